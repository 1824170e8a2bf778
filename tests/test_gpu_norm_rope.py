"""GPU parity: head norms, rotary positions and the paged E4M3 write (qk_norm_rope,
fp8_qk_norm_rope_kv_write) against the formula in 64 bits; cache bytes equal fp8_kv_write's of
the rounded keys."""
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
U24 = 2.0 ** -24


def setup_module(_):
    need_gpu()


def _table(npos, rot, gen):
    a = torch.rand((npos, max(rot // 2, 1)), generator=gen, device=DEV, dtype=F64) * 6.3
    return torch.cat([a.cos(), a.sin()], 1)[:, :rot].float().contiguous()


def _ref(x, w, eps, cs, pos, rot, inter, heads, d):
    """(y, bound) in binary64.  In binary32: the mean of D squares (D + 2 roundings at most), the
    root and quotient (3), two products, and the rotation's two products and sum (3), each of half
    a step relative to |n_a c| + |n_b s|; then half a bf16 step of y."""
    x = x.to(F64).reshape(-1, heads, d)
    n = x if w is None else x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.to(F64)
    y, size = n.clone(), n.abs()
    if rot:
        c, s = cs.to(F64)[pos][:, None, :rot // 2], cs.to(F64)[pos][:, None, rot // 2:]
        ia = torch.arange(0, rot, 2, device=DEV) if inter else torch.arange(rot // 2, device=DEV)
        ib = ia + 1 if inter else ia + rot // 2
        a, b = n[..., ia], n[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size = size.clone()
        size[..., ia] = (a * c).abs() + (b * s).abs()
        size[..., ib] = (b * c).abs() + (a * s).abs()
    bound = torch.finfo(BF16).eps / 2 * y.abs() + (d + 16) * U24 * size + 1e-30
    return y.reshape(x.shape[0], -1), bound.reshape(x.shape[0], -1)


def _check(got, ref):
    y, bound = ref
    err = (got.to(F64) - y).abs() / bound
    assert float(err.max()) <= 1.0, f"worst error / bound = {float(err.max()):.3f}"


CASES = [  # tokens, Hq, Hkv, D, rot, interleaved, norm, block size
    (1, 1, 1, 64, 64, False, True, 16), (16, 40, 4, 128, 128, False, True, 16),
    (7, 40, 4, 128, 128, True, True, 16), (33, 8, 8, 64, 32, True, False, 1),
    (5, 6, 2, 256, 64, False, True, 48), (19, 3, 1, 32, 16, False, True, 8),
    (3, 2, 1, 512, 512, True, True, 16), (257, 32, 8, 128, 0, False, True, 16),
    (9, 5, 5, 80, 40, False, True, 16), (11, 4, 2, 96, 96, True, True, 24),  # element-wise
    (6, 4, 2, 128, 24, False, False, 16), (4, 3, 3, 7, 6, False, True, 5),
    (1300, 40, 4, 128, 128, False, True, 16),
]


@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,norm,bs", CASES)
@pytest.mark.parametrize("layout", ["packed", "columns", "odd"])
def test_matches_the_formula_and_the_plain_write(t, hq, hkv, d, rot, inter, norm, bs, layout):
    g = torch.Generator(device=DEV).manual_seed(t * 7 + d + rot)
    pad = {"packed": 0, "columns": 64, "odd": 3}[layout]
    row = (hq + 2 * hkv) * d + pad
    qkv = (torch.randn((t, row), generator=g, device=DEV) * 3).to(BF16)
    if layout == "packed":
        q, k, v = (x.contiguous() for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = qkv[:, pad:].split([hq * d, hkv * d, hkv * d], 1)
    qw = (1 + torch.randn(d, generator=g, device=DEV) * 0.2).to(BF16) if norm else None
    kw = (1 + torch.randn(d, generator=g, device=DEV) * 0.2).to(BF16) if norm else None
    npos = 500
    cs = _table(npos, rot, g) if rot else None
    pos = torch.randint(0, npos, (t,), generator=g, device=DEV) if rot else None
    blocks = -(-t // bs) + 3
    slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:t].contiguous()
    slots[t // 2] = -1 if t % 2 else blocks * bs
    q_in, k_in = q.clone(), k.clone()
    qo, ko = fq.qk_norm_rope(q, k, pos, cs, hq, hkv, d, qw, kw, 1e-5, inter)
    _check(qo, _ref(q_in, qw, 1e-5, cs, pos, rot, inter, hq, d))
    _check(ko, _ref(k_in, kw, 1e-5, cs, pos, rot, inter, hkv, d))
    kc = torch.randint(0, 256, (blocks * bs * hkv * d,), generator=g, device=DEV, dtype=torch.uint8)
    vc = kc.flip(0).contiguous()
    kc2, vc2 = kc.clone(), vc.clone()
    ko2 = torch.empty_like(ko)
    qo2 = fq.fp8_qk_norm_rope_kv_write(q, k, v, pos, cs, kc, vc, slots, hq, hkv, d, bs, 0.03, 0.02,
                                       qw, kw, 1e-5, inter, k_out=ko2)
    fq.fp8_kv_write(ko, v, kc2, vc2, slots, hkv, d, bs, 0.03, 0.02,
                    value_stride=v.stride(0) if t > 1 else hkv * d)
    assert torch.equal(qo, qo2) and torch.equal(ko, ko2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert torch.equal(q, q_in) and torch.equal(k, k_in)
    # in place, and without k_out
    kc3, vc3 = kc.clone(), vc.clone()
    fq.fp8_qk_norm_rope_kv_write(q, k, v, pos, cs, kc3, vc3, slots, hq, hkv, d, bs, 0.03, 0.02, qw,
                                 kw, 1e-5, inter, q_out=q)
    assert torch.equal(kc, kc3) and torch.equal(vc, vc3) and torch.equal(q, qo)
    assert torch.equal(k, k_in)
    fq.qk_norm_rope(q_in, k, pos, cs, hq, hkv, d, qw, kw, 1e-5, inter, q_out=q, k_out=k)
    assert torch.equal(k, ko)


@pytest.mark.parametrize("d", [128, 80])
def test_tokens_outside_the_table_leave_everything_as_it_was(d):
    t, hq, hkv, bs = 6, 4, 2, 16
    q = torch.randn((t, hq * d), device=DEV).to(BF16)
    k = torch.randn((t, hkv * d), device=DEV).to(BF16)
    cs = torch.ones((50, d), device=DEV)
    pos = torch.tensor([0, -1, 49, 50, 1 << 40, -(1 << 62)], device=DEV)
    kc = torch.full((bs * 4 * hkv * d,), 7, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, 9)
    qo, ko = torch.full_like(q, 5.0), torch.full_like(k, 6.0)
    fq.fp8_qk_norm_rope_kv_write(q, k, k, pos, cs, kc, vc, torch.arange(t, device=DEV), hq, hkv, d,
                                 bs, 1.0, 1.0, q_out=qo, k_out=ko)
    for i in (1, 3, 4, 5):
        assert (qo[i] == 5).all() and (ko[i] == 6).all()
        assert (kc.view(-1, hkv * d)[i] == 7).all() and (vc.view(-1, hkv * d)[i] == 9).all()
    for i in (0, 2):
        assert not (qo[i] == 5).all() and not (kc.view(-1, hkv * d)[i] == 7).all()


def test_norm_of_zeros_and_of_large_values():
    d = 128
    q = torch.zeros((2, d), dtype=BF16, device=DEV)
    q[1] = 2.0 ** 60
    w = torch.ones(d, dtype=BF16, device=DEV)
    qo, _ = fq.qk_norm_rope(q, q.clone(), None, None, 1, 1, d, w, w)
    assert not qo[0].any() and torch.equal(qo[1], torch.ones_like(qo[1]))


def test_another_stream_and_a_replayed_graph():
    t, hq, hkv, d, bs = 16, 8, 2, 128, 16
    q = torch.randn((t, hq * d), device=DEV).to(BF16)
    k, v = (torch.randn((t, hkv * d), device=DEV).to(BF16) for _ in range(2))
    cs = _table(64, d, torch.Generator(device=DEV).manual_seed(1))
    pos, slots = torch.arange(t, device=DEV), torch.arange(t, device=DEV) + 5
    kc = torch.zeros(4 * bs * hkv * d, dtype=torch.uint8, device=DEV)
    vc, qo = torch.zeros_like(kc), torch.zeros_like(q)

    def step(**kw):
        fq.fp8_qk_norm_rope_kv_write(q, k, v, pos, cs, kc, vc, slots, hq, hkv, d, bs, 0.02, 0.02,
                                     q_out=qo, **kw)

    step()
    want = [x.clone() for x in (qo, kc, vc)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for x in (qo, kc, vc):
        x.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side.cuda_stream)
    alone = fq.qk_norm_rope(q, k, pos, cs, hq, hkv, d, stream=side.cuda_stream)[0]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((qo, kc, vc), want)) and torch.equal(alone, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in (qo, kc, vc):
            x.zero_()
        fq.qk_norm_rope(q, k, pos, cs, hq, hkv, d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((qo, kc, vc), want))


@pytest.mark.parametrize("d", [128, 96])
def test_rows_past_four_gib(d):
    """Rows 8 MiB apart give what packed rows give."""
    t, hq, hkv = 600, 2, 1
    g = torch.Generator(device=DEV).manual_seed(d)
    wide = torch.empty((t, 1 << 22), dtype=torch.bfloat16, device=DEV)
    q, k = wide[:, :hq * d], wide[:, 256:256 + hkv * d]
    for x in (q, k):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
    positions = torch.randint(0, 1000, (t,), generator=g, device=DEV)
    table = torch.randn((1000, 32), generator=g, device=DEV)
    want = fq.qk_norm_rope(q.contiguous(), k.contiguous(), positions, table, hq, hkv, d)
    got = fq.qk_norm_rope(q, k, positions, table, hq, hkv, d, q_out=wide[:, 512:512 + hq * d],
                          k_out=wide[:, 768:768 + hkv * d])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
