"""GPU: a served layer in a row, as one batch mixes them -- chunks of prompts, whole prompts, steps and
drafted tokens: norm with the residual's addition, W8A8 projections, head norms with rotary positions
and the paged write, attention over the pages, output projection, norm, gate and up projections, SiLU,
down projection.  Each step is held to its definition on the inputs that it got."""
import threading

import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from fp8_e4m3_quantization_amd import _lib
from tests import test_gpu_attn_chunk as chunk
from tests import test_gpu_norm_quant as norm
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
HQ, HKV, D, BS, K, INTER = 8, 2, 128, 16, 512, 640
KS = VS = 0.05


def setup_module(_):
    need_gpu()


def _weights(g, n, k):
    return fq.fp8_block_quant((torch.randn((n, k), generator=g, device=DEV) * 0.05).to(BF16))


def _product(q, s, w, ws, fn=None):
    """The product, held to its definition in 64 bits: 1e-2 of itself and 1e-3 of the rows' size."""
    fn = fn or (fq.w8a8_block_gemm if q.shape[0] <= 16 else fq.w8a8_block_gemm_prefill)
    out = fn(q, s, w, ws)
    a = q.view(torch.float8_e4m3fn).to(torch.float32).to(F64) * s.to(F64).repeat_interleave(128, 1)
    b = w.view(torch.float8_e4m3fn).to(torch.float32).to(F64)
    b = b * ws.to(F64).repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = a @ b.t()
    rms = want.square().mean().sqrt()
    assert ((out.to(F64) - want).abs() <= 1e-2 * want.abs() + 1e-3 * rms).all()
    return out


class Layer:
    def __init__(self, seed, blocks=64):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.qkv, self.o = _weights(g, (HQ + 2 * HKV) * D, K), _weights(g, K, HQ * D)
        self.gate_up, self.down = _weights(g, 2 * INTER, K), _weights(g, K, INTER)
        self.n1, self.n2 = ((1 + torch.randn(K, generator=g, device=DEV) * 0.2).to(BF16) for _ in range(2))
        self.qw, self.kw = ((1 + torch.randn(D, generator=g, device=DEV) * 0.1).to(BF16) for _ in range(2))
        angle = torch.arange(512, device=DEV, dtype=F64)[:, None] * \
            10000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=F64) / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.tables = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)[:36].view(3, 12).contiguous()
        self.kc = torch.full((blocks * BS * HKV * D,), 0x7F, dtype=torch.uint8, device=DEV)  # stale NaN
        self.vc = self.kc.clone()

    def slots(self, seq, pos):
        return self.tables[seq, pos // BS].long() * BS + pos % BS

    def run(self, x, residual, pos, slots, cu, lens, product=_product, lse=None):
        """(output, residual, what the attention was given and gave, both norms' inputs and outputs)."""
        q, s, r = fq.fp8_rms_norm_group_quant(x, self.n1, residual=residual)
        first = (x, self.n1, 1e-6, residual, q, s, r)
        qkv = product(q, s, *self.qkv)
        qh, kh, vh = qkv.split([HQ * D, HKV * D, HKV * D], 1)
        qh = fq.fp8_qk_norm_rope_kv_write(qh, kh, vh, pos, self.cos_sin, self.kc, self.vc, slots, HQ, HKV, D,
                                          BS, KS, VS, self.qw, self.kw)
        out = fq.fp8_attn_chunk(qh, self.kc, self.vc, self.tables, lens, cu, HQ, HKV, D, BS, KS, VS, lse=lse)
        y = product(*fq.fp8_group_quant(out), *self.o)
        before = x if r is None else r
        q, s, r = fq.fp8_rms_norm_group_quant(y, self.n2, residual=before)
        second = (y, self.n2, 1e-6, before, q, s, r)
        gate, up = product(q, s, *self.gate_up).split(INTER, 1)
        q, s = fq.fp8_silu_mul_group_quant(gate, up)
        return product(q, s, *self.down), r, (qh, out), (first, second, (gate, up, q, s))


def _check(layer, cu, lens, lse, attn, steps):
    qh, out = attn
    s = dict(q=qh, kc=layer.kc, vc=layer.vc, tables=layer.tables, bs=BS, cs=BS * HKV * D, hq=HQ, hkv=HKV, d=D,
             cu=cu, lens=lens)
    saved = chunk.KS, chunk.VS
    chunk.KS, chunk.VS = KS, VS
    try:
        chunk._check(s, out, lse)
    finally:
        chunk.KS, chunk.VS = saved
    for a in steps[:2]:
        norm._check_norm(*a, None)
    norm._check_silu(*steps[2], None)


# new tokens of the three sequences, call by call: a prompt's first chunk beside a whole prompt; its
# rest beside a step and a third prompt; four drafted tokens each; a step each
CALLS = [[60, 41, 0], [70, 1, 9], [4, 4, 4], [1, 1, 1]]


def _batch(g, new, have):
    """Rows, positions' sequence and place, starts and lengths of a call."""
    seq = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(new, device=DEV))
    pos = torch.cat([torch.arange(h, h + n, device=DEV) for h, n in zip(have, new)])
    have = [h + n for h, n in zip(have, new)]
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
    x = torch.randn((sum(new), K), generator=g, device=DEV).to(BF16)
    return x, seq, pos, cu, torch.tensor(have, dtype=torch.int32, device=DEV), have


def test_two_layers_over_chunks_steps_and_drafted_tokens():
    layers = [Layer(1), Layer(2)]
    g = torch.Generator(device=DEV).manual_seed(7)
    have = [0, 0, 0]
    queries = []
    for new in CALLS:
        x, seq, pos, cu, lens, have = _batch(g, new, have)
        residual = None
        for i, layer in enumerate(layers):
            lse = torch.empty((sum(new), HQ), device=DEV)
            x, residual, attn, steps = layer.run(x, residual, pos, layer.slots(seq, pos), cu, lens, lse=lse)
            _check(layer, cu, lens, lse, attn, steps)
            if i == 0:
                queries.append(attn[0][:new[0]])
    # the first sequence's queries of all calls at once see what they saw then
    q = torch.cat(queries)
    layer, lse = layers[0], torch.empty((len(q), HQ), device=DEV)
    cu = torch.tensor([0, len(q)], dtype=torch.int32, device=DEV)
    lens = torch.tensor(have[:1], dtype=torch.int32, device=DEV)
    assert len(q) == have[0]
    out = fq.fp8_attn_chunk(q, layer.kc, layer.vc, layer.tables[:1], lens, cu, HQ, HKV, D, BS, KS, VS, lse=lse)
    s = dict(q=q, kc=layer.kc, vc=layer.vc, tables=layer.tables[:1], bs=BS, cs=BS * HKV * D, hq=HQ, hkv=HKV,
             d=D, cu=cu, lens=lens)
    saved = chunk.KS, chunk.VS
    chunk.KS, chunk.VS = KS, VS
    try:
        chunk._check(s, out, lse)
    finally:
        chunk.KS, chunk.VS = saved


def test_a_captured_layer_replays():
    """The whole layer in one graph: every replay leaves the bits of the eager call, with eager work of
    other shapes between the replays."""
    layer = Layer(3)
    g = torch.Generator(device=DEV).manual_seed(8)
    x, seq, pos, cu, lens, have = _batch(g, [20, 5, 7], [100, 130, 3])
    slots = layer.slots(seq, pos)
    hist = torch.cat([layer.slots(b, torch.arange(n, device=DEV)) for b, n in enumerate([100, 130, 3])])
    k, v = (torch.randn((len(hist), HKV * D), generator=g, device=DEV).to(BF16) for _ in range(2))
    fq.fp8_kv_write(k, v, layer.kc, layer.vc, hist, HKV, D, BS, KS, VS)
    residual = torch.randn((32, K), generator=g, device=DEV).to(BF16)

    def product(q, s, w, ws):
        return fq.w8a8_block_gemm_prefill(q, s, w, ws)

    want = layer.run(x, residual, pos, slots, cu, lens, product)[:2]
    pools = layer.kc.clone(), layer.vc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.run(x, residual, pos, slots, cu, lens, product)[:2]
    for rep in range(4):
        for t in got:
            t.zero_()
        layer.run(x[:rep + 1], None, pos[:rep + 1], slots[:rep + 1], cu.clamp(max=rep + 1), lens, product)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
        assert torch.equal(layer.kc, pools[0]) and torch.equal(layer.vc, pools[1])


def test_two_threads_on_one_stream():
    """Each thread's calls enqueue two kernels with a workspace between them; calls of another thread on
    the same stream may come in between."""
    s = [chunk._setup([20, 1], [3000, 2000], 16, 2, 128, 16, seed=i) for i in range(2)]
    assert fq.fp8_attn_chunk_workspace_size(2, 21, 16, 2, 128) > 0
    want = [chunk._call(x) for x in s]
    got, spaces, start = [[], []], [None, None], threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(200):
            got[i].append(chunk._call(s[i]))
        spaces[i] = [t.data_ptr() for t in _lib._ATTN_WORKSPACES.of.values()]
        start.wait()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert spaces[0] and spaces[1] and not set(spaces[0]) & set(spaces[1])
    for i in range(2):
        assert len(got[i]) == 200 and all(torch.equal(x, want[i]) for x in got[i])
