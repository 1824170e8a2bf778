"""GPU: the operators in a row as a layer uses them -- W8A8 projections, head norms with rotary
positions and the paged write, attention over the prompt, then single-token steps over the cache,
and a second chunk behind the history read back from it."""
import threading

import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from fp8_e4m3_quantization_amd import _lib
from tests import attn_ref
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
HQ, HKV, D, BS, K = 8, 2, 128, 16, 512


def setup_module(_):
    need_gpu()


def test_prompt_then_steps_then_a_second_chunk():
    g = torch.Generator(device=DEV).manual_seed(11)
    lens = [37, 1, 130]
    wqkv = (torch.randn(((HQ + 2 * HKV) * D, K), generator=g, device=DEV) * 0.05).to(BF16)
    wo = (torch.randn((K, HQ * D), generator=g, device=DEV) * 0.05).to(BF16)
    wq, ws = fq.fp8_block_quant(wqkv)
    oq, os_ = fq.fp8_block_quant(wo)
    qw, kw = ((1 + torch.randn(D, generator=g, device=DEV) * 0.1).to(BF16) for _ in range(2))
    angle = torch.arange(512, device=DEV, dtype=F64)[:, None] * \
        10000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=F64) / D)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    blocks = 64
    tables = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)[:36].view(3, 12).contiguous()
    kc = torch.zeros(blocks * BS * HKV * D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks, vs = 0.05, 0.05

    def slots_of(seq, pos):
        return tables[seq, pos // BS].long() * BS + pos % BS

    def project(x):
        xq, xs = fq.fp8_group_quant(x)
        fn = fq.w8a8_block_gemm if x.shape[0] <= 16 else fq.w8a8_block_gemm_prefill
        return fn(xq, xs, wq, ws).split([HQ * D, HKV * D, HKV * D], 1)

    # the prompt
    seq = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(lens, device=DEV))
    pos = torch.cat([torch.arange(n, device=DEV) for n in lens])
    x = torch.randn((sum(lens), K), generator=g, device=DEV).to(BF16)
    q, k, v = project(x)
    ko = torch.empty((sum(lens), HKV * D), dtype=BF16, device=DEV)
    qo = fq.fp8_qk_norm_rope_kv_write(q, k, v, pos, cos_sin, kc, vc, slots_of(seq, pos), HQ, HKV, D,
                                      BS, ks, vs, qw, kw, k_out=ko)
    starts = [0, 37, 38, 168]
    cu = torch.tensor(starts, dtype=torch.int32, device=DEV)
    lse = torch.empty((sum(lens), HQ), device=DEV)
    out = fq.attn_prefill(qo, ko, v, cu, HQ, HKV, D, lse=lse)
    attn_ref.prefill(qo, ko, v, starts, starts, HQ, HKV, D, D ** -0.5, True, out, lse)
    y = fq.w8a8_block_gemm_prefill(*fq.fp8_group_quant(out), oq, os_)
    assert torch.isfinite(y.float()).all()

    # three single-token steps
    now = list(lens)
    for step in range(3):
        x = torch.randn((3, K), generator=g, device=DEV).to(BF16)
        q, k, v = project(x)
        pos = torch.tensor(now, device=DEV)
        qo = fq.fp8_qk_norm_rope_kv_write(q, k, v, pos, cos_sin, kc, vc,
                                          slots_of(torch.arange(3, device=DEV), pos), HQ, HKV, D, BS,
                                          ks, vs, qw, kw)
        now = [n + 1 for n in now]
        ctx = torch.tensor(now, dtype=torch.int32, device=DEV)
        lse = torch.empty((3, HQ), device=DEV)
        out = fq.fp8_attn_decode(qo, kc, vc, tables, ctx, HQ, HKV, D, BS, ks, vs, lse=lse)
        attn_ref.decode(qo, kc, vc, tables, now, HQ, HKV, D, BS, BS * HKV * D,
                        torch.tensor(ks).item(), torch.tensor(vs).item(), D ** -0.5, out, lse)
        y = fq.w8a8_block_gemm(*fq.fp8_group_quant(out), oq, os_)
        assert torch.isfinite(y.float()).all()

    # a second chunk of sequence 0: its history read back from the cache, its own rows in bf16
    n, more = now[0], 20
    pos = torch.arange(n, n + more, device=DEV)
    x = torch.randn((more, K), generator=g, device=DEV).to(BF16)
    q, k, v = project(x)
    hist = torch.arange(n, device=DEV)
    kall = torch.empty((n + more, HKV * D), dtype=BF16, device=DEV)
    vall = torch.empty_like(kall)
    fq.fp8_kv_read(kc, vc, slots_of(0, hist), HKV, D, BS, ks, vs, k_out=kall, v_out=vall)
    qo = fq.fp8_qk_norm_rope_kv_write(q, k, v, pos, cos_sin, kc, vc, slots_of(0, pos), HQ, HKV, D, BS,
                                      ks, vs, qw, kw, k_out=kall[n:])
    vall[n:] = v
    lse = torch.empty((more, HQ), device=DEV)
    out = fq.attn_prefill(qo, kall, vall, torch.tensor([0, more], dtype=torch.int32, device=DEV), HQ,
                          HKV, D, lse=lse,
                          cu_seqlens_k=torch.tensor([0, n + more], dtype=torch.int32, device=DEV))
    attn_ref.prefill(qo, kall, vall, [0, more], [0, n + more], HQ, HKV, D, D ** -0.5, True, out, lse)


def test_two_threads_on_one_stream():
    """Each thread's calls enqueue two kernels with a workspace between them; calls of another
    thread on the same stream may come in between."""
    g = torch.Generator(device=DEV).manual_seed(3)
    hq, hkv, d, bs, n = 16, 2, 128, 16, 3000
    blocks = n // bs + 1
    kc, vc = ((torch.randn((blocks * bs * hkv * d,), generator=g, device=DEV)).to(torch.float8_e4m3fn)
              .view(torch.uint8) for _ in range(2))
    tables = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu_q = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    k, v = (torch.randn((n, hkv * d), generator=g, device=DEV).to(BF16) for _ in range(2))
    qs = [torch.randn((20, hq * d), generator=g, device=DEV).to(BF16) for _ in range(2)]
    assert fq.attn_prefill_workspace_size(1, 20, n, hq, hkv, d) > 0

    def calls(q):
        return (fq.fp8_attn_decode(q[:1], kc, vc, tables, lens, hq, hkv, d, bs, 1.0, 1.0),
                fq.attn_prefill(q, k, v, cu_q, hq, hkv, d, cu_seqlens_k=cu_k))

    want = [calls(q) for q in qs]
    got = [[], []]
    spaces = [None, None]
    start = threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(200):
            got[i].append(calls(qs[i]))
        spaces[i] = [t.data_ptr() for t in _lib._ATTN_WORKSPACES.of.values()]
        start.wait()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert spaces[0] and spaces[1] and not set(spaces[0]) & set(spaces[1])
    for i in range(2):
        assert len(got[i]) == 200
        for pair in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(pair, want[i]))
