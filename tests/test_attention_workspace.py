"""Workspaces of the attention calls: attn_prefill's holds sums of real query rows, however the rows
are packed, and is bounded (CPU); the binding keeps few of them (GPU)."""
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from fp8_e4m3_quantization_amd import _lib

BF16 = torch.bfloat16
MOST_PARTS, MOST_BYTES = 64, 256 << 20


@pytest.mark.parametrize("seqs,tq,tk,hq,d", [
    (39, 39, 39 * 8192, 40, 128), (39, 39, 39 * 8192, 40, 256),  # one-token chunks behind histories
    (15, 15, 15 * 131072, 40, 256), (6, 24042, 2582747, 8, 256), (1, 9590, 2610032, 16, 256),
    (1, 3210, 912658, 40, 256), (2, 1526, 3044908, 40, 256), (1, 512, 8704, 40, 128),
    (1, 23, 2794, 10, 128), (1, 1, 1 << 30, 64, 256), (200, 200, 1 << 22, 8, 64)])
def test_prefill_workspace_is_what_its_rows_need(seqs, tq, tk, hq, d):
    need = fq.attn_prefill_workspace_size(seqs, tq, tk, hq, hq, d)
    row = 4 * d + 16  # its sums, and their reference and totals
    assert need % (tq * hq * row) == 0 and need // (tq * hq * row) <= MOST_PARTS
    assert need <= MOST_BYTES


def _decode_on(stream, s):
    with torch.cuda.stream(stream):
        return fq.fp8_attn_decode(*s, 8, 2, 128, 16, 1.0, 1.0)


@pytest.mark.gpu
def test_the_binding_keeps_few_workspaces():
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(2)
    q = torch.randn((2, 1024), generator=g, device=dev).to(BF16)
    kc, vc = (torch.randn(200 * 16 * 256, generator=g, device=dev).to(torch.float8_e4m3fn)
              .view(torch.uint8) for _ in range(2))
    s = (q, kc, vc, torch.arange(200, dtype=torch.int32, device=dev).view(2, 100),
         torch.tensor([1600, 1111], dtype=torch.int32, device=dev))
    want = _decode_on(torch.cuda.current_stream(), s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(20)]
    outs = [_decode_on(st, s) for st in streams for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert 1 <= len(_lib._ATTN_WORKSPACES.of) <= 8
    # a call that needs much: made for it, not kept
    tq, tk, hq, d = 1700, 30000, 40, 128
    assert fq.attn_prefill_workspace_size(1, tq, tk, hq, 4, d) > 64 << 20
    q, k, v = (torch.randn((n, h * d), generator=g, device=dev).to(BF16)
               for n, h in ((tq, hq), (tk, 4), (tk, 4)))
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=dev) for n in (tq, tk))
    a, b = (fq.attn_prefill(q, k, v, cu_q, hq, 4, d, cu_seqlens_k=cu_k) for _ in range(2))
    assert torch.equal(a, b)
    assert all(t.numel() <= 64 << 20 for t in _lib._ATTN_WORKSPACES.of.values())


def test_calls_of_too_many_sequences_are_refused():
    """Every workgroup searches all lengths: beyond 65536 sequences a call would run for seconds to
    minutes.  (Nothing is enqueued: the checks return before any pointer is looked at.)"""
    assert fq.fp8_attn_decode_workspace_size(1 << 16, 8, 2, 128) > 0
    assert fq.attn_prefill_workspace_size(1 << 16, 1 << 16, 1 << 16, 8, 2, 128) == 0
    n = (1 << 16) + 1
    for call in (lambda: fq.fp8_attn_decode_workspace_size(n, 8, 2, 128),
                 lambda: fq.attn_prefill_workspace_size(n, n, n, 8, 2, 128)):
        with pytest.raises(_lib.Fp8qError, match="-1"):
            call()
