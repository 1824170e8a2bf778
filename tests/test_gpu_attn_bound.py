"""GPU: the attention operators where their weights' roundings to bf16 add up as far as they can, and
fp8_attn_chunk on ordinary values, held to the bound of a quotient of sums of the same rounded weights."""
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests import attn_bound, attn_ref
from tests.gpu_util import DEV, need_gpu
from tests.test_gpu_attn_chunk import KS, VS, _call, _setup

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def setup_module(_):
    need_gpu()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [96, 192, 736, 1472])
def test_roundings_that_go_apart(n, d):
    q, k, v, scale = (x.to(DEV) if isinstance(x, torch.Tensor) else x for x in attn_bound.one_value(n, d))
    seen = torch.ones((1, n), dtype=torch.bool, device=DEV)
    want, bound = attn_bound.attend(q, k, v, scale, seen)
    kc, vc = (x.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1) for x in (k, v))
    table = torch.arange(n // 32, dtype=I32, device=DEV)[None]
    lens, cu_k = torch.tensor([n], dtype=I32, device=DEV), torch.tensor([0, n], dtype=I32, device=DEV)
    for rows in (1, 5, 40, 130):
        qs, cu = q.expand(rows, d).contiguous(), torch.tensor([0, rows], dtype=I32, device=DEV)
        out = fq.fp8_attn_chunk(qs, kc, vc, table, lens, cu, 1, 1, d, 32, 1.0, 1.0, softmax_scale=scale, causal=False)
        attn_ref.check(out, want.expand(rows, d), bound.expand(rows, d), f"chunk of {rows}")
        out = fq.attn_prefill(qs, k.to(BF16), v.to(BF16), cu, 1, 1, d, cu_seqlens_k=cu_k, softmax_scale=scale,
                              causal=False)
        attn_ref.check(out, want.expand(rows, d), bound.expand(rows, d), f"prompt of {rows}")
    out = fq.fp8_attn_decode(q, kc, vc, table, lens, 1, 1, d, 32, 1.0, 1.0, softmax_scale=scale)
    attn_ref.check(out, want, bound, "decode")


@pytest.mark.parametrize("q_lens,lens", [([1, 3, 17], [40, 700, 17]), ([70, 5], [300, 2100]), ([200], [200])])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 4, 4), (256, 4, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_of_ordinary_values(q_lens, lens, d, hq, hkv, causal):
    s = _setup(q_lens, lens, hq, hkv, d, 16)
    out = _call(s, causal=causal).view(-1, hq, d)
    ks, vs = torch.tensor(KS).item(), torch.tensor(VS).item()
    pools = [s[x].view(-1, 16, hkv, d) for x in ("kc", "vc")]
    first = 0
    for i, (lq, n) in enumerate(zip(q_lens, lens)):
        pos = torch.arange(n, device=DEV)
        ids = s["tables"][i].long()[pos // 16]
        seen = attn_ref.causal_mask(lq, n, DEV) if causal else torch.ones((lq, n), dtype=torch.bool, device=DEV)
        for h in range(hq):
            k, v = (attn_ref.e4m3_values(p[ids, pos % 16, h // (hq // hkv)]) for p in pools)
            rows = s["q"][first:first + lq].view(lq, hq, d)[:, h]
            want, bound = attn_bound.attend(rows, k, v, d ** -0.5 * ks, seen)
            attn_ref.check(out[first:first + lq, h], want * vs, bound * vs + want.abs() * vs * 4 * attn_ref.U24,
                           f"sequence {i} head {h}")
        first += lq
