"""GPU: what single weights do to attn_prefill's outputs -- one that is above all others, and ones
too small for binary32 beside values that are not finite."""
import math

import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests import attn_ref
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def setup_module(_):
    need_gpu()


def _cu(n):
    return torch.tensor([0, n], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,at", [(64, 300, 256), (20, 3000, 200)])  # whole, split over workgroups
def test_one_weight_above_all_others(d, lq, lk, at):
    """One key outweighs one other by 2^x, 0.5 <= x < 8, behind it, so that its weight against the
    running reference is 2^x and is rounded to bf16.  The rounding, by a factor 1 + e with
    |e| <= 2^-8, is in numerator and denominator: with w the true share and v = 0 at the other key,
    out = v w (1 + e) / (1 + w e) is off by at most v w (1 - w) 2^-8 (1 + 2^-7), and by its own
    rounding and a few binary32 steps.  All other keys' weights are below e^-150.  lse is off by
    its score's roundings ((d + 8) steps of at most 8 log 2) and a few of its own."""
    k = torch.full((lk, d), -448.0, device=DEV)
    k[0], k[at] = 0.0, 1.0
    v = torch.zeros((lk, d), device=DEV)
    v[at] = torch.arange(1, d + 1, device=DEV) * 4.0
    k, v = k.to(BF16), v.to(BF16)
    c = (torch.linspace(0.5, 7.9, lq, device=DEV) * math.log(2) / d).to(BF16)
    q = c[:, None].expand(lq, d).contiguous()
    assert (fq.attn_prefill_workspace_size(1, lq, lk, 1, 1, d) > 0) == (lk > 1000)
    lse = torch.empty((lq, 1), device=DEV)
    out = fq.attn_prefill(q, k, v, _cu(lq), 1, 1, d, cu_seqlens_k=_cu(lk), softmax_scale=1.0,
                          causal=False, lse=lse)
    s = c.double() * d
    w = torch.sigmoid(s)[:, None]
    top = v[at].double()
    bound = attn_ref.HALF_BF16 * w * top + 2.0 ** -8 * (1 + 2.0 ** -7) * w * (1 - w) * top + 2.0 ** -18 * top
    attn_ref.check(out, w * top, bound, "out")
    want = torch.log1p(torch.exp(s))
    attn_ref.check(lse[:, 0], want, ((d + 8) * 6 + 64) * attn_ref.U24 + 0 * want, "lse")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,causal", [(300, 300, True), (40, 300, False), (20, 3000, False)])
@pytest.mark.parametrize("at", [3, 130, -3])  # a tile that every query sees whole, one of few, the last
def test_values_that_are_not_finite_reach_all_that_see_them(d, lq, lk, causal, at):
    """Scores of 0 and +-200, so that most weights are 0 in binary32, before or behind the largest:
    an infinity reaches every query that sees it, in its columns, wherever its key lies and however
    the call is split; with one of the other sign beside it, or a NaN, the sum is NaN; a query with
    a score that is NaN is NaN throughout.  Nothing else changes."""
    g = torch.Generator(device=DEV).manual_seed(d + lq)
    at %= lk
    level = torch.randint(-1, 2, (lk, 1), generator=g, device=DEV) * 200.0
    sign = torch.randint(0, 2, (lq, 1), generator=g, device=DEV) * 2.0 - 1
    k, q = level.expand(lk, d).to(BF16).contiguous(), (sign / d).expand(lq, d).to(BF16).contiguous()
    v = torch.randn((lk, d), generator=g, device=DEV).to(BF16)
    sees = attn_ref.causal_mask(lq, lk, DEV) if causal else torch.ones((lq, lk), dtype=torch.bool, device=DEV)

    def run(k, v):
        return fq.attn_prefill(q, k, v, _cu(lq), 1, 1, d, cu_seqlens_k=_cu(lk), softmax_scale=1.0, causal=causal)

    want = run(k, v)
    assert torch.isfinite(want.float()).all()
    assert (fq.attn_prefill_workspace_size(1, lq, lk, 1, 1, d) > 0) == (lk > 1000)
    cols = torch.tensor([0, 5, 6, d - 1], device=DEV)
    for bad in (math.inf, -math.inf, math.nan):
        v2 = v.clone()
        v2[at, cols] = bad
        expect = want.clone()
        expect[:, cols] = torch.where(sees[:, at, None], bad, want[:, cols].float()).to(BF16)
        assert torch.equal(run(k, v2).nan_to_num(9e9, 8e9, 7e9), expect.nan_to_num(9e9, 8e9, 7e9)), bad
    other = (at + 90) % lk
    v2 = v.clone()
    v2[at, cols], v2[other, cols] = math.inf, -math.inf
    a, b = sees[:, at, None], sees[:, other, None]
    expect = want.clone()
    expect[:, cols] = torch.where(a & b, math.nan, torch.where(a, math.inf, torch.where(
        b, -math.inf, want[:, cols].float()))).to(BF16)
    assert torch.equal(run(k, v2).nan_to_num(9e9, 8e9, 7e9), expect.nan_to_num(9e9, 8e9, 7e9))
    k2 = k.clone()
    k2[other] = math.nan
    expect = torch.where(b, math.nan, expect.float()).to(BF16)
    assert torch.equal(run(k2, v2).nan_to_num(9e9, 8e9, 7e9), expect.nan_to_num(9e9, 8e9, 7e9))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,causal", [(300, 300, True), (33, 700, False), (20, 3000, False)])
@pytest.mark.parametrize("kinds,share", [((math.inf, -math.inf, math.nan), 0.002), ((math.inf,), 0.3),
                                         ((math.nan,), 1.0), ((math.inf, -math.inf), 0.6)])
def test_many_values_that_are_not_finite(d, lq, lk, causal, kinds, share):
    """What a query sees of a column decides: nothing but finite values, and the output is as if the
    others were finite too; else the sum of those that are not."""
    g = torch.Generator(device=DEV).manual_seed(d + lk)
    q, k, v = (torch.randn((n, d), generator=g, device=DEV).to(BF16) * std
               for n, std in ((lq, 30.0), (lk, 1.0), (lk, 1.0)))
    kind = torch.tensor(kinds, device=DEV).to(BF16)[torch.randint(0, len(kinds), (lk, d), generator=g, device=DEV)]
    hit = torch.rand((lk, d), generator=g, device=DEV) < share
    v2 = torch.where(hit, kind, v)
    sees = (attn_ref.causal_mask(lq, lk, DEV) if causal else torch.ones((lq, lk), dtype=torch.bool, device=DEV)).float()
    up, down, nan = (sees @ x.float() > 0 for x in (v2 == math.inf, v2 == -math.inf, torch.isnan(v2)))
    out = [fq.attn_prefill(q, k, x, _cu(lq), 1, 1, d, cu_seqlens_k=_cu(lk), causal=causal) for x in (v, v2)]
    expect = torch.where(nan | (up & down), math.nan, torch.where(up, math.inf, torch.where(
        down, -math.inf, out[0].float()))).to(BF16)
    assert torch.equal(out[1].nan_to_num(9e9, 8e9, 7e9), expect.nan_to_num(9e9, 8e9, 7e9))
