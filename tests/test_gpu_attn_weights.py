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
