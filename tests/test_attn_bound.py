"""CPU: what the roundings of attention's weights to bf16 can do to an output, in 64 bits but for those roundings."""
import pytest
import torch

from tests import attn_bound, attn_ref

F64 = torch.float64


@pytest.mark.parametrize("n", [96, 192, 384, 736, 1472])
def test_rounded_weights_in_numerator_and_denominator(n):
    """A quotient of sums of the same rounded weights stays within attn_bound's bound, and passes the one that
    attn_ref derives for a denominator of weights that are not rounded."""
    q, k, v, scale = attn_bound.one_value(n)
    seen = torch.ones((1, n), dtype=torch.bool)
    want, bound = attn_bound.attend(q, k, v, scale, seen)
    other, _, narrow, _ = attn_ref.attend(q, k, v, scale, seen)
    assert torch.equal(want, other)
    p = torch.exp(scale * (q.to(F64) @ k.to(F64).t())).float().to(torch.bfloat16).to(F64)
    out = (p @ v.to(F64) / p.sum(1, keepdim=True)).float().to(torch.bfloat16)
    attn_ref.check(out, want, bound, "out")
    assert ((out.to(F64) - want).abs() > narrow).any()
