"""GPU: the ends of what fp8_rms_norm_group_quant, fp8_silu_mul_group_quant and fp8_attn_chunk accept."""
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
U24 = 2.0 ** -24


def setup_module(_):
    need_gpu()


@pytest.mark.parametrize("k", [(1 << 31) - 16384 - 128, (1 << 31) - 16384, (1 << 31) - 128])
def test_norm_of_one_row_of_nearly_two_to_the_31_columns(k):
    """x is +-1 and +-2 in turn.  A lane's squares are whole numbers, 40 in 16 values, and add up exactly in its
    2^17 steps (below 2^24); the sums over 64 lanes and 16 waves round at most 22 times.  With the mean, its
    root and two products y is off by at most 30 u, and the scale by 2 u more; a group's codes are those of
    448 x / 2, which that does not move to a neighbour's."""
    g = torch.Generator(device=DEV).manual_seed(k % 1000)
    x = torch.empty((1, k), dtype=BF16, device=DEV)
    cell = torch.where(torch.rand((1, 128), generator=g, device=DEV) < 0.5, -1.0, 1.0)
    cell *= torch.tensor([1.0, 2.0], device=DEV).repeat(64)
    x.view(-1, 128)[:] = cell.to(BF16)
    x.view(-1, 128)[k // 128 - 1] = cell.flip(1)[0].to(BF16)  # the last group is another one
    q = torch.full((1, k), 0x7F, dtype=torch.uint8, device=DEV)
    s = torch.zeros((1, k // 128), device=DEV)
    fq.fp8_rms_norm_group_quant(x, None, eps=0.0, q=q, scales=s)
    want = 2.0 / 2.5 ** 0.5 / 448
    assert ((s.to(F64) - want).abs() <= 32 * U24 * want).all()
    codes = (cell * 224).to(torch.float8_e4m3fn).view(torch.uint8)[0]
    rows = q.view(-1, 128)
    assert torch.equal(rows[-1], codes.flip(0))
    for i in range(0, k // 128 - 1, 1 << 20):
        part = rows[i:min(i + (1 << 20), k // 128 - 1)]
        assert (part == codes).all(), i
