"""CPU checks of the ends of what fp8_rms_norm_group_quant, fp8_silu_mul_group_quant and
fp8_attn_chunk accept (nothing is enqueued: each call is refused for another reason)."""
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests.test_chunk_norm_checks import EALIGN, EINVAL, FAKE, _norm, _silu


@pytest.mark.parametrize("k", [128, 256, 384, 640, 5120, 16384 + 128, (1 << 31) - 128])
def test_most_rows(k):
    """m * (k / 128) < 2^31, to the last row."""
    most = ((1 << 31) - 1) // (k // 128)
    wide = dict(k=k, xs=k, rs=k, ros=k, nos=k)
    assert _norm(m=most, q=FAKE + 8, **wide) == EALIGN
    assert _norm(m=most + 1, q=FAKE + 8, **wide) == EINVAL
    wide = dict(k=k, gs=k, us=k, os=k)
    assert _silu(m=most, q=FAKE + 8, **wide) == EALIGN
    assert _silu(m=most + 1, q=FAKE + 8, **wide) == EINVAL


def test_binding_refuses_numbers_beyond_32_bits():
    """Their low halves would pass for a block of 16 positions, and for three sequences."""
    q, pool = torch.zeros((9, 1024), dtype=torch.bfloat16), torch.zeros(8 * 16 * 256, dtype=torch.uint8)
    tab, lens = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    cu = torch.tensor([0, 2, 5, 9], dtype=torch.int32)
    with pytest.raises(ValueError, match="block_size"):
        fq.fp8_attn_chunk(q, pool, pool, tab, lens, cu, 8, 2, 128, (1 << 32) + 16, 1.0, 1.0, cache_stride=16 * 256)
    many = (1 << 32) + 3
    wide, long, starts = (torch.empty(n, dtype=torch.int32, device="meta") for n in ((many, 4), many, many + 1))
    with pytest.raises(ValueError, match="sequences"):
        fq.fp8_attn_chunk(q, pool, pool, wide, long, starts, 8, 2, 128, 16, 1.0, 1.0)
