"""CPU checks of the ends of what fp8_rms_norm_group_quant, fp8_silu_mul_group_quant and
fp8_attn_chunk accept (nothing is enqueued: each call is refused for another reason)."""
import pytest

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
