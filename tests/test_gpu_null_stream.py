"""GPU: the attention operators on the null stream, given by its handle while another is current."""
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from fp8_e4m3_quantization_amd import _lib
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def setup_module(_):
    need_gpu()


def test_what_a_call_allocates_belongs_to_the_null_stream():
    g = torch.Generator(device=DEV).manual_seed(4)
    n, hq, hkv, d, bs = 40, 8, 2, 128, 16
    q, k, v = (torch.randn((n, h * d), generator=g, device=DEV).to(BF16) for h in (hq, hkv, hkv))
    kc, vc = (torch.randn(200 * bs * hkv * d, generator=g, device=DEV).to(torch.float8_e4m3fn)
              .view(torch.uint8) for _ in range(2))
    tables = torch.arange(200, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([3000], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 30], dtype=torch.int32, device=DEV)

    def calls(**kw):
        return [*fq.qk_norm_rope(q, k, None, None, hq, hkv, d, **kw),
                fq.attn_prefill(q, k, v, cu, hq, hkv, d, **kw),
                fq.fp8_attn_decode(q[:1], kc, vc, tables, lens, hq, hkv, d, bs, 1.0, 1.0, **kw)]

    assert torch.cuda.current_stream().cuda_stream == 0
    want = calls()
    torch.cuda.synchronize()
    _lib._ATTN_WORKSPACES.of.clear()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with _lib._on_stream(0, DEV):
            assert torch.cuda.current_stream().cuda_stream == 0
        got = calls(stream=0)
        assert torch.cuda.current_stream() == side
    torch.cuda.default_stream().synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert list(_lib._ATTN_WORKSPACES.of) == [(0, 0)]
