"""GPU parity: fp8_rms_norm_group_quant and fp8_silu_mul_group_quant against their definitions in
64 bits.

Bounds, with u = 2^-24.  Norm: a lane squares and adds 16 values in a tree (5 u), pieces and waves
add one after another (at most k / 16384 + 1 and 16), the wave in a tree (6): the mean is off by
(29 + k / 16384) u, with its division and eps 2 u more; the root halves that, v_rsq adds 2 u, the two
products 2 u: y is off by (20 + k / 16384) u, taken as (24 + k / 16384).  SiLU: the exponent's argument
is off by 2 u of itself, so the exponential by 2 u |gate| and 2 u of its own; sum, reciprocal and two
products add 6 u: (2 |gate| + 8) u, and where the reciprocal leaves binary32's normal numbers
2^-125 |gate up|.  A scale is off as its largest value, and by its division.  A code has to lie between
the codes of the 64-bit quotient times 1 -+ twice that (for value and scale) and a few u."""
import numpy as np
import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
U24 = 2.0 ** -24
HALF_BF16 = torch.finfo(BF16).eps / 2


def setup_module(_):
    need_gpu()


def _gen(*key):
    return torch.Generator(device=DEV).manual_seed(sum(x * 7919 ** i for i, x in enumerate(key)) % 2 ** 31)


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)


def _e4m3(t):
    return t.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float32)


def _check_groups(q, scales, y, off, tiny):
    """Codes and scales of the rows y (binary64), each value off by `off` of itself and by tiny."""
    m, k = y.shape
    g = y.view(m, k // 128, 128)
    off_g, tiny_g = off.view_as(g).amax(2), tiny.view_as(g).amax(2)
    top = g.abs().amax(2)
    want = top.clamp(min=1e-10) / 448
    got = scales.view(m, -1).to(F64)
    assert ((got - want).abs() <= want * (off_g + 2 * U24) + tiny_g / 448).all()
    share = (g / want[..., None])
    slack = share.abs() * (off.view_as(g) + off_g[..., None] + 8 * U24) + (tiny_g / want)[..., None] * 2
    codes = q.view(torch.float8_e4m3fn).to(torch.float32).view_as(g)
    assert torch.isfinite(codes).all()
    assert (codes >= _e4m3(share - slack)).all() and (codes <= _e4m3(share + slack)).all()


def _norm_ref(x, w, eps, residual):
    h = x if residual is None else (x.float() + residual.float()).to(BF16)
    y = h.to(F64)
    y = y / (y.square().mean(1, keepdim=True) + eps).sqrt()
    return h, y if w is None else y * w.to(F64)


def _check_norm(x, w, eps, residual, q, s, total, kept):
    h, y = _norm_ref(x, w, eps, residual)
    if residual is not None:
        assert torch.equal(total, h)
    off = torch.full_like(y, (24 + x.shape[1] / 16384) * U24)
    _check_groups(q, s, y, off, torch.zeros_like(y))
    if kept is not None:
        assert ((kept.to(F64) - y).abs() <= y.abs() * (HALF_BF16 + 2 * off)).all()


WIDTHS = [128, 256, 384, 896, 1024, 1152, 2048, 5120, 16384, 16512, 32768, 32896, 70016]


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_at_every_width(k, residual):
    for m in (1, 7, 16) if k > 4096 else (1, 3, 16, 130):
        g = _gen(m, k, residual)
        x, w = _normal(g, (m, k), 1.5), _normal(g, (k,), 1.0)
        r = _normal(g, (m, k), 4.0) if residual else None
        kept = torch.zeros((m, k), dtype=BF16, device=DEV)
        q, s, total = fq.fp8_rms_norm_group_quant(x, w, residual=r, norm_out=kept)
        assert (total is None) == (r is None)
        _check_norm(x, w, 1e-6, r, q, s, total, kept)


@pytest.mark.parametrize("m", [2000, 5000])
def test_norm_of_many_rows_and_the_same_bits_every_time(m):
    g = _gen(m)
    x, w, r = _normal(g, (m, 640)), _normal(g, (640,)), _normal(g, (m, 640), 3.0)
    first = fq.fp8_rms_norm_group_quant(x, w, residual=r)
    _check_norm(x, w, 1e-6, r, *first, None)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, fq.fp8_rms_norm_group_quant(x, w, residual=r)))


@pytest.mark.parametrize("k", [256, 5120, 40960])
def test_norm_strided_rows_in_place_and_no_weight(k):
    g = _gen(k, 3)
    m = 9
    wide = _normal(g, (m, k + 64), 2.0)
    x, r = wide[:, 16:16 + k], _normal(g, (m, 2 * k))[:, k:]
    out = torch.full((m, k + 8), 5.0, dtype=BF16, device=DEV)
    kept = torch.full((m, k + 24), 6.0, dtype=BF16, device=DEV)
    q, s, total = fq.fp8_rms_norm_group_quant(x, None, eps=1e-3, residual=r, residual_out=out[:, :k],
                                              norm_out=kept[:, 8:8 + k])
    _check_norm(x, None, 1e-3, r, q, s, total, kept[:, 8:8 + k])
    assert (out[:, k:] == 5).all() and (kept[:, :8] == 6).all() and (kept[:, 8 + k:] == 6).all()
    for place in (x, r):  # the sum takes the place of either
        a, b = x.clone(), r.clone()
        to = a if place is x else b
        again = fq.fp8_rms_norm_group_quant(a, None, eps=1e-3, residual=b, residual_out=to)
        assert again[2] is to and all(torch.equal(u, v) for u, v in zip(again, (q, s, total)))
    alone = torch.zeros((1, k + 64), dtype=BF16, device=DEV)[:, :k]  # one row: any stride
    assert not fq.fp8_rms_norm_group_quant(alone, None)[0].any()


def test_norm_of_zeros_and_of_small_and_large_rows():
    g = _gen(5)
    w = _normal(g, (512,))
    x = torch.zeros((6, 512), dtype=BF16, device=DEV)
    x[1] = _normal(g, (512,), 1e-18)
    x[2] = _normal(g, (512,), 1e17)
    x[3, 7] = 300.0
    x[4] = -0.0
    x[5] = _normal(g, (512,), 1e-3)
    q, s, _ = fq.fp8_rms_norm_group_quant(x, w, eps=0.01)
    _check_norm(x, w, 0.01, None, q, s, None, None)
    # one binary32 division, as numpy's (torch multiplies by the reciprocal of a number)
    floor = float(np.float32(1e-10) / np.float32(448))
    assert (s[0] == floor).all() and (q[[0, 4]] & 0x7F == 0).all()  # (0 times a negative weight: -0)
    q, s, _ = fq.fp8_rms_norm_group_quant(x, w, eps=0.0)  # rows of zeros: NaN
    _check_norm(x[1:4], w, 0.0, None, q[1:4], s[1:4], None, None)
    assert (q[0] & 0x7F == 0x7F).all() and (q[4] & 0x7F == 0x7F).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_norm_of_rows_that_are_not_finite(bad):
    """A NaN makes its row NaN; an infinity makes its own value NaN and the others 0.  Other rows
    do not change."""
    g = _gen(6)
    x, w = _normal(g, (5, 5120)), _normal(g, (5120,)).abs() + 0.1
    want = fq.fp8_rms_norm_group_quant(x, w)
    x[2, 1000] = bad
    kept = torch.zeros_like(x)
    q, s, _ = fq.fp8_rms_norm_group_quant(x, w, norm_out=kept)
    rest = [0, 1, 3, 4]
    assert torch.equal(q[rest], want[0][rest]) and torch.equal(s[rest], want[1][rest])
    nan = q[2] & 0x7F == 0x7F
    assert torch.equal(nan, torch.isnan(kept[2].float()))
    assert nan.all() if bad != bad else nan[1000] and int(nan.sum()) == 1 and (q[2][~nan] & 0x7F == 0).all()


def _check_silu(gate, up, q, s, kept):
    a, b = gate.to(F64), up.to(F64)
    y = a * torch.sigmoid(a) * b
    off = (2 * a.abs() + 8) * U24
    tiny = 2.0 ** -125 * (a * b).abs() + 2.0 ** -126
    _check_groups(q, s, y, off, tiny)
    if kept is not None:
        assert ((kept.to(F64) - y).abs() <= y.abs() * (HALF_BF16 + 2 * off) + 2 * tiny).all()


@pytest.mark.parametrize("k", [128, 256, 384, 1024, 1152, 5120, 16384, 17408])
@pytest.mark.parametrize("std", [1.0, 30.0])
def test_silu_at_every_width(k, std):
    for m in (1, 5, 67):
        g = _gen(m, k)
        gate, up = _normal(g, (m, k), std), _normal(g, (m, k), 2.0)
        kept = torch.zeros((m, k), dtype=BF16, device=DEV)
        q, s = fq.fp8_silu_mul_group_quant(gate, up, out=kept)
        _check_silu(gate, up, q, s, kept)
        again = fq.fp8_silu_mul_group_quant(gate, up)
        assert torch.equal(again[0], q) and torch.equal(again[1], s)


def test_silu_of_column_halves_and_strided_outputs():
    g = _gen(8)
    both = _normal(g, (33, 2 * 640 + 16), 2.0)
    gate, up = both[:, :640], both[:, 640:1280]
    out = torch.full((33, 648), 7.0, dtype=BF16, device=DEV)
    q, s = fq.fp8_silu_mul_group_quant(gate, up, out=out[:, :640])
    _check_silu(gate, up, q, s, out[:, :640])
    assert (out[:, 640:] == 7).all()


def test_silu_of_every_gate_value_and_of_what_is_not_finite():
    """All finite bf16 gates up to 2^60; infinities and NaNs as the formula has them."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device=DEV).to(torch.int16).view(BF16)
    gate = torch.where(torch.isfinite(bits.float()) & (bits.abs() < 2.0 ** 60), bits, 1.0).view(-1, 128)
    up = torch.ones_like(gate)
    kept = torch.zeros_like(gate)
    q, s = fq.fp8_silu_mul_group_quant(gate, up, out=kept)
    _check_silu(gate, up, q, s, kept)
    gate = torch.ones((3, 128), dtype=BF16, device=DEV)
    gate[0, 5], gate[1, 6], gate[2, 7] = float("inf"), float("-inf"), float("nan")
    up = torch.ones_like(gate)
    q, s = fq.fp8_silu_mul_group_quant(gate, up)
    nan = q & 0x7F == 0x7F
    assert nan.sum(1).tolist() == [1, 1, 1] and nan[0, 5] and nan[1, 6] and nan[2, 7]
    assert torch.isinf(s[0]).all() and (q[0] & 0x7F == 0).sum() == 127  # finite over infinite
    assert torch.isfinite(s[1:]).all()


def test_no_rows():
    none = torch.zeros((0, 256), dtype=BF16, device=DEV)
    q, s, total = fq.fp8_rms_norm_group_quant(none, None, residual=none)
    assert q.shape == (0, 256) and s.shape == (0, 2) and total.shape == (0, 256)
    assert fq.fp8_silu_mul_group_quant(none, none)[0].shape == (0, 256)


def test_rows_past_two_to_the_32_elements():
    """Offsets that 32 bits do not hold: the last rows of 2^21 + 40 of 2048."""
    m, k = (1 << 21) + 40, 2048
    g = _gen(11)
    x = torch.zeros((m, k), dtype=BF16, device=DEV)
    x[-3:] = _normal(g, (3, k))
    q, s, _ = fq.fp8_rms_norm_group_quant(x, None)
    _check_norm(x[-3:], None, 1e-6, None, q[-3:], s[-3:], None, None)
    assert not q[:100].any() and not q[-60:-3].any()
    gate = x
    q2, s2 = fq.fp8_silu_mul_group_quant(gate, gate, q=q, scales=s)
    _check_silu(x[-3:], x[-3:], q2[-3:], s2[-3:], None)


def test_streams_and_replayed_graphs():
    g = _gen(12)
    x, w, r = _normal(g, (40, 1024)), _normal(g, (1024,)), _normal(g, (40, 1024), 3.0)
    want = [*fq.fp8_rms_norm_group_quant(x, w, residual=r), *fq.fp8_silu_mul_group_quant(x, r)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [*fq.fp8_rms_norm_group_quant(x, w, residual=r, stream=side.cuda_stream),
           *fq.fp8_silu_mul_group_quant(x, r, stream=side.cuda_stream)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*fq.fp8_rms_norm_group_quant(x, w, residual=r), *fq.fp8_silu_mul_group_quant(x, r)]
    for _ in range(3):
        for t in got:
            t.zero_()
        fq.fp8_rms_norm_group_quant(r, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
