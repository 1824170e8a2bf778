"""GPU: the ends of what fp8_rms_norm_group_quant, fp8_silu_mul_group_quant and fp8_attn_chunk accept."""
import math

import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests import attn_ref
from tests.gpu_util import DEV, need_gpu
from tests.test_gpu_attn_chunk import _setup

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


@pytest.mark.parametrize("k_scale,scale", [(2.0 ** -64, 2.0 ** -149), (2.0 ** -64, 2.0 ** -100), (2.0 ** -64, 1e-30),
                                           (2.0 ** -64, 2.0 ** -86), (2.0 ** -64, 2.0 ** -70), (1.0, 2.0 ** -149)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 4, 4), (256, 4, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_of_the_smallest_scales(k_scale, scale, d, hq, hkv, causal):
    """Scores next to 0, be their scale's product below binary32's smallest number: out is the mean of V over the
    positions that a query sees, off by its own rounding and the sums' (n + 8) steps; lse the logarithm of their
    number.  With queries of 2^98 the scores reach 2^112 before a scale of at most 2^-134: weights off by
    2^-21 at most."""
    q_lens, lens = [1, 3, 40, 130, 5], [1, 700, 40, 300, 5000]
    s = _setup(q_lens, lens, hq, hkv, d, 16)
    s["tables"] = s["tables"].clone()
    s["tables"][3, 4] = -1
    nb = s["kc"].numel() // s["cs"]
    vp = s["vc"].view(nb, 16, hkv, d)
    for q in (s["q"], (s["q"].float() * 2.0 ** 96).to(BF16)):
        lse = torch.zeros((sum(q_lens), hq), device=DEV)
        out = fq.fp8_attn_chunk(q, s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], hq, hkv, d, 16, k_scale, 0.5,
                                softmax_scale=scale, causal=causal, lse=lse)
        first = 0
        for i, (lq, n) in enumerate(zip(q_lens, lens)):
            pos = torch.arange(n, device=DEV)
            ids = s["tables"][i].long()[pos // 16]
            good = ids >= 0
            seen = attn_ref.causal_mask(lq, n, DEV) if causal else torch.ones((lq, n), dtype=torch.bool, device=DEV)
            w = seen[:, good].to(F64)
            w /= w.sum(1, keepdim=True)
            for h in range(hq):
                v = 0.5 * attn_ref.e4m3_values(vp[ids[good], (pos % 16)[good], h // (hq // hkv)])
                bound = attn_ref.HALF_BF16 * (w @ v).abs() + ((n + 8) * U24 + 2.0 ** -20) * (w @ v.abs())
                attn_ref.check(out[first:first + lq].view(lq, hq, d)[:, h], w @ v, bound, f"sequence {i} out")
            want = torch.log(seen[:, good].sum(1).to(F64))[:, None].expand(lq, hq)
            attn_ref.check(lse[first:first + lq], want, 5 * U24 * want.abs() + 2.0 ** -20, f"sequence {i} lse")
            first += lq


@pytest.mark.parametrize("k", [512, 5120, 16384, 40960])
@pytest.mark.parametrize("place", ["new", "x", "residual"])
def test_norm_of_sums_that_are_not_finite(k, place):
    """A NaN or an infinity from x, from the residual, of both or of their sum's rounding to bf16: the sum is kept as
    torch has it; a NaN makes its row NaN codes, an infinity its own value NaN and the row's others 0."""
    g = torch.Generator(device=DEV).manual_seed(k)
    x, r = (torch.randn((9, k), generator=g, device=DEV).to(BF16) for _ in range(2))
    w = (torch.rand(k, generator=g, device=DEV) + 0.5).to(BF16)
    big = torch.finfo(BF16).max
    at = k - 7
    for row, (a, b) in enumerate([(math.nan, 1.0), (1.0, math.nan), (math.inf, 1.0), (1.0, -math.inf),
                                  (math.inf, -math.inf), (big, 2.0 ** 119), (-big, -big), (math.inf, math.nan)]):
        x[row, at], r[row, at] = a, b
    want = (x.float() + r.float()).to(BF16)
    assert torch.isnan(want[[0, 1, 4, 7], at]).all() and torch.isinf(want[[2, 3, 5, 6], at]).all()
    clean = fq.fp8_rms_norm_group_quant(x[8:], w, residual=r[8:])
    to = {"new": None, "x": x, "residual": r}[place]
    kept = torch.zeros_like(x)
    q, s, total = fq.fp8_rms_norm_group_quant(x, w, residual=r, residual_out=to, norm_out=kept)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(total), nan) and torch.equal(total[~nan], want[~nan])
    codes = q & 0x7F
    assert (codes[[0, 1, 4, 7]] == 0x7F).all()
    for row in (2, 3, 5, 6):
        assert codes[row, at] == 0x7F and int((codes[row] != 0).sum()) == 1, row
    assert torch.equal(torch.isnan(kept), codes == 0x7F)
    assert torch.equal(q[8:], clean[0]) and torch.equal(s[8:], clean[1])


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 8, 2), (256, 4, 2)])
@pytest.mark.parametrize("q_lens,lens", [([2], [150]), ([14], [150]), ([70], [150]), ([3, 30], [2000, 130])])
@pytest.mark.parametrize("gone", [False, True])
def test_a_nan_code_at_every_position_of_the_last_tiles(d, hq, hkv, q_lens, lens, gone):
    """One NaN code of a value at a time, at each of the last positions and behind the end: it reaches that value of the
    rows that see it and nothing else, also where a block does not exist (and the NaN codes of the pool's
    first block, read in its place, do not count)."""
    s = _setup(q_lens, lens, hq, hkv, d, 16)
    for p in ("kc", "vc"):
        s[p] = torch.where(s[p] & 0x7F == 0x7F, 0x31, s[p]).contiguous()
    if gone:
        s["tables"] = s["tables"].clone()
        used = s["tables"][0, 1].item()
        s["tables"][0, 1] = -1
        s["vc"][used * s["cs"]:(used + 1) * s["cs"]] = 0x7F
        blocks = [x for b, n in enumerate(lens) for x in s["tables"][b, :-(-n // 16)].tolist()]
        if 0 not in blocks:
            s["vc"][:s["cs"]] = 0xFF
    args = (s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], hq, hkv, d, 16, 0.02, 0.05)
    clean = fq.fp8_attn_chunk(*args).view(-1, hq, d)
    assert torch.isfinite(clean.float()).all()
    n, lq = lens[0], q_lens[0]
    for pos in range(n - 72, -(-n // 16) * 16):
        head, value = pos % hkv, (pos * 7) % d
        at = int(s["tables"][0, pos // 16]) * s["cs"] + (pos % 16 * hkv + head) * d + value
        old = int(s["vc"][at])
        s["vc"][at] = 0x7F
        want = torch.zeros(clean.shape, dtype=torch.bool, device=DEV)
        sees = torch.arange(lq, device=DEV) + n - lq >= pos
        want[:lq, head * (hq // hkv):(head + 1) * (hq // hkv), value] = (sees & (pos < n))[:, None]
        out = fq.fp8_attn_chunk(*args).view(-1, hq, d)
        s["vc"][at] = old
        assert torch.equal(torch.isnan(out.float()), want), pos
        assert torch.equal(out[~want], clean[~want]), pos


def test_time_does_not_go_by_codes_that_no_query_sees():
    """Steps behind a block that does not exist: NaN codes behind the sequences' ends, seen by no one, change nothing
    (a walk over all positions in search of them took 15 times as long; up to twice is taken for noise)."""
    lens = [500 + (i * 2339) % 7600 for i in range(64)]
    s = _setup([1] * 64, lens, 32, 8, 128, 32, nan_behind=False)
    s["tables"] = s["tables"].clone()
    s["tables"][:, 0] = -1
    s["vc"] = (s["vc"] & 0x77).contiguous()
    out, took = [], []
    for stale in (False, True):
        for b, n in enumerate(lens):
            if stale and n % 32:
                at = int(s["tables"][b, n // 32]) * s["cs"]
                s["vc"][at + n % 32 * 8 * 128:at + s["cs"]] = 0x7F
        best = math.inf
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                o = fq.fp8_attn_chunk(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], 32, 8, 128, 32, 0.02, 0.05)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        out.append(o)
        took.append(best)
    assert torch.equal(*out)
    assert took[1] < 2 * took[0], took
