"""GPU parity: fp8_attn_chunk against the definition in 64 bits (bounds derived in attn_ref)."""
import math

import pytest
import torch

import fp8_e4m3_quantization_amd as fq
from tests import attn_ref
from tests.gpu_util import DEV, need_gpu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
KS, VS = 0.02, 0.05


def setup_module(_):
    need_gpu()


def _setup(q_lens, lens, hq, hkv, d, bs, seed=0, pad=0, extra=0, cols=0, behind=0, nan_behind=True):
    """Sequences of q_lens new tokens and lens positions; NaN codes in every byte that no query may
    see (other blocks, blocks' padding, stale positions); `behind` rows of q after the last sequence."""
    g = torch.Generator(device=DEV).manual_seed(seed + sum(lens) + 31 * sum(q_lens) + d + bs)
    n = len(lens)
    need = [-(-x // bs) for x in lens]
    blocks = sum(need) + 2
    cs = bs * hkv * d + pad
    pools = []
    for _ in range(2):
        x = torch.full((blocks, cs), 0x7F, dtype=torch.uint8, device=DEV)
        val = (torch.randn((blocks, bs * hkv * d), generator=g, device=DEV) * 60).clamp(-448, 448)
        x[:, :bs * hkv * d] = val.to(torch.float8_e4m3fn).view(torch.uint8)
        x[blocks - 1] = 0x7F
        pools.append(x)
    width = max(need) + extra
    order = torch.randperm(blocks - 1, generator=g, device=DEV).to(torch.int32)  # last block: no one's
    tables = torch.full((n, width + cols), blocks - 1, dtype=torch.int32, device=DEV)
    first = 0
    for s in range(n):
        tables[s, :need[s]] = order[first:first + need[s]]
        first += need[s]
        if nan_behind and lens[s] % bs:
            last = int(tables[s, need[s] - 1])
            for p in pools:
                p[last, lens[s] % bs * hkv * d:] = 0xFF
    cu = torch.tensor([0] + list(q_lens)).cumsum(0).to(torch.int32).to(DEV)
    q = torch.randn((sum(q_lens) + behind, hq * d), generator=g, device=DEV).to(BF16)
    return dict(q=q, kc=pools[0].view(-1), vc=pools[1].view(-1), tables=tables[:, :width], bs=bs, cs=cs,
                hq=hq, hkv=hkv, d=d, cu=cu, lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def _call(s, **kw):
    return fq.fp8_attn_chunk(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], s["hq"],
                             s["hkv"], s["d"], s["bs"], KS, VS, cache_stride=s["cs"], **kw)


def _check(s, out, lse, scale=None, causal=True, some=None):
    """Holds out and lse of every sequence, head and query (or of `some` of the queries) to the
    definition; returns the rows that belong to a sequence."""
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    scale = d ** -0.5 if scale is None else scale
    ks, vs = torch.tensor(KS).item(), torch.tensor(VS).item()
    nb = s["kc"].numel() // s["cs"]
    kp, vp = (x.view(nb, s["cs"])[:, :bs * hkv * d].reshape(nb, bs, hkv, d) for x in (s["kc"], s["vc"]))
    cu = [min(max(x, 0), s["q"].shape[0]) for x in s["cu"].tolist()]
    covered = torch.zeros(s["q"].shape[0], dtype=torch.bool)
    q3, o3 = s["q"].view(-1, hq, d), out.view(-1, hq, d)
    for b, n in enumerate(s["lens"].tolist()):
        at, to = cu[b], max(cu[b], cu[b + 1])
        covered[at:to] = True
        if at == to:
            continue
        n = max(0, min(n, s["tables"].shape[1] * bs))
        lq = to - at
        pick = torch.arange(lq, device=DEV) if some is None else \
            torch.tensor([i for i in some if i < lq], device=DEV)
        pos = torch.arange(n, device=DEV)
        ids = s["tables"][b].long()[pos // bs]
        good = (ids >= 0) & (ids < nb)
        seen = attn_ref.causal_mask(lq, n, DEV)[pick] if causal else \
            torch.ones((len(pick), n), dtype=torch.bool, device=DEV)
        seen = seen[:, good]
        ids, off = ids[good], (pos % bs)[good]
        for h in range(hq):
            o, l = o3[at:to][pick, h], lse[at:to][pick, h]
            if ids.numel() == 0:
                assert not o.any() and (l == -math.inf).all()
                continue
            k, v = (attn_ref.e4m3_values(p[ids, off, h // (hq // hkv)]) for p in (kp, vp))
            want, wl, bound, lb = attn_ref.attend(q3[at:to][pick, h], k, v, scale * ks, seen)
            attn_ref.check(o, want * vs, bound * vs + want.abs() * vs * 4 * attn_ref.U24,
                           f"sequence {b} head {h} out")
            attn_ref.check(l, wl, lb, f"sequence {b} head {h} lse")
    return covered


def _run(q_lens, lens, hq, hkv, d, bs, causal=True, some=None, **kw):
    s = _setup(q_lens, lens, hq, hkv, d, bs, **kw)
    lse = torch.full((s["q"].shape[0], hq), 3.0, device=DEV)
    out = _call(s, lse=lse, causal=causal)
    _check(s, out, lse, causal=causal, some=some)
    return s, out, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bs", [1, 7, 16, 48, 128, 200])
def test_lengths_around_every_edge(d, bs):
    """Histories and chunks of one token to a few tiles, whole prompts among them, empty ones too."""
    _run([1, 1, 2, 3, 16, 1, 31, 33, 5, 0, 64, 65, 130, 40], [1, 2, 2, 15, 16, 31, 31, 33, 129, 50, 127, 128,
         130, 300], 4, 2, d, bs)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (8, 8), (10, 1), (16, 1), (17, 1), (40, 4), (36, 1),
                                    (64, 2), (12, 12), (24, 3), (16, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_head_groups(hq, hkv, d):
    """Tiles whose rows end inside a query's heads, heads that do not divide the 8 XCDs."""
    _run([3, 14, 1, 20], [5, 200, 64, 20], hq, hkv, d, 16)


@pytest.mark.parametrize("q_len", [1, 3, 4, 7, 8, 9, 13, 16, 17, 32, 33])
def test_rows_around_every_tile_form(q_len):
    """Rows of a tile from 4 to 132: one, two or four waves of rows."""
    _run([q_len, q_len], [700, q_len], 8, 2, 128, 16)


@pytest.mark.parametrize("q_lens,lens", [([4], [20000]), ([5, 3, 2, 1], [9000, 3, 2, 777]), ([2] * 7, [4096] * 7),
                                         ([300], [5000]), ([1, 250, 1], [6000, 3500, 1])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_histories_split_over_workgroups(q_lens, lens, d):
    s, out, lse = _run(q_lens, lens, 8, 2, d, 16, some=[0, 1, 2, 3, 4, 100, 249, 299])
    need = fq.fp8_attn_chunk_workspace_size(len(lens), sum(q_lens), 8, 2, d)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)  # any content will do
    for _ in range(3):  # the same bits every time
        again = _call(s, workspace=ws[:need])
        assert torch.equal(again, out) and (ws[need:] == 0xFF).all()


def test_whole_prompts_and_a_step_agree_with_the_other_kernels():
    """A prompt whose keys all lie in the cache is attn_prefill of the dequantized rows; one token a
    sequence is fp8_attn_decode: the same definition, so both within the sum of the bounds."""
    s, out, lse = _run([300, 41], [300, 41], 8, 2, 128, 16)
    t = s["q"].shape[0]
    slots = torch.cat([s["tables"][b].long()[torch.arange(n, device=DEV) // 16] * 16
                       + torch.arange(n, device=DEV) % 16 for b, n in enumerate([300, 41])])
    k, v = fq.fp8_kv_read(s["kc"], s["vc"], slots, 2, 128, 16, 1.0, 1.0)
    other = fq.attn_prefill(s["q"], k, v, s["cu"], 8, 2, 128, softmax_scale=128 ** -0.5 * KS)
    other = (other.float() * VS)
    assert ((other - out.float()).abs() <= 2.0 ** -6 * out.float().abs() + 0.02).all() and t == 341
    s, out, lse = _run([1, 1, 1], [777, 5, 1024], 8, 2, 128, 16)
    step = fq.fp8_attn_decode(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], 8, 2, 128, 16, KS, VS)
    assert ((step.float() - out.float()).abs() <= 2.0 ** -6 * out.float().abs() + 0.02).all()


@pytest.mark.parametrize("extra", [0, 1, 40])
@pytest.mark.parametrize("q_lens,lens", [([1], [256]), ([37], [255]), ([5, 1, 2], [256, 17, 250]), ([200], [256])])
def test_short_tables_and_wide_ones(q_lens, lens, extra):
    """Tables with room for 256 positions, one block more, and many: one kernel or two."""
    _run(q_lens, lens, 8, 2, 128, 16, extra=extra)


def test_chunks_without_a_causal_mask():
    _run([5, 40, 1, 200], [300, 40, 7, 250], 8, 2, 128, 16, causal=False)


@pytest.mark.parametrize("seqs", [63, 64, 65, 130, 256, 257, 300])
def test_many_sequences(seqs):
    q_lens = [(i * 7) % 4 for i in range(seqs)]
    _run(q_lens, [max(q, (i * 53) % 190) for i, q in enumerate(q_lens)], 4, 2, 64, 16)


@pytest.mark.parametrize("seqs", [100, 260])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (6, 6), (3, 3)])
@pytest.mark.parametrize("rows", [[129], [32, 33], [65, 1], [128, 129, 64, 257]])
def test_many_sequences_whose_tiles_are_barely_begun(seqs, hq, hkv, rows):
    """As many pieces as rows of such numbers can make: each finds a workgroup."""
    q_lens = [rows[i % len(rows)] for i in range(seqs)]
    s = _setup(q_lens, [q + i % 3 for i, q in enumerate(q_lens)], hq, hkv, 64, 16)
    out = torch.full_like(s["q"], math.nan)
    lse = torch.full((sum(q_lens), hq), math.nan, device=DEV)
    _call(s, out=out, lse=lse)
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()
    some = [s["cu"][i].item() for i in (0, 1, seqs - 1)]
    for i, at in zip((0, 1, seqs - 1), some):
        one = dict(s, q=s["q"][at:at + q_lens[i]].contiguous(), tables=s["tables"][i:i + 1].contiguous(),
                   lens=s["lens"][i:i + 1], cu=torch.tensor([0, q_lens[i]], dtype=torch.int32, device=DEV))
        _check(one, out[at:at + q_lens[i]], lse[at:at + q_lens[i]])


def test_a_serving_batch():
    """One chunk beside single steps and a whole prompt, wide tables, strides, rows behind the last."""
    q_lens, lens = [1] * 12 + [200, 1, 90], [40 + 300 * i for i in range(12)] + [1900, 5, 90]
    s = _setup(q_lens, lens, 8, 2, 128, 16, pad=256, extra=5, cols=3, behind=6)
    n, e = s["q"].shape[0], 8 * 128
    wide = torch.full((n, e + 64), 9.0, dtype=BF16, device=DEV)
    lse = torch.full((n, 8), 3.0, device=DEV)
    _call(s, out=wide[:, :e], lse=lse)
    covered = _check(s, wide[:, :e].contiguous(), lse, some=[0, 1, 88, 89, 127, 128, 199])
    assert (wide[:, e:] == 9).all() and (wide[-6:] == 9).all() and (lse[-6:] == 3).all()
    assert covered.tolist() == [True] * (n - 6) + [False] * 6
    s["q"] = torch.cat([s["q"], s["q"]], 1)[:, :e]
    assert torch.equal(_call(s)[:-6], wide[:-6, :e]) and not _call(s)[-6:].any()


def test_lengths_starts_and_blocks_out_of_range():
    """Lengths are clamped to the table and starts to the rows; positions in blocks that do not exist
    do not count; queries before the history's start see nothing."""
    s = _setup([10, 10, 10, 10, 10], [64, 64, 64, 64, 64], 4, 2, 128, 16, nan_behind=False)
    s["lens"] = torch.tensor([-3, 64, 1 << 30, 64, 7], dtype=torch.int32, device=DEV)
    s["tables"] = s["tables"].clone()
    s["tables"][1, 1] = -1
    s["tables"][1, 3] = 1 << 30
    s["tables"][3] = s["kc"].numel() // s["cs"]
    lse = torch.zeros((50, 4), device=DEV)
    out = _call(s, lse=lse)
    _check(s, out, lse)
    assert not out[:10].any() and not out[30:40].any() and not out[40:43].any() and out[43:].any()
    for causal in (True, False):
        out = _call(s, lse=lse, causal=causal)
        _check(s, out, lse, causal=causal)
    s["cu"] = torch.tensor([-5, 10, 20, 1000, 30, 70], dtype=torch.int32, device=DEV)
    out = _call(s, lse=lse)  # the third sequence takes rows 20 to 49, the fourth none, the last 30 to 49
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("q_lens,lens", [([20], [140]), ([150], [150]), ([3], [2000]), ([140], [4000])])
def test_nan_codes_reach_the_queries_that_see_them(q_lens, lens):
    """A NaN code of a value reaches that value of the queries that see its position, however small its
    weight; one of a key all values of them; in tiles seen whole, in part, and in parts of a history."""
    for back in (1, 5, q_lens[0], lens[0] - 1, lens[0]):
        pos = lens[0] - back
        if pos < 0:
            continue
        s = _setup(q_lens, lens, 4, 2, 128, 16)
        clean = _call(s)
        at = int(s["tables"][0, pos // 16]) * s["cs"] + pos % 16 * 256
        sees = torch.arange(q_lens[0], device=DEV) + lens[0] - q_lens[0] >= pos
        s["vc"][at + 128 + 77] = 0xFF  # KV head 1, value 77
        out = _call(s)
        want = torch.zeros((q_lens[0], 4, 128), dtype=torch.bool, device=DEV)
        want[sees, 2:, 77] = True
        assert torch.equal(torch.isnan(out.float()), want.flatten(1)), (back, "value")
        assert torch.equal(out[~want.flatten(1)], clean[~want.flatten(1)])
        s["q"] = s["q"] * 40  # weights of 0 in binary32
        assert torch.equal(torch.isnan(_call(s).float()), want.flatten(1)), (back, "small weights")
        s["kc"][at + 128 + 3] = 0x7F
        want[sees, 2:] = True
        lse = torch.zeros((q_lens[0], 4), device=DEV)
        assert torch.equal(torch.isnan(_call(s, lse=lse).float()), want.flatten(1)), (back, "key")
        assert torch.equal(torch.isnan(lse), want[:, :, 0])


def test_nan_codes_beside_blocks_that_do_not_exist():
    s = _setup([30], [300], 4, 2, 128, 16)
    s["tables"] = s["tables"].clone()
    at = int(s["tables"][0, 2]) * s["cs"]
    s["vc"][at + 9] = 0x7F
    s["tables"][0, 3] = -7
    out = _call(s).view(30, 4, 128)
    assert torch.isnan(out[:, :2, 9].float()).all() and int(torch.isnan(out.float()).sum()) == 60


def test_empty_table_and_no_queries():
    s = _setup([2, 3], [2, 3], 4, 2, 128, 16)
    s["tables"] = torch.zeros((2, 0), dtype=torch.int32, device=DEV)
    lse = torch.zeros((5, 4), device=DEV)
    assert not _call(s, lse=lse).any() and (lse == -math.inf).all()
    s["cu"] = torch.zeros(3, dtype=torch.int32, device=DEV)
    out = torch.full_like(s["q"], 4.0)
    assert (_call(s, out=out) == 4).all()
    none = torch.zeros((0, 512), dtype=BF16, device=DEV)
    assert fq.fp8_attn_chunk(none, s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], 4, 2, 128, 16, 1.0,
                             1.0).shape == (0, 512)


@pytest.mark.parametrize("scale", [1e-4, 0.5])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales(scale, d):
    s = _setup([40, 9], [130, 9], 4, 1, d, 16)
    lse = torch.zeros((49, 4), device=DEV)
    _check(s, _call(s, lse=lse, softmax_scale=scale), lse, scale)


@pytest.mark.parametrize("unit", [2.0 ** 10, 2.0 ** 40, 2.0 ** 64])  # k_scale's largest
@pytest.mark.parametrize("q_lens,lens", [([3, 70], [3000, 70]), ([50, 1], [300, 1])])
def test_huge_scores_pick_the_largest(q_lens, lens, unit):
    """Scores that are exact multiples of `unit` in binary32: out is the mean of V over the ties.  Scores
    of ties are equal, so that a fused product leaves each the same weight, 1 + e with a rounding to
    bf16 that numerator and denominator share: out is off by its own rounding and the sums' (n + 8)
    steps; lse by its rounding, 5 steps as in the other kernels' tests."""
    s = _setup(q_lens, lens, 4, 2, 64, 16)
    codes = torch.randint(-2, 3, s["kc"].shape, device=DEV).float().to(torch.float8_e4m3fn)
    s["kc"] = codes.view(torch.uint8)
    s["q"] = torch.randint(-2, 3, s["q"].shape, device=DEV).to(BF16)
    lse = torch.zeros((sum(q_lens), 4), device=DEV)
    out = fq.fp8_attn_chunk(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], 4, 2, 64, 16, unit,
                            0.5, softmax_scale=1.0, lse=lse)
    kp, vp = (attn_ref.e4m3_values(s[x]).view(-1, 16, 2, 64) for x in ("kc", "vc"))
    first = 0
    for i, (lq, n) in enumerate(zip(q_lens, lens)):
        pos = torch.arange(n, device=DEV)
        ids = s["tables"][i].long()[pos // 16]
        seen = attn_ref.causal_mask(lq, n, DEV)
        for h in range(4):
            k, v = kp[ids, pos % 16, h // 2], 0.5 * vp[ids, pos % 16, h // 2]
            q = s["q"][first:first + lq].double().view(lq, 4, 64)[:, h]
            score = torch.where(seen, unit * (q @ k.t()), -math.inf)
            top = score.amax(1, keepdim=True)
            best = (score == top).double()
            w = best / best.sum(1, keepdim=True)
            want = w @ v
            bound = attn_ref.HALF_BF16 * want.abs() + (n + 8) * attn_ref.U24 * (w @ v.abs()) + 1e-30
            attn_ref.check(out[first:first + lq].view(lq, 4, 64)[:, h], want, bound, "out")
            want = top[:, 0] + torch.log(best.sum(1))
            attn_ref.check(lse[first:first + lq, h], want, 5 * attn_ref.U24 * want.abs() + 2.0 ** -20, "lse")
        first += lq


@pytest.mark.parametrize("q_lens,lens", [([30], [1000]), ([200], [300])])
def test_one_weight_above_all_others(q_lens, lens):
    """One position outweighs one other by 2^x, 0.5 <= x < 8, behind it in the same wave.  The weight's
    rounding to bf16, by a factor 1 + e with |e| <= 2^-8, is in numerator and denominator: with w the true
    share and V = 0 at the other position, out = V w (1 + e) / (1 + w e) is off by at most
    V w (1 - w) 2^-8 (1 + 2^-7), and by its own rounding and a few binary32 steps."""
    lq, n, d, bs, at = q_lens[0], lens[0], 64, 4, 72
    nb = n // bs
    kc = torch.full((nb, bs, d), -448.0, device=DEV)
    vc = torch.zeros((nb, bs, d), device=DEV)
    kc[0, 0] = 0.0
    kc[at // bs, 0] = 1.0
    vc[at // bs, 0] = torch.arange(1, d + 1, device=DEV) * 4.0
    kc, vc = (x.to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1) for x in (kc, vc))
    c = (torch.linspace(0.5, 7.9, lq, device=DEV) * math.log(2) / d).to(BF16)
    q = c[:, None].expand(lq, d).contiguous()
    tables = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    cu = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
    out = fq.fp8_attn_chunk(q, kc, vc, tables, torch.tensor([n], dtype=torch.int32, device=DEV), cu, 1, 1, d,
                            bs, 1.0, 1.0, softmax_scale=1.0)
    sees = torch.arange(lq, device=DEV) + n - lq >= at
    w = torch.where(sees, torch.sigmoid(c.double() * d), 0.0)[:, None]
    v = attn_ref.e4m3_values(vc).view(-1, d)[at]
    bound = attn_ref.HALF_BF16 * w * v + 2.0 ** -8 * (1 + 2.0 ** -7) * w * (1 - w) * v + 2.0 ** -18 * v
    attn_ref.check(out, w * v, bound, "out")


def test_cache_past_four_gib():
    """Blocks whose byte offsets pass 2^32."""
    bs, hkv, d = 16, 4, 128
    cs = bs * hkv * d
    blocks = (1 << 32) // cs + 40
    kc = torch.empty(blocks * cs, dtype=torch.uint8, device=DEV)
    vc = torch.empty_like(kc)
    g = torch.Generator(device=DEV).manual_seed(5)
    n = 50
    table = torch.arange(blocks - 4, blocks, device=DEV, dtype=torch.int32)[None].contiguous()
    for p in (kc, vc):
        x = (torch.randn(4 * cs, generator=g, device=DEV) * 50).clamp(-448, 448)
        p[-4 * cs:] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    s = dict(q=torch.randn((20, 8 * d), generator=g, device=DEV).to(BF16), kc=kc, vc=vc, tables=table,
             lens=torch.tensor([n], dtype=torch.int32, device=DEV), hq=8, hkv=hkv, d=d, bs=bs, cs=cs,
             cu=torch.tensor([0, 20], dtype=torch.int32, device=DEV))
    lse = torch.zeros((20, 8), device=DEV)
    out = _call(s, lse=lse)
    small = dict(s, kc=kc[-4 * cs:].clone(), vc=vc[-4 * cs:].clone(), tables=table - (blocks - 4))
    _check(small, out, lse)


def test_another_stream_and_two_replayed_graphs():
    """Two graphs captured one after the other, replayed on two streams at once: each has its own
    workspace; eager calls of other shapes go on between the replays."""
    a = _setup([5, 3], [5000, 300], 8, 2, 128, 16)
    b = _setup([6, 2], [7000, 64], 8, 2, 128, 16, seed=9)
    want = [_call(a), _call(b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _call(a, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want[0])
    outs, graphs = [], []
    for s in (a, b):
        out = torch.zeros_like(want[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _call(s, out=out)
        outs.append(out)
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for o in outs:
            o.zero_()
        _run([3, 1], [(rep * 997) % 3000 + 3, 40], 4, 1, 128, 16)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_graph_replayed_over_growing_histories():
    """Lengths, starts and tables are read at replay: the same graph serves step after step, whether its
    histories are cut or not, and as many new tokens as the rows hold."""
    s = _setup([2, 2, 60], [6000, 40, 900], 8, 2, 128, 16, extra=8, nan_behind=False)
    for p in ("kc", "vc"):
        s[p] = (s[p] & 0x77).contiguous()  # no NaN codes: stale positions become real ones
    s["tables"] = s["tables"].contiguous()
    tables, lens, cu = s["tables"].clone(), s["lens"].clone(), s["cu"].clone()
    out, lse = torch.zeros_like(s["q"]), torch.zeros((64, 8), device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(s, out=out, lse=lse)
    for step, starts in enumerate([[0, 2, 4, 64], [0, 1, 2, 3], [0, 0, 64, 64], [0, 2, 4, 64], [0, 0, 0, 0]]):
        s["cu"].copy_(torch.tensor(starts))
        s["lens"].copy_(torch.tensor([6000 - 2500 * step, 64 + step, 100 + 200 * step]).clamp(min=0))
        s["tables"].copy_(tables.flip(0) if step == 3 else tables)
        if step == 3:  # (the first row's blocks for the last sequence: the same ones, another order)
            s["lens"].copy_(torch.tensor([0, 64, 6000]))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        eager, elog = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        _call(s, out=eager, lse=elog)
        assert torch.equal(out, eager) and torch.equal(lse, elog), step
        covered = _check(s, out, lse, some=[0, 1, 31, 32, 59, 63])
        assert (out[~covered] == 7).all() and (lse[~covered] == 7).all()
    s["lens"].copy_(lens)
    s["cu"].copy_(cu)
    s["tables"].copy_(tables)
    graph.replay()
    _check(s, out, lse, some=[0, 1, 59])


@pytest.mark.parametrize("q_lens,lens", [([3, 4, 1, 70], [600, 640, 33, 700]), ([200, 2], [900, 901])])
def test_blocks_shared_by_sequences_and_named_twice(q_lens, lens):
    """A prefix that several sequences share, and one block that a table names again."""
    s = _setup(q_lens, lens, 8, 2, 128, 16, nan_behind=False)
    for p in ("kc", "vc"):
        s[p] = (s[p] & 0x77).contiguous()
    s["tables"] = s["tables"].clone()
    s["tables"][1:, :2] = s["tables"][0, :2]
    s["tables"][0, 5] = s["tables"][0, 4]
    s["tables"][0, 6] = s["tables"][0, 0]
    lse = torch.zeros((sum(q_lens), 8), device=DEV)
    _check(s, _call(s, lse=lse), lse, some=[0, 1, 2, 3, 69, 127, 128, 199])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("q_lens,lens", [([3], [2000]), ([40], [300]), ([100], [2000])])
def test_a_query_that_is_not_finite_stays_alone(q_lens, lens, bad):
    for d, hq, hkv in ((64, 8, 2), (128, 8, 8), (256, 4, 1)):
        s = _setup(q_lens, lens, hq, hkv, d, 16)
        clean = _call(s).view(-1, hq, d)
        s["q"].view(-1, hq, d)[q_lens[0] // 2, hq - 1, 5] = bad
        out = _call(s).view(-1, hq, d)
        hit = torch.zeros((q_lens[0], hq), dtype=torch.bool, device=DEV)
        hit[q_lens[0] // 2, hq - 1] = True
        assert torch.equal(out[~hit], clean[~hit])
        if math.isnan(bad):
            assert torch.isnan(out[hit].float()).all()


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 8), (128, 16, 4), (256, 4, 4), (256, 8, 2), (128, 200, 1)])
@pytest.mark.parametrize("q_lens,lens", [([3], [700]), ([7, 30], [2000, 90])])
def test_nan_codes_of_heads_that_share_a_piece(d, hq, hkv, q_lens, lens):
    s = _setup(q_lens, lens, hq, hkv, d, 16)
    clean = _call(s).view(-1, hq, d)
    pos, head, value = lens[0] - 2, hkv - 1, d - 3
    s["vc"][int(s["tables"][0, pos // 16]) * s["cs"] + (pos % 16 * hkv + head) * d + value] = 0x7F
    out = _call(s).view(-1, hq, d)
    want = torch.zeros((sum(q_lens), hq, d), dtype=torch.bool, device=DEV)
    want[q_lens[0] - 2:q_lens[0], head * (hq // hkv):, value] = True
    assert torch.equal(torch.isnan(out.float()), want) and torch.equal(out[~want], clean[~want])


def test_more_query_heads_than_a_tile_holds():
    _run([1, 3, 9], [300, 3, 1000], 200, 1, 128, 16, some=[0, 2, 8])
