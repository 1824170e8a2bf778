"""GPU parity: attn_prefill against the definition in 64 bits (bounds derived in attn_ref)."""
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


def _starts(lens, base=0):
    out = [base]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _run(q_lens, k_lens, hq, hkv, d, causal=True, scale=None, seed=0, pad=0, tail=0, spread=2.0):
    """Calls the operator on random data with `pad` extra columns and `tail` rows behind the last
    sequence (keys and values there are NaN), and holds it to the definition."""
    g = torch.Generator(device=DEV).manual_seed(seed + sum(q_lens) + d)
    cu_q, cu_k = _starts(q_lens), _starts(k_lens)
    tq, tk = cu_q[-1] + tail, cu_k[-1] + tail

    def rows(n, heads, std):
        x = (torch.randn((n, heads * d + pad), generator=g, device=DEV) * std).to(BF16)
        return x[:, :heads * d]

    q, k, v = rows(tq, hq, spread), rows(tk, hkv, 1.0), rows(tk, hkv, 3.0)
    k[cu_k[-1]:] = math.nan
    v[cu_k[-1]:] = math.nan
    out = torch.full((tq, hq * d + pad), 11.0, dtype=BF16, device=DEV)
    lse = torch.full((tq, hq), 13.0, device=DEV)
    a = torch.tensor(cu_q, dtype=torch.int32, device=DEV)
    b = torch.tensor(cu_k, dtype=torch.int32, device=DEV)
    fq.attn_prefill(q, k, v, a, hq, hkv, d, cu_seqlens_k=b, softmax_scale=scale, causal=causal,
                    out=out[:, :hq * d], lse=lse)
    scale = d ** -0.5 if scale is None else scale
    covered = attn_ref.prefill(q, k, v, cu_q, cu_k, hq, hkv, d, scale, causal, out[:, :hq * d], lse)
    assert (out[:, hq * d:] == 11).all()
    assert (out[~covered] == 11).all() and (lse[~covered] == 13).all()
    return q, k, v, a, b, out[:, :hq * d], lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_one_sequence_of_every_tile_edge(n, d):
    _run([n], [n], 4, 2, d, tail=3)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (8, 8), (16, 2), (40, 4), (5, 5)])
def test_head_groups(hq, hkv):
    _run([70, 5], [70, 5], hq, hkv, 128)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_sequences_with_histories_and_empty_ones(d, causal):
    """Queries behind histories, sequences without queries, without keys, and with fewer keys than
    queries (whose first queries see nothing)."""
    _run([40, 0, 1, 130, 7, 0, 64, 9], [40, 5, 300, 513, 0, 0, 50, 9], 4, 2, d, causal=causal, tail=70)


@pytest.mark.parametrize("lq,lk", [(1, 1000), (128, 2000), (100, 99), (300, 10), (65, 4096)])
def test_chunks(lq, lk):
    _run([lq], [lk], 4, 1, 128)
    _run([lq], [lk], 2, 2, 64, causal=False)


@pytest.mark.parametrize("q_lens,k_lens,hq,hkv,d", [
    ([1], [9000], 4, 1, 128), ([130], [5000], 10, 2, 64), ([40], [3000], 2, 1, 256),
    ([20, 0, 200, 5], [6000, 4000, 30, 7000], 4, 2, 128), ([3000], [3000], 1, 1, 128),
    ([300], [20000], 8, 8, 64)])
def test_few_queries_over_long_keys_are_split(q_lens, k_lens, hq, hkv, d):
    """Keys split over workgroups (with sequences too short to split among them): the same bits in
    any workspace, and what lies behind the sequences does not reach them."""
    need = fq.attn_prefill_workspace_size(len(q_lens), sum(q_lens) + 9, sum(k_lens) + 9, hq, hkv, d)
    assert need > 0
    q, k, v, a, b, out, lse = _run(q_lens, k_lens, hq, hkv, d, tail=9)
    n = sum(q_lens)
    for fill in (0, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        got = fq.attn_prefill(q, k, v, a, hq, hkv, d, cu_seqlens_k=b, workspace=ws)
        assert torch.equal(got[:n], out[:n])
    _run(q_lens, k_lens, hq, hkv, d, causal=False, seed=5)


@pytest.mark.parametrize("seqs", [64, 65, 256, 257, 700])
def test_many_sequences(seqs):
    """More sequences than a wave has lanes, and than the ordered search takes."""
    lens = [(i * 37) % 9 + (150 if i % 97 == 3 else 0) for i in range(seqs)]
    _run(lens, [n + i % 3 for i, n in enumerate(lens)], 2, 1, 64)


def test_long_prompt():
    _run([2500], [2500], 8, 1, 128, spread=1.0)


@pytest.mark.parametrize("pad", [8, 128])
def test_strided_rows(pad):
    _run([77, 130], [77, 200], 4, 2, 128, pad=pad, tail=5)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 2.0 ** -40])
def test_scales(scale):
    _run([100], [100], 2, 1, 128, scale=scale, spread=1.0)


def test_large_scores_move_the_reference():
    """Scores of hundreds, growing along the keys: the running reference moves many times."""
    d, n = 128, 300
    q = torch.ones((n, d), device=DEV).to(BF16)
    k = (torch.arange(n, device=DEV)[:, None] * 0.25 - 30).expand(n, d).to(BF16).contiguous()
    v = torch.randn((n, d), device=DEV).to(BF16)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lse = torch.empty((n, 1), device=DEV)
    out = fq.attn_prefill(q, k, v, cu, 1, 1, d, lse=lse)
    attn_ref.prefill(q, k, v, [0, n], [0, n], 1, 1, d, d ** -0.5, True, out, lse)


@pytest.mark.parametrize("unit", [2.0 ** 10, 2.0 ** 22, 2.0 ** 40, 2.0 ** 80])
@pytest.mark.parametrize("d,lq,lk,causal", [(64, 200, 200, True), (128, 200, 200, True),
                                            (256, 200, 200, True), (128, 20, 3000, False)])
def test_huge_scores_pick_the_largest(d, lq, lk, causal, unit):
    """Scores that are exact multiples of `unit` in binary32: the weights are 1 at the largest
    and 0 elsewhere, so out is the mean of v over the ties.  Tolerance: a mean of at most lk terms
    in binary32 and one rounding to bf16; and, as in attn_ref, half a bf16 step of sum w|v|: the
    tied weights are 2^e with the reference's rounding e in the exponent, not 1, and are rounded to
    bf16 in the numerator alone, by a factor within 1 +- 2^-8.  lse: five roundings (scale to log2
    units, its product, the reference's sum with the log, the constant and product back)."""
    g = torch.Generator(device=DEV).manual_seed(d + lk)
    q = (torch.randint(-2, 3, (lq, 2 * d), generator=g, device=DEV) * unit ** 0.5).to(BF16)
    k = (torch.randint(-2, 3, (lk, d), generator=g, device=DEV) * unit ** 0.5).to(BF16)
    v = torch.randn((lk, d), generator=g, device=DEV).to(BF16)
    a = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
    b = torch.tensor([0, lk], dtype=torch.int32, device=DEV)
    lse = torch.empty((lq, 2), device=DEV)
    out = fq.attn_prefill(q, k, v, a, 2, 1, d, cu_seqlens_k=b, softmax_scale=1.0, causal=causal, lse=lse)
    for h in range(2):
        s = q[:, h * d:(h + 1) * d].double() @ k.double().t()
        if causal:
            s = torch.where(attn_ref.causal_mask(lq, lk, DEV), s, -math.inf)
        best = (s == s.amax(1, keepdim=True)).double()
        w = best / best.sum(1, keepdim=True)
        want, size = w @ v.double(), w @ v.double().abs()
        bound = attn_ref.HALF_BF16 * (want.abs() + size) + (lk + 8) * attn_ref.U24 * size
        attn_ref.check(out[:, h * d:(h + 1) * d], want, bound, "out")
        want = s.amax(1) + torch.log(best.sum(1))
        attn_ref.check(lse[:, h], want, 5 * attn_ref.U24 * want.abs() + 2.0 ** -20, "lse")


@pytest.mark.parametrize("causal", [True, False])
def test_smallest_scale(causal):
    """The smallest scale that a binary32 holds: every seen key counts the same."""
    n, d = 100, 128
    q, k, v = (torch.randn((n, d), device=DEV).to(BF16) for _ in range(3))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lse = torch.empty((n, 1), device=DEV)
    out = fq.attn_prefill(q, k, v, cu, 1, 1, d, softmax_scale=2.0 ** -149, causal=causal, lse=lse)
    attn_ref.prefill(q, k, v, [0, n], [0, n], 1, 1, d, 2.0 ** -149, causal, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_infinities_and_nans_stay_where_they_are(bad, d):
    """A value row that is not finite reaches the queries that see it, in its columns, and no
    other; a key row that is not finite likewise."""
    n, at = 150, 100
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn((n, d), generator=g, device=DEV).to(BF16) for _ in range(3))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    want = fq.attn_prefill(q, k, v, cu, 1, 1, d)
    v2 = v.clone()
    v2[at, 5:9] = bad
    got = fq.attn_prefill(q, k, v2, cu, 1, 1, d)
    assert torch.equal(got[:at], want[:at])
    keep = [c for c in range(d) if not 5 <= c < 9]
    assert torch.equal(got[:, keep], want[:, keep])
    seen = got[at:, 5:9].float()
    assert torch.isnan(seen).all() if bad != bad else (seen == bad).all()
    k2 = k.clone()
    k2[at] = math.nan
    got = fq.attn_prefill(q, k2, v, cu, 1, 1, d)
    assert torch.equal(got[:at], want[:at]) and torch.isnan(got[at:].float()).all()


def test_bad_starts_are_clamped():
    """Entries outside the rows are clamped to them: nothing outside is read or written."""
    d, n = 64, 50
    q, k, v = (torch.randn((n, d), device=DEV).to(BF16) for _ in range(3))
    cu = torch.tensor([-5, 20, 1 << 30], dtype=torch.int32, device=DEV)
    fixed = torch.tensor([0, 20, n], dtype=torch.int32, device=DEV)
    assert torch.equal(fq.attn_prefill(q, k, v, cu, 1, 1, d), fq.attn_prefill(q, k, v, fixed, 1, 1, d))


def test_another_stream_and_a_replayed_graph():
    q, k, v, a, b, out, lse = _run([200, 33], [250, 33], 4, 2, 128)
    want, want_lse = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fq.attn_prefill(q, k, v, a, 4, 2, 128, cu_seqlens_k=b, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.attn_prefill(q, k, v, a, 4, 2, 128, cu_seqlens_k=b, out=out, lse=lse)
    for _ in range(3):
        out.zero_()
        lse.zero_()
        fq.attn_prefill(q, k, v, a, 4, 2, 128)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_rows_past_four_gib():
    """Rows 8 MiB apart: the last lie 5.5 GiB behind the first."""
    n, hq, hkv, d = 700, 2, 1, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    wide = torch.empty((n, 1 << 22), dtype=BF16, device=DEV)
    cols = [0, 256, 384, 512]
    q, k, v, out = (wide[:, c:c + w] for c, w in zip(cols, (256, 128, 128, 256)))
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    starts = [0, 30, n]
    cu = torch.tensor(starts, dtype=torch.int32, device=DEV)
    lse = torch.empty((n, hq), device=DEV)
    fq.attn_prefill(q, k, v, cu, hq, hkv, d, out=out, lse=lse)
    attn_ref.prefill(q, k, v, starts, starts, hq, hkv, d, d ** -0.5, True, out, lse)


def test_two_graphs_of_split_calls():
    """Each graph has its own sums, whichever order they are replayed in, beside eager calls."""
    hq, hkv, d, lk = 8, 2, 128, 3000
    g = torch.Generator(device=DEV).manual_seed(6)
    cu_k = torch.tensor([0, lk], dtype=torch.int32, device=DEV)
    k, v = (torch.randn((lk, hkv * d), generator=g, device=DEV).to(BF16) for _ in range(2))
    calls = []
    for lq in (20, 33):
        assert fq.attn_prefill_workspace_size(1, lq, lk, hq, hkv, d) > 0
        q = torch.randn((lq, hq * d), generator=g, device=DEV).to(BF16)
        cu = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
        want = fq.attn_prefill(q, k, v, cu, hq, hkv, d, cu_seqlens_k=cu_k)
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            fq.attn_prefill(q, k, v, cu, hq, hkv, d, cu_seqlens_k=cu_k, out=out)
        calls.append((q, cu, want, out, graph))
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for _, _, _, out, _ in calls:
            out.zero_()
        for i in order:
            calls[i][4].replay()
        q, cu, want, _, _ = calls[order[0]]
        assert torch.equal(fq.attn_prefill(q, k, v, cu, hq, hkv, d, cu_seqlens_k=cu_k), want)
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(calls[i][3], calls[i][2])
