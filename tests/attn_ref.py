"""Plain 64-bit definitions of the attention operators, and the error bounds the tests hold
their outputs to (torch, any device; no code of the library)."""
import math

import torch

F64 = torch.float64
U24 = 2.0 ** -24   # half a binary32 step
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def attend(q, k, v, scale, seen):
    """q [n, D], k / v [m, D], seen [n, m] bool -> (out, lse, out's bound, lse's bound), binary64.

    Bounds, with u = 2^-24 and z = scale sum |q||k| of the largest seen key.  A score is a sum of
    D exact products in binary32 in any order, scaled and shifted by a reference of at most z:
    off by (D + 8) u z.  exp2 adds 2^-22, a sum over n keys n u (taken up to 4096: a longer sum is
    made of partial sums), a few scalings 8 u; together a weight is off by a factor 1 + d.  The
    numerator is a sum of weights rounded to bf16 (half a step) times v, the denominator a sum of
    unrounded weights: out is off by (half + 3 d) sum w|v| before its own rounding, half |out|.
    lse is off by 2 d, and by its own few roundings."""
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    s = scale * (q @ k.t())
    size = scale * (q.abs() @ k.abs().t())
    s = torch.where(seen, s, -math.inf)
    any_seen = seen.any(1)
    top = torch.where(any_seen, s.amax(1), 0.0)
    p = torch.where(seen, torch.exp(s - top[:, None]), 0.0)
    total = p.sum(1)
    safe = torch.where(total > 0, total, 1.0)
    w = p / safe[:, None]
    vz = torch.where(torch.isfinite(v), v, 0.0)
    out = w @ vz
    lse = top + torch.log(total)
    n = seen.sum(1).to(F64)
    biggest = torch.where(seen, size, 0.0).amax(1)
    d = (q.shape[1] + 8) * U24 * biggest + (8 + n.clamp(max=4096)) * U24 + 2.0 ** -21
    out_bound = HALF_BF16 * out.abs() + (HALF_BF16 + 3 * d)[:, None] * (w @ vz.abs()) + 1e-30
    lse_bound = 2 * d + 8 * U24 * lse.abs().nan_to_num(0, 0, 0)
    return out, lse, out_bound, lse_bound


def causal_mask(lq, lk, device):
    i = torch.arange(lq, device=device)[:, None]
    return torch.arange(lk, device=device)[None, :] <= i + lk - lq


def check(got, want, bound, what):
    """|got - want| <= bound element-wise, infinities and NaNs in the same places."""
    got = got.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: infinities or NaNs differ"
    assert torch.equal(got[~fine].nan_to_num(7.0), want[~fine].nan_to_num(7.0)), what
    err = (got - want).abs()[fine] / bound.expand_as(want)[fine]
    if err.numel():
        assert float(err.max()) <= 1.0, f"{what}: worst error / bound = {float(err.max()):.3f}"


def prefill(q, k, v, cu_q, cu_k, hq, hkv, d, scale, causal, out, lse, rows=None):
    """Holds out (and lse) of every sequence and head to the definition; returns the rows that
    belong to some sequence."""
    covered = torch.zeros(q.shape[0], dtype=torch.bool)
    q3, k3, v3 = q.reshape(-1, hq, d), k.reshape(-1, hkv, d), v.reshape(-1, hkv, d)
    for s in range(len(cu_q) - 1):
        a, b, c, e = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        covered[a:b] = True
        if a == b:
            continue
        seen = causal_mask(b - a, e - c, q.device) if causal else \
            torch.ones((b - a, e - c), dtype=torch.bool, device=q.device)
        for h in range(hq):
            if e == c:
                o = torch.zeros((b - a, d), dtype=F64, device=q.device)
                check(out[a:b].reshape(b - a, hq, d)[:, h], o, o + 1e-30, "no keys")
                assert torch.equal(lse[a:b, h], torch.full_like(lse[a:b, h], -math.inf))
                continue
            m = h // (hq // hkv)
            o, l, ob, lb = attend(q3[a:b, h], k3[c:e, m], v3[c:e, m], scale, seen)
            check(out[a:b].reshape(b - a, hq, d)[:, h], o, ob, f"sequence {s} head {h} out")
            check(lse[a:b, h], l, lb, f"sequence {s} head {h} lse")
    return covered


def e4m3_values(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32).to(F64)


def decode(q, kc, vc, tables, lens, hq, hkv, d, bs, cs, ks, vs, scale, out, lse):
    """Holds out and lse of every sequence and head to the definition (pools [blocks, cs])."""
    nb = kc.numel() // cs
    kp, vp = (x.view(nb, cs)[:, :bs * hkv * d].reshape(nb, bs, hkv, d) for x in (kc, vc))
    for s, n in enumerate(lens):
        n = max(0, min(n, tables.shape[1] * bs))
        pos = torch.arange(n, device=q.device)
        ids = tables[s].long()[pos // bs]
        good = (ids >= 0) & (ids < nb)
        ids, off = ids[good], pos[good] % bs
        for m in range(hkv):
            heads = slice(m * (hq // hkv), (m + 1) * (hq // hkv))
            qq = q[s].reshape(hq, d)[heads]
            if ids.numel() == 0:
                assert not out[s].reshape(hq, d)[heads].any()
                assert torch.equal(lse[s, heads], torch.full_like(lse[s, heads], -math.inf))
                continue
            k, v = e4m3_values(kp[ids, off, m]), e4m3_values(vp[ids, off, m])
            seen = torch.ones((qq.shape[0], ids.numel()), dtype=torch.bool, device=q.device)
            o, l, ob, lb = attend(qq, k, v, scale * ks, seen)
            check(out[s].reshape(hq, d)[heads], o * vs, ob * vs + o.abs() * vs * 4 * U24,
                  f"sequence {s} KV head {m} out")
            check(lse[s, heads], l, lb, f"sequence {s} KV head {m} lse")
