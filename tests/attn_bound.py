"""The bound of attention outputs whose numerator and denominator take the same rounded weights, and a case that
comes near it (torch, any device; no code of the library)."""
import math

import torch

from tests import attn_ref

F64 = torch.float64
HALF = attn_ref.HALF_BF16


def attend(q, k, v, scale, seen):
    """q [n, D], k / v [m, D], seen [n, m] bool -> (out, its bound), binary64, finite values.

    With weights w (their sum 1) that bf16 takes to w (1 + e), |e| <= half, out is
    sum w (1 + e) v / sum w (1 + e) = out + sum w e (v - out) / (1 + sum w e): off by at most
    half / (1 - half) sum w |v - out|.  The binary32 steps' share, 3 d sum w |v|, is attn_ref.attend's, and out's
    own rounding half of what it rounds."""
    out, _, _, _ = attn_ref.attend(q, k, v, scale, seen)
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    s = torch.where(seen, scale * (q @ k.t()), -math.inf)
    w = torch.nan_to_num(torch.softmax(s, 1), 0.0)
    size = torch.where(seen, scale * (q.abs() @ k.abs().t()), 0.0).amax(1)
    d = (q.shape[1] + 8) * attn_ref.U24 * size + (8 + seen.sum(1).clamp(max=4096)) * attn_ref.U24 + 2.0 ** -21
    apart = torch.stack([w[i] @ (v - out[i]).abs() for i in range(len(w))])
    bound = (HALF / (1 - HALF) * apart + 3 * d[:, None] * (w @ v.abs())) * (1 + HALF) + HALF * out.abs() + 1e-30
    return out, bound


def one_value(n, d=64, at=77):
    """q [1, d], k and v [n, d], softmax scale: of every 32 positions the first has the score 0 and the weight 1, the
    others (1/2 + 2^-9) (1 - 2^-17), which bf16 takes down to 1/2; at `at` it is that times about 1 + 2^-16, which
    goes up, and the only value that is not 0.  Numerator and denominator go apart as far as they can."""
    q, k, v = torch.zeros((1, d)), torch.zeros((n, d)), torch.zeros((n, d))
    scale = -math.log((0.5 + 2.0 ** -9) * (1 - 2.0 ** -17))
    q[0, 0], q[0, 1] = -1.0, 2.0 ** -10
    k[:, 0] = 1.0
    k[::32, 0] = 0.0
    k[at, 1] = 2.0 ** -6 * 1.5
    v[at] = (1 + torch.arange(d) % 8 / 8) * 2.0 ** (torch.arange(d) // 8 % 2)
    return q.to(torch.bfloat16), k, v, scale
