"""Cases of the attention layer around the paged E4M3 cache, and their plain forms.

Three operators: head norms and rotary positions with the paged E4M3 write ("rope"), causal
attention over packed prompts ("prefill"), single-token attention over the paged E4M3 cache
("decode").  `run` computes them in elementary torch operations in binary32, or, where `own`
is true, through the package's entry points.  `exact` computes them in binary64.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
TABLE_POSITIONS = 32768
ROPE_BASE = 1.0e6


def listed():
    return [
        # a decode step of 16 rows: one token of each of 16 sequences (launch latency)
        rope("rope_step_16", 16, 40, 4, 128, 128, False, True, 16),
        # a prompt of 4593 tokens, the prefill length of the quantizer's benchmark
        rope("rope_prompt_4593", 4593, 40, 4, 128, 128, False, True, 16),
        # rotation alone, pairs side by side over half of a 64-wide head, odd token count
        rope("rope_part_1021", 1021, 32, 8, 64, 32, True, False, 16),
        # one short question (latency)
        prefill("prefill_short_37", "37", "37", 40, 4, 128),
        # one long prompt
        prefill("prefill_prompt_4593", "4593", "4593", 40, 4, 128),
        # a batch of prompts of very different lengths, one token among them
        prefill("prefill_packed_6072", "2048,1,777,333,1536,64,2,1311",
                "2048,1,777,333,1536,64,2,1311", 32, 8, 128),
        # a chunk of a prompt behind a history already in the cache
        prefill("prefill_chunk_512", "512", "8704", 40, 4, 128),
        # two prompts of a model with 64-wide heads
        prefill("prefill_d64_2x2500", "2500,2500", "2500,2500", 32, 8, 64),
        # one sequence, short history (latency)
        decode("decode_1_777", "777", 40, 4, 128, 16),
        # the decode step of 16 rows over ragged histories
        decode("decode_16_ragged", "8192,1023,4096,5121,1,7777,2048,6500,3333,8000,512,4444,"
               "6001,1500,7169,2900", 40, 4, 128, 16),
        # a full serving batch
        decode("decode_64_ragged", ",".join(str(500 + (i * 2339) % 7600) for i in range(64)),
               32, 8, 128, 32),
        # two very long documents
        decode("decode_2_long", "131072,100003", 40, 4, 128, 16),
    ]


def rope(name, tokens, q_heads, kv_heads, dim, rot, interleaved, norm, block):
    return dict(name=name, op="rope", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                rot=rot, interleaved=interleaved, norm=norm, block=block)


def prefill(name, q_lens, k_lens, q_heads, kv_heads, dim):
    return dict(name=name, op="prefill", q_lens=q_lens, k_lens=k_lens, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim)


def decode(name, lens, q_heads, kv_heads, dim, block):
    return dict(name=name, op="decode", lens=lens, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                block=block)


def log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def shares(rng, total, count):
    """`count` lengths >= 1 that add up to about `total`."""
    w = [rng.random() ** 2 + 0.01 for _ in range(count)]
    return [max(1, int(total * x / sum(w))) for x in w]


def draw(rng):
    op = rng.choice(("rope", "prefill", "decode"))
    dim = rng.choice((64, 128, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8, 10, 16))
    while kv * group > 40:
        group = rng.choice((1, 2, 4, 5, 8, 10))
    heads = kv * group
    block = rng.choice((1, 8, 16, 16, 32, 48, 64, 128))
    if op == "rope":
        rot = rng.choice((dim, dim // 2, dim // 4))
        most = 4593 * 48 * 128 // (dim * (heads + 2 * kv))
        c = rope("", log_uniform(rng, 1, min(16384, most)), heads, kv, dim, rot,
                 rng.random() < 0.4, rng.random() < 0.7, block)
    elif op == "prefill":
        total = log_uniform(rng, 1, 4593 if dim <= 128 else 2300)
        lens = shares(rng, total, rng.choice((1, 1, 2, 3, 5, 9, 14)))
        behind = rng.random() < 0.3
        more = [n + (rng.randrange(0, 1 + (4593 if dim <= 128 else 2300) // len(lens)) if behind else 0)
                for n in lens]
        c = prefill("", ",".join(map(str, lens)), ",".join(map(str, more)), heads, kv, dim)
    else:
        most = 240000 * 1024 // (kv * dim)  # tokens whose codes the largest listed cases hold
        count = rng.choice((1, 1, 2, 3, 7, 16, 33, 64, 128))
        total = log_uniform(rng, count, min(most, count * 65536) // 2)
        c = decode("", ",".join(map(str, shares(rng, total, count))), heads, kv, dim, block)
    del c["name"]
    return c


def ints(text):
    return [int(x) for x in text.split(",")]


def pairs(case):
    """(query, key) pairs of the causal mask: query i of Lq sees keys 0 .. i + Lk - Lq."""
    return sum(max(0, lk - lq) * lq + sum(range(1, lq + 1)) if lk >= lq else lk * (lk + 1) // 2
               for lq, lk in zip(ints(case["q_lens"]), ints(case["k_lens"])))


def work(case):
    h, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        # q, k, v in; q out; codes out; the table's row, position and slot of each token
        row = 2 * (h + 2 * kv) * d + 2 * h * d + 2 * kv * d + 4 * case["rot"] + 16
        return {"bytes": t * row, "flops": t * (h + kv) * d * 8}
    if case["op"] == "prefill":
        tq, tk = sum(ints(case["q_lens"])), sum(ints(case["k_lens"]))
        return {"bytes": 4 * tq * h * d + 4 * tk * kv * d + 4 * tq * h,
                "flops": 4 * d * h * pairs(case)}
    lens = ints(case["lens"])
    return {"bytes": 2 * sum(lens) * kv * d + len(lens) * (4 * h * d + 4 * h + 4)
            + 4 * sum(-(-n // case["block"]) for n in lens),
            "flops": 4 * d * h * sum(lens)}


# ---------------------------------------------------------------------------------- inputs


def normal(g, shape, std=1.0, p=0.0, factor=1.0):
    """bf16 normal values; an independent share p of them multiplied by `factor`."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=F32) * std
    if p:
        x = torch.where(torch.rand(shape, generator=g, device="cuda") < p, x * factor, x)
    return x.to(BF16)


def starts(lens):
    t = torch.tensor([0] + lens, dtype=torch.int64)
    return t.cumsum(0).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    s = dict(case)
    if case["op"] == "rope":
        t, bs, r = case["tokens"], case["block"], case["rot"]
        # q, k and v are columns of one projection's output
        s["qkv"] = normal(g, (t, (h + 2 * kv) * d), 3.0, 0.002, 40.0)
        s["q"], s["k"], s["v"] = s["qkv"].split([h * d, kv * d, kv * d], dim=1)
        s["qw"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(BF16) if case["norm"] else None
        s["kw"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(BF16) if case["norm"] else None
        angle = (torch.arange(TABLE_POSITIONS, device="cuda", dtype=F64)[:, None]
                 * ROPE_BASE ** (-torch.arange(0, r, 2, device="cuda", dtype=F64) / r))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(F32)
        blocks = 2 * (-(-t // bs)) + 8
        if t <= 256:  # one token of each of t sequences
            s["positions"] = torch.randint(0, TABLE_POSITIONS, (t,), generator=g, device="cuda")
            s["slots"] = torch.randperm(blocks * bs, generator=g, device="cuda")[:t].contiguous()
        else:  # a prompt: consecutive positions, pages in any order
            s["positions"] = torch.arange(t, device="cuda")
            page = torch.randperm(blocks, generator=g, device="cuda")
            at = torch.arange(t, device="cuda")
            s["slots"] = page[at // bs] * bs + at % bs
        s["k_scale"] = 12.0 / 448 if case["norm"] else 1.5 * float(s["k"].abs().max()) / 448
        s["v_scale"] = float(s["v"].abs().max()) / 448
        s["k_cache"] = torch.zeros(blocks * bs * kv * d, dtype=torch.uint8, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["out"] = torch.empty((t, h * d), dtype=BF16, device="cuda")
    elif case["op"] == "prefill":
        q_lens, k_lens = ints(case["q_lens"]), ints(case["k_lens"])
        tq, tk = sum(q_lens), sum(k_lens)
        # normed heads: unit variance; the query's factor gives scores a spread of 2.5
        s["q"] = normal(g, (tq, h * d), 2.5)
        s["k"] = normal(g, (tk, kv * d))
        s["v"] = normal(g, (tk, kv * d), 3.0, 0.002, 40.0)
        s["starts_q"], s["starts_k"] = starts(q_lens), starts(k_lens)
        s["out"] = torch.empty((tq, h * d), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((tq, h), dtype=F32, device="cuda")
    else:
        lens, bs = ints(case["lens"]), case["block"]
        need = [-(-n // bs) for n in lens]
        blocks = sum(need) + 8
        page = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
        first = torch.tensor([0] + need).cumsum(0)[:-1].cuda()
        column = torch.arange(max(need), device="cuda")
        at = (first[:, None] + column).clamp(max=blocks - 1)
        s["tables"] = page[at]  # columns past a sequence's own blocks name other blocks
        s["lens_dev"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["q"] = normal(g, (len(lens), h * d), 2.5)
        for name, std, p in (("k", 1.0, 0.0), ("v", 3.0, 0.002)):
            x = normal(g, (blocks * bs * kv * d,), std, p, 40.0)
            s[name + "_scale"] = float(x.abs().max()) / 448
            s[name + "_cache"] = (x.float() / s[name + "_scale"]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        s["out"] = torch.empty((len(lens), h * d), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((len(lens), h), dtype=F32, device="cuda")
    return s


# --------------------------------------------------------------------- the framework's calls


def own_rope(s):
    import fp8_e4m3_quantization_amd as fq
    fq.fp8_qk_norm_rope_kv_write(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"],
                                 s["v_cache"], s["slots"], s["q_heads"], s["kv_heads"], s["dim"],
                                 s["block"], s["k_scale"], s["v_scale"], q_weight=s["qw"],
                                 k_weight=s["kw"], eps=EPS, interleaved=s["interleaved"],
                                 q_out=s["out"])
    return s["out"], s["k_cache"].view(E4M3), s["v_cache"].view(E4M3)


def own_prefill(s):
    import fp8_e4m3_quantization_amd as fq
    fq.attn_prefill(s["q"], s["k"], s["v"], s["starts_q"], s["q_heads"], s["kv_heads"], s["dim"],
                    cu_seqlens_k=s["starts_k"], causal=True, out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def own_decode(s):
    import fp8_e4m3_quantization_amd as fq
    fq.fp8_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens_dev"], s["q_heads"],
                       s["kv_heads"], s["dim"], s["block"], s["k_scale"], s["v_scale"],
                       out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


# -------------------------------------------------------------------------- the plain forms


def turned(x, cos, sin, rot, interleaved):
    """Rotation of the first `rot` of each head's values; x [t, heads, d], cos / sin [t, 1, rot/2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def plain_rope(s):
    d, r = s["dim"], s["rot"]
    table = s["cos_sin"][s["positions"]][:, None]
    cos, sin = table[..., :r // 2], table[..., r // 2:]

    def head(x, w):
        x = x.float().unflatten(1, (-1, d))
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return turned(x, cos, sin, r, s["interleaved"]).flatten(1).to(BF16)

    q, k = head(s["q"], s["qw"]), head(s["k"], s["kw"])
    for x, pool, scale in ((k, "k_cache", "k_scale"), (s["v"], "v_cache", "v_scale")):
        codes = (x.float() / s[scale]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        s[pool].view(-1, x.shape[1])[s["slots"]] = codes
    return q, s["k_cache"].view(E4M3), s["v_cache"].view(E4M3)


def weigh(scores, seen, v):
    """Softmax over the last axis of what `seen` leaves, times v; rows with nothing give 0."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out, (top + torch.log(total)).squeeze(-1)


def plain_prefill(s):
    h, kv, d = s["q_heads"], s["kv_heads"], s["dim"]
    q = s["q"].float().unflatten(1, (h, d)).transpose(0, 1)
    k = s["k"].float().unflatten(1, (kv, d)).permute(1, 2, 0).repeat_interleave(h // kv, 0).contiguous()
    v = s["v"].float().unflatten(1, (kv, d)).transpose(0, 1).repeat_interleave(h // kv, 0).contiguous()
    at_q = torch.arange(q.shape[1], device="cuda", dtype=torch.int32)
    at_k = torch.arange(v.shape[1], device="cuda", dtype=torch.int32)
    seq_q = torch.searchsorted(s["starts_q"], at_q, right=True) - 1
    seq_k = torch.searchsorted(s["starts_k"], at_k, right=True) - 1
    # a query's distance from its sequence's end, and a key's: causal from the end
    left_q, left_k = s["starts_q"][seq_q + 1] - at_q, s["starts_k"][seq_k + 1] - at_k
    seen = (seq_q[:, None] == seq_k) & (left_k >= left_q[:, None])
    out, lse = weigh(torch.matmul(q.contiguous(), k) * d ** -0.5, seen, v)
    return out.transpose(0, 1).flatten(1).to(BF16), lse.t().contiguous()


def plain_decode(s):
    h, kv, d, bs = s["q_heads"], s["kv_heads"], s["dim"], s["block"]
    at = torch.arange(s["tables"].shape[1] * bs, device="cuda")
    rows = s["tables"][:, at // bs].long() * bs + at % bs
    seen = at < s["lens_dev"][:, None]

    def read(pool, scale):
        codes = pool.view(-1, kv * d)[rows].view(E4M3)
        return codes.float().unflatten(2, (kv, d)).transpose(1, 2) * scale

    q = s["q"].float().unflatten(1, (kv, h // kv, d))
    k = read(s["k_cache"], s["k_scale"]).transpose(2, 3).contiguous()
    v = read(s["v_cache"], s["v_scale"]).contiguous()
    out, lse = weigh(torch.matmul(q, k) * d ** -0.5, seen[:, None, None], v)
    return out.flatten(1).to(BF16), lse.flatten(1)


def run(state):
    if own:
        return {"rope": own_rope, "prefill": own_prefill, "decode": own_decode}[state["op"]](state)
    return {"rope": plain_rope, "prefill": plain_prefill, "decode": plain_decode}[state["op"]](state)


# ------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    h, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        half = case["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        table = s["cos_sin"].double()[s["positions"]]
        turn = torch.complex(table[:, :half], table[:, half:])[:, None]

        def head(x, w):
            y = x.double().reshape(case["tokens"], -1, d).clone()
            if w is not None:
                y *= w.double() / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y.reshape(case["tokens"], -1)

        pools = []
        for x, scale in ((head(s["k"], s["kw"]), s["k_scale"]), (s["v"].double(), s["v_scale"])):
            pool = torch.zeros((s["k_cache"].numel() // (kv * d), kv * d), dtype=F64, device="cuda")
            pool[s["slots"]] = (x / scale).clamp(-448, 448)
            pools.append(pool.flatten())
        return head(s["q"], s["qw"]), pools[0], pools[1]

    def one(q, k, v, behind):
        """One head of one sequence: query i sees the first i + 1 + behind keys."""
        x = q.double() @ k.double().t() / math.sqrt(d)
        i = torch.arange(x.shape[0], device="cuda")[:, None]
        x.masked_fill_(torch.arange(x.shape[1], device="cuda") > i + behind, -math.inf)
        lse = torch.logsumexp(x, 1)
        p = (x - lse[:, None].clamp(min=-1e300)).exp()
        return p @ v.double(), lse

    if case["op"] == "prefill":
        out = torch.zeros((s["q"].shape[0], h, d), dtype=F64, device="cuda")
        lse = torch.full((s["q"].shape[0], h), -math.inf, dtype=F64, device="cuda")
        q, k, v = s["q"].view(-1, h, d), s["k"].view(-1, kv, d), s["v"].view(-1, kv, d)
        i = j = 0
        for lq, lk in zip(ints(case["q_lens"]), ints(case["k_lens"])):
            for n in range(h):
                m = n // (h // kv)
                out[i:i + lq, n], lse[i:i + lq, n] = one(q[i:i + lq, n], k[j:j + lk, m],
                                                         v[j:j + lk, m], lk - lq)
            i, j = i + lq, j + lk
        return out.flatten(1), lse
    bs = case["block"]
    lens = ints(case["lens"])
    out = torch.zeros((len(lens), h, d), dtype=F64, device="cuda")
    lse = torch.full((len(lens), h), -math.inf, dtype=F64, device="cuda")
    pools = [s[n + "_cache"].view(-1, bs, kv, d) for n in ("k", "v")]
    q = s["q"].view(-1, kv, h // kv, d)
    for b, n in enumerate(lens):
        pages = s["tables"][b, :-(-n // bs)].long()
        k, v = (p[pages].view(E4M3).double().view(-1, kv, d)[:n] * s[c + "_scale"]
                for c, p in zip("kv", pools))
        for m in range(kv):
            g = slice(m * (h // kv), (m + 1) * (h // kv))
            out[b, g], lse[b, g] = one(q[b, m], k[:, m], v[:, m], n)
    return out.flatten(1), lse
