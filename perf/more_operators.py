"""Cases of what a layer does between its products and over its paged cache, and their plain forms.

Three operators: RMS norm with the residual's addition and E4M3 groups ("norm"), SiLU of the gate
times the up projection with E4M3 groups ("silu"), attention of chunks of new tokens over the paged
E4M3 cache ("chunk").  `run` computes them in elementary torch operations in binary32, or, where
`own` is true, through the package's entry points.  `exact` computes them in binary64.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
GROUP = 128
FLOOR = 1e-10  # smallest group maximum


def listed():
    return [
        # a decode step of 16 rows (launch latency)
        norm("norm_step_16", 16, 5120, True, False),
        # a prompt of 4593 tokens, the prefill length of the quantizer's benchmark
        norm("norm_prompt_4593", 4593, 5120, True, False),
        # the first layer's norm of a wide model: no residual yet, the bf16 rows kept too, odd count
        norm("norm_wide_517", 517, 16384, False, True),
        # the same three for the products' gate: a step, a prompt, an odd count of narrow rows
        silu("silu_step_16", 16, 16384, False),
        silu("silu_prompt_4593", 4593, 16384, False),
        silu("silu_part_1021", 1021, 1024, True),
        # one sequence, five drafted tokens behind a short history (latency)
        chunk("chunk_1x5_777", "5", "777", 40, 4, 128, 16),
        # a step of 16 sequences with four drafted tokens each over ragged histories
        chunk("chunk_16x4_ragged", ",".join(["4"] * 16), "8192,1023,4096,5121,4,7777,2048,6500,3333,"
              "8000,512,4444,6001,1500,7169,2900", 40, 4, 128, 16),
        # a chunk of a prompt behind its history
        chunk("chunk_512_8704", "512", "8704", 40, 4, 128, 16),
        # a serving batch: one prompt's chunk beside the steps of 23 other sequences
        chunk("chunk_mixed_24", "509" + ",1" * 23, "4605," + ",".join(str(500 + (i * 2339) % 7600) for i in
              range(23)), 32, 8, 128, 32),
        # two prompts of a model with 64-wide heads, one from its start, one behind a history
        chunk("chunk_d64_2", "700,1300", "700,5300", 32, 8, 64, 16),
        # a question of 64 tokens about a very long document
        chunk("chunk_64_100003", "64", "100003", 40, 4, 128, 16),
    ]


def norm(name, rows, width, residual, keep):
    return dict(name=name, op="norm", rows=rows, width=width, residual=residual, keep=keep)


def silu(name, rows, width, keep):
    return dict(name=name, op="silu", rows=rows, width=width, keep=keep)


def chunk(name, q_lens, lens, q_heads, kv_heads, dim, block):
    return dict(name=name, op="chunk", q_lens=q_lens, lens=lens, q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, block=block)


def log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def shares(rng, total, count):
    """`count` lengths >= 1 that add up to about `total`."""
    w = [rng.random() ** 2 + 0.01 for _ in range(count)]
    return [max(1, int(total * x / sum(w))) for x in w]


def draw(rng):
    op = rng.choice(("norm", "silu", "chunk", "chunk"))
    if op != "chunk":
        width = GROUP * log_uniform(rng, 1, 160)
        rows = log_uniform(rng, 1, min(32768, 4593 * 5120 // width))
        c = norm("", rows, width, rng.random() < 0.7, rng.random() < 0.3) if op == "norm" else \
            silu("", rows, width, rng.random() < 0.3)
        del c["name"]
        return c
    dim = rng.choice((64, 128, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 8, 10, 16))
    while kv * group > 40:
        group = rng.choice((1, 2, 4, 5, 8, 10))
    heads = kv * group
    block = rng.choice((1, 8, 16, 16, 32, 48, 64, 128))
    count = rng.choice((1, 1, 2, 3, 7, 16, 33, 64))
    # new tokens and (token, position) pairs, of all sequences, within the largest listed case's
    total = log_uniform(rng, count, 2048)
    q_lens = [rng.randint(1, 8) for _ in range(count)] if rng.random() < 0.4 else shares(rng, total, count)
    most = 64 * 100003 * 40 * 128 // (sum(q_lens) * heads * dim)
    behind = shares(rng, log_uniform(rng, 1, max(2, min(most, 131072) // 2)), count)
    lens = [q + (n if rng.random() < 0.8 else 0) for q, n in zip(q_lens, behind)]
    c = chunk("", ",".join(map(str, q_lens)), ",".join(map(str, lens)), heads, kv, dim, block)
    del c["name"]
    return c


def ints(text):
    return [int(x) for x in text.split(",")]


def pairs(case):
    """(query, position) pairs of the causal mask: query i of Lq sees positions 0 .. i + len - Lq."""
    return sum((n - q) * q + q * (q + 1) // 2 for q, n in zip(ints(case["q_lens"]), ints(case["lens"])))


def work(case):
    if case["op"] == "chunk":
        h, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
        q_lens, lens = ints(case["q_lens"]), ints(case["lens"])
        return {"bytes": 2 * sum(lens) * kv * d + sum(q_lens) * (4 * h * d + 4 * h) + 8 * len(lens)
                + 4 * sum(-(-n // case["block"]) for n in lens),
                "flops": 4 * d * h * pairs(case)}
    values = case["rows"] * case["width"]
    out = values + 4 * (values // GROUP) + (2 * values if case["keep"] else 0)
    if case["op"] == "silu":
        return {"bytes": 4 * values + out, "flops": 6 * values}
    return {"bytes": (6 if case["residual"] else 2) * values + 2 * case["width"] + out, "flops": 6 * values}


# ---------------------------------------------------------------------------------- inputs


def normal(g, shape, std=1.0, p=0.0, factor=1.0):
    """bf16 normal values; an independent share p of them multiplied by `factor`."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=F32) * std
    if p:
        x = torch.where(torch.rand(shape, generator=g, device="cuda") < p, x * factor, x)
    return x.to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "chunk":
        h, kv, d, bs = case["q_heads"], case["kv_heads"], case["dim"], case["block"]
        q_lens, lens = ints(case["q_lens"]), ints(case["lens"])
        tokens = sum(q_lens)
        need = [-(-n // bs) for n in lens]
        blocks = sum(need) + 8
        page = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
        first = torch.tensor([0] + need).cumsum(0)[:-1].cuda()
        column = torch.arange(max(need), device="cuda")
        at = (first[:, None] + column).clamp(max=blocks - 1)
        s["tables"] = page[at]  # columns past a sequence's own blocks name other blocks
        s["lens_dev"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["starts"] = torch.tensor([0] + q_lens).cumsum(0).to(torch.int32).cuda()
        # normed heads: unit variance; the query's factor gives scores a spread of 2.5
        s["q"] = normal(g, (tokens, h * d), 2.5)
        for name, std, p in (("k", 1.0, 0.0), ("v", 3.0, 0.002)):
            x = normal(g, (blocks * bs * kv * d,), std, p, 40.0)
            s[name + "_scale"] = float(x.abs().max()) / 448
            s[name + "_cache"] = (x.float() / s[name + "_scale"]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        s["out"] = torch.empty((tokens, h * d), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((tokens, h), dtype=F32, device="cuda")
        return s
    t, k = case["rows"], case["width"]
    s["codes"] = torch.empty((t, k), dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty((t, k // GROUP), dtype=F32, device="cuda")
    s["kept"] = torch.empty((t, k), dtype=BF16, device="cuda") if case["keep"] else None
    if case["op"] == "silu":
        # the two halves of one projection's output
        s["both"] = normal(g, (t, 2 * k), 1.5, 0.001, 20.0)
        s["gate"], s["up"] = s["both"].split(k, dim=1)
        return s
    s["x"] = normal(g, (t, k), 1.0, 0.001, 20.0)
    s["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device="cuda")).to(BF16)
    s["residual"] = s["sum"] = None
    if case["residual"]:
        # a residual stream has a few channels that are large in every row
        channel = torch.where(torch.rand(k, generator=g, device="cuda") < 0.002, 30.0, 1.0)
        s["residual"] = (normal(g, (t, k), 3.0).float() * channel).to(BF16)
        s["sum"] = torch.empty_like(s["residual"])
    return s


# --------------------------------------------------------------------- the framework's calls


def rows_of(s, first):
    return [x for x in (s["codes"].view(E4M3), s["scales"], s["kept"], first) if x is not None]


def own_norm(s):
    import fp8_e4m3_quantization_amd as fq
    fq.fp8_rms_norm_group_quant(s["x"], s["weight"], eps=EPS, residual=s["residual"], q=s["codes"],
                                scales=s["scales"], residual_out=s["sum"], norm_out=s["kept"])
    return rows_of(s, s["sum"])


def own_silu(s):
    import fp8_e4m3_quantization_amd as fq
    fq.fp8_silu_mul_group_quant(s["gate"], s["up"], q=s["codes"], scales=s["scales"], out=s["kept"])
    return rows_of(s, None)


def own_chunk(s):
    import fp8_e4m3_quantization_amd as fq
    fq.fp8_attn_chunk(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens_dev"], s["starts"],
                      s["q_heads"], s["kv_heads"], s["dim"], s["block"], s["k_scale"], s["v_scale"],
                      out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


# -------------------------------------------------------------------------- the plain forms


def grouped(y, keep):
    """binary32 rows -> their E4M3 values, the groups' scales, and the rows in bf16 where kept."""
    groups = y.unflatten(1, (-1, GROUP))
    scales = groups.abs().amax(-1).clamp(min=FLOOR) / 448
    codes = (groups / scales[..., None]).clamp(-448, 448).to(E4M3).flatten(1)
    return [codes, scales] + ([y.to(BF16)] if keep else [])


def plain_norm(s):
    h = s["x"].float()
    total = None
    if s["residual"] is not None:
        total = (h + s["residual"].float()).to(BF16)
        h = total.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    return grouped(y, s["keep"]) + ([] if total is None else [total])


def plain_silu(s):
    gate = s["gate"].float()
    return grouped(gate / (1 + torch.exp(-gate)) * s["up"].float(), s["keep"])


def plain_chunk(s):
    h, kv, d, bs = s["q_heads"], s["kv_heads"], s["dim"], s["block"]
    lens, starts = s["lens_dev"], s["starts"]
    # all histories, end to end: each position's sequence, place and row in the pools
    ends = lens.cumsum(0)
    at = torch.arange(sum(ints(s["lens"])), device="cuda")
    seq = torch.searchsorted(ends, at, right=True)
    place = at - (ends - lens)[seq]
    rows = s["tables"][seq, place // bs].long() * bs + place % bs
    # each new token's sequence, and the positions that it sees of it
    token = torch.arange(s["q"].shape[0], device="cuda")
    own_seq = torch.searchsorted(starts, token, right=True) - 1
    sees = token - starts[own_seq + 1] + lens[own_seq] + 1
    seen = (own_seq[:, None] == seq) & (place < sees[:, None])

    def read(pool, scale):
        return pool.view(-1, kv, d)[rows].view(E4M3).float() * scale

    q = s["q"].float().unflatten(1, (kv, h // kv, d)).permute(1, 2, 0, 3).flatten(1, 2).contiguous()
    k = read(s["k_cache"], s["k_scale"]).permute(1, 2, 0).contiguous()
    v = read(s["v_cache"], s["v_scale"]).transpose(0, 1).contiguous()
    x = torch.matmul(q, k).unflatten(1, (h // kv, -1)).mul_(d ** -0.5)
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(1, 2), v).unflatten(1, (h // kv, -1)) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    return out.permute(2, 0, 1, 3).flatten(1).to(BF16), lse.flatten(0, 1).t().contiguous()


def run(state):
    if own:
        return {"norm": own_norm, "silu": own_silu, "chunk": own_chunk}[state["op"]](state)
    return {"norm": plain_norm, "silu": plain_silu, "chunk": plain_chunk}[state["op"]](state)


# ------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "chunk":
        if case["op"] == "norm":
            total = None
            y = s["x"].double()
            if case["residual"]:
                total = y + s["residual"].double()
                y = total.to(F32).to(BF16).double()  # what the layer keeps, and norms
            y = y / (y.pow(2).sum(1, keepdim=True) / case["width"] + EPS).sqrt() * s["weight"].double()
        else:
            total = None
            y = s["up"].double() * s["gate"].double() * torch.sigmoid(s["gate"].double())
        most = y.abs().reshape(case["rows"], -1, GROUP).max(2).values
        scales = torch.maximum(most, torch.full_like(most, FLOOR)) / 448
        codes = y / scales.repeat_interleave(GROUP, 1)
        return [x for x in (codes, scales, y if case["keep"] else None, total) if x is not None]
    h, kv, d, bs = case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    g = h // kv
    pools = [s[n + "_cache"].view(-1, bs, kv, d) for n in ("k", "v")]
    q = s["q"].view(-1, kv, g, d)
    out = torch.zeros((q.shape[0], kv, g, d), dtype=F64, device="cuda")
    lse = torch.full((q.shape[0], kv, g), -math.inf, dtype=F64, device="cuda")
    i = 0
    for b, (lq, n) in enumerate(zip(ints(case["q_lens"]), ints(case["lens"]))):
        pages = s["tables"][b, :-(-n // bs)].long()
        k, v = (p[pages].view(E4M3).double().view(-1, kv, d)[:n] * s[c + "_scale"]
                for c, p in zip("kv", pools))
        hidden = torch.arange(n, device="cuda") > torch.arange(n - lq, n, device="cuda")[:, None]
        for m in range(h):
            x = q[i:i + lq, m // g, m % g].double() @ k[:, m // g].t() / math.sqrt(d)
            x.masked_fill_(hidden, -math.inf)
            lse[i:i + lq, m // g, m % g] = z = torch.logsumexp(x, 1)
            out[i:i + lq, m // g, m % g] = (x - z[:, None]).exp_() @ v[:, m // g]
        i += lq
    return out.flatten(1), lse.flatten(1)
