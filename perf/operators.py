"""What is measured of the paged K/V path: rotary positions, the insert into a K/V pool, and dense attention over it.

Each case is one call on data of a decode step (one new token per request), a speculative-verify step (a few rows per
request) or a prefill chunk.  `run` computes it in plain torch operations, or with `own` by the framework's calls.
"""
import math

import torch

own = False

INTERLEAVED, HALF = 0, 1  # pairs (2i, 2i + 1), or (i, i + rot / 2)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # attention: the first answer after a short prompt, where latency is all there is
        dict(name="attend_one_short", op="attend", rows=1, group=1, kv_heads=4, hpg=16, dim=128, page=128, fmt="fp8",
             lo=257, hi=257),
        # one request of 4,096 tokens, 16-bit cache
        dict(name="attend_one_4k", op="attend", rows=1, group=1, kv_heads=4, hpg=16, dim=128, page=64, fmt="bf16",
             lo=4096, hi=4096),
        # the batched decode: 32 requests of 16K to 64K tokens, FP8 cache in the block-sparse variant's pages
        dict(name="attend_b32_16k_64k", op="attend", rows=32, group=1, kv_heads=4, hpg=16, dim=128, page=128,
             fmt="fp8", lo=16384, hi=65536),
        # eight long requests, 16-bit cache
        dict(name="attend_b8_128k", op="attend", rows=8, group=1, kv_heads=4, hpg=8, dim=128, page=64, fmt="bf16",
             lo=131072, hi=131072),
        # speculative verify: four rows of each of four requests share one read of the cache
        dict(name="attend_verify_4x4_64k", op="attend", rows=16, group=4, kv_heads=4, hpg=16, dim=128, page=128,
             fmt="fp8", lo=60000, hi=65536),
        # a padded batch of ragged, partly empty rows with an odd number of heads per KV head and small pages
        dict(name="attend_ragged_d64", op="attend", rows=23, group=1, kv_heads=3, hpg=5, dim=64, page=16, fmt="bf16",
             lo=0, hi=9001),
        # insert: one decode step's tokens, rotated keys and queries, FP8 pool
        dict(name="insert_decode_8", op="insert", tokens=8, kv_heads=4, hpg=16, dim=128, page=128, fmt="fp8", rot=64,
             layout=HALF, scaled="yarn", pos=131072),
        # an odd chunk without rotation into a 16-bit pool
        dict(name="insert_plain_333", op="insert", tokens=333, kv_heads=3, hpg=5, dim=64, page=16, fmt="bf16", rot=0,
             layout=HALF, scaled="none", pos=4096),
        # a prefill chunk of 8,192 tokens on a 56K prefix
        dict(name="insert_prefill_8k", op="insert", tokens=8192, kv_heads=4, hpg=16, dim=128, page=128, fmt="fp8",
             rot=128, layout=HALF, scaled="none", pos=65536),
        # rotary positions of one token: 96 query heads' last 64 of 576 dims, its latent's and its index key's
        dict(name="rope_decode_1", op="rope", tokens=1, heads=96, dim=576, rot=64, layout=INTERLEAVED, dtype="bf16",
             scaled="none", pos=4096),
        # 16 verify rows at positions near a million, stretched by YaRN
        dict(name="rope_verify_1m", op="rope", tokens=16, heads=96, dim=576, rot=64, layout=INTERLEAVED, dtype="bf16",
             scaled="yarn", pos=1048576),
        # a prefill chunk of 8,192 tokens
        dict(name="rope_prefill_8k", op="rope", tokens=8192, heads=96, dim=576, rot=64, layout=INTERLEAVED,
             dtype="bf16", scaled="none", pos=65536),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "insert", "rope"))
    scaled = rng.choice(("none", "linear", "ntk", "yarn"))
    if op == "attend":
        group = rng.choice((1, 1, 2, 4))
        rows = group * _log(rng, 1, 32 // group)
        dim, fmt = rng.choice((64, 128)), rng.choice(("bf16", "fp8"))
        kv_heads, hpg = _log(rng, 1, 8), _log(rng, 1, 16)
        # the cache of all rows stays within that of the eight long requests
        most = min(131072, (1 << 30) // (rows * kv_heads * dim * 2))
        hi = _log(rng, 1, most)
        return dict(op=op, rows=rows, group=group, kv_heads=kv_heads, hpg=hpg, dim=dim, page=rng.choice((16, 32, 64, 128)),
                    fmt=fmt, lo=round(hi * rng.choice((0.0, 0.25, 1.0))), hi=hi)
    if op == "insert":
        dim = rng.choice((64, 128))
        rot = rng.choice((0, dim // 2, dim))
        return dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=_log(rng, 1, 8), hpg=_log(rng, 1, 8), dim=dim,
                    page=rng.choice((16, 32, 64, 128)), fmt=rng.choice(("bf16", "fp8")), rot=rot,
                    layout=rng.choice((INTERLEAVED, HALF)), scaled=scaled if rot else "none", pos=_log(rng, 16, 1048576))
    rot = 2 * _log(rng, 4, 64)
    return dict(op=op, tokens=_log(rng, 1, 8192), heads=_log(rng, 1, 96), dim=rot + rng.choice((0, 64, 448)), rot=rot,
                layout=rng.choice((INTERLEAVED, HALF)), dtype=rng.choice(("bf16", "fp32")), scaled=scaled,
                pos=_log(rng, 16, 1048576))


def _contexts(case):
    """The rows' visible tokens, spread over [lo, hi]; the rows of a group end one token apart, as verify rows do."""
    n, lo, hi = case["rows"] // case["group"], case["lo"], case["hi"]
    last = [lo + round((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    last[-1] = hi
    return [max(0, t - (case["group"] - 1 - g)) for t in last for g in range(case["group"])]


def _bytes(fmt):
    return {"fp8": 1, "bf16": 2, "fp32": 4}[fmt]


def work(case):
    if case["op"] == "attend":
        ctx, g = _contexts(case), case["group"]
        heads = case["kv_heads"] * case["hpg"]
        keys = sum(max(ctx[i:i + g]) for i in range(0, len(ctx), g))
        rows = case["rows"] * heads * (case["dim"] * 4 + 4)
        table = 4 * sum(-(-max(ctx[i:i + g]) // case["page"]) for i in range(0, len(ctx), g))
        return {"bytes": keys * case["kv_heads"] * 2 * case["dim"] * _bytes(case["fmt"]) + rows + table,
                "flops": 4 * sum(ctx) * heads * case["dim"]}
    if case["op"] == "insert":
        n, d, kv = case["tokens"], case["dim"], case["kv_heads"]
        q = n * kv * case["hpg"] * case["rot"]
        return {"bytes": n * kv * 2 * d * (2 + _bytes(case["fmt"])) + q * 4 + n * 8,
                "flops": 3 * (q + n * kv * case["rot"]) + 2 * n * kv * d}
    x = case["tokens"] * case["rot"] * (case["heads"] + 2)
    return {"bytes": x * 2 * _bytes(case["dtype"]) + case["tokens"] * 4, "flops": 3 * x}


# ------------------------------------------------------------------ inputs

THETA, FACTOR, TRAINED = 10000.0, 32.0, 4096  # the base, and the stretch of a 4,096-token model's positions


def _frequencies(rot, scaled, device):
    """Radians per position of each pair (64 bits), and the factor on the rotated values."""
    e = torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot
    if scaled == "ntk":
        return torch.pow(THETA * FACTOR ** (rot / max(rot - 2, 1)), -e), 1.0
    f = torch.pow(THETA, -e)
    if scaled == "linear":
        return f / FACTOR, 1.0
    if scaled == "yarn":
        at = [rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(THETA)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64, device=device) - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


K_SCALE, V_SCALE = 1.0 / 72.0, 1.0 / 80.0  # about amax / 448 of normal values


def _pool(case, gen, pages):
    """A pool [pages, KV heads, K and V, page, dim] of normal values."""
    shape = (pages, case["kv_heads"], 2, case["page"], case["dim"])
    if case["fmt"] == "bf16":
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    pool = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
    step = max(1, (1 << 27) // (shape[1] * 2 * shape[3] * shape[4]))
    for p in range(0, pages, step):
        x = torch.randn((min(step, pages - p),) + shape[1:], generator=gen, device="cuda", dtype=torch.bfloat16)
        pool[p:p + step] = (x * 76.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "attend":
        ctx, g, page = _contexts(case), case["group"], case["page"]
        groups = [max(ctx[i:i + g]) for i in range(0, len(ctx), g)]
        s["max_ctx"] = max(max(ctx), 1)
        width = -(-s["max_ctx"] // page)
        need = [-(-t // page) for t in groups]
        pages = sum(need) + max(2, sum(need) // 8)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["table"] = torch.full((len(groups), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        pool = _pool(case, gen, pages)
        bits = pool.view(torch.int16 if case["fmt"] == "bf16" else torch.uint8)
        for i, n in enumerate(need):
            s["table"][i, :n] = order[at:at + n]
            if groups[i] % page:  # slots that hold no token yet are NaN codes
                bits[order[at + n - 1].long(), :, :, groups[i] % page:] = 0x7FFF if case["fmt"] == "bf16" else 0x7F
            at += n
        s["pool"] = pool
        s["row_req"] = torch.arange(len(ctx), device="cuda", dtype=torch.int32) // g
        s["row_ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["q"] = _normal(gen, case["rows"], case["kv_heads"] * case["hpg"], case["dim"])
        s["scales"] = (K_SCALE, V_SCALE) if case["fmt"] == "fp8" else (1.0, 1.0)
        if own:  # the handle, outputs and workspace that a program keeps
            import prefill_dsa_indexer_gb300 as P
            s["kv"] = P.KvCache(pool, *s["scales"])
            heads = case["kv_heads"] * case["hpg"]
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((case["rows"], heads), device="cuda")
            s["ws"] = torch.empty(max(256, P.kv_attention_workspace_size(s["kv"], case["rows"], heads, s["max_ctx"])),
                                  dtype=torch.uint8, device="cuda")
        return s
    n, rot = case["tokens"], case["rot"]
    # tokens of a chunk follow one another; few tokens are of different requests
    if n > 64:
        first = max(0, case["pos"] - n)
        s["positions"] = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
    else:
        s["positions"] = torch.randint(0, case["pos"], (n,), generator=gen, device="cuda", dtype=torch.int32)
    if rot:
        s["freq"], s["factor"] = _frequencies(rot, case["scaled"], "cuda")
        if own:
            import prefill_dsa_indexer_gb300 as P
            s["rope"] = P.rope_table(rot, THETA, scaling=case["scaled"], factor=FACTOR, trained_ctx=TRAINED)
    if case["op"] == "insert":
        kv, d, page = case["kv_heads"], case["dim"], case["page"]
        heads = kv * case["hpg"]
        qkv = _normal(gen, n, heads + 2 * kv, d)  # one projection's output; q, k and v are parts of its rows
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        pages = -(-n // page) + 3
        s["pool"] = _pool(case, gen, pages)
        s["slots"] = torch.randperm(pages * page, generator=gen, device="cuda")[:n].to(torch.int32)
        if n > 64:  # a chunk fills whole pages in order
            order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
            t = torch.arange(n, device="cuda")
            s["slots"] = order[t // page] * page + (t % page).to(torch.int32)
        s["q_out"] = torch.empty((n, heads, rot), dtype=torch.bfloat16, device="cuda") if rot else None
        s["scales"] = (K_SCALE, V_SCALE) if case["fmt"] == "fp8" else (1.0, 1.0)
        if own:
            s["kv"] = _handle(s)
        return s
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    q = _normal(gen, n, case["heads"], case["dim"], dtype=dtype)
    lat = _normal(gen, n, 1, case["dim"], dtype=dtype)
    key = _normal(gen, n, 1, 2 * rot, dtype=dtype)
    # the rotary part: the last dims of each query head and latent, the first of the index key
    s["x"] = [q[..., case["dim"] - rot:], lat[..., case["dim"] - rot:], key[..., :rot]]
    s["layouts"] = [case["layout"], case["layout"], HALF]
    s["out"] = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in s["x"]]
    return s


def _handle(s):
    import prefill_dsa_indexer_gb300 as P
    return P.KvCache(s["pool"], *s["scales"])


# ------------------------------------------------------------------ one pass

def _rotate(x, s, layout):
    """x [tokens, heads, rot] rotated by its tokens' angles, in 32 bits."""
    a = s["positions"].to(torch.float64)[:, None, None] * s["freq"]
    c, d = (torch.cos(a) * s["factor"]).float(), (torch.sin(a) * s["factor"]).float()
    x = x.float()
    if layout == HALF:
        x0, x1 = x.chunk(2, dim=-1)
        return torch.cat((x0 * c - x1 * d, x0 * d + x1 * c), dim=-1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * c - x1 * d, x0 * d + x1 * c), dim=-1).flatten(-2)


def _attend(s):
    case, pool = s["case"], s["pool"]
    R, kv, g, d, page = case["rows"], case["kv_heads"], case["hpg"], case["dim"], case["page"]
    t = torch.arange(s["max_ctx"], device="cuda")
    seen = t[None] < s["row_ctx"][:, None]
    at = s["table"][s["row_req"].long()][:, t // page].clamp_min(0).long()
    bits = pool.view(torch.uint8) if case["fmt"] == "fp8" else pool
    off = (t % page)[None].expand_as(at)
    k = bits[at, :, 0, off].view(pool.dtype).float()  # [R, T, KV heads, d]
    score = torch.matmul(s["q"].float().view(R, kv, g, d), k.permute(0, 2, 3, 1))
    del k
    score = score * ((d ** -0.5) * s["scales"][0])
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], bits[at, :, 1, off].view(pool.dtype).float(), 0.0)
    out = torch.matmul(p, v.transpose(1, 2)) * s["scales"][1]
    out = torch.where(total > 0, out / total, 0.0)
    return {"out": out.reshape(R, kv * g, d).to(torch.bfloat16), "lse": (top + torch.log(total)).reshape(R, kv * g)}


def _insert(s):
    case, pool = s["case"], s["pool"]
    rot, page = case["rot"], case["page"]
    k, v = s["k"].float(), s["v"].float()
    q = None
    if rot:
        k = torch.cat((_rotate(s["k"][..., :rot], s, case["layout"]), k[..., rot:]), dim=-1)
        q = _rotate(s["q"][..., :rot], s, case["layout"]).to(torch.bfloat16)
    at, off = (s["slots"] // page).long(), (s["slots"] % page).long()
    if case["fmt"] == "fp8":
        k, v = (x.div(c).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, c in zip((k, v), s["scales"]))
        bits = pool.view(torch.uint8)
    else:
        k, v, bits = k.to(torch.bfloat16), v.to(torch.bfloat16), pool
    bits[at, :, 0, off] = k
    bits[at, :, 1, off] = v
    return {"pool": pool, "q": q}


def run(s):
    case = s["case"]
    if own:
        import prefill_dsa_indexer_gb300 as P
        if case["op"] == "attend":
            out, lse = P.kv_attention(s["kv"], s["table"], s["row_req"], s["row_ctx"], s["max_ctx"], s["q"],
                                      rows_per_group=case["group"], out=s["out"], lse=s["lse"], workspace=s["ws"])
            return {"out": out, "lse": lse}
        if case["op"] == "insert":
            if not case["rot"]:
                P.kv_insert(s["kv"], s["slots"], s["k"], s["v"])
            else:
                P.kv_insert(s["kv"], s["slots"], s["k"], s["v"], rope=s["rope"], positions=s["positions"],
                            layout=case["layout"], q=s["q"][..., :case["rot"]], q_out=s["q_out"])
            return {"pool": s["pool"], "q": s["q_out"]}
        return P.rope(s["x"], s["rope"], s["positions"], layout=s["layouts"], out=s["out"])
    if case["op"] == "attend":
        return _attend(s)
    if case["op"] == "insert":
        return _insert(s)
    return [_rotate(x, s, layout).to(x.dtype) for x, layout in zip(s["x"], s["layouts"])]


# ------------------------------------------------------------------ in 64 bits

def _angles(s):
    """cos and sin of every token and pair, from the definition, one pair at a time on the host."""
    case = s["case"]
    rot, kind = case["rot"], case["scaled"]
    per, gain = [], 1.0
    for i in range(rot // 2):
        base = THETA * FACTOR ** (rot / max(rot - 2, 1)) if kind == "ntk" else THETA
        w = base ** (-2.0 * i / rot)
        if kind == "linear":
            w = w / FACTOR
        elif kind == "yarn":
            # pairs of fewer than one turn over the trained length are stretched, of more than 32 kept
            edge = lambda turns: rot * math.log(TRAINED / (2 * math.pi * turns)) / (2 * math.log(THETA))  # noqa: E731
            a, b = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), rot - 1)
            mix = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            w = w / FACTOR * mix + w * (1.0 - mix)
            gain = 1.0 + 0.1 * math.log(FACTOR)
        per.append(w)
    turn = torch.outer(s["positions"].double().cpu(), torch.tensor(per, dtype=torch.float64))
    return (gain * torch.cos(turn)).cuda(), (gain * torch.sin(turn)).cuda()


def _turned(x, cos, sin, layout):
    y = x.double().clone()
    n = y.shape[-1] // 2
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if layout == INTERLEAVED else (i, i + n)
        u, w = x[..., a].double(), x[..., b].double()
        y[..., a] = u * cos[:, i:i + 1] - w * sin[:, i:i + 1]
        y[..., b] = u * sin[:, i:i + 1] + w * cos[:, i:i + 1]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        cos, sin = _angles(s)
        return [_turned(x, cos, sin, layout) for x, layout in zip(s["x"], s["layouts"])]
    if case["op"] == "insert":
        k, v, q = s["k"].double(), s["v"].double(), None
        if case["rot"]:
            cos, sin = _angles(s)
            k = torch.cat((_turned(s["k"][..., :case["rot"]], cos, sin, case["layout"]), k[..., case["rot"]:]), -1)
            q = _turned(s["q"][..., :case["rot"]], cos, sin, case["layout"])
        pool = s["pool"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            pool[slot // case["page"], :, 0, slot % case["page"]] = k[i] / s["scales"][0]
            pool[slot // case["page"], :, 1, slot % case["page"]] = v[i] / s["scales"][1]
        if case["fmt"] == "fp8":
            pool = pool.clamp(-448, 448)
        return {"pool": pool, "q": q}
    # attention, one row and KV head at a time over the tokens that it sees
    g, page = case["hpg"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(_contexts(case)):
        if n == 0:
            continue
        pages = s["table"][r // case["group"], :-(-n // page)].long()
        for h in range(case["kv_heads"]):
            kv = s["pool"][pages, h] if case["fmt"] == "bf16" else \
                s["pool"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn)
            k = kv[:, 0].reshape(-1, case["dim"])[:n].double() * s["scales"][0]
            v = kv[:, 1].reshape(-1, case["dim"])[:n].double() * s["scales"][1]
            x = s["q"][r, h * g:(h + 1) * g].double() @ k.T / math.sqrt(case["dim"])
            lse[r, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
            out[r, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}
