"""What is measured of the batch step around the paged K/V path: the step's rows, slots and pages from request
lengths, rotary positions with several axes, and attention of a batch that shares a long prefix.

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
        # the rows of a decode step of eight requests: one token each, latency is all there is
        dict(name="plan_decode_8", op="plan", requests=8, lo=1, hi=1, cached=131072, page=64, group=1, ended=0,
             segments=1, rows=8, short=False),
        # a verify step of 257 requests with 0 to 4 drafted tokens in groups of four rows; one in nine has ended
        dict(name="plan_verify_257", op="plan", requests=257, lo=0, hi=4, cached=9001, page=16, group=4, ended=9,
             segments=5, rows=1100, short=False),
        # 2,048 requests that get 0 to 15 tokens each, a mixed step into 128-token pages
        dict(name="plan_mixed_2k", op="plan", requests=2048, lo=0, hi=15, cached=16384, page=128, group=1, ended=50,
             segments=64, rows=16384, short=False),
        # a decode step's tokens among an image's: keys into an FP8 pool and queries, time, height and width
        dict(name="axes_insert_8", op="insert", tokens=8, kv_heads=4, hpg=16, dim=128, page=128, fmt="fp8", rot=128,
             layout=HALF, sections="16,24,24", order="split", restart=False, pos=131072),
        # an odd chunk of image patches, height and width with frequencies of their own, half of the dims
        dict(name="axes_insert_333", op="insert", tokens=333, kv_heads=3, hpg=5, dim=64, page=16, fmt="bf16", rot=32,
             layout=INTERLEAVED, sections="8,8", order="split", restart=True, pos=4096),
        # a prefill chunk of 8,192 tokens of text and images on a 56K prefix, axes in turn
        dict(name="axes_rope_8k", op="rope", tokens=8192, heads=96, dim=576, rot=64, layout=INTERLEAVED, dtype="bf16",
             sections="12,10,10", order="cycle", restart=False, pos=65536),
        # four short continuations of one prompt of 2,048 tokens, 16-bit cache
        dict(name="shared_4_2k", op="attend", rows=4, group=1, kv_heads=4, hpg=16, dim=128, page=64, fmt="bf16",
             segments=1, pre_lo=2048, pre_hi=2048, own_lo=1, own_hi=200, pad=0),
        # the batched decode over a common prompt of 32K tokens, FP8 cache
        dict(name="shared_32_32k", op="attend", rows=32, group=1, kv_heads=4, hpg=16, dim=128, page=128, fmt="fp8",
             segments=1, pre_lo=32768, pre_hi=32768, own_lo=100, own_hi=4096, pad=0),
        # 64 samples of one 64K context, 16-bit cache
        dict(name="shared_64_64k", op="attend", rows=64, group=1, kv_heads=4, hpg=8, dim=128, page=64, fmt="bf16",
             segments=1, pre_lo=65536, pre_hi=65536, own_lo=1, own_hi=1000, pad=0),
        # verify rows of sixteen requests over four prompts
        dict(name="shared_verify_4x4x4", op="attend", rows=64, group=4, kv_heads=4, hpg=16, dim=128, page=128,
             fmt="fp8", segments=4, pre_lo=8192, pre_hi=16384, own_lo=10, own_hi=2000, pad=0),
        # a padded batch of 45 rows over five prompts of ragged lengths, an odd number of heads, small pages
        dict(name="shared_ragged_d64", op="attend", rows=45, group=1, kv_heads=3, hpg=5, dim=64, page=16, fmt="bf16",
             segments=5, pre_lo=0, pre_hi=9001, own_lo=1, own_hi=777, pad=3),
        # 256 rows over 64K tokens: the products of the prefix are the whole cost
        dict(name="shared_256_64k", op="attend", rows=256, group=1, kv_heads=4, hpg=16, dim=128, page=128, fmt="fp8",
             segments=1, pre_lo=65536, pre_hi=65536, own_lo=64, own_hi=1024, pad=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _split(rng, pairs):
    """Sections of one to four axes that make up `pairs` pairs."""
    axes = rng.randint(1, min(4, pairs))
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(("attend", "attend", "plan", "insert", "rope"))
    if op == "plan":
        n, group = _log(rng, 1, 2048), rng.choice((1, 1, 2, 4))
        lo = rng.choice((0, 1))
        hi = max(lo, _log(rng, 1, max(1, 16384 // n)))
        rows = max(group, n * -(-hi // group) * group)
        return dict(op=op, requests=n, lo=lo, hi=hi, cached=_log(rng, 16, min(131072, (1 << 26) // n)),
                    page=rng.choice((16, 32, 64, 128)), group=group, ended=rng.choice((0, 2, 9, 50)),
                    segments=rng.randint(0, min(n, 64)), rows=rng.choice((rows, rows + 3 * group, max(1, rows // (2 * group)) * group)),
                    short=rng.choice((False, False, True)))
    if op == "attend":
        group = rng.choice((1, 1, 1, 2, 4))
        rows = group * _log(rng, 1, 256 // group)
        dim, fmt = rng.choice((64, 128)), rng.choice(("bf16", "fp8"))
        kv_heads, hpg = _log(rng, 1, 8), _log(rng, 1, 16)
        segments = rng.randint(1, min(6, rows // group))
        # products and scores within those of the 256 rows, the cache of all rows within 2 GB
        most = min(65536, (1 << 30) // (rows * kv_heads * hpg))
        pre_hi = _log(rng, 1, most)
        own_hi = _log(rng, 1, min(4096, max(1, (1 << 31) // (rows // group * kv_heads * dim * 4))))
        return dict(op=op, rows=rows, group=group, kv_heads=kv_heads, hpg=hpg, dim=dim,
                    page=rng.choice((16, 32, 64, 128)), fmt=fmt, segments=segments,
                    pre_lo=round(pre_hi * rng.choice((0.0, 0.25, 1.0))), pre_hi=pre_hi,
                    own_lo=max(1, round(own_hi * rng.choice((0.0, 0.25, 1.0)))), own_hi=own_hi,
                    pad=rng.choice((0, 0, 1, 5)))
    restart, order = rng.choice((False, True)), rng.choice(("split", "cycle"))
    if op == "insert":
        dim = rng.choice((64, 128))
        rot = rng.choice((dim // 2, dim))
        return dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=_log(rng, 1, 8), hpg=_log(rng, 1, 8), dim=dim,
                    page=rng.choice((16, 32, 64, 128)), fmt=rng.choice(("bf16", "fp8")), rot=rot,
                    layout=rng.choice((INTERLEAVED, HALF)), sections=_split(rng, rot // 2), order=order,
                    restart=restart, pos=_log(rng, 16, 1048576))
    rot = 2 * _log(rng, 4, 64)
    return dict(op=op, tokens=_log(rng, 1, 8192), heads=_log(rng, 1, 96), dim=rot + rng.choice((0, 64, 448)), rot=rot,
                layout=rng.choice((INTERLEAVED, HALF)), dtype=rng.choice(("bf16", "fp32")),
                sections=_split(rng, rot // 2), order=order, restart=restart, pos=_log(rng, 16, 1048576))


def _spread(lo, hi, n, turn):
    """n whole numbers over [lo, hi], the last one hi."""
    v = [lo + round((hi - lo) * ((i * turn) % 1.0)) for i in range(n)]
    return v[:-1] + [hi] if n else v


def _batch(case):
    """(first group of each segment and the end, shared tokens of each, tokens of each request beyond them)."""
    n, k = case["rows"] // case["group"], case["segments"]
    first = [i * n // k for i in range(k + 1)]
    return (first, _spread(case["pre_lo"], case["pre_hi"], k, 0.6180339887498949),
            _spread(case["own_lo"], case["own_hi"], n, 0.7548776662466927))


def _contexts(case):
    """The rows' visible tokens; the rows of a group end one token apart, as verify rows do; padding rows see none."""
    first, pre, beyond = _batch(case)
    ctx = []
    for s in range(case["segments"]):
        for i in range(first[s], first[s + 1]):
            ctx += [max(pre[s] + beyond[i] - (case["group"] - 1 - g), 0) for g in range(case["group"])]
    return ctx + [0] * (case["pad"] * case["group"])


def _bytes(fmt):
    return {"fp8": 1, "bf16": 2, "fp32": 4}[fmt]


def _sections(case):
    """The pairs of each axis."""
    return tuple(int(n) for n in case["sections"].split(","))


def _axis_of(case):
    """The axis of each pair: the axes' sections one after another, or the axes in turn while they have pairs left."""
    sections = _sections(case)
    if case["order"] == "split":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def work(case):
    if case["op"] == "plan":
        n, new = case["requests"], case["requests"] * (case["lo"] + case["hi"]) // 2
        # lengths in and out, grants, starts; four numbers a row; a page id in and out for each page begun
        return {"bytes": 4 * (6 * n + 4 * case["rows"] + 3 * (new // case["page"])), "flops": case["rows"]}
    if case["op"] == "attend":
        ctx, g = _contexts(case), case["group"]
        first, pre, beyond = _batch(case)
        heads = case["kv_heads"] * case["hpg"]
        tokens = sum(pre) + sum(beyond)
        rows = len(ctx) * heads * (case["dim"] * 4 + 4)
        table = 4 * (sum(-(-t // case["page"]) for t in pre) + sum(-(-t // case["page"]) for t in beyond))
        return {"bytes": tokens * case["kv_heads"] * 2 * case["dim"] * _bytes(case["fmt"]) + rows + table,
                "flops": 4 * sum(ctx) * heads * case["dim"]}
    if case["op"] == "insert":
        n, d, kv = case["tokens"], case["dim"], case["kv_heads"]
        q = n * kv * case["hpg"] * case["rot"]
        return {"bytes": n * kv * 2 * d * (2 + _bytes(case["fmt"])) + q * 4 + n * 4 * (1 + len(_sections(case))),
                "flops": 3 * (q + n * kv * case["rot"]) + 2 * n * kv * d}
    x = case["tokens"] * case["rot"] * (case["heads"] + 2)
    return {"bytes": x * 2 * _bytes(case["dtype"]) + case["tokens"] * 4 * len(_sections(case)), "flops": 3 * x}


# ------------------------------------------------------------------ inputs

THETA = 10000.0
K_SCALE, V_SCALE = 1.0 / 72.0, 1.0 / 80.0  # about amax / 448 of normal values


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


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


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_plan(case, gen):
    n, page = case["requests"], case["page"]
    s = dict(case=case)
    s["context"] = torch.randint(0, case["cached"] + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    s["new"] = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    i = torch.arange(n, device="cuda")
    if case["ended"]:
        s["new"][i % case["ended"] == case["ended"] // 2] = -1
    had = (s["context"] + page - 1) // page
    # the first quarter of every third request's pages belongs to a shared prefix
    s["first_own"] = torch.where(i % 3 == 0, had // 4, 0).to(torch.int32)
    width = -(-(case["cached"] + case["hi"]) // page)
    pages = n * width
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    listed = torch.arange(width, device="cuda")[None] < had[:, None]
    s["table"] = torch.where(listed, order.view(n, width), -1).contiguous()
    # the pages that no table lists are free
    free = order[~listed.flatten()]
    count = free.numel()
    if case["short"]:  # about half of what the step asks for
        count = min(count, max(0, n * (case["lo"] + case["hi"]) // (4 * page)))
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:count] = free[:count]
    s["count"] = _int([count])
    s["segments"] = _int([j * n // case["segments"] for j in range(case["segments"] + 1)]) if case["segments"] else None
    s["num_pages"] = pages
    if own:  # the outputs that a program keeps
        import prefill_dsa_indexer_gb300 as P
        s["plan"] = P.KvPlan(n, case["rows"], page, pages, rows_per_group=case["group"],
                             num_segments=case["segments"])
    return s


def _prepare_attend(case, gen):
    page, g = case["page"], case["group"]
    s = dict(case=case)
    first, pre, beyond = _batch(case)
    ctx = _contexts(case)
    total = [pre[k] + beyond[i] for k in range(case["segments"]) for i in range(first[k], first[k + 1])]
    s["max_ctx"] = max(max(total), 1)
    width = -(-s["max_ctx"] // page)
    # whole pages of the shared tokens are listed by every request of the segment; what lies behind them, the rest of
    # the shared tokens among it, is in pages of the request's own
    whole = [p // page for p in pre]
    need = sum(whole) + sum(-(-total[i] // page) - whole[k] for k in range(case["segments"])
                            for i in range(first[k], first[k + 1]))
    pages = need + 2
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    pool = _pool(case, gen, pages)
    bits = pool.view(torch.int16 if case["fmt"] == "bf16" else torch.uint8)
    table = torch.full((len(total), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for k in range(case["segments"]):
        common = order[at:at + whole[k]]
        at += whole[k]
        rest = pre[k] - whole[k] * page
        kept = None
        for i in range(first[k], first[k + 1]):
            mine = order[at:at + -(-total[i] // page) - whole[k]]
            at += mine.numel()
            table[i, :whole[k]] = common
            table[i, whole[k]:whole[k] + mine.numel()] = mine
            if rest:  # the shared tokens of the page that is begun are the same in every request's copy of it
                if kept is None:
                    kept = bits[mine[0].long(), :, :, :rest].clone()
                bits[mine[0].long(), :, :, :rest] = kept
            if total[i] % page:  # slots that hold no token yet are NaN codes
                last = mine[-1] if mine.numel() else common[-1]
                bits[last.long(), :, :, total[i] % page:] = 0x7FFF if case["fmt"] == "bf16" else 0x7F
    s["pool"], s["table"] = pool, table
    s["row_req"] = _int([min(r // g, len(total) - 1) if c else 0 for r, c in enumerate(ctx)])
    s["row_ctx"] = _int(ctx)
    s["segment_rows"], s["segment_ctx"] = _int([f * g for f in first]), _int(pre)
    heads = case["kv_heads"] * case["hpg"]
    s["q"] = _normal(gen, len(ctx), heads, case["dim"])
    s["scales"] = (K_SCALE, V_SCALE) if case["fmt"] == "fp8" else (1.0, 1.0)
    if own:  # the handle, outputs and workspace that a program keeps
        import prefill_dsa_indexer_gb300 as P
        s["kv"] = P.KvCache(pool, *s["scales"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((len(ctx), heads), device="cuda")
        size = P.kv_attention_shared_workspace_size(s["kv"], len(ctx), heads, s["max_ctx"], case["segments"])
        s["ws"] = torch.empty(max(256, size), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, gen)
    if case["op"] == "attend":
        return _prepare_attend(case, gen)
    s = dict(case=case)
    n, rot, axes = case["tokens"], case["rot"], len(_sections(case))
    # few tokens are of different requests; a chunk is a third of text, whose axes agree, and patches of images in rows
    # of 40 at one time
    if n > 64:
        text, i = n // 3, torch.arange(n, device="cuda", dtype=torch.int32)
        first = max(0, case["pos"] - n)
        at = torch.where(i < text, i, text)
        patch = (i - text).clamp_min(0)
        grid = [torch.zeros_like(i), patch // 40, patch % 40, patch // 1600]
        s["positions"] = torch.stack([first + at + (grid[a] if axes > 1 else patch) for a in range(axes)])
    else:
        s["positions"] = torch.randint(0, case["pos"], (axes, n), generator=gen, device="cuda", dtype=torch.int32)
    axis = _axis_of(case)
    if case["restart"]:  # each axis counts its own pairs
        e = [axis[:i].count(a) / _sections(case)[a] for i, a in enumerate(axis)]
    else:
        e = [2 * i / rot for i in range(rot // 2)]
    s["freq"] = torch.pow(THETA, -torch.tensor(e, dtype=torch.float64, device="cuda"))
    s["axis"] = torch.tensor(axis, device="cuda")
    if own:
        import prefill_dsa_indexer_gb300 as P
        s["rope"] = P.rope_table(rot, THETA, sections=_sections(case), order=case["order"], restart=case["restart"])
    if case["op"] == "insert":
        kv, d, page = case["kv_heads"], case["dim"], case["page"]
        heads = kv * case["hpg"]
        qkv = _normal(gen, n, heads + 2 * kv, d)  # one projection's output; q, k and v are parts of its rows
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        pages = -(-n // page) + 3
        s["pool"] = _pool(case, gen, pages)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        t = torch.arange(n, device="cuda")
        s["slots"] = order[t // page] * page + (t % page).to(torch.int32)
        s["q_out"] = torch.empty((n, heads, rot), dtype=torch.bfloat16, device="cuda")
        s["scales"] = (K_SCALE, V_SCALE) if case["fmt"] == "fp8" else (1.0, 1.0)
        if own:
            s["kv"] = P.KvCache(s["pool"], *s["scales"])
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


# ------------------------------------------------------------------ one pass

def _plan(s):
    """Whole-number torch operations on [requests, pages] and [rows]."""
    case, table = s["case"], s["table"]
    page, group, rows = case["page"], case["group"], case["rows"]
    ctx, new = s["context"].long(), s["new"].long()
    ended = new == -1
    had = (ctx + page - 1) // page
    k = torch.arange(table.shape[1], device="cuda")[None]
    # what ended requests give back goes on the stack of free pages, in order
    back = torch.where(ended, (had - s["first_own"]).clamp_min(0), 0)
    place = s["count"] + (back.cumsum(0) - back)[:, None] + k - s["first_own"][:, None]
    given = ended[:, None] & (k >= s["first_own"][:, None]) & (k < had[:, None])
    stack = torch.cat((s["free"], s["free"].new_zeros(1)))
    stack[torch.where(given, place, s["free"].numel())] = table
    free = stack[:-1]
    count = s["count"] + back.sum()
    # pages and rows of the others; who comes behind the last page or row gets none
    n = torch.where(ended, 0, new)
    need = (ctx + n + page - 1) // page - had
    need = torch.where(ended, 0, need)
    wide = (n + group - 1) // group * group
    pages_end, rows_end = need.cumsum(0), wide.cumsum(0)
    ok = ((need == 0) | (pages_end <= count)) & ((wide == 0) | (rows_end <= rows)) & ~ended
    granted = torch.where(ok, n, 0)
    start = torch.cat((rows_end.new_zeros(1), rows_end)).clamp_max(rows)
    nth = (pages_end - need)[:, None] + k - had[:, None]
    taken = ok[:, None] & (k >= had[:, None]) & (k < (had + need)[:, None])
    table = torch.where(taken, free[(count - 1 - nth).clamp(0, free.numel() - 1)], table)
    r = torch.arange(rows, device="cuda")
    req = torch.searchsorted(rows_end, r, right=True)
    inside = req < ctx.numel()
    req = torch.where(inside, req, 0)
    j = r - (rows_end - wide)[req]
    live = inside & (j < granted[req])
    pos = torch.where(live, ctx[req] + j, -1)
    p = pos.clamp_min(0)
    slot = torch.where(live, table[req, (p // page).clamp_max(table.shape[1] - 1)] * page + p % page, -1)
    out = dict(row_req=req, row_ctx=pos + 1, positions=pos, slots=slot, row_start=start, granted=granted,
               context=torch.where(ended, 0, ctx + granted), free_count=count - torch.where(ok, need, 0).sum(),
               block_table=table, free_pages=free)
    out["segment_rows"] = start[s["segments"].long()] if s["segments"] is not None else start[:0]
    return {name: x.to(torch.int32) for name, x in out.items()}


def _rotate(x, s, layout):
    """x [tokens, heads, rot] rotated by its tokens' angles, in 32 bits."""
    a = (s["positions"].to(torch.float64)[s["axis"]].T * s["freq"])[:, None]
    c, d = torch.cos(a).float(), torch.sin(a).float()
    x = x.float()
    if layout == HALF:
        x0, x1 = x.chunk(2, dim=-1)
        return torch.cat((x0 * c - x1 * d, x0 * d + x1 * c), dim=-1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * c - x1 * d, x0 * d + x1 * c), dim=-1).flatten(-2)


def _insert(s):
    case, pool = s["case"], s["pool"]
    rot, page = case["rot"], case["page"]
    v = s["v"].float()
    k = torch.cat((_rotate(s["k"][..., :rot], s, case["layout"]), s["k"][..., rot:].float()), dim=-1)
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


def _attend(s):
    """A segment at a time: its shared tokens against all of its rows, each request's others against its own rows."""
    case, pool = s["case"], s["pool"]
    kv, g, d, page, group = case["kv_heads"], case["hpg"], case["dim"], case["page"], case["group"]
    first, pre, beyond = _batch(case)
    bits = pool.view(torch.uint8) if case["fmt"] == "fp8" else pool
    out = torch.zeros((s["q"].shape[0], kv, g, d), device="cuda")
    lse = torch.full((s["q"].shape[0], kv, g), -math.inf, device="cuda")
    for i in range(case["segments"]):
        a, b, n = first[i], first[i + 1], pre[i]
        rows, m = slice(a * group, b * group), max(beyond[a:b])
        q = s["q"][rows].float().view(b - a, group, kv, g, d) * (d ** -0.5 * s["scales"][0])
        q = q.permute(2, 0, 1, 3, 4).reshape(kv, -1, d)                     # [KV heads, requests x rows x heads, d]
        t = torch.arange(n, device="cuda")
        at, off = s["table"][a, t // page].long(), t % page
        k, v = (bits[at, :, y, off].view(pool.dtype).float().transpose(0, 1) for y in (0, 1))
        ctx = s["row_ctx"][rows].view(1, b - a, group, 1, 1)
        seen = t < ctx
        x = torch.matmul(q, k.transpose(1, 2)).view(kv, b - a, group, g, n)
        x = torch.where(seen, x, -math.inf)
        t = torch.arange(n, n + m, device="cuda")
        at, off = s["table"][a:b, (t // page).clamp_max(s["table"].shape[1] - 1)].clamp_min(0).long(), t % page
        off = off.expand_as(at)
        seen = t < ctx
        ko, vo = (bits[at, :, y, off].view(pool.dtype).float().permute(2, 0, 1, 3) for y in (0, 1))
        y = torch.matmul(q.view(kv, b - a, group * g, d), ko.transpose(2, 3)).view(kv, b - a, group, g, m)
        y = torch.where(seen, y, -math.inf)
        vo = torch.where(t[None, :, None] < ctx.amax(2)[:, :, :, 0, None], vo, 0.0)
        top = torch.maximum(x.amax(-1, keepdim=True) if n else y.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
        base = torch.where(top == -math.inf, 0.0, top)
        x, y = torch.exp(x - base), torch.exp(y - base)
        total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = torch.matmul(x.reshape(kv, (b - a) * group * g, n), v).view(kv, b - a, group, g, d)
        o = o + torch.matmul(y.view(kv, b - a, group * g, m), vo).view(o.shape)
        o = torch.where(total > 0, o * s["scales"][1] / total, 0.0)
        out[rows] = o.permute(1, 2, 0, 3, 4).reshape(-1, kv, g, d)
        lse[rows] = (top + torch.log(total))[..., 0].permute(1, 2, 0, 3).reshape(-1, kv, g)
    return {"out": out.to(torch.bfloat16).view(s["q"].shape), "lse": lse.view(s["q"].shape[:2])}


def run(s):
    case = s["case"]
    if own:
        import prefill_dsa_indexer_gb300 as P
        if case["op"] == "plan":
            p = s["plan"]
            p.run(s["context"], s["new"], s["table"], s["free"], s["count"], first_own=s["first_own"],
                  segment_requests=s["segments"])
            return dict(row_req=p.row_req, row_ctx=p.row_ctx, positions=p.positions, slots=p.slots,
                        row_start=p.row_start, granted=p.granted, context=p.context, free_count=p.free_count[0],
                        block_table=s["table"], free_pages=s["free"], segment_rows=p.segment_rows)
        if case["op"] == "attend":
            out, lse = P.kv_attention_shared(s["kv"], s["table"], s["row_req"], s["row_ctx"], s["max_ctx"], s["q"],
                                             s["segment_rows"], s["segment_ctx"], rows_per_group=case["group"],
                                             out=s["out"], lse=s["lse"], workspace=s["ws"])
            return {"out": out, "lse": lse}
        if case["op"] == "insert":
            P.kv_insert(s["kv"], s["slots"], s["k"], s["v"], rope=s["rope"], positions=s["positions"],
                        layout=case["layout"], q=s["q"][..., :case["rot"]], q_out=s["q_out"])
            return {"pool": s["pool"], "q": s["q_out"]}
        return P.rope(s["x"], s["rope"], s["positions"], layout=s["layouts"], out=s["out"])
    if case["op"] == "plan":
        out = _plan(s)
        out["free_count"] = out["free_count"][0]
        return out
    if case["op"] == "attend":
        return _attend(s)
    if case["op"] == "insert":
        return _insert(s)
    return [_rotate(x, s, layout).to(x.dtype) for x, layout in zip(s["x"], s["layouts"])]


# ------------------------------------------------------------------ from the definitions

def _exact_plan(s):
    """One request after another, on the host."""
    case = s["case"]
    page, group, rows = case["page"], case["group"], case["rows"]
    table, free, count = s["table"].tolist(), s["free"].tolist(), int(s["count"])
    ctx, new, kept = s["context"].tolist(), s["new"].tolist(), s["first_own"].tolist()
    for i, n in enumerate(new):
        if n == -1:
            for p in table[i][kept[i]:-(-ctx[i] // page)]:
                free[count] = p
                count += 1
    o = dict(row_req=[], positions=[], slots=[], row_start=[0], granted=[], context=[])
    asked, row, taken = 0, 0, 0
    for i, n in enumerate(new):
        if n == -1:
            o["granted"].append(0)
            o["context"].append(0)
            o["row_start"].append(min(row, rows))
            continue
        need, wide = -(-(ctx[i] + n) // page) - -(-ctx[i] // page), -(-n // group) * group
        asked, row = asked + need, row + wide
        ok = (need == 0 or asked <= count) and (wide == 0 or row <= rows)
        if ok:
            for j in range(need):
                table[i][-(-ctx[i] // page) + j] = free[count - 1 - taken - j]
            taken += need
        o["granted"].append(n if ok else 0)
        o["context"].append(ctx[i] + o["granted"][-1])
        for j in range(wide):
            if len(o["row_req"]) < rows:
                pos = ctx[i] + j if j < o["granted"][-1] else -1
                o["row_req"].append(i)
                o["positions"].append(pos)
                o["slots"].append(table[i][pos // page] * page + pos % page if pos >= 0 else -1)
        o["row_start"].append(min(row, rows))
    more = rows - len(o["row_req"])
    o["row_req"] += [0] * more
    o["positions"] += [-1] * more
    o["slots"] += [-1] * more
    o["row_ctx"] = [p + 1 for p in o["positions"]]
    o["segment_rows"] = [o["row_start"][j] for j in s["segments"].tolist()] if s["segments"] is not None else []
    o.update(free_count=count - taken, block_table=table, free_pages=free)
    return {name: _int(x) for name, x in o.items()}


def _angles(s):
    """cos and sin of every token and pair, from the definition, one pair at a time on the host."""
    case = s["case"]
    left = {a: 0 for a in range(len(_sections(case)))}
    cos, sin = [], []
    for i, a in enumerate(_axis_of(case)):
        w = THETA ** (-left[a] / _sections(case)[a] if case["restart"] else -2.0 * i / case["rot"])
        left[a] += 1
        t = s["positions"][a].cpu().double() * w
        cos.append(torch.cos(t))
        sin.append(torch.sin(t))
    return torch.stack(cos, 1).cuda(), torch.stack(sin, 1).cuda()


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
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "rope":
        cos, sin = _angles(s)
        return [_turned(x, cos, sin, layout) for x, layout in zip(s["x"], s["layouts"])]
    if case["op"] == "insert":
        cos, sin = _angles(s)
        rot, page = case["rot"], case["page"]
        k = torch.cat((_turned(s["k"][..., :rot], cos, sin, case["layout"]), s["k"][..., rot:].double()), -1)
        q, v, pool = _turned(s["q"][..., :rot], cos, sin, case["layout"]), s["v"].double(), s["pool"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            pool[slot // page, :, 0, slot % page] = k[i] / s["scales"][0]
            pool[slot // page, :, 1, slot % page] = v[i] / s["scales"][1]
        return {"pool": pool.clamp(-448, 448) if case["fmt"] == "fp8" else pool, "q": q}
    # attention, one row and KV head at a time over the tokens that the row's own table lists
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
