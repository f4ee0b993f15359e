"""Paged attention in the corners of its formula, against 64-bit evaluations of it."""
import math

import pytest
import torch

import prefill_dsa_indexer_gb300 as P
from tests.test_gpu_kv_path import Case, bits

pytestmark = pytest.mark.gpu


def weight_error(fmt, dim):
    """A softmax weight as it multiplies V: (relative to itself, against its part's largest).  bf16 pools: two bf16
    terms, 2^-9 2^-8.  FP8 pools: fp16, half a step being 2^-11, with a smallest step of 2^-16 or 2^-24 where the
    largest weight is at least 2^13 or 2^7."""
    if fmt == "bf16":
        return 2.0 ** -16, 0.0
    return 2.0 ** -11, 2.0 ** -29 if dim == 128 else 2.0 ** -32


def check_weights(c, out, lse, rows=None):
    """Case.check with the weights' own errors."""
    for r in range(len(c.rows)) if rows is None else rows:
        n = c.rows[r]
        if n == 0:
            assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
            continue
        for h in range(c.q.shape[1] // c.hpg):
            at = slice(h * c.hpg, (h + 1) * c.hpg)
            k, v = c.tokens(r, h)
            q = c.q[r, at].double()
            s = q @ k.T * c.sm
            p = torch.softmax(s, -1)
            ref, mag = p @ v, p @ v.abs()
            big = (q.abs() @ k.abs().T * c.sm).amax(-1, keepdim=True)
            # scores: fp32 sums; over FP8 pools of head_dim 128 q is two e4m3 terms, which leave 2^-10 where the
            # largest element is above 224; of head_dim 64 fp16, which leaves 2^-25 where it is at least 2^13
            ds = (c.dim + 8) * 2.0 ** -24 * big
            if c.fmt == "fp8":
                step = 2.0 ** -10 / 224 if c.dim == 128 else 2.0 ** -25 / 2 ** 13
                ds = ds + step * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).max() * c.sm
            own, floor = weight_error(c.fmt, c.dim)
            w = own + 2.0 ** -22 + n * 2.0 ** -24
            # (a part's weights against the row's largest: no part has a larger one)
            sub = floor * p.amax(-1, keepdim=True) * v.abs().sum(0)
            bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * ((w + 2 * ds) * mag + sub) + 1e-30
            off = (out[r, at].double() - ref).abs()
            assert (off <= bound).all(), (r, h, (off / bound).max().item())
            want = torch.logsumexp(s, -1)
            lb = ds[:, 0] + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * want.abs()
            assert ((lse[r, at].double() - want).abs() <= lb).all(), (r, h)


# ------------------------------------------------------------------ parts in which a row sees nothing

def shift_scores(c, nats):
    """Every key of the case gets a first element that adds `nats` (negative) to all scores: a constant that the softmax
    does not see."""
    code = -448.0 if c.fmt == "fp8" else -32.0
    c.pool.view(torch.uint8 if c.fmt == "fp8" else torch.int16)[:, :, 0, :, 0] = \
        bits(torch.tensor([code], device="cuda").to(c.pool.dtype)).item()
    c.q[..., 0] = nats / (code * c.ks * c.sm)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nats", [-150.0, -1000.0])
@pytest.mark.parametrize("group, row_ctx", [
    (2, [256, 257]), (2, [257, 256]), (2, [64, 5000, 511, 513]), (4, [8190, 8191, 8192, 8193]),
    (4, [100, 8193, 300, 5000]), (8, [0, 1, 255, 256, 257, 512, 513, 20000])])
@pytest.mark.parametrize("hpg", [2, 16])
def test_rows_whose_last_parts_are_empty(fmt, dim, nats, group, row_ctx, hpg):
    ctx = [max(row_ctx[i:i + group]) for i in range(0, len(row_ctx), group)]
    c = Case(61, fmt, ctx, 2, hpg, dim, 64, group=group, row_ctx=row_ctx)
    shift_scores(c, nats)
    check_weights(c, *c.run())


@pytest.mark.parametrize("dim", [64, 128])
def test_a_part_whose_scores_are_all_minus_infinity(dim):
    c = Case(62, "bf16", [1500], 1, 4, dim, 16)
    shift_scores(c, -200.0)
    hidden = range(256, 512)  # one part of the row
    for t in hidden:
        c.pool[c.table[0, t // 16].item(), :, 0, t % 16, 0] = -math.inf
    out, lse = c.run()
    keep = torch.ones(1500, dtype=torch.bool, device="cuda")
    keep[256:512] = False
    k, v = (x[keep] for x in c.tokens(0, 0))
    s = c.q[0].double() @ k.T * c.sm
    p = torch.softmax(s, -1)
    # fp32 scores of size 200: 2^-24 (dim + 8) of them each; the output's rounding
    ds = (dim + 8) * 2.0 ** -24 * 300
    assert ((out[0].double() - p @ v).abs() <= 2.0 ** -8 * (p @ v).abs() + (2 * ds + 2.0 ** -12) * (p @ v.abs())).all()
    assert ((lse[0].double() - torch.logsumexp(s, -1)).abs() <= ds + 2.0 ** -14).all()


# ------------------------------------------------------------------ rows that are refused on the device

@pytest.mark.parametrize("fmt, dim", [("bf16", 64), ("bf16", 128), ("fp8", 64), ("fp8", 128)])
@pytest.mark.parametrize("bad", ["request below", "request above", "two requests", "context above", "context below"])
def test_a_refused_group_is_answered_with_nothing(fmt, dim, bad):
    """Out is 0 and lse -inf, whatever the workspace holds, and the other groups keep their bits."""
    group = 2
    c = Case(63, fmt, [5000, 9000, 700], 2, 4, dim, 32, group=group)
    need = P.kv_attention_workspace_size(c.kv, 6, 8, c.max_ctx)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    want = [x.clone() for x in c.run(workspace=ws)]
    c.check(*want)
    req, ctx = c.row_req.clone(), c.row_ctx.clone()
    if bad == "request below":
        req[2:4] = -1
    elif bad == "request above":
        req[2:4] = 3
    elif bad == "two requests":
        req[3] = 0
    elif bad == "context above":
        ctx[3] = c.max_ctx + 1
    else:
        ctx[2] = -1
    for fill in (0xFF, None):  # NaN, and what the call before left there
        if fill is not None:
            ws.fill_(fill)
        status = P.new_status()
        out, lse = P.kv_attention(c.kv, c.table, req, ctx, c.max_ctx, c.q, rows_per_group=group, workspace=ws,
                                  status=status)
        torch.cuda.synchronize()
        assert status.item() == P.ERR_BOUNDS
        assert (out[2:4] == 0).all() and (lse[2:4] == -math.inf).all()
        for got, w in zip((out, lse), want):
            assert torch.equal(got[:2], w[:2]) and torch.equal(got[4:], w[4:])
        c.run(workspace=ws)


# ------------------------------------------------------------------ small weights beside large ones

@pytest.mark.parametrize("fmt, dim", [("fp8", 128), ("fp8", 64), ("bf16", 128)])
@pytest.mark.parametrize("kv_heads, hpg, group", [(4, 13, 1), (4, 13, 2), (4, 13, 4), (8, 13, 1), (8, 13, 8)])
@pytest.mark.parametrize("ctx", [500, 32768, 131072])
@pytest.mark.parametrize("noise", [0.0, 0.5])
def test_the_background_behind_an_attention_sink(fmt, dim, kv_heads, hpg, group, ctx, noise):
    """The first token 8 to 20 log2 units ahead of all others, a head each, and values of one sign: the many small
    weights come to as much as the large one."""
    c = Case(64, fmt, [ctx], kv_heads, hpg, dim, 128, group=group)
    raw = bits(c.pool)
    code = lambda x: bits(torch.tensor([x], device="cuda").to(c.pool.dtype)).item()  # noqa: E731
    first = c.table[0, 0].item()
    raw[:, :, 1] = code(64.0)
    raw[first, :, 1, 0] = code(-64.0)
    key = c.pool[:, :, 0].float() * noise
    key[..., 0] = 0.0
    key = key.to(c.pool.dtype)
    key[first, :, 0, 0] = 64.0
    c.pool[:, :, 0].copy_(key) if fmt == "bf16" else raw[:, :, 0].copy_(key.view(torch.uint8))
    ahead = 8.0 + torch.arange(hpg, device="cuda").float().repeat(kv_heads)
    c.q[..., 0] = (ahead * math.log(2.0) / (64.0 * c.ks * c.sm)).to(torch.bfloat16)
    check_weights(c, *c.run(), rows=range(0, group, 3))


@pytest.mark.parametrize("fmt, dim", [("fp8", 128), ("fp8", 64), ("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("kv_heads, hpg, group", [(2, 7, 1), (2, 16, 2), (1, 33, 2), (2, 4, 8), (1, 128, 1)])
@pytest.mark.parametrize("q_scale", [0.3, 1.0, 4.0])
def test_weights_keep_their_bits(fmt, dim, kv_heads, hpg, group, q_scale):
    c = Case(65, fmt, [group + 1, 140, 1000, 6000], kv_heads, hpg, dim, 64, group=group, q_scale=q_scale)
    check_weights(c, *c.run())


# ------------------------------------------------------------------ values that are no numbers

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hpg, group", [(1, 1), (5, 1), (16, 2), (7, 4)])
@pytest.mark.parametrize("ctx", [40, 3000])
def test_infinite_values_that_a_row_sees(dim, hpg, group, ctx):
    """bf16 pools: an infinity of V makes its dim infinite, two of opposite signs make it NaN."""
    c = Case(66, "bf16", [ctx], 2, hpg, dim, 16, group=group)
    at = [(t, d) for d, t in enumerate((0, 3, 17, ctx - group, ctx // 2, ctx // 3))]
    for sign, (t, d) in zip((1, -1, 1, -1, 1, -1), at):
        c.pool[c.table[0, t // 16].item(), :, 1, t % 16, d] = sign * math.inf
    for t, sign in ((5, 1), (30, -1)):
        c.pool[c.table[0, t // 16].item(), :, 1, t % 16, 20] = sign * math.inf
    out, lse = c.run()
    for r in range(group):
        for h in range(2):
            k, v = c.tokens(r, h)
            ref = torch.softmax(c.q[r, h * hpg:(h + 1) * hpg].double() @ k.T * c.sm, -1) @ v
            got = out[r, h * hpg:(h + 1) * hpg].double()
            assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.isnan(ref[:, 20]).all()
            odd = torch.isinf(ref)
            assert torch.equal(torch.isinf(got), odd) and odd.sum() >= 5 * hpg and torch.equal(got[odd], ref[odd])
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("fmt, dim", [("bf16", 64), ("bf16", 128), ("fp8", 64), ("fp8", 128)])
@pytest.mark.parametrize("hpg, group", [(5, 1), (16, 2), (16, 4)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_head_of_no_numbers_leaves_other_groups_their_bits(fmt, dim, hpg, group, value):
    c = Case(49, fmt, [700, 90], 2, hpg, dim, 32, group=group)
    want = c.run()
    q = c.q.clone()
    q[-1, hpg + 2, 3] = value
    got = c.run(q=q)
    for a, b in zip(got, want):
        assert torch.equal(a[:group], b[:group])
        assert torch.equal(a[group:, :hpg], b[group:, :hpg])  # (the other KV head)
    # the other heads of its block: either answer is within its rounding and its weights' of the formula's (values up to
    # 448 / 90 or 6)
    rest = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    rest[-1, hpg + 2] = False
    a, b = (x[0][rest].float() for x in (got, want))
    assert ((a - b).abs() <= 2 * (2.0 ** -8 * b.abs() + 2.0 ** -10 * 6)).all()


# ------------------------------------------------------------------ tensors that share a buffer

def test_rope_takes_parts_of_one_buffer_that_do_not_overlap():
    """Random pairs of tensors in one buffer: refused if and only if an output meets anything but its own input."""
    g = torch.Generator().manual_seed(5)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    table = P.rope_table(8)
    refused = 0
    for case in range(400):
        n, step = pick(1, 4), pick(40, 90)
        buffer = torch.arange(step * 8, device="cuda").to(torch.bfloat16)
        positions = torch.arange(n, device="cuda", dtype=torch.int32)

        def view():
            heads = pick(1, 3)
            head = pick(8, min(16, (step - 8) // max(heads - 1, 1)))
            return buffer.as_strided((n, heads, 8), (step, head, 1), pick(0, step * 3))

        xs = [view(), view()]
        outs = [x if pick(0, 1) else buffer.as_strided(x.shape, x.stride(), pick(0, step * 3)) for x in xs]
        index = torch.arange(buffer.numel())
        used = lambda t: set(index.as_strided(t.shape, t.stride(), t.storage_offset()).flatten().tolist())  # noqa: E731
        meets = bool(used(outs[0]) & used(outs[1]))
        for i in range(2):
            same = outs[i].storage_offset() == xs[i].storage_offset()
            meets |= bool(used(outs[i]) & used(xs[1 - i])) or (not same and bool(used(outs[i]) & used(xs[i])))
        before = buffer.clone()
        if meets:
            refused += 1
            with pytest.raises(P.DsaError):
                P.rope(xs, table, positions, out=outs)
            continue
        want = [P.rope(x.contiguous(), table, positions) for x in xs]
        P.rope(xs, table, positions, out=outs)
        rest = torch.ones_like(buffer, dtype=torch.bool)
        for o, w in zip(outs, want):
            assert torch.equal(o, w), case
            rest.as_strided(o.shape, o.stride(), o.storage_offset()).fill_(False)
        assert torch.equal(buffer[rest], before[rest]), case
    assert 50 < refused < 350


def test_outputs_beside_their_inputs_in_one_buffer():
    """A step whose queries, keys, values, rotated queries and answers are parts of one buffer."""
    c = Case(67, "bf16", [300, 90], 2, 4, 64, 16)
    R, H, D = 2, 8, 64
    wide = R * (3 * H + 2) * D
    buffer = torch.zeros(wide + R * H * D, dtype=torch.bfloat16, device="cuda")
    rows = buffer[:wide].view(R, 3 * H + 2, D)
    q, k, v, turned = rows[:, :H], rows[:, H:H + 2], rows[:, H + 2:H + 4], rows[:, 2 * H:3 * H]
    q.copy_(c.q)
    k.copy_(c.q[:, :2])
    v.copy_(c.q[:, 2:4])
    out = buffer[wide:].view(R, H, D)
    slots = torch.tensor([c.table[r, (n - 1) // 16].item() * 16 + (n - 1) % 16 for r, n in enumerate(c.rows)],
                         dtype=torch.int32, device="cuda")
    positions = (c.row_ctx - 1).contiguous()
    P.kv_insert(c.kv, slots, k, v, rope=P.rope_table(D), positions=positions, q=q, q_out=turned)
    _, lse = P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, turned, out=out)
    c.q = turned.clone()
    check_weights(c, out, lse)
    with pytest.raises(P.DsaError):
        P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, out=c.q)
    with pytest.raises(P.DsaError):
        P.kv_insert(c.kv, slots, k, v, rope=P.rope_table(D), positions=positions, q=q, q_out=rows[:, H - 1:2 * H - 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [P.ROPE_INTERLEAVED, P.ROPE_HALF])
@pytest.mark.parametrize("heads, rot, pad", [(5, 64, 0), (5, 64, 1), (24, 32, 8), (1, 34, 0)])
def test_rope_tiles_of_either_size(dtype, layout, heads, rot, pad):
    """Around the number of pieces (of 16 bytes; of a pair where the rows are not aligned) from which a tile is larger: the
    same bits as the same tokens' in small calls."""
    g = torch.Generator(device="cuda").manual_seed(heads)
    vec = (rot if layout == P.ROPE_INTERLEAVED else rot // 2) % (16 // dtype.itemsize) == 0 and pad != 1
    pieces = rot * dtype.itemsize // (16 if layout == P.ROPE_INTERLEAVED else 32) if vec else rot // 2
    most = -(-(1 << 17) // (heads * pieces))
    table = P.rope_table(rot)
    x = torch.randn((most + 3, heads, pad + rot), generator=g, device="cuda").to(dtype)[..., pad:]
    positions = torch.randint(0, 1 << 20, (most + 3,), generator=g, device="cuda", dtype=torch.int32)
    want = torch.cat([P.rope(x[i:i + 97], table, positions[i:i + 97], layout=layout,
                             out=torch.empty_like(x[i:i + 97], memory_format=torch.contiguous_format))
                      for i in range(0, most + 3, 97)])
    for n in (most - 1, most, most + 3):
        out = torch.full((n, heads, rot), 7.0, dtype=dtype, device="cuda")
        P.rope(x[:n], table, positions[:n], layout=layout, out=out)
        assert torch.equal(out, want[:n])


# ------------------------------------------------------------------ values past a row's context, in many tiles

@pytest.mark.parametrize("fmt, dim", [("fp8", 128), ("fp8", 64), ("bf16", 128)])
@pytest.mark.parametrize("kv_heads, hpg, group, row_ctx", [
    (2, 5, 2, [700, 3000, 128, 129]),                # 10 columns
    (2, 7, 4, [64, 700, 1300, 700, 0, 5, 2000, 257]),  # 28
    (1, 16, 4, [9000, 300, 8999, 4100]),             # 64
    (1, 20, 8, [1, 255, 256, 257, 511, 900, 1400, 40]),  # two blocks of columns and a rest
    (4, 8, 8, [20000, 19999, 19871, 19872, 19873, 5000, 19744, 64])])
def test_nan_values_in_tiles_that_some_rows_see(fmt, dim, kv_heads, hpg, group, row_ctx):
    """NaN in V behind each row's context, in tiles where the others' sums go on: rows keep their bits, and each sees its
    own NaN alone."""
    ctx = [max(row_ctx[i:i + group]) for i in range(0, len(row_ctx), group)]
    make = lambda: Case(68, fmt, ctx, kv_heads, hpg, dim, 32, group=group, row_ctx=row_ctx)  # noqa: E731
    want = make().run()
    nan = {"fp8": 0x7F, "bf16": 0x7FFF}[fmt]
    for at in sorted(set(row_ctx)):
        c = make()
        struck = [r for r, n in enumerate(row_ctx) if n > at]  # token `at` is the first that a row of context `at` misses
        if not struck:
            continue
        for req, longest in enumerate(ctx):
            for t in range(at, longest, 97):  # and many behind it
                bits(c.pool)[c.table[req, t // 32].item(), :, 1, t % 32, 3] = nan
        out, lse = c.run()
        assert torch.equal(lse, want[1])
        for r in range(len(row_ctx)):
            if r in struck:
                assert out[r, :, 3].isnan().all()
                rest = [d for d in range(dim) if d != 3]
                assert torch.equal(out[r][:, rest], want[0][r][:, rest])
            else:
                assert torch.equal(out[r], want[0][r])
