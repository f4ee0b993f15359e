"""A batch's rows, slots and pages from request lengths (dsa_kv_plan) on the GPU against plain whole numbers, and rotary
positions with several axes (dsa_rope_with_axes, dsa_kv_insert_with_axes) against their formulas in 64 bits."""
import random

import pytest
import torch

import prefill_dsa_indexer_gb300 as P
from tests.test_gpu_kv_path import bits, checked, gen, new_pool, randn, ref_rotate, rope_bound

pytestmark = pytest.mark.gpu


def ints(values, shape=None):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


# ------------------------------------------------------------------ plans

class Step:
    """A step's requests, and what it has to make of them, one request after another."""

    def __init__(self, context, new, page, rows, group=1, first_own=None, free=None, count=None, segments=None,
                 width=None, pages=None):
        self.context, self.new, self.page, self.rows, self.group = context, new, page, rows, group
        n = len(context)
        had = [max(0, -(-c // page)) for c in context]
        self.width = width or max([1] + [-(-(max(c, 0) + max(t, 0)) // page) for c, t in zip(context, new)])
        rng = random.Random(n * 1000 + page + rows)
        self.pages = pages or n * self.width + 8
        ids = list(range(self.pages))
        rng.shuffle(ids)
        self.table = [[-7] * self.width for _ in range(n)]
        for i in range(n):
            for p in range(min(had[i], self.width)):
                self.table[i][p] = ids.pop()
        self.free = [-9] * (self.pages if free is None else free)
        self.count = min(len(ids), len(self.free)) if count is None else count
        for k in range(max(0, min(self.count, len(self.free)))):
            self.free[k] = ids.pop()
        self.first_own, self.segments = first_own, segments

    def want(self):
        page, rows, group = self.page, self.rows, self.group
        table, free, count = [list(r) for r in self.table], list(self.free), self.count
        bad = count < 0 or count > len(free)
        count = min(max(count, 0), len(free))
        fresh = []
        for i, (c, n) in enumerate(zip(self.context, self.new)):
            own = self.first_own[i] if self.first_own else 0
            wrong = c < 0 or c > self.width * page or n < -1 or c + n > self.width * page or own < 0
            bad |= wrong
            fresh.append(0 if wrong or n == -1 else n)
            if n == -1 and not wrong:
                for p in table[i][own:-(-c // page)]:
                    if count < len(free):
                        free[count] = p
                        count += 1
                    else:
                        bad = True
        o = dict(row_req=[], positions=[], slots=[], row_start=[0], granted=[], context=[])
        asked = row = taken = 0
        for i, (c, n) in enumerate(zip(self.context, fresh)):
            need, wide = -(-(c + n) // page) - -(-c // page), -(-n // group) * group
            asked, row = asked + need, row + wide
            ok = (need == 0 or asked <= count) and (wide == 0 or row <= rows)
            if ok:
                for j in range(need):
                    table[i][-(-c // page) + j] = free[count - 1 - taken - j]
                taken += need
            o["granted"].append(n if ok else 0)
            o["context"].append(0 if self.new[i] == -1 else c + o["granted"][-1])
            for j in range(wide):
                if len(o["row_req"]) < rows:
                    pos = c + j if j < o["granted"][-1] else -1
                    slot = -1
                    if pos >= 0:
                        if 0 <= table[i][pos // page] < self.pages:
                            slot = table[i][pos // page] * page + pos % page
                        else:
                            bad = True
                    o["row_req"].append(i)
                    o["positions"].append(pos)
                    o["slots"].append(slot)
            o["row_start"].append(min(row, rows))
        more = rows - len(o["row_req"])
        o["row_req"] += [0] * more
        o["positions"] += [-1] * more
        o["slots"] += [-1] * more
        o["row_ctx"] = [p + 1 for p in o["positions"]]
        o["free_count"], self.bad = [count - taken], bad
        if self.segments is not None:
            o["segment_rows"] = []
            for s in self.segments:
                self.bad |= s < 0 or s > len(self.context)
                o["segment_rows"].append(o["row_start"][min(max(s, 0), len(self.context))])
        return o, table, free

    def tensors(self):
        n = len(self.context)
        return (ints(self.context, (n,)), ints(self.new, (n,)), ints(self.table, (n, self.width)),
                ints(self.free, (len(self.free),)), ints([self.count]))

    def plan(self):
        return P.KvPlan(len(self.context), self.rows, self.page, self.pages, self.group,
                        len(self.segments) - 1 if self.segments else 0)

    def check(self, plan, table, free):
        o, t, f = self.want()
        torch.cuda.synchronize()
        for name, v in o.items():
            assert getattr(plan, name).tolist() == v, name
        assert table.tolist() == t and free.tolist() == f
        assert plan.status.item() == (P.ERR_BOUNDS if self.bad else P.OK)

    def run(self):
        context, new, table, free, count = self.tensors()
        plan = self.plan()
        plan.run(context, new, table, free, count, None if self.first_own is None else ints(self.first_own),
                 None if self.segments is None else ints(self.segments))
        self.check(plan, table, free)
        assert context.tolist() == self.context and count.tolist() == [self.count]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_plan_of_a_few_requests(page, group):
    context = [0, 1, page - 1, page, page + 1, 5 * page, 3 * page - 2, 0, 7]
    new = [1, 0, 1, 1, page, 3 * page + 1, 2, -1, -1]
    step = Step(context, new, page, 8 * page, group, first_own=[0, 0, 0, 0, 0, 0, 0, 0, 1], segments=[0, 0, 3, 8, 9])
    step.run()


@pytest.mark.parametrize("n, page, group, most, rows", [
    (1, 16, 1, 1, 1), (1, 128, 1, 9001, 9001), (31, 16, 4, 5, 300), (33, 64, 1, 40, 700), (1000, 16, 2, 3, 3000),
    (1025, 32, 1, 20, 12000), (2049, 128, 8, 8, 16400), (16384, 16, 1, 2, 20000), (5000, 64, 1, 1, 1024),
    (300, 64, 1, 200, 1032)])
def test_plan_of_many_requests(n, page, group, most, rows):
    rng = random.Random(n + page)
    context = [rng.randint(0, 40 * page) for _ in range(n)]
    new = [rng.choice((-1, 0, rng.randint(0, most), most)) for _ in range(n)]
    own = [rng.choice((0, 0, 3, 50)) for _ in range(n)]
    cuts = sorted(rng.randint(0, n) for _ in range(min(n, 20) + 1))
    Step(context, new, page, rows // group * group, group, first_own=own, segments=cuts).run()


@pytest.mark.parametrize("count", [0, 1, 2, 5, 6, 7])
def test_plan_with_too_few_pages(count):
    """Requests get their pages in order until one does not fit; those that need none go on."""
    step = Step([16, 3, 32, 17, 48, 5, 64], [1, 4, 33, 2, 17, 0, 1], 16, 64, count=count)
    step.run()
    assert not step.bad


@pytest.mark.parametrize("rows", [0, 1, 5, 8, 9, 40, 41, 64])
@pytest.mark.parametrize("group", [1, 2])
def test_plan_with_too_few_rows(rows, group):
    Step([16, 3, 32, 0, 17], [5, 4, 33, 0, 1], 16, rows // group * group, group).run()


def test_plan_gives_pages_on_that_ended_requests_gave_back():
    step = Step([100, 40, 33, 16], [-1, 30, -1, 60], 16, 128, first_own=[2, 0, 0, 0], count=1)
    step.run()
    Step([100, 40, 33, 16], [-1, 30, -1, 60], 16, 128, count=0).run()
    step = Step([100, 40], [-1, 0], 16, 8, free=4, count=2)  # the stack is too short
    step.run()
    assert step.bad


@pytest.mark.parametrize("free", [None, 30000])
def test_plan_takes_back_the_pages_of_long_requests(free):
    """Runs of them much longer than what a warp goes through at once, beside short and empty ones; or more than the stack
    has room for."""
    rng = random.Random(9)
    context = [rng.choice((0, 1, 500, 40000 + 17 * i, 16 * 257)) for i in range(60)]
    new = [-1 if i % 3 else rng.randint(0, 200) for i in range(60)]
    Step(context, new, 16, 4000, first_own=[rng.choice((0, 5, 300)) for _ in range(60)], free=free, count=free and 29000).run()


def test_plan_refuses_lengths_that_cannot_be():
    for context, new, extra in (([-1, 20], [3, 4], {}), ([5, 20], [-2, 4], {}), ([40, 20], [9, 13], dict(width=2)),
                                ([33, 20], [-1, 4], dict(width=2)), ([5, 20], [2147483647, 4], dict(width=4)),
                                ([5, 20], [-1, 4], dict(first_own=[-1, 0])), ([20, 5], [1, 2], dict(segments=[-1, 3])),
                                ([-2147483648, 20], [-1, 4], {}), ([20, 5], [4, 2], dict(count=-3)),
                                ([20, 5], [40, 2], dict(free=3, count=9))):
        step = Step(context, new, 16, 64, **extra) if new[0] < 1 << 20 else Step(context, [0, 4], 16, 64, **extra)
        step.new = new
        step.run()
        assert step.bad, (context, new)
    step = Step([20, 5, 16], [4, 2, 1], 16, 16)
    step.pages = 1  # most ids are outside such a pool
    step.run()
    assert step.bad
    context, new, table, free, count = Step([16, 16], [1, 1], 16, 4, count=1).tensors()
    rows, status = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), P.new_status()
    P.kv_plan(context, new, table, free, count, 16, 100, rows[0], rows[1], status=status)  # no `granted` to tell
    assert status.item() == P.ERR_BOUNDS and rows.tolist() == [[0, 1, 0, 0], [17, 0, 0, 0]]


@pytest.mark.parametrize("wrong", ["first_own", "context"])
def test_pages_of_an_ended_request_with_lengths_that_cannot_be_can_be_given_back(wrong):
    """Contexts in place: the request ends without giving a page back, its row of the table still lists them, and a call
    with its lengths put right gives them back, to the next request that needs some."""
    first = Step([70, 20, 5], [-1, 40, 1], 16, 64, first_own=[1, 0, 0], width=5, count=3)
    context, new, table, free, count = first.tensors()
    plan, own = first.plan(), ints([1, 0, 0])
    plan.context.copy_(context)
    plan.free_count.copy_(count)
    if wrong == "first_own":
        first.first_own[0] = own[0] = -1
    else:
        first.context[0] = plan.context[0] = 81  # the table lists 80
    plan.run(plan.context, new, table, free, plan.free_count, own)
    first.check(plan, table, free)
    assert first.bad and plan.context.tolist() == [0, 60, 6] and table[0].tolist() == first.table[0]
    assert plan.free_count.item() == 1
    plan.context[0], own[0] = 70, 1
    plan.status.zero_()
    again = Step([70, 60, 6], [-1, 5, 60], 16, 96, first_own=[1, 0, 0], width=5, pages=first.pages)
    again.table, again.free, again.count = table.tolist(), free.tolist(), 1
    new.copy_(ints(again.new))
    plan = again.plan()
    plan.context.copy_(ints(again.context))
    plan.free_count.fill_(1)
    plan.run(plan.context, new, table, free, plan.free_count, own)
    again.check(plan, table, free)
    assert not again.bad and plan.granted.tolist() == [0, 5, 60] and plan.free_count.item() == 0


def test_plan_without_requests_or_rows():
    Step([], [], 16, 5, free=3, count=2).run()
    Step([], [], 16, 0, free=0, count=0).run()
    Step([4, 5], [0, 0], 16, 0, segments=[0, 2]).run()


@pytest.mark.parametrize("n, most", [(5, 40), (1500, 9)])
@pytest.mark.parametrize("graph", [False, True])
def test_plans_that_follow_one_another_in_place(n, most, graph):
    """Contexts and the count of free pages are the plan's own of the step before."""
    rng = random.Random(n)
    page, steps = 16, 5
    context = [rng.randint(0, 60) for _ in range(n)]
    first = Step(context, [0] * n, page, 8 * n, width=-(-(60 + steps * most) // page))
    context, new, table, free, count = first.tensors()
    plan = first.plan()
    plan.context.copy_(context)
    plan.free_count.copy_(count)
    step = lambda: plan.run(plan.context, new, table, free, plan.free_count)  # noqa: E731
    if graph:
        saved = [t.clone() for t in (plan.context, table, free, plan.free_count)]
        with torch.cuda.stream(torch.cuda.Stream()):
            step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for t, v in zip((plan.context, table, free, plan.free_count), saved):
            t.copy_(v)
    for _ in range(steps):
        now = Step(first.context, [rng.choice((-1, 0, 1, most)) for _ in range(n)], page, first.rows,
                   width=first.width, pages=first.pages)
        now.table, now.free, now.count = table.tolist(), free.tolist(), plan.free_count.item()
        new.copy_(ints(now.new))
        captured.replay() if graph else step()
        now.check(plan, table, free)
        first.context = plan.context.tolist()


def test_plan_refusals_of_the_binding():
    step = Step([4, 5], [1, 2], 16, 4, segments=[0, 2])
    plan, (context, new, table, free, count) = step.plan(), step.tensors()
    seg = ints(step.segments)
    call = lambda **k: plan.run(**{**dict(context=context, new_tokens=new, block_table=table, free_pages=free,  # noqa: E731
                                          free_count=count, segment_requests=seg), **k})
    for bad in (dict(context=context.long()), dict(new_tokens=new[:1]), dict(block_table=table[0]), dict(block_table=table[:1]),
                dict(block_table=table.t()), dict(free_pages=free.cpu()), dict(free_count=count[:0]), dict(first_own=new[:1]),
                dict(segment_requests=None), dict(segment_requests=seg[:1]), dict(context=plan.granted),
                dict(free_pages=plan.row_req), dict(new_tokens=plan.context)):
        with pytest.raises(P.DsaError):
            call(**bad)
    with pytest.raises(P.DsaError):
        plan.slots = plan.row_req
    call()
    step.check(plan, table, free)


def test_plans_on_two_streams_at_once():
    steps = [Step([7 * i % 90 for i in range(n)], [i % 5 for i in range(n)], 16, 4 * n) for n in (70, 1300)]
    runs = [(s, s.plan(), s.tensors(), torch.cuda.Stream()) for s in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, plan, t, stream in runs:
            plan.run(*t, stream=stream)
    torch.cuda.synchronize()
    for s, plan, t, _ in runs:
        s.check(plan, t[2], t[3])


# ------------------------------------------------------------------ positions with several axes

def axis_list(sections, order):
    if order == "split":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def ref_axes(x, positions, axis, freq, scale, layout):
    """ref_rotate with pair i's own position: one pair at a time."""
    n, ref, mag = x.shape[-1] // 2, torch.empty_like(x, dtype=torch.float64), torch.empty_like(x, dtype=torch.float64)
    for i, a in enumerate(axis):
        at = [i, i + n] if layout == P.ROPE_HALF else [2 * i, 2 * i + 1]
        ref[..., at], mag[..., at] = ref_rotate(x[..., at], positions[a], freq[i:i + 1], scale, layout)
    return ref, mag


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [P.ROPE_INTERLEAVED, P.ROPE_HALF])
@pytest.mark.parametrize("tokens, heads, rot, pad, sections, order, restart", [
    (1, 1, 2, 0, (1,), "split", False), (5, 3, 10, 7, (2, 3), "cycle", False),
    (33, 96, 64, 512, (12, 10, 10), "cycle", False), (7, 128, 256, 0, (64, 0, 30, 34), "split", False),
    (300, 2, 48, 16, (12, 12), "split", True), (2048, 9, 64, 64, (2, 15, 15), "cycle", True),
    (130, 4, 128, 0, (16, 24, 24), "split", False)])
def test_rope_with_axes(dtype, layout, tokens, heads, rot, pad, sections, order, restart):
    g = gen(tokens * 1000 + rot)
    full = randn(g, tokens, heads, pad + rot, dtype=dtype)
    x = full[..., pad:]
    positions = torch.randint(0, 1 << 20, (len(sections), tokens), generator=g, device="cuda", dtype=torch.int32)
    table = P.rope_table(rot, 10000.0, "yarn", 32.0, 4096, sections=sections, order=order, restart=restart)
    axis = axis_list(sections, order)
    freq, scale = P.rope_frequencies(rot, 10000.0, "yarn", 32.0, 4096)
    if restart:
        own = [P.rope_frequencies(2 * n, 10000.0, "yarn", 32.0, 4096)[0] for n in sections]
        freq = torch.stack([own[a][axis[:i].count(a)] for i, a in enumerate(axis)])
    assert P.rope_sections(sections, order).tolist() == axis
    ref, mag = ref_axes(x, positions, axis, freq, scale, layout)
    before = full.clone()
    out = torch.empty((tokens, heads, rot), dtype=dtype, device="cuda")
    P.rope(x, table, positions, layout=layout, out=out)
    torch.cuda.synchronize()
    assert torch.equal(full, before)
    assert ((out.double() - ref).abs() <= rope_bound(ref, mag, scale, dtype)).all()
    P.rope(x, table, positions, layout=layout)  # in place: the same bits, and nothing else touched
    torch.cuda.synchronize()
    assert torch.equal(x, out) and torch.equal(full[..., :pad], before[..., :pad])


@pytest.mark.parametrize("layout", [P.ROPE_INTERLEAVED, P.ROPE_HALF])
def test_axes_that_agree_are_one_position(layout):
    """Text tokens: the bits of the call with one position, also from one row of positions for all axes."""
    g = gen(5)
    x = randn(g, 70, 6, 64)
    one = torch.randint(0, 1 << 20, (70,), generator=g, device="cuda", dtype=torch.int32)
    want = P.rope(x, P.rope_table(64), one, layout=layout, out=torch.empty_like(x))
    table = P.rope_table(64, sections=(12, 10, 10), order="cycle")
    for positions in (one.expand(3, 70), one.repeat(3, 1), one.repeat(3, 2)[:, :70]):
        assert torch.equal(P.rope(x, table, positions, layout=layout, out=torch.empty_like(x)), want)


def test_tokens_with_a_negative_position_on_any_axis_are_left_alone():
    g = gen(6)
    q, k = randn(g, 6, 5, 64), randn(g, 6, 1, 129)[..., 65:]
    positions = ints([[5, -1, 0, 9, 7, 9], [1, 4, 131071, -1, 2, 0], [0, 3, 8, 8, -2147483648, 1]])
    table, live = P.rope_table(64, sections=(10, 11, 11)), torch.tensor([0, 2, 5], device="cuda")
    axis, freq = axis_list((10, 11, 11), "split"), P.rope_frequencies(64, 10000.0)[0]
    before = [q.clone(), k.clone()]
    P.rope([q, k], table, positions, layout=[P.ROPE_HALF, P.ROPE_INTERLEAVED])
    for x, b, layout in ((q, before[0], P.ROPE_HALF), (k, before[1], P.ROPE_INTERLEAVED)):
        ref, mag = ref_axes(b, positions.clamp_min(0), axis, freq, 1.0, layout)
        assert ((x.double() - ref).abs() <= rope_bound(ref, mag, 1.0, x.dtype))[live].all()
        assert torch.equal(x[[1, 3, 4]], b[[1, 3, 4]])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("tokens, kv_heads, hpg, dim, page, rot, off, sections, order", [
    (1, 1, 1, 64, 16, 2, 3, (0, 1), "split"), (8, 4, 16, 128, 128, 128, 0, (16, 24, 24), "split"),
    (333, 3, 5, 64, 16, 32, 16, (8, 8), "cycle"), (2100, 2, 3, 128, 64, 90, 5, (20, 15, 10), "cycle"),
    (9000, 8, 2, 128, 64, 64, 64, (32,), "split")])
def test_insert_with_axes_is_rope_with_axes_and_insert(fmt, tokens, kv_heads, hpg, dim, page, rot, off, sections, order):
    """Bit for bit the two calls one after the other, K rotated in 32 bits (so by way of a K in 32 bits), and no other
    byte of the pool written."""
    g = gen(tokens + rot)
    heads = kv_heads * hpg
    qkv = randn(g, tokens, heads + 2 * kv_heads, dim)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    pool = new_pool(g, fmt, -(-tokens // page) + 2, kv_heads, page, dim)
    kv = P.KvCache(pool, *((1 / 72, 1 / 90) if fmt == "fp8" else (1.0, 1.0)))
    slots = torch.randperm(pool.shape[0] * page, generator=g, device="cuda")[:tokens].int()
    positions = torch.randint(0, 1 << 20, (len(sections), tokens), generator=g, device="cuda", dtype=torch.int32)
    slots[0], positions[-1, 0] = -1, -1  # a padding token
    table = P.rope_table(rot, sections=sections, order=order)
    for layout in (P.ROPE_HALF, P.ROPE_INTERLEAVED):
        want = bits(pool).clone()
        k32 = k.float()
        P.rope(k32[..., off:off + rot], table, positions, layout=layout)
        at = [(s // page, s % page) for s in slots.tolist()]
        q_out, status = torch.full((tokens, heads, rot), 7.0, dtype=torch.bfloat16, device="cuda"), P.new_status()
        P.kv_insert(kv, slots, k, v, rope=table, positions=positions, layout=layout, rot_offset=off,
                    q=q[..., off:off + rot], q_out=q_out, status=status)
        checked(status)
        i, j = (torch.tensor(x, device="cuda")[1:] for x in zip(*at))
        for y, x, s in ((0, k32, kv.k_scale), (1, v.float(), kv.v_scale)):
            x = bits((x / s).clamp(-448, 448).to(torch.float8_e4m3fn) if fmt == "fp8" else x.to(torch.bfloat16))
            want[i, :, y, j] = x[1:]
        assert torch.equal(bits(pool), want)
        ref = P.rope(q[..., off:off + rot], table, positions, layout=layout, out=torch.full_like(q_out, 7.0))
        assert torch.equal(q_out, ref)


def test_tables_without_an_axis_are_refused():
    freq, _ = P.rope_frequencies(64, 10000.0)
    turns, axis = P.rope_turns(freq).cuda(), P.rope_sections((12, 10, 10))
    for bad in (dict(axis=axis, num_axes=0), dict(axis=axis, num_axes=-1), dict(axis=axis[:16]), dict(axis=axis.int()),
                dict(axis=axis.cuda())):
        with pytest.raises(P.DsaError):
            P.RopeTable(turns, **bad)
    x, at = torch.zeros(3, 1, 64, device="cuda"), ints([0, 1, 2]).expand(3, 3)
    for axes in (2, 5):  # fewer than the pairs name; more than there may be
        with pytest.raises(P.DsaError):
            P.rope(x, P.RopeTable(turns, axis=axis, num_axes=axes), ints([0, 1, 2]).expand(axes, 3))
    with pytest.raises(P.DsaError):
        P.rope(x, P.RopeTable(turns, axis=axis), at[:2])
    P.rope(x, P.RopeTable(turns, axis=axis), at)


def test_insert_reports_a_slot_of_a_token_without_a_place():
    g = gen(9)
    pool = new_pool(g, "bf16", 2, 1, 16, 64)
    before, k, status = pool.clone(), randn(g, 2, 1, 64), P.new_status()
    table = P.rope_table(64, sections=(16, 16))
    P.kv_insert(P.KvCache(pool), ints([3, 4]), k, k, rope=table, positions=ints([[1, 1], [2, -1]]), status=status)
    torch.cuda.synchronize()
    assert status.item() == P.ERR_BOUNDS and torch.equal(pool[0, 0, 1, 3], k[0, 0])
    assert torch.equal(pool[0, :, :, 4:], before[0, :, :, 4:])
