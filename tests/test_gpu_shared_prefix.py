"""Attention over shared prefixes on the GPU (dsa_kv_attention_shared) against its formula in 64 bits, and a run of a
batch's step: plan, rotary positions with several axes, insert, attention."""
import math
import random

import pytest
import torch

import prefill_dsa_indexer_gb300 as P
from tests.test_gpu_kv_path import bits, checked, gen, new_pool, randn, ref_rotate, rope_bound

pytestmark = pytest.mark.gpu


def ints(values, shape=None):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t if shape is None else t.view(shape)


# ------------------------------------------------------------------ attention over shared prefixes

class Shared:
    """Segments of (shared tokens, tokens of each request) in shuffled pages: whole pages of the shared tokens are listed
    by every request of the segment, what lies behind them is in its own; slots that hold no token are NaN."""

    def __init__(self, seed, fmt, segments, kv_heads, hpg, dim, page, group=1, before=(), after=(), pad=0, q_scale=1.0,
                 row_ctx=None):
        g = gen(seed)
        self.fmt, self.dim, self.page, self.hpg, self.group = fmt, dim, page, hpg, group
        batch = [(0, list(before))] + list(segments) + [(0, list(after))]  # (first and last: in no segment)
        lens = [n for _, own in batch for n in own]
        need = sum(-(-n // page) for n in lens) + 3
        pool = new_pool(g, fmt, need, kv_heads, page, dim)
        self.ks, self.vs = (1 / 72, 1 / 90) if fmt == "fp8" else (1.0, 1.0)
        order = torch.randperm(need, generator=g, device="cuda").int()
        self.max_ctx = max(lens + [1])
        self.table = torch.full((len(lens), -(-self.max_ctx // page)), 0x7FFFFFF, dtype=torch.int32, device="cuda")
        nan, b, at, r = 0x7F if fmt == "fp8" else 0x7FFF, bits(pool), 0, 0
        starts, shared = [], []
        for s, (pre, own) in enumerate(batch):
            if 0 < s <= len(segments):
                starts.append(r * group)
                shared.append(pre)
            whole = min([pre // page] + [n // page for n in own]) if own else 0
            common = order[at:at + whole]
            at += whole
            kept = {}
            for n in own:
                mine = order[at:at + -(-n // page) - whole]
                at += mine.numel()
                self.table[r, :whole] = common
                self.table[r, whole:whole + mine.numel()] = mine
                for y, p in enumerate(mine.tolist()):  # shared tokens in pages of the request's own: the same in each
                    have = min(pre - (whole + y) * page, page)
                    if have > 0:
                        kept.setdefault(y, b[p].clone())
                        b[p, :, :, :have] = kept[y][:, :, :have]
                if n % page:
                    b[self.table[r, n // page].item(), :, :, n % page:] = nan
                r += 1
        starts.append((r - len(after)) * group)
        for p in order[at:].tolist():
            b[p] = nan
        self.pool, self.kv = pool, P.KvCache(pool, self.ks, self.vs)
        self.rows = row_ctx or [max(0, n - (group - 1 - i)) for n in lens for i in range(group)]
        self.rows = self.rows + [0] * (pad * group)
        self.row_req = (torch.arange(len(self.rows), dtype=torch.int32, device="cuda") // group) % max(len(lens), 1)
        self.row_ctx, self.starts, self.shared = ints(self.rows), ints(starts), ints(shared)
        self.q = (randn(g, len(self.rows), kv_heads * hpg, dim).float() * q_scale).to(torch.bfloat16)
        self.sm = dim ** -0.5

    def run(self, **kw):
        """Shared wherever there is anything to share, unless `least_saved` says otherwise."""
        status = P.new_status()
        kw.setdefault("least_saved", 1)
        a = dict(starts=self.starts, shared=self.shared, q=self.q)
        a.update({k: kw.pop(k) for k in tuple(kw) if k in a})
        got = P.kv_attention_shared(self.kv, self.table, self.row_req, self.row_ctx, self.max_ctx, a["q"], a["starts"],
                                    a["shared"], rows_per_group=self.group, status=status, **kw)
        checked(status)
        return got

    def check(self, out, lse, rows=None):
        for r in range(len(self.rows)) if rows is None else rows:
            n = self.rows[r]
            if n == 0:
                assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
                continue
            pages = self.table[self.row_req[r], :-(-n // self.page)].long()
            kv = bits(self.pool)[pages].view(self.pool.dtype).double()  # [pages, KV heads, 2, page, dim]
            k, v = (kv[:, :, y].transpose(0, 1).flatten(1, 2)[:, :n] * s for y, s in ((0, self.ks), (1, self.vs)))
            q = self.q[r].double().view(-1, self.hpg, self.dim)
            s = q @ k.transpose(1, 2) * self.sm
            p = torch.softmax(s, -1)
            ref, mag = p @ v, p @ v.abs()
            # scores: `dim` fp32 sums of products up to big; over FP8 pools q is two e4m3 terms, which leave 2^-10 where
            # the largest element is above 224
            big = torch.where(s > -math.inf, q.abs() @ k.abs().transpose(1, 2) * self.sm, 0.0).amax(-1, keepdim=True)
            ds = (self.dim + 8) * 2.0 ** -24 * big
            if self.fmt == "fp8":
                ds = ds + 2.0 ** -10 / 224 * q.abs().amax(-1, keepdim=True) * \
                    k.abs().sum(-1).amax(-1)[:, None, None] * self.sm
            # weights rounded to bf16 (2^-8), or to fp16 (2^-11) in steps of 2^-24 where the largest is at least 2^7;
            # rows' own tokens over FP8 pools of head_dim 128 keep 2^-29 of their part's largest; sums in fp32
            w = (2.0 ** -11 if self.fmt == "fp8" else 2.0 ** -8) + 2.0 ** -22 + n * 2.0 ** -24
            sub = 2.0 ** -29 * p.amax(-1, keepdim=True) * v.abs().sum(1, keepdim=True) if self.fmt == "fp8" else 0
            bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * ((w + 2 * ds) * mag + sub) + 1e-30
            off = (out[r].double().view_as(ref) - ref).abs()
            assert (off <= bound).all(), (r, (off / bound).max().item())
            want = torch.logsumexp(s, -1)
            lb = ds[..., 0] + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * want.abs()
            assert ((lse[r].double().view_as(want) - want).abs() <= lb).all(), r


SHAPES = [(1, 1, 64, 16), (4, 16, 128, 128), (4, 8, 128, 64), (3, 5, 64, 32), (2, 7, 128, 16), (1, 33, 64, 64),
          (2, 64, 128, 128), (1, 128, 64, 128)]
FORMATS = ["bf16", "fp8"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kv_heads, hpg, dim, page", SHAPES)
def test_shared_short_prefixes(fmt, kv_heads, hpg, dim, page):
    """Around the tile of 128 tokens, segments of one to nine requests, rows in no segment, padding rows."""
    segments = [(n, [n + m for m in own]) for n, own in (
        (0, [5, 1]), (1, [1, 2]), (127, [128, 200, 127]), (128, [129]), (128, [128, 129, 500]), (129, [300, 257]),
        (255, [256, 255, 511, 3000]), (256, [1, 7]), (257, [300 * i + 1 for i in range(9)]), (640, [1, 130]))]
    c = Shared(11, fmt, segments, kv_heads, hpg, dim, page, before=[77, 300], after=[1, 129], pad=2)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kv_heads, hpg, dim, page", SHAPES)
@pytest.mark.parametrize("prefix, rows", [(4096, 7), (9001, 40), (20000, 3)])
def test_shared_long_prefixes(fmt, kv_heads, hpg, dim, page, prefix, rows):
    c = Shared(12, fmt, [(prefix, [prefix + 1 + 37 * i % 500 for i in range(rows)])], kv_heads, hpg, dim, page)
    out, lse = c.run()
    c.check(out, lse, rows=sorted({0, 1, 2, rows // 2, rows - 1}))
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group, kv_heads, hpg, dim, page", [(2, 2, 3, 64, 16), (4, 2, 16, 128, 128), (8, 1, 4, 128, 64),
                                                            (8, 2, 16, 64, 32), (2, 1, 16, 128, 32)])
def test_shared_verify_rows(fmt, group, kv_heads, hpg, dim, page):
    """Rows whose own tokens begin inside the group, and rows that end before the shared tokens do."""
    segments = [(1000, [1001, 1500, 1000 + group]), (300, [300]), (2000, [2000, 2003, 1990, 4000]), (128, [128, 131])]
    c = Shared(13, fmt, segments, kv_heads, hpg, dim, page, group=group, pad=1)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_rows_that_see_less_than_the_prefix(fmt):
    """Of a row's context below the shared tokens, and of none: a padding row among the others."""
    ctx = [5000, 0, 700, 4999, 5200, 0, 1, 6000, 5999, 5000, 4100, 4096]
    lens = [5000, 5000, 5000, 5200, 5200, 5001, 5001, 6000, 6000, 5000, 5000, 5000]
    segments = [(5000, lens[:4]), (5000, lens[4:7]), (5000, lens[7:])]
    c = Shared(14, fmt, segments, 2, 4, 128, 64, row_ctx=ctx)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_scale", [0.0, 30.0, 1e-3])
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_peaked_and_flat_scores(fmt, q_scale, dim):
    c = Shared(15, fmt, [(2500, [2501, 2600, 2777]), (640, [641] * 20)], 2, 8, dim, 64, q_scale=q_scale)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_without_a_segment_is_the_plain_call(fmt):
    c = Shared(16, fmt, [(300, [301, 5000])], 2, 4, 128, 64)
    want = P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q)
    got = c.run(starts=ints([0]), shared=ints([], (0,)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*c.run(starts=ints([2, 2]), shared=ints([300])))  # an empty segment behind the last row


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("starts, shared", [([0, 3, 2, 4], [300, 300, 300]), ([-1, 2], [300]), ([0, 5], [300]),
                                            ([0, 2, 4], [300, -5]), ([4, 0], [300])])
@pytest.mark.parametrize("least", [0, 1])
def test_shared_segments_that_cannot_be_are_reported(fmt, starts, shared, least):
    """And their rows are answered as if in none."""
    c = Shared(17, fmt, [(300, [301, 500, 302, 900])], 2, 4, 128, 64)
    status = P.new_status()
    out, lse = P.kv_attention_shared(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, ints(starts), ints(shared),
                                     status=status, least_saved=least)
    torch.cuda.synchronize()
    assert status.item() == P.ERR_BOUNDS
    c.check(out, lse)


def test_shared_segments_that_cut_a_group_are_reported():
    c = Shared(18, "bf16", [(300, [301, 500])], 2, 4, 128, 64, group=2)
    status = P.new_status()
    out, lse = P.kv_attention_shared(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, ints([0, 3]), ints([300]),
                                     rows_per_group=2, status=status, least_saved=1)
    torch.cuda.synchronize()
    assert status.item() == P.ERR_BOUNDS
    c.check(out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_device_errors_are_reported(fmt):
    """A context or a request out of range answers its own rows with nothing and leaves the segment's others alone; a
    page id outside the pool is reported."""
    for what in ("ctx", "negative", "request", "page", "own page"):
        c = Shared(19, fmt, [(640, [700, 900, 641])], 2, 4, 128, 64)
        status, rows = P.new_status(), [0, 2]
        if what == "ctx":
            c.row_ctx[1] = c.max_ctx + 1
        if what == "negative":
            c.row_ctx[1] = -4
        if what == "request":
            c.row_req[1] = 3
        if what == "page":
            c.table[0, 3] = c.pool.shape[0]
        if what == "own page":
            c.table[1, 11] = -1
        out, lse = P.kv_attention_shared(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, c.starts, c.shared,
                                         status=status, least_saved=1)
        torch.cuda.synchronize()
        assert status.item() == P.ERR_BOUNDS, what
        if what in ("ctx", "negative", "request"):
            assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
        if what != "page":
            c.check(out, lse, rows=rows)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_shared_a_head_of_no_numbers_stays_alone(fmt, dim, value):
    c = Shared(20, fmt, [(700, [800, 701, 900, 1000])], 2, 5, dim, 32)
    q = c.q.clone()
    q[2, 7, 3] = value
    out, lse = c.run(q=q)
    assert torch.isnan(out[2, 7]).any() and not torch.isfinite(lse[2, 7])
    c.check(out, lse, rows=[0, 1, 3])
    rest = torch.ones(10, dtype=torch.bool, device="cuda")
    rest[7] = False
    assert torch.isfinite(out[2, rest].float()).all() and torch.isfinite(lse[2, rest]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_values_of_no_numbers_reach_their_dim_alone(fmt, dim):
    """A NaN (and, in a bf16 pool, an infinity) of V among the shared tokens reaches every row there, no other dim, and
    no other segment."""
    c = Shared(21, fmt, [(700, [800, 701]), (700, [900, 1000, 701])], 2, 5, dim, 32)
    b, nan = bits(c.pool), 0x7F if fmt == "fp8" else 0x7FFF
    b[c.table[0, 3].item(), 1, 1, 5, 9] = nan
    if fmt == "bf16":
        c.pool[c.table[0, 2].item(), 0, 1, 5, 3] = math.inf
    out, lse = c.run()
    assert torch.isnan(out[:2, 5:, 9]).all() and torch.isfinite(lse).all()
    if fmt == "bf16":
        assert (out[:2, :5, 3] == math.inf).all()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:2, 5:, 9] = True
    bad[:2, :5, 3] = fmt == "bf16"
    assert torch.isfinite(out[~bad].float()).all()
    c.check(out, lse, rows=[2, 3, 4])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nats", [-150.0, -1000.0, 300.0])
@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_scores_far_from_zero(fmt, dim, nats):
    """A constant that the softmax does not see on all scores: parts without a base of their own would vanish."""
    c = Shared(22, fmt, [(1000, [1001, 1000, 2000]), (300, [290, 5000])], 2, 6, dim, 64)
    code = (-448.0 if fmt == "fp8" else -32.0) * (1 if nats < 0 else -1)
    b = bits(c.pool)
    b[:, :, 0, :, 0] = bits(torch.tensor([code], device="cuda").to(c.pool.dtype)).item()
    c.q[..., 0] = nats / (code * c.ks * c.sm)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [64, 128])
def test_shared_scores_of_minus_infinity_weigh_nothing(dim):
    """Keys of an infinity: the tokens that hold it score -inf, on shared tiles as a whole and in part."""
    c = Shared(23, "bf16", [(512, [600, 700])], 1, 3, dim, 128)
    c.q[..., 0] = c.q[..., 0].abs().clamp_min(0.5)
    pages = c.table[0, :4].long()
    c.pool[pages[0], :, 0, :, 0] = -math.inf         # all of a tile
    c.pool[pages[2], :, 0, 5:100, 0] = -math.inf     # most of another
    c.check(*c.run())
    c.pool[pages, :, 0, :, 0] = -math.inf            # all that is shared
    c.check(*c.run())
    c.pool[c.table[0, 4].long(), :, 0, :, 0] = -math.inf  # and all of the first row's own
    out, lse = c.run()
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    c.check(out, lse, rows=[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_background_behind_a_first_token_that_takes_most(fmt):
    """A first token 11 nats ahead of many others whose values it opposes: what lies far below it counts."""
    n = 32768
    c = Shared(24, fmt, [(n, [n + 1, n + 2])], 1, 2, 128, 128)
    c.pool.view(torch.uint8 if fmt == "fp8" else torch.int16).zero_()
    first = c.table[0, 0].item()
    one = torch.ones(1, device="cuda")
    code = lambda x: (one * x).to(c.pool.dtype)  # noqa: E731
    b = bits(c.pool)
    b[:, :, 1] = bits(code(1.0 / c.vs if fmt == "fp8" else 1.0)).item()
    b[first, :, 1, 0] = bits(code(-0.5 / c.vs if fmt == "fp8" else -0.5)).item()
    k = 80.0 if fmt == "fp8" else 1.0
    b[first, :, 0, 0, 0] = bits(code(k)).item()
    c.q.zero_()
    c.q[..., 0] = 11.0 / (k * c.ks * c.sm)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_of_many_segments_and_rows(fmt):
    rng = random.Random(3)
    segments = []
    for s in range(90):
        n = rng.choice((0, 100, 128, 400, 1500))
        segments.append((n, [n + rng.randint(1, 60) for _ in range(rng.choice((0, 1, 2, 3, 17)))]))
    c = Shared(25, fmt, segments, 2, 4, 64, 16, pad=3)
    out, lse = c.run()
    c.check(out, lse, rows=range(0, len(c.rows), 7))
    empty = torch.tensor([n == 0 for n in c.rows], device="cuda")
    assert (out[empty] == 0).all() and torch.isfinite(lse[~empty]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_segments_bits_do_not_depend_on_the_others(fmt, dim):
    one = (1500, [1501 + 9 * i for i in range(21)])
    a = Shared(26, fmt, [one], 2, 8, dim, 64)
    want = a.run()
    b = Shared(27, fmt, [(900, [901, 1000]), one, (4000, [4001] * 5)], 2, 8, dim, 64, after=[3000])
    # the same tokens and queries in the other batch's pages
    for r in range(21):
        for p in range(-(-a.rows[r] // 64)):
            bits(b.pool)[b.table[2 + r, p].item()] = bits(a.pool)[a.table[r, p].item()]
    b.q[2:23] = a.q
    got = b.run()
    assert torch.equal(got[0][2:23], want[0]) and torch.equal(got[1][2:23], want[1])


def test_shared_rows_of_a_packed_projection_and_other_scales():
    c = Shared(28, "bf16", [(513, [600, 514, 2000])], 4, 8, 128, 64)
    packed = torch.zeros(3, 32 + 8, 128, dtype=torch.bfloat16, device="cuda")
    packed[:, :32] = c.q
    a, b = c.run(q=packed[:, :32]), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.sm = 0.3
    c.check(*c.run(sm_scale=0.3))


def test_shared_calls_in_graphs_on_streams_and_at_once():
    """Each call has a workspace of its own; graphs replay while an eager call runs."""
    cases = [Shared(29, "fp8", [(3000, [3001, 3100, 5000]), (400, [500, 600])], 2, 8, 128, 64),
             Shared(30, "bf16", [(5000, [5001 + i for i in range(30)])], 2, 8, 128, 64),
             Shared(31, "bf16", [(700, [701, 1000])], 4, 4, 64, 32, group=2)]
    want = [c.run() for c in cases]
    graphs = []
    for c in cases:
        need = P.kv_attention_shared_workspace_size(c.kv, c.q.shape[0], c.q.shape[1], c.max_ctx, c.shared.numel())
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        o, l = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            P.kv_attention_shared(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, c.starts, c.shared,
                                  rows_per_group=c.group, out=o, lse=l, workspace=ws, least_saved=1)
        graphs.append((graph, o, l, ws, torch.cuda.Stream()))
    for _ in range(4):
        for _, o, l, ws, _ in graphs:
            o.fill_(7.0)
            l.fill_(7.0)
            ws.fill_(0xFF)
        torch.cuda.synchronize()
        for graph, _, _, _, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        eager = cases[1].run(stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        for (_, o, l, _, _), w in zip(graphs, want):
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])
        assert torch.equal(eager[0], want[1][0]) and torch.equal(eager[1], want[1][1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_calls_beside_other_work(fmt, dim):
    """SMs that other kernels hold: whichever are left to the rows' own tokens, all of those are read."""
    c = Shared(46, fmt, [(4000, [4001 + 97 * i for i in range(40)])], 4, 8, dim, 64)
    want, stream = c.run(), torch.cuda.Stream()
    c.check(*want, rows=[0, 17, 39])
    a = torch.randn(2048, 2048, device="cuda", dtype=torch.bfloat16)
    for i in range(20):
        with torch.cuda.stream(stream):
            for _ in range(1 + i % 4):
                a @ a
                a.sum()
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_where_it_pays(fmt):
    """The library's choice: a call too small by its shapes is the plain one, bit for bit, and a segment that saves too
    little beside one that saves enough is as if it shared nothing."""
    c = Shared(33, fmt, [(700, [701, 900, 1000])], 2, 4, 128, 64)
    got, want = c.run(least_saved=0), P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    token, least = 2 * 2 * 128 * (1 if fmt == "fp8" else 2), (100 if fmt == "fp8" else 160) << 20
    n = -(-least // (4 * 15 * token * 128)) * 128  # the least that pays for 16 rows, of two segments
    c = Shared(34, fmt, [(n, [n + i for i in range(16)]), (n - 128, [n] * 16)], 2, 2, 128, 128)
    assert 31 * c.max_ctx * token < least  # too little by its shapes
    got, plain = c.run(least_saved=0), P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    c = Shared(34, fmt, [(n, [n + i for i in range(16)]), (n - 128, [n] * 16)], 2, 2, 128, 128, after=[64, 4 * n])
    (out, lse), first, both = c.run(least_saved=0), c.run(shared=ints([n, 0])), c.run()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and not torch.equal(lse[16:32], both[1][16:32])
    c.check(out, lse, rows=[0, 7, 15, 16, 31, 32, 33])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kv_heads, hpg, rows", [(40, 1, 130), (33, 3, 100), (5, 16, 600), (160, 1, 5)])
def test_shared_of_many_heads(fmt, kv_heads, hpg, rows):
    """More items than CTAs in every part, or nearly."""
    c = Shared(35, fmt, [(700, [701 + i % 50 for i in range(rows)]), (400, [401, 500])], kv_heads, hpg, 64, 64)
    out, lse = c.run()
    c.check(out, lse, rows=[0, 1, rows // 2, rows - 1, rows, rows + 1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hpg, rows", [(8, 4), (8, 5), (1, 40), (5, 20), (16, 9)])
def test_shared_items_that_follow_one_another(fmt, dim, hpg, rows):
    """Several items a CTA, of columns that leave some of its warps with little or nothing to write, which are at the next
    item's queries while the others write."""
    segments = [(300 + 150 * s, [310 + 160 * s + i for i in range(rows)]) for s in range(12)]
    c = Shared(45, fmt, segments, 40, hpg, dim, 64)
    out, lse = c.run()
    c.check(out, lse, rows=range(0, len(c.rows), 11))
    for _ in range(10):
        again = c.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_of_very_many_rows(fmt):
    """More rows than the segments' kernel keeps in shared memory."""
    c = Shared(36, fmt, [(520, [528 + i % 9 for i in range(1040)]), (130, [140] * 2)], 1, 2, 64, 16, group=8, pad=2)
    out, lse = c.run()
    c.check(out, lse, rows=[0, 1, 4099, 8191, 8192, 8319, 8320, 8335, 8336, 8351])
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_shared_calls_that_follow_one_another_in_one_workspace():
    """Of different segments, pools and shapes, without a wait between them: nothing of one call is taken for another's."""
    cases = [Shared(37, "fp8", [(1500, [1501 + i for i in range(9)]), (400, [500, 600])], 2, 8, 128, 64),
             Shared(38, "fp8", [(300, [301] * 3), (2000, [2001 + i for i in range(30)])], 2, 8, 128, 64),
             Shared(39, "bf16", [(900, [901, 1000]), (500, [501, 700]), (2500, [2600] * 20)], 2, 8, 128, 64)]
    want = [c.run() for c in cases]
    need = max(P.kv_attention_shared_workspace_size(c.kv, c.q.shape[0], c.q.shape[1], c.max_ctx, c.shared.numel())
               for c in cases)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for i in range(60):
        c = cases[(i * 7 + i // 5) % 3]
        got.append(((i * 7 + i // 5) % 3, P.kv_attention_shared(
            c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, c.starts, c.shared, rows_per_group=c.group, workspace=ws,
            least_saved=1)))
    torch.cuda.synchronize()
    for i, (o, l) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_rows_of_one_request(fmt):
    """A chunk of a prompt, row by row over what its request has in the cache: one request in all rows of a segment."""
    c = Shared(41, fmt, [(2000, [2300])], 4, 8, 128, 64)
    c.rows = list(range(2001, 2301))
    c.row_ctx, c.row_req, c.starts = ints(c.rows), ints([0] * 300), ints([0, 300])
    c.q = randn(gen(42), 300, 32, 128).to(torch.bfloat16)
    c.check(*c.run(), rows=[0, 1, 46, 47, 48, 175, 299])


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_pages_of_a_large_pool(fmt):
    """Pages whose elements lie beyond 2^31, and their bytes beyond 2^32."""
    c = Shared(43, fmt, [(700, [701, 900, 1500]), (300, [301, 400])], 4, 8, 128, 128)
    (out, lse), far = c.run(), (1 << 32) // (2 * 4 * 128 * 128 * c.pool.element_size())
    big = torch.empty(far + c.pool.shape[0], *c.pool.shape[1:], dtype=c.pool.dtype, device="cuda")
    bits(big)[far:] = bits(c.pool)
    c.table = torch.where(c.table < c.pool.shape[0], c.table + far, c.table)
    c.pool, c.kv = big, P.KvCache(big, c.ks, c.vs)
    got = c.run()
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("graph", [False, True])
def test_shared_calls_whose_inputs_change_in_place(fmt, graph):
    """Lengths, segments and block table stand at the same addresses in every call of one workspace, and each call finds
    other ones there: nothing that an earlier call read is taken for this one's (merges and the shared tokens' kernel read
    before they wait).  Few rows, so that many SMs run none of the kernels that wait first."""
    cases = [Shared(47, fmt, [(1500, [1501 + 9 * i for i in range(6)]), (400, [500, 600])], 2, 4, 128, 64),
             Shared(48, fmt, [(300, [310, 460, 610]), (2000, [2100 + 90 * i for i in range(5)])], 2, 4, 128, 64),
             Shared(49, fmt, [(0, [1, 9, 5, 700]), (0, [4000, 3, 2500, 128])], 2, 4, 128, 64)]
    most, width = max(c.max_ctx for c in cases), max(c.table.shape[1] for c in cases)
    H, names = cases[0].q.shape[1], ("table", "row_req", "row_ctx", "starts", "shared")
    for c in cases:
        c.table = torch.nn.functional.pad(c.table, (0, width - c.table.shape[1]))
    ours = {n: torch.empty_like(getattr(cases[0], n)) for n in names}
    need = P.kv_attention_shared_workspace_size(cases[0].kv, 8, H, most, 2)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")

    def both(c, a, ws):
        shared = P.kv_attention_shared(c.kv, a["table"], a["row_req"], a["row_ctx"], most, c.q, a["starts"], a["shared"],
                                       workspace=ws, least_saved=1)
        return shared + P.kv_attention(c.kv, a["table"], a["row_req"], a["row_ctx"], most, c.q, workspace=ws)
    want = []
    for c in cases:
        want.append(both(c, {n: getattr(c, n) for n in names}, None))
        torch.cuda.synchronize()

    def calls():
        got = []
        for i in (0, 1, 2, 1, 0, 2, 0, 1):
            for n in names:
                ours[n].copy_(getattr(cases[i], n))
            got.append((i, both(cases[i], ours, ws)))
        return got
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = calls()
    for _ in range(5):
        captured.replay() if graph else None
        got = got if graph else calls()
        torch.cuda.synchronize()
        for i, tensors in got:
            assert all(torch.equal(x, y) for x, y in zip(tensors, want[i])), i


def test_layer_takes_both_of_its_segments_tensors():
    c = Shared(44, "bf16", [(300, [301, 302])], 2, 4, 128, 64)
    layer = P.KvLayer(c.kv, c.table, c.max_ctx, 2, 8, num_segments=1)
    slots, k = ints([-1, -1]), torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(segment_rows=c.starts), dict(segment_ctx=c.shared)):
        with pytest.raises(P.DsaError):
            layer.run(c.row_req, c.row_ctx, slots, None, c.q, k, k, **bad)
    want, got = c.run(), layer.run(c.row_req, c.row_ctx, slots, None, c.q, k, k, segment_rows=c.starts, segment_ctx=c.shared)
    torch.testing.assert_close(got[0], want[0], atol=2e-2, rtol=2e-2)


def test_shared_calls_without_a_row():
    c = Shared(32, "bf16", [(300, [301, 302])], 2, 4, 128, 64)
    none = ints([], (0,))
    out, lse = P.kv_attention_shared(c.kv, c.table, none, none, c.max_ctx, c.q[:0], ints([0, 0]), ints([300]))
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)


# ------------------------------------------------------------------ a run of them

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_batch_over_a_shared_prefix(fmt, graph):
    """Three steps of five requests over two prefixes: plan, rotate with axes, insert, attend over what was shared,
    captured once and replayed, or eagerly; one request ends on the way and its pages go to another."""
    g = gen(40)
    page, dim, kv_heads, hpg, n, rows = 16, 128, 2, 4, 5, 8
    H, width = kv_heads * hpg, 40
    prefix = [300, 150]              # tokens of requests 0 - 2 and 3 - 4
    pages = 120
    pool = new_pool(g, fmt, pages, kv_heads, page, dim)
    kv = P.KvCache(pool, *((1 / 72, 1 / 90) if fmt == "fp8" else (1.0, 1.0)))
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    whole = [p // page for p in prefix]
    table[:3, :whole[0]] = ids[:whole[0]]
    table[3:, :whole[1]] = ids[whole[0]:whole[0] + whole[1]]
    used, kept = sum(whole), [whole[0] * page] * 3 + [whole[1] * page] * 2
    free, count = torch.full((pages,), -1, dtype=torch.int32, device="cuda"), pages - used
    free[:count] = ids[used:]
    plan = P.KvPlan(n, rows, page, pages, num_segments=2)
    plan.context.copy_(ints(kept))
    plan.free_count.fill_(count)
    first_own, seg_req, seg_ctx = ints([whole[0]] * 3 + [whole[1]] * 2), ints([0, 3, 5]), ints([w * page for w in whole])
    rope = P.rope_table(64, sections=(12, 10, 10), order="cycle")
    layer = P.KvLayer(kv, table, width * page, rows, H, rope=rope, rot_offset=32, num_segments=2)
    new, qkv = ints([0] * n), torch.zeros(rows, H + 2 * kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    parts = qkv[:, :H], qkv[:, H:H + kv_heads], qkv[:, H + kv_heads:]

    def step():
        plan.run(plan.context, new, table, free, plan.free_count, first_own, seg_req)
        layer.run(plan.row_req, plan.row_ctx, plan.slots, plan.positions.expand(3, rows), *parts,
                  segment_rows=plan.segment_rows, segment_ctx=seg_ctx)
    if graph:
        with torch.cuda.stream(torch.cuda.Stream()):
            step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    ctx = list(kept)
    for i, fresh in enumerate(([1, 1, 2, 1, 3], [1, -1, 2, 2, 1], [4, 0, 1, 1, 1])):
        new.copy_(ints(fresh))
        qkv.copy_(randn(g, rows, H + 2 * kv_heads, dim))
        raw = qkv.clone()
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        checked(plan.status)
        checked(layer.status)
        r = 0
        for j, t in enumerate(fresh):
            if t == -1:
                ctx[j] = 0
                continue
            for _ in range(t):
                assert (plan.row_req[r].item(), plan.positions[r].item()) == (j, ctx[j])
                slot = plan.slots[r].item()
                assert slot // page == table[j, ctx[j] // page].item() and slot % page == ctx[j] % page
                assert torch.equal(bits(pool)[slot // page, :, 1, slot % page], bits(
                    (raw[r, H + kv_heads:].float() / kv.v_scale).clamp(-448, 448).to(pool.dtype) if fmt == "fp8" else
                    raw[r, H + kv_heads:]))
                ctx[j] += 1
                r += 1
        assert plan.context.tolist() == ctx and (plan.slots[r:] == -1).all()
        assert torch.equal(qkv[r:], raw[r:]) and (layer.out[r:] == 0).all()
        freq, _ = P.rope_frequencies(64, 10000.0)
        ref, mag = ref_rotate(raw[:r, :H, 32:96], plan.positions[:r], freq, 1.0, P.ROPE_HALF)
        assert ((qkv[:r, :H, 32:96].double() - ref).abs() <= rope_bound(ref, mag, 1.0, torch.bfloat16)).all()
        c = object.__new__(Shared)
        c.fmt, c.dim, c.page, c.hpg, c.pool, c.table, c.sm = fmt, dim, page, hpg, pool, table, dim ** -0.5
        c.ks, c.vs, c.rows, c.row_req, c.q = kv.k_scale, kv.v_scale, plan.row_ctx.tolist(), plan.row_req, qkv[:, :H]
        c.check(layer.out, layer.lse)
        own = (table[2, whole[0]:-(-ctx[2] // page)].tolist(), table[0, whole[0]:-(-ctx[0] // page)].tolist())
        assert not set(own[0]) & set(own[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_layer_shares_what_it_is_told_to(fmt, dim):
    """A layer's call is kv_attention_shared's, bit for bit, by the layer's least_saved; by the library's choice these few
    rows are read one by one."""
    c = Shared(50, fmt, [(1500, [1501, 1700, 2000]), (640, [650 + i for i in range(4)])], 2, 4, dim, 64, after=[30])
    slots, k = ints([-1] * 8), torch.zeros(8, 2, dim, dtype=torch.bfloat16, device="cuda")
    plain = P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q)
    for least, want in ((1, c.run()), (0, plain)):
        layer = P.KvLayer(c.kv, c.table, c.max_ctx, 8, 8, num_segments=2, least_saved=least)
        got = layer.run(c.row_req, c.row_ctx, slots, None, c.q, k, k, segment_rows=c.starts, segment_ctx=c.shared)
        checked(layer.status)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        c.check(*got)
    assert not torch.equal(c.run()[0], plain[0])


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_layer_with_a_long_bound_can_keep_to_the_plain_call(fmt):
    """By its bound the library shares (as far as there is anything to share), with more to save than its shapes leave it is
    dsa_kv_attention with that bound, bit for bit, and still reports segments that cannot be."""
    c = Shared(54, fmt, [(700, [701, 900, 1000, 2000])], 4, 8, 128, 64)
    most, slots = 131072, ints([-1] * 4)
    c.table = torch.nn.functional.pad(c.table, (0, most // 64 - c.table.shape[1]))
    k = torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda")
    want = P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, most, c.q)
    for least in (0, 1 << 40):
        layer = P.KvLayer(c.kv, c.table, most, 4, 32, num_segments=1, least_saved=least)
        got = layer.run(c.row_req, c.row_ctx, slots, None, c.q, k, k, segment_rows=c.starts, segment_ctx=c.shared)
        checked(layer.status)
        c.check(*got)
        if least:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        layer.run(c.row_req, c.row_ctx, slots, None, c.q, k, k, segment_rows=ints([3, 2]), segment_ctx=c.shared)
        torch.cuda.synchronize()
        assert layer.status.item() == P.ERR_BOUNDS


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("group", [1, 2])
def test_steps_of_a_batch_that_reads_its_prefixes_once(fmt, graph, group):
    """Steps of five requests over two prefixes of several tiles, by the kernels of shared tokens: plan, rotate, insert
    and attend, captured once and replayed, or eagerly.  The plan's segments are those of its requests, the layer's outputs
    the formula's and, bit for bit, those of the attention call on what the plan made."""
    g = gen(51)
    page, dim, kv_heads, hpg, n, rows = 16, 128, 2, 4, 5, 16
    H, width, prefix = kv_heads * hpg, 110, [1500, 700]  # tokens of requests 0 - 2 and 3 - 4
    whole = [p // page for p in prefix]
    pages = sum(whole) + 60
    pool = new_pool(g, fmt, pages, kv_heads, page, dim)
    kv = P.KvCache(pool, *((1 / 72, 1 / 90) if fmt == "fp8" else (1.0, 1.0)))
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[:3, :whole[0]] = ids[:whole[0]]
    table[3:, :whole[1]] = ids[whole[0]:sum(whole)]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:60] = ids[sum(whole):]
    plan = P.KvPlan(n, rows, page, pages, group, num_segments=2)
    kept = [w * page for w in whole]
    ctx = [kept[0]] * 3 + [kept[1]] * 2
    plan.context.copy_(ints(ctx))
    plan.free_count.fill_(60)
    first_own, seg_req, seg_ctx = ints([whole[0]] * 3 + [whole[1]] * 2), ints([0, 3, 5]), ints(kept)
    rope = P.rope_table(64, sections=(12, 10, 10), order="cycle")
    layer = P.KvLayer(kv, table, width * page, rows, H, rope=rope, rot_offset=32, rows_per_group=group, num_segments=2,
                      least_saved=1)
    new, qkv = ints([0] * n), torch.zeros(rows, H + 2 * kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    parts = qkv[:, :H], qkv[:, H:H + kv_heads], qkv[:, H + kv_heads:]

    def step():
        plan.run(plan.context, new, table, free, plan.free_count, first_own, seg_req)
        layer.run(plan.row_req, plan.row_ctx, plan.slots, plan.positions.expand(3, rows), *parts,
                  segment_rows=plan.segment_rows, segment_ctx=seg_ctx)
    if graph:
        with torch.cuda.stream(torch.cuda.Stream()):
            step()  # (of no tokens)
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    wide = lambda t: -(-t // group) * group  # noqa: E731
    for fresh in ([1, 1, 2, 1, 3], [1, -1, 2, 2, 1], [4, 0, 1, 1, 1], [2, 0, 3, 1, 0], [1, 0, 1, 1, 4]):
        new.copy_(ints(fresh))
        qkv.copy_(randn(g, rows, H + 2 * kv_heads, dim))
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        checked(plan.status)
        checked(layer.status)
        ctx = [0 if t == -1 else x + t for x, t in zip(ctx, fresh)]
        starts = [sum(wide(max(t, 0)) for t in fresh[:i]) for i in (0, 3, 5)]
        assert plan.context.tolist() == ctx and plan.segment_rows.tolist() == starts
        q = parts[0].contiguous()
        call = lambda f, *a, **k: f(kv, table, plan.row_req, plan.row_ctx, width * page, q, *a,  # noqa: E731
                                    rows_per_group=group, **k)
        want = call(P.kv_attention_shared, plan.segment_rows, seg_ctx, least_saved=1)
        assert torch.equal(layer.out, want[0]) and torch.equal(layer.lse, want[1])
        assert not torch.equal(layer.out, call(P.kv_attention)[0])
        c = object.__new__(Shared)
        c.fmt, c.dim, c.page, c.hpg, c.pool, c.table, c.sm = fmt, dim, page, hpg, pool, table, dim ** -0.5
        c.ks, c.vs, c.rows, c.row_req, c.q = kv.k_scale, kv.v_scale, plan.row_ctx.tolist(), plan.row_req, q
        c.check(layer.out, layer.lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("segments", [1, 3])
def test_a_rows_bits_depend_on_its_segment_and_the_shapes_alone(fmt, dim, segments):
    """Two calls of the same shapes, with one segment of 24 rows over many parts the same and everything else of other
    lengths, prefixes, values and places, so that SMs and items are shared out otherwise."""
    one = (9000, [9001 + 41 * i for i in range(24)])
    others = [([(300, [301 + i for i in range(8)]), one, (128, [200] * 8)], [5000 + 700 * i for i in range(6)]),
              ([(6000, [6001 + 300 * i for i in range(8)]), one, (700, [5, 3000] + [701] * 6)], [1 + i for i in range(6)])]
    cases = [Shared(52 + i, fmt, s if segments == 3 else [one], 4, 8, dim, 64, after=after if segments == 3 else
                    after + [n for _, own in (s[0], s[2]) for n in own]) for i, (s, after) in enumerate(others)]
    a, b = cases
    at = 8 if segments == 3 else 0
    most = max(c.max_ctx for c in cases)
    for c in cases:
        c.table = torch.nn.functional.pad(c.table, (0, -(-most // 64) - c.table.shape[1]))
        c.max_ctx = most
    assert len(a.rows) == len(b.rows) == 46 and a.rows != b.rows
    for r in range(at, at + 24):  # the same tokens and queries in the other batch's pages
        for p in range(-(-a.rows[r] // 64)):
            bits(b.pool)[b.table[r, p].item()] = bits(a.pool)[a.table[r, p].item()]
    b.q[at:at + 24] = a.q[at:at + 24]
    want, got = a.run(), b.run()
    assert torch.equal(got[0][at:at + 24], want[0][at:at + 24]) and torch.equal(got[1][at:at + 24], want[1][at:at + 24])
    a.check(*want, rows=[0, at, at + 11, at + 23, 45])
    b.check(*got, rows=[0, at, at + 11, at + 23, 45])
