"""The dense K/V path on the GPU against plain 64-bit evaluations of its formulas: rotary positions
(dsa_rope), the K/V insert (dsa_kv_insert), paged attention (dsa_kv_attention), and a run of them."""
import math

import pytest
import torch

import prefill_dsa_indexer_gb300 as P

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def checked(status):
    torch.cuda.synchronize()
    P.check_status(status)


# ------------------------------------------------------------------ rotary positions

def ref_rotate(x, positions, freq, scale, layout):
    """(rotated x in 64 bits, |a| + |b| of each element's pair)."""
    t = positions.double()[:, None, None] * freq.cuda()
    c, s = torch.cos(t) * scale, torch.sin(t) * scale
    x = x.double()
    n = x.shape[-1] // 2
    a, b = (x[..., :n], x[..., n:]) if layout == P.ROPE_HALF else (x[..., 0::2], x[..., 1::2])
    u, w, m = a * c - b * s, a * s + b * c, a.abs() + b.abs()
    if layout == P.ROPE_HALF:
        return torch.cat((u, w), -1), torch.cat((m, m), -1)
    return torch.stack((u, w), -1).flatten(-2), torch.stack((m, m), -1).flatten(-2)


def rope_bound(ref, mag, scale, dtype):
    """Half a step of the stored type, and before it: the phase rounded to 2^-26 turn (2^-23.3 rad), cos
    and sin to 2 ulp (2^-23) and their factor, two products and a sum (2^-24 each)."""
    return torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -21 * abs(scale) * mag + 1e-30


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [P.ROPE_INTERLEAVED, P.ROPE_HALF])
@pytest.mark.parametrize("tokens, heads, rot, pad, scaling", [
    (1, 1, 2, 0, "none"), (1, 96, 64, 512, "none"), (5, 3, 10, 7, "linear"), (33, 96, 64, 512, "yarn"),
    (7, 128, 256, 0, "ntk"), (300, 2, 48, 16, "yarn"), (2048, 9, 64, 64, "none")])
def test_rope(dtype, layout, tokens, heads, rot, pad, scaling):
    g = gen(tokens * 1000 + rot)
    full = randn(g, tokens, heads, pad + rot, dtype=dtype)
    x = full[..., pad:]
    positions = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    positions[0] = (1 << 20) - 1
    freq, scale = P.rope_frequencies(rot, 10000.0, scaling, 32.0, 4096)
    table = P.rope_table(rot, 10000.0, scaling, 32.0, 4096)
    ref, mag = ref_rotate(x, positions, freq, scale, layout)
    before = full.clone()
    out = torch.empty((tokens, heads, rot), dtype=dtype, device="cuda")
    P.rope(x, table, positions, layout=layout, out=out)
    torch.cuda.synchronize()
    assert torch.equal(full, before)
    assert ((out.double() - ref).abs() <= rope_bound(ref, mag, scale, dtype)).all()
    P.rope(x, table, positions, layout=layout)  # in place: the same bits, and nothing else touched
    torch.cuda.synchronize()
    assert torch.equal(x, out)
    assert torch.equal(full[..., :pad], before[..., :pad])


@pytest.mark.parametrize("dtype, heads, rot, pad", [(torch.bfloat16, 20, 128, 0), (torch.bfloat16, 33, 64, 512),
                                                    (torch.float32, 3, 256, 64), (torch.bfloat16, 1, 256, 0)])
@pytest.mark.parametrize("layout", [P.ROPE_INTERLEAVED, P.ROPE_HALF])
def test_rope_of_a_long_prefill(dtype, heads, rot, pad, layout):
    """Tiles of many pieces a thread, more in flight than fit its ring, with padding tokens among them."""
    g = gen(heads)
    tokens = 8195 if heads > 1 else 40001
    x = randn(g, tokens, heads, pad + rot, dtype=dtype)[..., pad:]
    positions = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    positions[torch.randint(0, tokens, (500,), generator=g, device="cuda")] = -1
    live = positions >= 0
    table, freq = P.rope_table(rot, 500000.0), P.rope_frequencies(rot, 500000.0)[0]
    out = torch.full((tokens, heads, rot), 7.0, dtype=dtype, device="cuda")
    P.rope(x, table, positions, layout=layout, out=out)
    for a in range(0, tokens, 5000):
        at = slice(a, a + 5000)
        ref, mag = ref_rotate(x[at], positions[at], freq, 1.0, layout)
        assert ((out[at].double() - ref).abs() <= rope_bound(ref, mag, 1.0, dtype))[live[at]].all()
    assert (out[~live] == 7.0).all()
    kept = x[~live].clone()
    P.rope(x, table, positions, layout=layout)
    assert torch.equal(x[live], out[live]) and torch.equal(x[~live], kept)


def test_rope_of_heads_before_tokens():
    """Tensors that lie in memory as [heads, tokens, dims], in and out."""
    g = gen(4)
    x = randn(g, 5, 40, 64).transpose(0, 1)
    positions = torch.arange(40, dtype=torch.int32, device="cuda") * 77
    table, freq = P.rope_table(64), P.rope_frequencies(64, 10000.0)[0]
    out = P.rope(x, table, positions, out=torch.empty(5, 40, 64, dtype=x.dtype, device="cuda").transpose(0, 1))
    ref, mag = ref_rotate(x, positions, freq, 1.0, P.ROPE_INTERLEAVED)
    assert ((out.double() - ref).abs() <= rope_bound(ref, mag, 1.0, x.dtype)).all()


def test_rope_several_tensors_in_one_call_and_padding_tokens():
    g = gen(3)
    n, table = 6, P.rope_table(64)
    q, lat, key, odd = randn(g, n, 96, 576), randn(g, n, 1, 576), randn(g, n, 1, 128), randn(g, n, 3, 65)
    positions = torch.tensor([5, -1, 0, 131071, -7, 9], dtype=torch.int32, device="cuda")
    xs = [q[..., 512:], lat[..., 512:], key[..., :64], odd[..., 1:]]
    layouts = [P.ROPE_INTERLEAVED, P.ROPE_INTERLEAVED, P.ROPE_HALF, P.ROPE_HALF]
    before = [x.clone() for x in xs]
    P.rope(xs, table, positions, layout=layouts)
    torch.cuda.synchronize()
    freq, scale = P.rope_frequencies(64, 10000.0)
    live = positions >= 0
    for x, b, layout in zip(xs, before, layouts):
        ref, mag = ref_rotate(b, positions, freq, scale, layout)
        assert ((x.double() - ref).abs() <= rope_bound(ref, mag, scale, x.dtype))[live].all()
        assert torch.equal(x[~live], b[~live])


@pytest.mark.parametrize("pos", [0, 1, 65535, 1048575, (1 << 31) - 1])
def test_rope_far_positions_keep_their_precision(pos):
    """Against the exact phase (integers of any size), where 32-bit angles would be off by radians."""
    table = P.rope_table(64)
    x = torch.ones(1, 1, 64, device="cuda")
    out = P.rope(x, table, torch.tensor([pos], dtype=torch.int32, device="cuda"), out=torch.empty_like(x))
    turns = [int(v) % (1 << 64) for v in table.turns.tolist()]
    for i, v in enumerate(turns):
        t = 2 * math.pi * ((pos * v % (1 << 64)) / 2.0 ** 64)
        want = (math.cos(t) - math.sin(t), math.sin(t) + math.cos(t))
        for got, w in zip(out[0, 0, 2 * i:2 * i + 2].tolist(), want):
            assert abs(got - w) <= 2.0 ** -23 * abs(w) + 2.0 ** -20


def test_rope_inverts_by_the_negative_angles():
    g = gen(9)
    freq, _ = P.rope_frequencies(64, 10000.0)
    there, back = P.rope_table(64), P.RopeTable(P.rope_turns(-freq).cuda())
    x = randn(g, 50, 4, 64, dtype=torch.float32)
    positions = torch.arange(50, dtype=torch.int32, device="cuda") * 1001
    y = P.rope(P.rope(x, there, positions, out=torch.empty_like(x)), back, positions)
    mag = (x[..., 0::2].abs() + x[..., 1::2].abs()).repeat_interleave(2, -1)
    assert ((y - x).abs() <= 2 * 2 * 2.0 ** -21 * mag).all()  # twice the bound, each of two terms


# ------------------------------------------------------------------ K/V insert

def codes(x, scale):
    return (x.float() / scale).clamp(-448, 448).to(F8)


def new_pool(g, fmt, pages, kv_heads, page, dim):
    x = randn(g, pages, kv_heads, 2, page, dim)
    return x if fmt == "bf16" else codes(x, 1 / 80)


def bits(t):
    return t.view(torch.uint8) if t.dtype == F8 else t.view(torch.int16)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("tokens, kv_heads, heads, dim, page, rot, off, layout", [
    (1, 1, 1, 64, 16, 0, 0, P.ROPE_HALF), (1, 4, 64, 128, 128, 64, 0, P.ROPE_HALF),
    (37, 3, 5, 64, 32, 64, 0, P.ROPE_INTERLEAVED), (70, 2, 6, 128, 64, 32, 96, P.ROPE_HALF),
    (9, 2, 2, 128, 64, 18, 3, P.ROPE_HALF), (9, 2, 3, 128, 64, 22, 7, P.ROPE_INTERLEAVED),
    (1000, 8, 8, 128, 128, 128, 0, P.ROPE_HALF), (8195, 4, 33, 128, 128, 64, 32, P.ROPE_HALF),
    (8195, 8, 70, 64, 16, 64, 0, P.ROPE_INTERLEAVED)])
def test_kv_insert(fmt, tokens, kv_heads, heads, dim, page, rot, off, layout):
    g = gen(tokens + dim + rot)
    pages = tokens // page + 4
    pool = new_pool(g, fmt, pages, kv_heads, page, dim)
    ks, vs = (1 / 72, 1 / 90) if fmt == "fp8" else (1.0, 1.0)
    qkv = randn(g, tokens, heads + 2 * kv_heads, dim)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].to(torch.int32)
    if tokens > 5:
        slots[3] = -1
    positions = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    before, q_before, status = pool.clone(), qkv.clone(), P.new_status()
    cache = P.KvCache(pool, ks, vs)
    if rot:
        table = P.rope_table(rot, 10000.0, "yarn", 8.0, 4096)
        part = q[..., off:off + rot]
        P.kv_insert(cache, slots, k, v, rope=table, positions=positions, layout=layout, rot_offset=off, q=part,
                    status=status)
    else:
        P.kv_insert(cache, slots, k, v, status=status)
    checked(status)
    live = slots >= 0
    at, row = (slots[live] // page).long(), (slots[live] % page).long()
    # V, and K's dims outside the rotary part: the exact bytes
    store = (lambda x, s: codes(x, s)) if fmt == "fp8" else (lambda x, s: x)
    assert torch.equal(bits(pool)[at, :, 1, row], bits(store(v[live].contiguous(), vs)))
    plain = [d for d in range(dim) if not off <= d < off + rot]
    assert torch.equal(bits(pool)[at, :, 0, row][..., plain], bits(store(k[live].contiguous(), ks))[..., plain])
    if rot:
        freq, scale = P.rope_frequencies(rot, 10000.0, "yarn", 8.0, 4096)
        ref, mag = ref_rotate(k[..., off:off + rot], positions, freq, scale, layout)
        ref, mag = ref[live] / ks, mag[live] / ks
        got = bits(pool)[at, :, 0, row][..., off:off + rot].contiguous().view(pool.dtype).double()
        eps = 2.0 ** -4 if fmt == "fp8" else 2.0 ** -8
        # half a step of the format (e4m3: at least 2^-10, saturating), the division, the rotation's fp32
        bound = eps * ref.abs() + (2.0 ** -10 if fmt == "fp8" else 0) + (2.0 ** -21 * scale + 2.0 ** -23) * mag
        top = 448 if fmt == "fp8" else math.inf
        assert ((got - ref.clamp(-top, top)).abs() <= bound).all()
        qr, qm = ref_rotate(q_before[:, :heads][..., off:off + rot], positions, freq, scale, layout)
        assert ((q[..., off:off + rot].double() - qr).abs() <= rope_bound(qr, qm, scale, torch.bfloat16)).all()
        q_before[:, :heads, off:off + rot] = q[..., off:off + rot]
    assert torch.equal(qkv, q_before)  # nothing but q's rotary part changed
    bits(before)[at, :, :, row] = bits(pool)[at, :, :, row]
    assert torch.equal(bits(pool), bits(before))  # nor any other slot


def test_kv_insert_saturates_and_keeps_nan():
    pool = torch.zeros(1, 1, 2, 16, 64, dtype=torch.uint8, device="cuda")
    k = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    k[0, 0, :6] = torch.tensor([1e30, -1e30, math.inf, -math.inf, math.nan, -0.0])
    P.kv_insert(P.KvCache(pool), torch.tensor([5], dtype=torch.int32, device="cuda"), k, k)
    got = pool[0, 0, 0, 5, :6].tolist()
    assert got[:4] == [0x7E, 0xFE, 0x7E, 0xFE] and got[4] & 0x7F == 0x7F and got[5] == 0x80


def test_kv_insert_reports_bad_slots_and_writes_the_others():
    g = gen(1)
    pool = new_pool(g, "bf16", 3, 2, 16, 64)
    before = pool.clone()
    k, v = randn(g, 4, 2, 64), randn(g, 4, 2, 64)
    table = P.rope_table(64)
    for slots, positions, good in (([48, 7, -1, 2147483647], [1, 2, 3, 4], {7: 1}),
                                   ([3, 9, 20, -1], [1, -1, 2, -1], {3: 0, 20: 2})):
        pool.copy_(before)
        status = P.new_status()
        P.kv_insert(P.KvCache(pool), torch.tensor(slots, dtype=torch.int32, device="cuda"), k, v, rope=table,
                    positions=torch.tensor(positions, dtype=torch.int32, device="cuda"), status=status)
        torch.cuda.synchronize()
        assert status.item() == P.ERR_BOUNDS
        rest = before.clone()
        for s, i in good.items():
            assert torch.equal(pool[s // 16, :, 1, s % 16], v[i])
            rest[s // 16, :, :, s % 16] = pool[s // 16, :, :, s % 16]
        assert torch.equal(pool, rest)


# ------------------------------------------------------------------ attention

class Case:
    """Requests of given contexts in shuffled pages; slots that hold no token are NaN."""

    def __init__(self, seed, fmt, ctx, kv_heads, hpg, dim, page, group=1, row_ctx=None, q_scale=1.0):
        g = gen(seed)
        self.fmt, self.dim, self.page, self.hpg, self.group = fmt, dim, page, hpg, group
        need = [-(-n // page) for n in ctx]
        pages = sum(need) + 2
        pool = new_pool(g, fmt, pages, kv_heads, page, dim)
        self.ks, self.vs = (1 / 72, 1 / 90) if fmt == "fp8" else (1.0, 1.0)
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.max_ctx = max(max(ctx), 1)
        self.table = torch.full((len(ctx), -(-self.max_ctx // page)), 0x7FFFFFF, dtype=torch.int32, device="cuda")
        nan = 0x7F if fmt == "fp8" else 0x7FFF
        at = 0
        b = bits(pool)
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            if n and ctx[i] % page:
                b[order[at + n - 1].item(), :, :, ctx[i] % page:] = nan
            at += n
        for p in order[at:].tolist():
            b[p] = nan
        self.pool, self.kv = pool, P.KvCache(pool, self.ks, self.vs)
        self.rows = row_ctx if row_ctx is not None else [max(0, n - (group - 1 - i)) for n in ctx for i in range(group)]
        self.row_req = torch.arange(len(self.rows), dtype=torch.int32, device="cuda") // group
        self.row_ctx = torch.tensor(self.rows, dtype=torch.int32, device="cuda")
        self.q = (randn(g, len(self.rows), kv_heads * hpg, dim).float() * q_scale).to(torch.bfloat16)
        self.sm = dim ** -0.5

    def run(self, **kw):
        status = P.new_status()
        got = P.kv_attention(self.kv, self.table, self.row_req, self.row_ctx, self.max_ctx, kw.pop("q", self.q),
                             rows_per_group=self.group, status=status, **kw)
        checked(status)
        return got

    def tokens(self, r, h):
        """K and V of row r's KV head h in 64 bits, over the tokens that the row sees."""
        n = self.rows[r]
        pages = self.table[r // self.group, :-(-n // self.page)].long()
        kv = bits(self.pool)[pages, h].contiguous().view(self.pool.dtype).double()
        return [kv[:, i].reshape(-1, self.dim)[:n] * s for i, s in ((0, self.ks), (1, self.vs))]

    def check(self, out, lse, rows=None):
        H = self.q.shape[1]
        assert out.shape == (len(self.rows), H, self.dim) and lse.shape == (len(self.rows), H)
        for r in range(len(self.rows)) if rows is None else rows:
            n = self.rows[r]
            if n == 0:
                assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
                continue
            for h in range(H // self.hpg):
                at = slice(h * self.hpg, (h + 1) * self.hpg)
                k, v = self.tokens(r, h)
                q = self.q[r, at].double()
                s = q @ k.T * self.sm
                p = torch.softmax(s, -1)
                ref, mag = p @ v, p @ v.abs()
                # scores: `dim` fp32 sums of products up to big, and the exponent's argument
                big = (q.abs() @ k.abs().T * self.sm).amax(-1, keepdim=True)
                ds = (self.dim + 8) * 2.0 ** -24 * big
                # weights: two bf16 terms (2^-16), two e4m3 terms (each rounds to 4 significant bits, half a
                # step being 2^-4: 2^-8; and half of e4m3's smallest step, 2^-10, where the largest weight is at
                # least 2^6 / 2), exp2 (2^-22), sums over n tokens in fp32
                w = (2.0 ** -8 if self.fmt == "fp8" else 2.0 ** -16) + 2.0 ** -22 + n * 2.0 ** -24
                sub = 2.0 ** -15 * p.amax(-1, keepdim=True) * v.abs().sum(0) if self.fmt == "fp8" else 0
                bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * ((w + 2 * ds) * mag + sub) + 1e-30
                off = (out[r, at].double() - ref).abs()
                assert (off <= bound).all(), (r, h, (off / bound).max().item())
                want = torch.logsumexp(s, -1)
                lb = ds[:, 0] + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * want.abs()
                assert ((lse[r, at].double() - want).abs() <= lb).all(), (r, h)


SHAPES = [(1, 1, 64, 16), (4, 16, 128, 128), (4, 8, 128, 64), (3, 5, 64, 32), (2, 7, 128, 16), (1, 33, 64, 64),
          (2, 64, 128, 128), (1, 128, 64, 128)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("kv_heads, hpg, dim, page", SHAPES)
def test_attention_short_and_odd_contexts(fmt, kv_heads, hpg, dim, page):
    c = Case(11, fmt, [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300], kv_heads, hpg, dim, page)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("kv_heads, hpg, dim, page", [(4, 16, 128, 128), (2, 5, 64, 16), (1, 40, 128, 64)])
def test_attention_long_ragged_contexts(fmt, kv_heads, hpg, dim, page):
    c = Case(12, fmt, [4096, 1000, 8192, 8193, 0, 20001, 33000], kv_heads, hpg, dim, page)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("group, kv_heads, hpg, dim, page", [(2, 2, 3, 64, 16), (4, 2, 16, 128, 128), (8, 1, 4, 128, 64),
                                                            (8, 2, 16, 64, 32), (2, 2, 16, 128, 32), (4, 1, 7, 128, 16),
                                                            (8, 1, 16, 128, 128)])
def test_attention_verify_rows(fmt, group, kv_heads, hpg, dim, page):
    c = Case(13, fmt, [group, 70, 129, 8192 + group // 2, 3000], kv_heads, hpg, dim, page, group=group)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_attention_group_of_very_different_contexts(fmt):
    c = Case(14, fmt, [5000, 400], 2, 4, 128, 64, group=4, row_ctx=[0, 5000, 64, 1300, 400, 1, 399, 130])
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("q_scale", [0.0, 30.0, 1e-3])
def test_attention_peaked_and_flat_scores(fmt, q_scale):
    c = Case(15, fmt, [2500, 130], 2, 6, 128, 64, q_scale=q_scale)
    c.check(*c.run())


def test_attention_huge_queries_over_an_fp8_pool():
    """bf16 queries far outside fp16's range on both sides."""
    c = Case(16, "fp8", [700], 2, 4, 128, 64)
    c.sm = 1e-30
    c.q = (c.q.float() * 1e30).to(torch.bfloat16)
    c.check(*c.run(sm_scale=1e-30))
    c.q = (c.q.float() * 1e-32 * 1e-28).to(torch.bfloat16)
    c.sm = 1e28
    c.check(*c.run(sm_scale=1e28))


@pytest.mark.parametrize("fmt, dim", [("bf16", 64), ("bf16", 128), ("fp8", 64), ("fp8", 128)])
@pytest.mark.parametrize("hpg, group", [(5, 1), (16, 2), (16, 4)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attention_a_head_of_no_numbers_stays_alone(fmt, dim, hpg, group, value):
    """A NaN or an infinity in one head's query reaches neither its neighbours nor the other rows of its group."""
    c = Case(49, fmt, [700, 90], 2, hpg, dim, 32, group=group)
    want = c.run()
    q, r, h = c.q.clone(), len(c.rows) - 1, hpg + 2
    q[r, h, 3] = value
    out, lse = c.run(q=q)
    assert torch.isnan(out[r, h]).any() and not torch.isfinite(lse[r, h])
    rest = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    rest[r, h] = False
    c.check(out, lse, rows=range(r))
    assert torch.isfinite(out[rest].float()).all()
    assert torch.equal(out[:r], want[0][:r]) or fmt == "fp8"  # (an FP8 group's bases move together)


def test_attention_rows_of_a_packed_projection():
    c = Case(17, "bf16", [513, 77, 2000], 4, 8, 128, 64)
    packed = torch.zeros(3, 32 + 8, 128, dtype=torch.bfloat16, device="cuda")
    packed[:, :32] = c.q
    a, b = c.run(q=packed[:, :32]), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_of_very_many_rows(fmt, dim):
    """More row groups than a launch keeps running costs for, most of them short or empty."""
    g = gen(21)
    ctx = torch.randint(0, 40, (1301,), generator=g, device="cuda").tolist()
    for i in range(0, 1301, 97):
        ctx[i] = 3 * i
    c = Case(22, fmt, ctx, 2, 3, dim, 16)
    out, lse = c.run()
    c.check(out, lse, rows=list(range(0, 1301, 97)) + list(range(5, 1301, 41)) + [1299, 1300])
    empty = torch.tensor([n == 0 for n in ctx], device="cuda")
    assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all() and torch.isfinite(lse[~empty]).all()
    assert torch.equal(c.run()[0], out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_attention_when_no_row_sees_anything(fmt):
    c = Case(23, fmt, [0, 0, 0], 2, 16, 128, 64)
    c.max_ctx, c.table = 70000, torch.full((3, 1094), 0x7FFFFFF, dtype=torch.int32, device="cuda")
    out, lse = c.run()
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_attention_row_does_not_depend_on_its_batch(fmt):
    ctx = [9000, 128, 40000, 1, 700]
    c = Case(18, fmt, ctx, 2, 8, 128, 64)
    out, lse = c.run()
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for r, n in enumerate(ctx):  # alone, and with the tightest bound on its length
        one, l1 = P.kv_attention(c.kv, c.table, c.row_req[r:r + 1].contiguous(), c.row_ctx[r:r + 1].contiguous(), n,
                                 c.q[r:r + 1].contiguous())
        torch.cuda.synchronize()
        assert torch.equal(one[0], out[r]) and torch.equal(l1[0], lse[r])


@pytest.mark.parametrize("fmt, value", [("bf16", math.nan), ("bf16", math.inf), ("bf16", -math.inf), ("fp8", math.nan)])
@pytest.mark.parametrize("dim, hpg", [(64, 5), (128, 5), (128, 7), (128, 16)])
@pytest.mark.parametrize("what", ["k", "v", "both"])
def test_attention_values_past_a_rows_context_never_reach_it(fmt, value, dim, hpg, what):
    """A verify group whose newer tokens are not finite: the rows that do not see them are unharmed."""
    ctx = [200, 64, 130]
    clean = Case(19, fmt, ctx, 2, hpg, dim, 16, group=4)
    want = clean.run()
    c = Case(19, fmt, ctx, 2, hpg, dim, 16, group=4)
    side = {"k": slice(0, 1), "v": slice(1, 2), "both": slice(0, 2)}[what]
    for req, n in enumerate(ctx):
        for t in (n - 2, n - 1):  # seen by the last two rows, and by the last alone
            c.pool[c.table[req, t // 16].item(), :, side, t % 16] = value
    got = c.run()
    for r in (0, 1, 4, 5, 8, 9):
        assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1][r], want[1][r])
    if value != value:
        for r in (2, 3, 6, 7, 10, 11):
            assert got[0][r].isnan().all()
            assert got[1][r].isnan().all() or (what == "v" and torch.equal(got[1][r], want[1][r]))


def test_attention_scores_of_minus_infinity_weigh_nothing():
    c = Case(20, "bf16", [300, 90], 1, 4, 64, 16)
    c.q = c.q.abs() + 0.5
    for t in list(range(0, 300, 3)):
        c.pool[c.table[0, t // 16].item(), :, 0, t % 16] = -math.inf
    for t in range(90):
        c.pool[c.table[1, t // 16].item(), :, 0, t % 16] = -math.inf
    out, lse = c.run(q=c.q)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    keep = [t for t in range(300) if t % 3]
    k, v = (x[keep] for x in c.tokens(0, 0))
    s = c.q[0].double() @ k.T * c.sm
    ref = torch.softmax(s, -1) @ v
    assert ((out[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * v.abs().amax()).all()
    assert ((lse[0].double() - torch.logsumexp(s, -1)).abs() <= 2.0 ** -17).all()


def test_attention_agrees_with_the_block_sparse_layer_that_keeps_every_block():
    """At most 16 blocks: dsa_msa_attention attends to every token of the same pool."""
    from prefill_dsa_indexer_gb300 import inputs as I
    wl = I.small_msa_workload("all", [2048, 1500, 77])
    m = I.make_msa_inputs(wl).to("cuda")
    R, sm = wl.num_rows, 128 ** -0.5
    blocks = torch.full((R, 4, 16), -1, dtype=torch.int32, device="cuda")
    for r, n in enumerate(wl.ctx):
        nb = -(-n // 128)
        blocks[r, :, :nb] = torch.arange(nb, dtype=torch.int32, device="cuda")
    a, la = P.msa_attention(m.kv_pool, m.k_scale, m.v_scale, m.block_table, m.row_req, m.row_ctx, max(wl.ctx), m.q,
                            m.q_scale, blocks, sm)
    q = m.q.view(F8).to(torch.bfloat16)  # e4m3 codes are exact in bf16
    kv = P.KvCache(m.kv_pool.view(-1, 4, 2, 128, 128), m.k_scale, m.v_scale)
    b, lb = P.kv_attention(kv, m.block_table, m.row_req, m.row_ctx, max(wl.ctx), q, sm_scale=sm * m.q_scale)
    torch.cuda.synchronize()
    # both round their weights to fp16 (2^-11 of values up to max|V|), the second its output to bf16
    big = 448 * m.v_scale
    assert ((a - b.float()).abs() <= 2.0 ** -8 * a.abs() + 2 * 2.0 ** -10 * big).all()
    assert ((la - lb).abs() <= 2e-3).all()


def test_device_errors_of_attention_are_reported():
    c = Case(21, "fp8", [300, 300], 2, 4, 128, 64)
    def status_of(table=c.table, req=c.row_req, ctx=c.row_ctx, max_ctx=c.max_ctx, group=1):
        st = P.new_status()
        P.kv_attention(c.kv, table, req, ctx, max_ctx, c.q, rows_per_group=group, status=st)
        torch.cuda.synchronize()
        return st.item()
    assert status_of() == P.OK
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for page in (-1, c.pool.shape[0], 2 ** 31 - 1):
        t = c.table.clone()
        t[1, 2] = page
        assert status_of(table=t) == P.ERR_BOUNDS
    assert status_of(ctx=i32(300, 301)) == P.ERR_BOUNDS
    assert status_of(ctx=i32(-1, 300)) == P.ERR_BOUNDS
    assert status_of(req=i32(0, 2)) == P.ERR_BOUNDS
    assert status_of(req=i32(0, -1)) == P.ERR_BOUNDS
    assert status_of(group=2) == P.ERR_BOUNDS  # rows of one group, two requests
    c.check(*c.run())


def test_slots_past_32_bit_offsets():
    """A pool of more than 4 GiB whose tokens are in its last pages: insert, then attend."""
    pages, page, heads, dim = 36000, 128, 4, 128  # 4.4 GiB of codes, 9.0 GiB of bf16
    for dtype in (torch.bfloat16, torch.uint8):
        pool = torch.empty((pages, heads, 2, page, dim), dtype=dtype, device="cuda")
        kv = P.KvCache(pool, *((1 / 72, 1 / 90) if dtype == torch.uint8 else ()))
        g = gen(4)
        n = 200
        k, v, q = randn(g, n, heads, dim), randn(g, n, heads, dim), randn(g, 1, 8, dim)
        table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
        t = torch.arange(n, device="cuda", dtype=torch.int32)
        st = P.new_status()
        P.kv_insert(kv, table[0][(t // page).long()] * page + t % page, k, v, status=st)
        one = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = P.kv_attention(kv, table, one, one + n, n, q, status=st)
        checked(st)
        far = out.clone(), lse.clone()
        small = torch.empty((2, heads, 2, page, dim), dtype=dtype, device="cuda")
        kv2 = P.KvCache(small, kv.k_scale, kv.v_scale)
        table2 = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
        P.kv_insert(kv2, table2[0][(t // page).long()] * page + t % page, k, v, status=st)
        out, lse = P.kv_attention(kv2, table2, one, one + n, n, q, status=st)
        checked(st)
        assert torch.equal(out, far[0]) and torch.equal(lse, far[1])
        del pool, kv


# ------------------------------------------------------------------ a run of them

def step_inputs(g, R, heads, kv_heads, dim):
    qkv = randn(g, R, heads + 2 * kv_heads, dim)
    return qkv, (qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_steps_over_a_growing_cache(fmt, graph):
    """Four steps of three requests (and a padding row): rotate, insert, attend, against the formulas over
    everything that was put in; captured once and replayed for every step, or eagerly."""
    g = gen(30)
    dim, page, kv_heads, hpg = 128, 32, 2, 4
    H, ctx, steps = kv_heads * hpg, [126, 1, 700], 4
    c = Case(31, fmt, [n + steps for n in ctx], kv_heads, hpg, dim, page)
    table = P.rope_table(64)
    layer = P.KvLayer(c.kv, c.table, c.max_ctx, 4, H, rope=table, rot_offset=32)
    req = torch.tensor([0, 1, 2, 0], dtype=torch.int32, device="cuda")
    bufs = dict(row_ctx=torch.zeros(4, dtype=torch.int32, device="cuda"),
                slots=torch.full((4,), -1, dtype=torch.int32, device="cuda"),
                positions=torch.full((4,), -1, dtype=torch.int32, device="cuda"),
                qkv=torch.zeros(4, H + 2 * kv_heads, dim, dtype=torch.bfloat16, device="cuda"))
    parts = bufs["qkv"][:, :H], bufs["qkv"][:, H:H + kv_heads], bufs["qkv"][:, H + kv_heads:]
    step = lambda: layer.run(req, bufs["row_ctx"], bufs["slots"], bufs["positions"], *parts)  # noqa: E731
    if graph:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for i in range(steps):
        pos = [n + i for n in ctx]
        slots = [c.table[r, p // page].item() * page + p % page for r, p in enumerate(pos)]
        bufs["positions"].copy_(torch.tensor(pos + [-1], dtype=torch.int32))
        bufs["slots"].copy_(torch.tensor(slots + [-1], dtype=torch.int32))
        bufs["row_ctx"].copy_(torch.tensor([p + 1 for p in pos] + [0], dtype=torch.int32))
        qkv, _ = step_inputs(g, 4, H, kv_heads, dim)
        bufs["qkv"].copy_(qkv)
        layer.out.fill_(7.0)
        captured.replay() if graph else step()
        checked(layer.status)
        # the padding row: q untouched, an empty answer
        assert torch.equal(bufs["qkv"][3], qkv[3]) and (layer.out[3] == 0).all() and (layer.lse[3] == -math.inf).all()
        freq, _ = P.rope_frequencies(64, 10000.0)
        ref, mag = ref_rotate(qkv[:3, :H, 32:96], bufs["positions"][:3], freq, 1.0, P.ROPE_HALF)
        assert ((bufs["qkv"][:3, :H, 32:96].double() - ref).abs() <= rope_bound(ref, mag, 1.0, torch.bfloat16)).all()
        # attention over what the pool now holds, by the queries as they were rotated
        c.rows, c.q = [p + 1 for p in pos], bufs["qkv"][:3, :H].clone()
        c.check(layer.out[:3], layer.lse[:3])


def test_calls_on_another_stream_and_two_at_once():
    a, b = Case(40, "bf16", [5000, 12], 2, 8, 128, 64), Case(41, "fp8", [9000, 300], 4, 4, 64, 32)
    want = a.run(), b.run()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, st in zip((a, b), s):
            with torch.cuda.stream(st):
                got.append(P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, stream=st))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_calls_on_a_stream_that_is_not_current():
    """What a call allocates for itself belongs to the stream that it is given."""
    c = Case(46, "bf16", [30000, 4000], 2, 8, 128, 64)
    want, st = c.run(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, stream=st))
        torch.full((4 << 20,), 7.0, device="cuda")  # the current stream's own allocations
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_two_captured_graphs_and_an_eager_call_at_once():
    """Each capture has a workspace of its own, so they may run beside each other and beside an eager call."""
    a, b = Case(42, "fp8", [9000, 12, 300], 2, 8, 128, 64, group=2), Case(43, "bf16", [20000], 4, 4, 64, 32)
    want = a.run(), b.run()
    graphs, outs, spaces = [], [], []  # (a graph does not keep its workspace alive)
    for c in (a, b, a):
        need = P.kv_attention_workspace_size(c.kv, c.q.shape[0], c.q.shape[1], c.max_ctx)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        o, l = torch.empty_like(want[0][0] if c is a else want[1][0]), torch.empty_like(want[0][1] if c is a else want[1][1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            P.kv_attention(c.kv, c.table, c.row_req, c.row_ctx, c.max_ctx, c.q, rows_per_group=c.group, out=o, lse=l,
                           workspace=ws)
        graphs.append(graph)
        outs.append((o, l))
        spaces.append(ws)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for o, l in outs:
            o.fill_(7.0)
            l.fill_(7.0)
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
                graph.replay()
        eager = b.run()
        torch.cuda.synchronize()
        for (o, l), w in zip(outs + [eager], (want[0], want[1], want[0], want[1])):
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_layer_without_rotary_positions():
    g = gen(44)
    c = Case(45, "bf16", [33, 64], 2, 4, 64, 16)
    layer = P.KvLayer(c.kv, c.table, c.max_ctx, 2, 8)
    slots = torch.tensor([c.table[r, p // 16].item() * 16 + p % 16 for r, p in enumerate((32, 63))], dtype=torch.int32,
                         device="cuda")
    k, v = randn(g, 2, 2, 64), randn(g, 2, 2, 64)
    out, lse = layer.run(c.row_req, c.row_ctx, slots, None, c.q, k, v)
    checked(layer.status)
    for r, s in enumerate(slots.tolist()):
        assert torch.equal(c.pool[s // 16, :, 0, s % 16], k[r]) and torch.equal(c.pool[s // 16, :, 1, s % 16], v[r])
    c.check(out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_calls_without_a_token(fmt):
    """No token, no row: nothing is launched or touched."""
    g = gen(47)
    c = Case(48, fmt, [20], 2, 4, 128, 16)
    table, none = P.rope_table(64), torch.empty(0, dtype=torch.int32, device="cuda")
    before = bits(c.pool).clone()
    k = randn(g, 0, 2, 128)
    q = randn(g, 0, 8, 128)[..., :64]
    assert P.kv_insert(c.kv, none, k, k, rope=table, positions=none, q=q).shape == (0, 8, 64)
    assert P.kv_insert(c.kv, none, k, k) is None
    assert P.rope(q, table, none).shape == (0, 8, 64)
    out, lse = P.kv_attention(c.kv, c.table, none, none, c.max_ctx, randn(g, 0, 8, 128))
    torch.cuda.synchronize()
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8) and torch.equal(bits(c.pool), before)


def test_binding_refusals():
    c = Case(50, "bf16", [100], 2, 4, 64, 16)
    call = lambda **k: P.kv_attention(**{**dict(kv=c.kv, block_table=c.table, row_req=c.row_req, row_ctx=c.row_ctx,  # noqa: E731
                                                max_ctx=c.max_ctx, q=c.q), **k})
    for bad in (dict(q=c.q.half()), dict(q=c.q[..., :32]), dict(q=c.q.transpose(0, 1)), dict(q=c.q.cpu()),
                dict(block_table=c.table.long()), dict(row_ctx=c.row_ctx.long()), dict(row_req=c.row_req[:0]),
                dict(out=c.q.float()), dict(max_ctx=10 ** 6), dict(rows_per_group=3), dict(sm_scale=0.0),
                dict(block_table=c.table[0])):
        with pytest.raises(P.DsaError):
            call(**bad)
    k = randn(gen(1), 3, 2, 64)
    slots, pos = (torch.arange(3, dtype=torch.int32, device="cuda") for _ in range(2))
    ins = lambda **kw: P.kv_insert(**{**dict(kv=c.kv, slots=slots, k=k, v=k), **kw})  # noqa: E731
    table = P.rope_table(64)
    for bad in (dict(k=k.float()), dict(k=k[:2]), dict(k=k.transpose(1, 2)), dict(slots=slots.long()),
                dict(rope=table), dict(q=k), dict(rope=table, positions=pos[:2]), dict(rope=table, positions=pos, rot_offset=8),
                dict(rope=table, positions=pos, q=k[:2]), dict(rope=table, positions=pos, q=k.float())):
        with pytest.raises(P.DsaError):
            ins(**bad)
    for bad in (dict(slots=slots[:, None]), dict(slots=slots[:2]), dict(slots=torch.arange(6, dtype=torch.int32,
                                                                                           device="cuda")[::2]),
                dict(slots=slots.cpu()), dict(v=k.cpu()), dict(v=k[..., :32])):
        with pytest.raises(P.DsaError):
            ins(**bad)
    rope = lambda x=k, pos=pos, **kw: P.rope(x, table, pos, **kw)  # noqa: E731
    for bad in (dict(x=[]), dict(x=[k] * 5), dict(x=k[0]), dict(x=k.half()), dict(x=k.cpu()), dict(x=k[..., :32]),
                dict(x=[k, k]), dict(x=[k, k[:2]]), dict(x=[k, k.float()], out=[k.clone(), k.float()]),
                dict(layout=[0]), dict(x=[k], layout=[0, 1]), dict(out=k[:2].clone()), dict(out=k.float()),
                dict(pos=pos[:2]), dict(pos=pos.long()), dict(pos=pos[:, None]), dict(layout=7),
                dict(x=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(P.DsaError):
            rope(**bad)
    x = randn(gen(1), 3, 2, 64)
    for bad in (dict(x=x.half()), dict(x=x[..., :32]), dict(x=[x] * 5), dict(x=[x, x[:2]]), dict(x=x[0]),
                dict(x=x, out=x.float()), dict(x=x, out=x[:2]), dict(x=x.cpu()), dict(x=[x], layout=[0, 1])):
        with pytest.raises(P.DsaError):
            P.rope(table=table, positions=pos, **bad)
