"""The dense K/V path (rotary positions, K/V insert, paged attention) as far as it needs no GPU: the
host helpers against their formulas in 64 bits, and every refusal of the C ABI and of the binding."""
import ctypes
import math

import pytest
import torch

import prefill_dsa_indexer_gb300 as P
from prefill_dsa_indexer_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P.load_library()


FAKE, ODD = 0x10000, 0x10008


def kv(base=FAKE, fmt=P.KV_FP8, page=64, pages=10, heads=4, dim=128, ks=1.0, vs=1.0):
    return P._KvCache(base, fmt, page, pages, heads, dim, ks, vs)


def rows(n=1, ctx=256, stride=4, g=1, table=FAKE, reqs=1):
    return P._Rows(table, stride, reqs, FAKE, FAKE, n, ctx, g)


# ------------------------------------------------------------------ host helpers

@pytest.mark.parametrize("rot", [2, 10, 64, 256])
@pytest.mark.parametrize("scaling", list(P.ROPE_SCALINGS))
def test_frequencies_follow_their_formulas(lib, rot, scaling):
    theta, factor, trained = 10000.0, 32.0, 4096
    got, scale = P.rope_frequencies(rot, theta, scaling, factor, trained)
    for i in range(rot // 2):
        base = theta * factor ** (rot / max(rot - 2, 1)) if scaling == "ntk" else theta
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            e = [rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (32.0, 1.0)]
            lo, hi = max(math.floor(e[0]), 0), min(math.ceil(e[1]), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        # a handful of 64-bit operations and one pow of an exponent up to ln(1e7)
        assert abs(got[i].item() - f) <= 64 * 2.0 ** -53 * f
    assert scale == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=2.0 ** -23)


def test_yarn_of_factor_one_changes_nothing(lib):
    a, s = P.rope_frequencies(64, 10000.0, "yarn", 1.0, 4096)
    b, _ = P.rope_frequencies(64, 10000.0)
    assert s == 1.0 and torch.allclose(a, b, rtol=2.0 ** -50, atol=0)


def test_turns_are_the_fraction_of_a_turn_and_wrap_exactly(lib):
    f = torch.tensor([0.0, 2 * math.pi, 1.0, 1e-4, 7.0, -1.0, -1e-30, 3.25], dtype=torch.float64)
    t = [v % (1 << 64) for v in P.rope_turns(f).tolist()]
    assert t[0] == 0 and t[6] == 0
    for x, v in zip(f.tolist(), t):
        for pos in (1, 4095, (1 << 20) + 7):
            # the phase of pos, whole turns dropped, against pos * x in 64 bits: x / 2 pi is rounded
            # once (2^-53 of it, at least 2^-54 of a turn), and so is the product compared with
            got = pos * v % (1 << 64) / 2.0 ** 64
            want = (pos * x / (2 * math.pi)) % 1.0
            d = abs(got - want)
            assert min(d, 1 - d) <= pos * (abs(x) + 1) * 2.0 ** -50


def test_helper_refusals(lib):
    d, s = (ctypes.c_double * 128)(), ctypes.c_float()
    ok = lambda *a: lib.dsa_rope_frequencies(*a, d, ctypes.byref(s))  # noqa: E731
    assert ok(64, 1e4, 0, 0.0, 0) == P.OK
    for bad in ((0, 1e4, 0, 1.0, 0), (7, 1e4, 0, 1.0, 0), (64, 1.0, 0, 1.0, 0), (64, float("nan"), 0, 1.0, 0),
                (64, float("inf"), 0, 1.0, 0), (64, 1e4, 1, 0.5, 0), (64, 1e4, 1, float("nan"), 0),
                (64, 1e4, 3, 2.0, 0), (64, 1e300, 2, 1e300, 0)):
        assert ok(*bad) == P.ERR_INVALID_ARG, bad
    assert ok(258, 1e4, 0, 1.0, 0) == P.ERR_UNSUPPORTED
    assert ok(64, 1e4, 4, 1.0, 0) == P.ERR_UNSUPPORTED
    assert lib.dsa_rope_frequencies(64, 1e4, 0, 1.0, 0, None, ctypes.byref(s)) == P.ERR_INVALID_ARG
    x = (ctypes.c_double * 1)(float("inf"))
    assert lib.dsa_rope_turns(x, 1, (ctypes.c_uint64 * 1)()) == P.ERR_INVALID_ARG
    assert lib.dsa_rope_turns(None, 1, None) == P.ERR_INVALID_ARG
    assert lib.dsa_rope_turns(None, 0, None) == P.OK
    with pytest.raises(P.DsaError):
        P.rope_frequencies(64, 1e4, "other")
    with pytest.raises(P.DsaError):
        P.rope_turns(torch.zeros(4))


# ------------------------------------------------------------------ C-ABI refusals (no launch)

def test_rope_refusals(lib):
    spec = P._RopeSpec(FAKE, FAKE, 64, 1.0)
    t = lambda x=FAKE, out=FAKE, heads=4, layout=0, xs=(256, 64), os=(256, 64): \
        P._RopeTensor(x, out, heads, layout, *xs, *os)  # noqa: E731
    call = lambda sp, ts, n=1, dt=1, tok=3: lib.dsa_rope(sp, ts, n, dt, tok, None)  # noqa: E731
    one = (P._RopeTensor * 1)(t())
    assert call(spec, one, tok=0) == P.OK
    assert call(spec, one, tok=-1) == P.ERR_INVALID_ARG
    assert call(spec, one, n=0) == P.ERR_INVALID_ARG
    assert call(spec, one, n=5) == P.ERR_UNSUPPORTED
    assert call(spec, one, dt=3) == P.ERR_UNSUPPORTED
    assert call(spec, None) == P.ERR_INVALID_ARG
    assert call(None, one) == P.ERR_INVALID_ARG
    for bad in (P._RopeSpec(None, FAKE, 64, 1.0), P._RopeSpec(FAKE, None, 64, 1.0), P._RopeSpec(FAKE, FAKE, 0, 1.0),
                P._RopeSpec(FAKE, FAKE, 63, 1.0), P._RopeSpec(FAKE, FAKE, 64, float("nan"))):
        assert call(bad, one) == P.ERR_INVALID_ARG
    assert call(P._RopeSpec(FAKE, FAKE, 258, 1.0), one) == P.ERR_UNSUPPORTED
    for bad in (t(x=None), t(out=None), t(heads=0), t(x=FAKE + 1), t(os=(512, 64)), t(out=2 * FAKE, os=(-256, 64))):
        assert call(spec, (P._RopeTensor * 1)(bad)) == P.ERR_INVALID_ARG
    assert call(spec, (P._RopeTensor * 1)(t(x=FAKE + 2)), dt=2) == P.ERR_INVALID_ARG
    assert call(spec, (P._RopeTensor * 1)(t(layout=2))) == P.ERR_UNSUPPORTED
    assert call(spec, (P._RopeTensor * 1)(t(heads=4097))) == P.ERR_UNSUPPORTED


def test_rope_outputs_that_overlap_are_refused(lib):
    spec = P._RopeSpec(FAKE, FAKE, 64, 1.0)
    t = lambda x, out, heads=4, xs=(256, 64), os=(256, 64): P._RopeTensor(x, out, heads, 0, *xs, *os)  # noqa: E731
    call = lambda *ts, tok=3: lib.dsa_rope(spec, (P._RopeTensor * len(ts))(*ts), len(ts), 1, tok, None)  # noqa: E731
    # one tensor at two outputs' address, one's output at another's input
    assert call(t(FAKE, 2 * FAKE), t(3 * FAKE, 2 * FAKE)) == P.ERR_INVALID_ARG
    assert call(t(FAKE, FAKE), t(FAKE, FAKE)) == P.ERR_INVALID_ARG
    assert call(t(FAKE, 2 * FAKE), t(2 * FAKE, 3 * FAKE)) == P.ERR_INVALID_ARG
    assert call(t(FAKE, 2 * FAKE), t(3 * FAKE, FAKE)) == P.ERR_INVALID_ARG
    # strides that fold an output's tokens or heads onto each other
    for heads, os in ((4, (0, 64)), (4, (256, 0)), (4, (255, 64)), (4, (256, 63)), (4, (64, 191)), (1, (63, 1 << 20)),
                      (4, (192, 128))):
        assert call(t(FAKE, 2 * FAKE, heads, os=os)) == P.ERR_INVALID_ARG, os
    assert call(t(FAKE, 2 * FAKE, 4, os=(7, 63)), tok=1) == P.ERR_INVALID_ARG


def test_rope_outputs_that_overlap_in_part_are_refused(lib):
    """Tensors whose tokens lie at one distance, and single tokens."""
    spec = P._RopeSpec(FAKE, FAKE, 64, 1.0)
    t = lambda x, out, heads=4, xs=(256, 64), os=(256, 64): P._RopeTensor(x, out, heads, 0, *xs, *os)  # noqa: E731
    call = lambda *ts, tok=3, dt=1: lib.dsa_rope(spec, (P._RopeTensor * len(ts))(*ts), len(ts), dt, tok, None)  # noqa: E731
    # an output a little ahead of or behind its own input; tokens are 512 bytes apart
    for shift in (2, -2, 64, 126, 512, -1024, 1026, 512 * 3 - 2):
        assert call(t(4 * FAKE, 4 * FAKE + shift)) == P.ERR_INVALID_ARG, shift
    # a packed row of 8 heads of 128 (2,048 bytes): outputs of heads 0-3 and 3-6, and of a later token's
    packed = lambda at, heads=4, x=FAKE: t(x, 4 * FAKE + at, heads, os=(1024, 128))  # noqa: E731
    for at in (3 * 256, 3 * 256 + 126, 256, 2048 + 256, 2 * 2048 + 3 * 256):
        assert call(packed(0), packed(at, x=2 * FAKE)) == P.ERR_INVALID_ARG, at
        assert call(packed(at), packed(0, x=2 * FAKE)) == P.ERR_INVALID_ARG, at
    # an output over another tensor's input
    assert call(packed(0), t(4 * FAKE + 130, 8 * FAKE, 4, xs=(1024, 128))) == P.ERR_INVALID_ARG
    assert call(t(4 * FAKE - 1922, 8 * FAKE, 4, xs=(1024, 128)), packed(0)) == P.ERR_INVALID_ARG
    # single tokens of any strides, fp32
    assert call(t(FAKE, 4 * FAKE, 4, os=(0, 100)), t(2 * FAKE, 4 * FAKE + 1000, 2, os=(0, 64)), tok=1, dt=2) == \
        P.ERR_INVALID_ARG


def test_insert_and_attention_outputs_that_overlap_are_refused(lib):
    spec = P._RopeSpec(FAKE, FAKE, 64, 1.0)
    base = 16 * FAKE  # the pool: 10 pages of 64 tokens, 655,360 bytes
    call = lambda out, k=FAKE, v=2 * FAKE, ks=2048: lib.dsa_kv_insert(  # noqa: E731
        kv(base=base), FAKE, 3, P._KvRows(k, v, ks, ks, 0, 0), spec, P._RopeTensor(out, out, 4, 0, 2048, 128, 2048, 128),
        None, None)
    for out in (base, base + 655360 - 128, base - 128 + 16, base - 2 * 4096 - 768):
        assert call(out) == P.ERR_INVALID_ARG, out
    assert call(FAKE + 1000) == P.ERR_INVALID_ARG and call(2 * FAKE + 4096 - 768) == P.ERR_INVALID_ARG
    att = lambda q, out, lse=None, n=3, stride=8192: lib.dsa_kv_attention(  # noqa: E731
        kv(base=base), rows(n=n), q, stride, 64, 0.1, out, lse, None, 0, None, None)
    for q, out, lse in ((FAKE, FAKE, None), (FAKE, FAKE + 16, None), (FAKE + 3 * 16384 - 16, FAKE, None),
                        (8 * FAKE, FAKE, 8 * FAKE + 4), (8 * FAKE, FAKE, FAKE + 3 * 16384 - 4)):
        assert att(q, out, lse) == P.ERR_INVALID_ARG
    # out over the second row of a q whose rows lie further apart
    assert att(FAKE, FAKE + 32768 - 16, n=2, stride=16384) == P.ERR_INVALID_ARG


BAD_CACHES = [(dict(fmt=P.KEY_FP8), P.ERR_UNSUPPORTED), (dict(page=8), P.ERR_UNSUPPORTED),
              (dict(page=48), P.ERR_UNSUPPORTED), (dict(page=256), P.ERR_UNSUPPORTED), (dict(dim=96), P.ERR_UNSUPPORTED),
              (dict(dim=256), P.ERR_UNSUPPORTED), (dict(heads=0), P.ERR_INVALID_ARG), (dict(pages=0), P.ERR_INVALID_ARG),
              (dict(heads=257), P.ERR_UNSUPPORTED), (dict(pages=1 << 22), P.ERR_UNSUPPORTED),
              (dict(ks=0.0), P.ERR_INVALID_ARG), (dict(vs=-1.0), P.ERR_INVALID_ARG),
              (dict(ks=float("inf")), P.ERR_INVALID_ARG), (dict(vs=float("nan")), P.ERR_INVALID_ARG)]


def test_the_largest_pool(lib):
    """Of rows of head_dim, counted exactly: num_pages * kv_heads * 2 * page_size < 2^31."""
    most = ((1 << 31) - 1) // (3 * 2 * 16)
    assert most * 3 * 2 * 16 < 1 << 31 <= (most + 1) * 3 * 2 * 16
    size = lambda n: lib.dsa_kv_attention_workspace_size(kv(heads=3, page=16, pages=n), 1, 3, 1 << 20)  # noqa: E731
    assert size(most) > 0 and size(most + 1) == 0
    assert lib.dsa_kv_attention_workspace_size(kv(heads=4, page=16, pages=1 << 24), 1, 4, 1 << 20) == 0


@pytest.mark.parametrize("change, want", BAD_CACHES)
def test_cache_refusals(lib, change, want):
    c = kv(**change)
    r = P._KvRows(FAKE, FAKE, 1 << 20, 1 << 20, 0, 0)
    assert lib.dsa_kv_insert(c, FAKE, 1, r, None, None, None, None) == want
    assert lib.dsa_kv_attention(c, rows(), FAKE, 1 << 20, 1024, 0.1, FAKE, None, FAKE, 1 << 30, None, None) == want
    assert lib.dsa_kv_attention_workspace_size(c, 1, 64, 1 << 20) == 0


def test_insert_refusals(lib):
    r = lambda k=FAKE, v=FAKE, ks=512, vs=512, off=0, lay=0: P._KvRows(k, v, ks, vs, off, lay)  # noqa: E731
    spec = P._RopeSpec(FAKE, FAKE, 64, 1.0)
    q = P._RopeTensor(FAKE, FAKE, 4, 0, 256, 64, 256, 64)
    call = lambda c=None, slots=FAKE, n=1, kvr=None, rope=None, qt=None: \
        lib.dsa_kv_insert(c or kv(), slots, n, kvr or r(), rope, qt, None, None)  # noqa: E731
    assert call(n=0) == P.OK
    assert call(n=-1) == P.ERR_INVALID_ARG
    assert lib.dsa_kv_insert(None, FAKE, 1, r(), None, None, None, None) == P.ERR_INVALID_ARG
    assert lib.dsa_kv_insert(kv(), FAKE, 1, None, None, None, None, None) == P.ERR_INVALID_ARG
    assert call(slots=None) == P.ERR_INVALID_ARG
    for bad in (r(k=None), r(v=None), r(ks=511), r(vs=511), r(k=FAKE + 1)):
        assert call(kvr=bad) == P.ERR_INVALID_ARG
    assert call(c=kv(base=None)) == P.ERR_INVALID_ARG
    assert call(c=kv(base=ODD)) == P.ERR_INVALID_ARG
    assert call(qt=q) == P.ERR_INVALID_ARG  # q without rope
    assert call(kvr=r(off=65), rope=spec) == P.ERR_INVALID_ARG
    assert call(kvr=r(off=-2), rope=spec) == P.ERR_INVALID_ARG
    assert call(kvr=r(lay=2), rope=spec) == P.ERR_UNSUPPORTED
    assert call(rope=P._RopeSpec(FAKE, FAKE, 130, 1.0)) == P.ERR_INVALID_ARG  # wider than a head
    assert call(rope=spec, qt=P._RopeTensor(FAKE, None, 4, 0, 256, 64, 256, 64)) == P.ERR_INVALID_ARG


def test_attention_refusals(lib):
    def call(c=None, rw=None, q=FAKE, stride=8192, heads=64, sm=0.1, out=FAKE, ws=FAKE, wb=1 << 40):
        return lib.dsa_kv_attention(c or kv(), rw or rows(), q, stride, heads, sm, out, None, ws, wb, None, None)
    assert call(rw=rows(n=0)) == P.OK
    assert lib.dsa_kv_attention(None, rows(), FAKE, 8192, 64, 0.1, FAKE, None, FAKE, 1, None, None) == P.ERR_INVALID_ARG
    for bad in (dict(heads=0), dict(heads=62), dict(sm=0.0), dict(sm=float("nan")), dict(sm=float("inf")),
                dict(q=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(stride=8191), dict(stride=8196),
                dict(rw=rows(n=-1)), dict(rw=rows(ctx=-1)), dict(rw=rows(stride=3)), dict(rw=rows(n=3, g=2)),
                dict(rw=rows(table=None)), dict(c=kv(base=None)), dict(c=kv(base=ODD))):
        assert call(**bad) == P.ERR_INVALID_ARG, bad
    assert call(heads=4 * 129, stride=1 << 20) == P.ERR_UNSUPPORTED
    assert call(rw=rows(n=3, g=3)) == P.ERR_UNSUPPORTED
    assert call(rw=rows(ctx=(1 << 30) + 1, stride=1 << 28)) == P.ERR_UNSUPPORTED
    long = rows(ctx=1 << 20, stride=1 << 14)
    need = lib.dsa_kv_attention_workspace_size(kv(), 1, 64, 1 << 20)
    assert need > 0
    assert call(rw=long, ws=None, wb=0) == P.ERR_WORKSPACE
    assert call(rw=long, wb=need - 1) == P.ERR_WORKSPACE
    assert call(rw=long, ws=FAKE + 16) == P.ERR_INVALID_ARG


def test_workspace_size_is_host_logic(lib):
    size = lambda n, h, ctx: lib.dsa_kv_attention_workspace_size(kv(), n, h, ctx)  # noqa: E731
    assert size(0, 64, 4096) == 0 and size(4, 0, 4096) == 0 and size(4, 64, 0) == 0
    assert size(4, 64, 1) == 0  # one part: nothing to merge
    assert size(8, 64, 131072) >= 2 * 8 * 64 * 128 * 4
    assert all(size(2, 64, n) <= size(2, 64, n + 128) for n in range(1, 300000, 4999))


# ------------------------------------------------------------------ the binding

def test_binding_refuses_cpu_tensors():
    with pytest.raises(P.DsaError):
        P.KvCache(torch.zeros(2, 1, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(P.DsaError):
        P.RopeTable(torch.zeros(32, dtype=torch.int64))
    with pytest.raises(P.DsaError):
        P.KvCache(torch.zeros(2, 1, 3, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(P.DsaError):
        P.KvCache(torch.zeros(2, 1, 2, 16, 64))
