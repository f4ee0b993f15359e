"""A batch's step (plans, rotary positions with several axes, attention over shared prefixes) as far as it needs no GPU:
host helpers and every refusal of the C ABI and of the binding."""
import ctypes

import pytest
import torch

import prefill_dsa_indexer_gb300 as P
from tests.test_kv_path import BAD_CACHES, FAKE, ODD, kv, lib, rows  # noqa: F401

WORDS = 0x100000  # between the fake arrays


def step(**change):
    """A step of 5 requests with 3 pages each, 8 rows, 2 segments."""
    names = ("context", "new_tokens", "first_own", "block_table", "free_pages", "free_count", "segment_requests",
             "row_req", "row_ctx", "positions", "slots", "row_start", "granted", "context_out", "free_count_out",
             "segment_rows")
    s = P._KvStep(num_requests=5, page_size=16, num_pages=100, bt_stride=3, free_capacity=40, num_segments=2, max_rows=8,
                  rows_per_group=1, **{n: FAKE + i * WORDS for i, n in enumerate(names)})
    for n, v in change.items():
        setattr(s, n, v)
    return s


def test_plan_refusals(lib):  # noqa: F811
    call = lambda **change: lib.dsa_kv_plan(step(**change), None, None)  # noqa: E731
    assert lib.dsa_kv_plan(None, None, None) == P.ERR_INVALID_ARG
    for name in ("num_requests", "num_pages", "bt_stride", "free_capacity", "num_segments", "max_rows"):
        assert call(**{name: -1}) == P.ERR_INVALID_ARG, name
    for name in ("context", "new_tokens", "block_table", "free_pages", "free_count", "segment_requests", "row_req",
                 "row_ctx", "segment_rows"):
        assert call(**{name: None}) == P.ERR_INVALID_ARG, name
        assert call(**{name: FAKE + 2}) == P.ERR_INVALID_ARG, name
    assert call(rows_per_group=4, max_rows=10) == P.ERR_INVALID_ARG
    for change in (dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(rows_per_group=3),
                   dict(rows_per_group=0), dict(num_requests=P.KV_PLAN_MAX_REQUESTS + 1), dict(num_pages=1 << 27),
                   dict(bt_stride=(1 << 31) + 1)):
        assert call(**change) == P.ERR_UNSUPPORTED, change


def test_plan_outputs_that_overlap_are_refused(lib):  # noqa: F811
    base = step()
    call = lambda **change: lib.dsa_kv_plan(step(**change), None, None)  # noqa: E731
    # an output over an input or another output, exactly or by its last or first word
    for out, words in (("row_req", 8), ("row_ctx", 8), ("positions", 8), ("slots", 8), ("row_start", 6), ("granted", 5),
                       ("segment_rows", 3)):
        for other, n in (("context", 5), ("new_tokens", 5), ("first_own", 5), ("block_table", 15), ("free_pages", 40),
                         ("free_count", 1), ("segment_requests", 3), ("context_out", 5), ("free_count_out", 1)):
            at = getattr(base, other)
            for to in (at, at + 4 * n - 4, at - 4 * words + 4):
                assert call(**{out: to}) == P.ERR_INVALID_ARG, (out, other)
    assert call(context_out=base.context + 4) == P.ERR_INVALID_ARG
    assert call(context_out=base.new_tokens) == P.ERR_INVALID_ARG
    assert call(free_count_out=base.free_pages + 16) == P.ERR_INVALID_ARG
    assert call(block_table=base.free_pages) == P.ERR_INVALID_ARG
    assert lib.dsa_kv_plan(step(), base.granted + 16, None) == P.ERR_INVALID_ARG


def test_sections(lib):  # noqa: F811
    assert P.rope_sections((2, 1, 3)).tolist() == [0, 0, 1, 2, 2, 2]
    assert P.rope_sections((2, 1, 3), "cycle").tolist() == [0, 1, 2, 0, 2, 2]
    assert P.rope_sections((0, 2), "cycle").tolist() == [1, 1]
    assert P.rope_sections((128,)).tolist() == [0] * 128
    i32, axis = lambda *v: (ctypes.c_int32 * len(v))(*v), (ctypes.c_uint8 * 128)()  # noqa: E731
    call = lambda s, n, order=0, pairs=4, out=axis: lib.dsa_rope_sections(s, n, order, pairs, out)  # noqa: E731
    assert call(i32(1, 3), 2) == P.OK and list(axis[:4]) == [0, 1, 1, 1]
    assert call(None, 2) == call(i32(1, 3), 2, out=None) == call(i32(1, 2), 2) == P.ERR_INVALID_ARG
    assert call(i32(5, -1), 2) == call(i32(4), 0) == call(i32(0, 0), 2, pairs=0) == P.ERR_INVALID_ARG
    assert call(i32(1, 1, 1, 1, 0), 5) == call(i32(4), 1, order=2) == call(i32(129), 1, pairs=129) == P.ERR_UNSUPPORTED
    for bad in (((1, 2), "other"), ((1, -1), "split"), ((), "split"), ((129,), "split"), ((1,) * 5, "split")):
        with pytest.raises(P.DsaError):
            P.rope_sections(*bad)
    with pytest.raises(P.DsaError):
        P.rope_table(64, sections=(10, 10, 10), device="cpu")


def test_rope_with_axes_refusals(lib):  # noqa: F811
    axis = (ctypes.c_uint8 * 32)(*([0] * 16 + [1] * 16))
    one = (P._RopeTensor * 1)(P._RopeTensor(FAKE, FAKE, 4, 0, 256, 64, 256, 64))
    row = P._KvRows(FAKE, FAKE, 512, 512, 0, 0)

    def both(want, tok=3, **change):
        f = dict(turns=FAKE, positions=FAKE, axis_stride=8, axis=ctypes.addressof(axis), num_axes=2, rot_dim=64, scale=1.0)
        spec = P._RopeAxes(**{**f, **change})
        assert lib.dsa_rope_with_axes(spec, one, 1, 1, tok, None) == want, change
        assert lib.dsa_kv_insert_with_axes(kv(), FAKE, tok, row, spec, None, None, None) == want, change
    both(P.OK, tok=0)
    for change in (dict(turns=None), dict(positions=None), dict(axis=None), dict(axis_stride=-1), dict(num_axes=0),
                   dict(num_axes=1), dict(rot_dim=0), dict(rot_dim=63), dict(scale=float("inf"))):
        both(P.ERR_INVALID_ARG, **change)
    both(P.ERR_UNSUPPORTED, num_axes=5)
    both(P.ERR_UNSUPPORTED, rot_dim=258)
    assert lib.dsa_rope_with_axes(None, one, 1, 1, 3, None) == P.ERR_INVALID_ARG
    spec = P._RopeAxes(FAKE, FAKE, 8, ctypes.addressof(axis), 2, 64, 1.0)
    for n, dt, tok, want in ((0, 1, 3, P.ERR_INVALID_ARG), (5, 1, 3, P.ERR_UNSUPPORTED), (1, 3, 3, P.ERR_UNSUPPORTED),
                             (1, 1, -1, P.ERR_INVALID_ARG)):
        assert lib.dsa_rope_with_axes(spec, one, n, dt, tok, None) == want


def segments(first=FAKE, ctx=FAKE, n=2, least=0):
    return P._KvSegments(first, ctx, n, least)


def test_shared_attention_refusals(lib):  # noqa: F811
    def call(c=None, rw=None, seg=None, q=FAKE, stride=8192, heads=64, sm=0.1, out=FAKE << 4, ws=FAKE, wb=1 << 40):
        return lib.dsa_kv_attention_shared(c or kv(), rw or rows(), seg or segments(), q, stride, heads, sm, out, None, ws,
                                           wb, None, None)
    assert call(rw=rows(n=0)) == P.OK
    assert lib.dsa_kv_attention_shared(None, rows(), segments(), FAKE, 8192, 64, 0.1, FAKE, None, FAKE, 1, None, None) == \
        P.ERR_INVALID_ARG
    assert lib.dsa_kv_attention_shared(kv(), rows(), None, FAKE, 8192, 64, 0.1, FAKE, None, FAKE, 1, None, None) == \
        P.ERR_INVALID_ARG
    for bad in (dict(heads=0), dict(heads=62), dict(sm=0.0), dict(sm=float("nan")), dict(q=None), dict(out=None),
                dict(q=ODD), dict(out=ODD), dict(stride=8191), dict(stride=8196), dict(rw=rows(n=-1)),
                dict(rw=rows(n=3, g=2)), dict(rw=rows(table=None)), dict(c=kv(base=ODD)), dict(seg=segments(first=None)),
                dict(seg=segments(ctx=None)), dict(seg=segments(n=-1)), dict(seg=segments(least=-1)),
                dict(out=FAKE)):
        assert call(**bad) == P.ERR_INVALID_ARG, bad
    assert call(heads=4 * 129, stride=1 << 20) == P.ERR_UNSUPPORTED
    size = lib.dsa_kv_attention_shared_workspace_size
    long, need = rows(n=4, ctx=1 << 20, stride=1 << 14), size(kv(), 4, 64, 1 << 20, 2)
    assert need > 0
    assert call(rw=long, ws=None, wb=0) == P.ERR_WORKSPACE
    assert call(rw=long, wb=need - 1) == P.ERR_WORKSPACE
    assert call(rw=long, ws=FAKE + 16) == P.ERR_INVALID_ARG


@pytest.mark.parametrize("change, want", BAD_CACHES)
def test_shared_attention_cache_refusals(lib, change, want):  # noqa: F811
    c = kv(**change)
    assert lib.dsa_kv_attention_shared(c, rows(), segments(), FAKE, 1 << 20, 1024, 0.1, FAKE, None, FAKE, 1 << 30, None,
                                       None) == want
    assert lib.dsa_kv_attention_shared_workspace_size(c, 1, 64, 1 << 20, 1) == 0


def test_shared_workspace_size_is_host_logic(lib):  # noqa: F811
    size = lambda n, h, ctx, s: lib.dsa_kv_attention_shared_workspace_size(kv(), n, h, ctx, s)  # noqa: E731
    assert size(0, 64, 4096, 1) == size(4, 0, 4096, 1) == size(4, 64, 0, 1) == size(4, 64, 4096, -1) == 0
    assert size(4, 64, 4096, 0) == lib.dsa_kv_attention_workspace_size(kv(), 4, 64, 4096)
    assert size(8, 64, 131072, 1) >= lib.dsa_kv_attention_workspace_size(kv(), 8, 64, 131072)
    assert all(size(6, 64, n, 2) <= size(6, 64, n + 128, 2) for n in range(1, 300000, 4999))


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(P.DsaError):
        P.kv_plan(z, z, z[None], z, z[:1], 16, 4, z, z)
    with pytest.raises(P.DsaError):
        P.RopeTable(torch.zeros(32, dtype=torch.int64), axis=torch.zeros(32, dtype=torch.uint8))
