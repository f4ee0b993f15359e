"""The dense K/V path's calls beside the sparse ones: rotary positions feed the sparse attention's queries, latents and
index keys, and the K/V insert fills the pool that the block-sparse attention reads."""

import numpy as np
import pytest
import torch

import oracle
import prefill_dsa_indexer_gb300 as P
from prefill_dsa_indexer_gb300 import inputs as I
from tests import gpu_util as U
from tests.test_gpu_kv_path import codes, gen, randn, ref_rotate, rope_bound

pytestmark = pytest.mark.gpu


def test_block_sparse_attention_over_a_pool_that_the_insert_filled():
    """At most 16 blocks a row, so the block-sparse attention sees every token that the insert wrote; against the formula
    and the dense attention over the same pool."""
    ctx = [2048, 1300, 77]
    m = I.make_msa_inputs(I.small_msa_workload("filled", ctx)).to("cuda")
    m.kv_pool.fill_(0x7F)  # NaN wherever nothing is inserted
    pool = m.kv_pool.view(-1, 4, 2, 128, 128)
    ks, vs = 1 / 72, 1 / 90
    kv, table, status = P.KvCache(pool, ks, vs), P.rope_table(64, 500000.0), P.new_status()
    g, rot = gen(70), slice(32, 96)
    keys, values = [], []
    for r, n in enumerate(ctx):
        k, v = randn(g, n, 4, 128), randn(g, n, 4, 128)
        t = torch.arange(n, device="cuda", dtype=torch.int32)
        slots = m.block_table[r][(t // 128).long()] * 128 + t % 128
        P.kv_insert(kv, slots, k, v, rope=table, positions=t, layout=P.ROPE_HALF, rot_offset=32, status=status)
        turned = k.double()
        turned[..., rot] = ref_rotate(k[..., rot], t, P.rope_frequencies(64, 500000.0)[0], 1.0, P.ROPE_HALF)[0]
        keys.append(turned)
        values.append(codes(v, vs).double() * vs)
    R, sm = len(ctx), 128 ** -0.5
    blocks = torch.full((R, 4, 16), -1, dtype=torch.int32, device="cuda")
    for r, n in enumerate(ctx):
        blocks[r, :, :-(-n // 128)] = torch.arange(-(-n // 128), dtype=torch.int32, device="cuda")
    a, la = P.msa_attention(m.kv_pool, ks, vs, m.block_table, m.row_req, m.row_ctx, max(ctx), m.q, m.q_scale, blocks, sm,
                            status=status)
    q = m.q.view(torch.float8_e4m3fn).to(torch.bfloat16)  # (codes are exact in bf16)
    b, lb = P.kv_attention(kv, m.block_table, m.row_req, m.row_ctx, max(ctx), q, sm_scale=sm * m.q_scale, status=status)
    torch.cuda.synchronize()
    P.check_status(status)
    # one pool and one q: weights rounded to fp16 on both sides (2^-11 of values up to 448 vs), b's output to bf16
    assert ((a - b.float()).abs() <= 2.0 ** -8 * a.abs() + 2 * 2.0 ** -10 * 448 * vs).all()
    assert ((la - lb).abs() <= 2e-3).all()
    hpg = q.shape[1] // 4
    for r in range(R):
        for h in range(4):
            k, v = keys[r][:, h], values[r][:, h]
            x = q[r, h * hpg:(h + 1) * hpg].double() * m.q_scale
            s = x @ k.T * sm
            p = torch.softmax(s, -1)
            # keys rounded to e4m3: 2^-4 of each element, 2^-10 steps at least (times ks): both ways in a weight's exponent
            ds = (x.abs() @ (2.0 ** -4 * k.abs() + 2.0 ** -10 * ks).T * sm).amax(-1, keepdim=True)
            bound = torch.expm1(2 * ds) * (p @ v.abs() + (p @ v).abs()) + 2.0 ** -8 * (p @ v).abs() + 2.0 ** -9
            assert ((b[r, h * hpg:(h + 1) * hpg].double() - p @ v).abs() <= bound).all()


def test_rotated_queries_latents_and_index_keys_in_the_sparse_path():
    """A step's last 64 of 576 query and latent dims and the first 64 index key dims, rotated in place, inserted, scored
    and attended to, against the oracle on the same bytes."""
    n = 700
    wl = I.small_workload("turned", [n], seed=4)
    inp = I.make_inputs(wl).to("cuda")
    g, table, freq = gen(71), P.rope_table(64), P.rope_frequencies(64, 10000.0)[0]
    keys, lats = randn(g, n, 128), randn(g, n, 576)
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    before = [keys.clone(), lats.clone()]
    P.rope([lats[:, None, 512:], keys[:, None, :64]], table, t, layout=[P.ROPE_INTERLEAVED, P.ROPE_HALF])
    for x, old, part, layout in ((lats, before[1], slice(512, 576), P.ROPE_INTERLEAVED),
                                 (keys, before[0], slice(0, 64), P.ROPE_HALF)):
        ref, mag = ref_rotate(old[:, None, part], t, freq, 1.0, layout)
        assert ((x[:, None, part].double() - ref).abs() <= rope_bound(ref, mag, 1.0, torch.bfloat16)).all()
        old[:, part] = x[:, part]
        assert torch.equal(x, old)
    q = inp.q_mla.view(torch.bfloat16)
    P.rope(q[..., 512:], table, inp.row_ctx - 1)
    slots = (inp.block_table[0][(t // 64).long()] * 64 + t % 64).to(torch.int32)
    P.cache_insert(inp.idx_pool, wl.key_fmt, inp.lat_pool, wl.lat_fmt, inp.tensor_scale, slots, keys.view(torch.int16),
                   lats.view(torch.int16))
    lg = P.indexer_logits(inp.idx_pool, wl.key_fmt, inp.block_table, inp.row_req, inp.row_ctx, inp.max_ctx, inp.q_idx,
                          inp.head_w)
    chosen = torch.full((1, 2048), -1, dtype=torch.int32, device="cuda")
    chosen[0, :n] = slots
    out, lse = P.sparse_mla_decode(inp.lat_pool, wl.lat_fmt, inp.tensor_scale, inp.q_mla, chosen, U.SM_SCALE)
    torch.cuda.synchronize()
    ref, bound = U.oracle_logits(inp)[0, :n], U.logit_bound(inp, [0])[0][:n]
    assert np.all(np.abs(lg.cpu().numpy()[0, :n].astype(np.float64) - ref) <= bound)
    ref_o, ref_l = oracle.sparse_mla(inp.np("lat_pool"), U.ORACLE_FMT[wl.lat_fmt], inp.tensor_scale, inp.np("q_mla"),
                                     chosen.cpu().numpy(), U.SM_SCALE)
    max_abs, rel = U.mla_errors(out.cpu().numpy(), ref_o)
    assert max_abs <= 2e-2 and rel <= 1e-2, (max_abs, rel)
    assert np.all(np.abs(lse.cpu().numpy() - ref_l) <= 2e-3)
