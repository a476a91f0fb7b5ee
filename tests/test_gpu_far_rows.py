"""The tree and block calls over a pool of more than 2^32 bytes whose sequences
lie at its far end: row offsets need 64 bits."""

import numpy as np
import pytest
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from tests.operators_harness import (LITE, V2, attention_bounds, dev, handle, host, ints, ok, shape, stored, within,
                                     words)

pytestmark = pytest.mark.gpu

PAGES = 2 ** 32 // (64 * 576 * 2) + 200      # of 73728 bytes


@pytest.fixture(scope="module", autouse=True)
def _built():
    from head_latent_attention_09_b200 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("aligned", [True, False])      # tensor cores, CUDA cores
@pytest.mark.parametrize("sh", [shape(LITE), shape(V2)])
def test_far_end_of_a_large_pool(sh, aligned):
    rng = np.random.default_rng(3)
    ctx, T, k, blocks, n_h = [150, 64], 4, 2, 3, sh["n_h"]
    rows = [stored(sh, rng.standard_normal((n + T, 576))) for n in ctx]
    skip = 0 if aligned else 1
    raw = torch.empty(PAGES * 64 * 576 + 8, dtype=torch.bfloat16, device="cuda")
    raw.fill_(float("nan"))
    pool = raw[skip:skip + PAGES * 64 * 576].view(PAGES, 64, 576)
    order = PAGES - 1 - rng.permutation(150)[:2 * blocks].reshape(2, blocks)
    table, lens = ints(order), ints(ctx)
    for b, r in enumerate(rows):
        d = dev(sh, r)
        for p in range(0, len(r), 64):
            pool[order[b, p // 64], :len(r[p:p + 64])] = d[p:p + 64]
    args = (pool, PAGES, table, blocks)
    h = handle(sh, 64, strict=aligned)
    scale = O.softmax_scale(sh["d_h"], sh["d_r"])

    keys = torch.zeros(2, blocks, 576, dtype=torch.bfloat16, device="cuda")
    M.mla_block_keys(h, *args, None, lens, 2, 150, keys, blocks)
    ok(h)
    for b, n in enumerate(ctx):
        want, mass = O.block_means(rows[b][:n]), O.block_means(np.abs(rows[b][:n]))
        within(host(keys)[b, :len(want)], want, 2.0 ** -8 * 1.01 * np.abs(want) + 65 * 2.0 ** -24 * mass, "means")

    q = stored(sh, rng.standard_normal((2, n_h, 576)) * 0.7)
    sel = [[0, 2], [0]]
    ws = torch.empty(M.mla_decode_workspace_size(h, 2, 0), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(2, n_h, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, n_h, device="cuda")
    M.mla_decode_attn_sparse(h, dev(sh, q), *args, lens, ints([[0, 2], [0, -1]]), ints([2, 1]), k, 2, 0, ws, ws.numel())
    M.mla_combine_splits(h, ws, ws.numel(), 2, 0, out, lse)
    ok(h)
    for b, n in enumerate(ctx):
        mine = np.concatenate([rows[b][:n][64 * j:64 * j + 64] for j in sel[b]]).astype(np.float64)
        qb = q[b].astype(np.float64)
        want, z = O.latent_attention(qb, mine, d_c=512, scale=scale)
        bo, bl = attention_bounds(sh, qb, mine, scale, want, z)
        within(host(out)[b], want, bo, "sparse ctx_lat")
        within(host(lse)[b], z, bl, "sparse lse")

    bits = O.tree_bits([-1, 0, 0, 1])
    q = stored(sh, rng.standard_normal((2, T, n_h, 576)) * 0.7)
    out, lse = torch.empty(2, T, n_h, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, T, n_h, device="cuda")
    ws = torch.empty(M.mla_tree_workspace_size(h, 2, T), dtype=torch.uint8, device="cuda")
    M.mla_tree_attn(h, dev(sh, q), *args, lens, words([bits] * 2), 2, T, 0, out, lse, ws, ws.numel())
    ok(h)
    for b, n in enumerate(ctx):
        r, qb = rows[b].astype(np.float64), q[b].astype(np.float64)
        want, z = O.tree_attention(qb, r[:n], r[n:], bits, d_c=512, scale=scale)
        for t in range(T):
            bo, bl = attention_bounds(sh, qb[t], r, scale, want[t], z[t])
            within(host(out)[b, t], want[t], bo, "tree ctx_lat")
            within(host(lse)[b, t], z[t], bl, "tree lse")

    M.mla_tree_accept(h, *args, lens, ints([[0, 1, 3, 0]] * 2), ints([3, 3]), 2, T, lens)
    ok(h)
    assert lens.tolist() == [n + 3 for n in ctx]
    for b, n in enumerate(ctx):
        got = np.stack([host(pool[order[b, p // 64], p % 64]) for p in range(n + T)])
        assert np.array_equal(got, O.tree_accept(rows[b], n, [0, 1, 3]))

    x = stored(sh, rng.standard_normal((2, 1, sh["d_model"])))
    w = stored(sh, rng.standard_normal((576, sh["d_model"])) * sh["d_model"] ** -0.5)
    M.mla_cache_append_tree(h, dev(sh, x), 2, 1, lens, ints([[0], [0]]), dev(sh, w[:512]), dev(sh, w[512:]), *args)
    ok(h)
    M.mla_destroy(h)
    for b, n in enumerate(ctx):
        p = n + 3
        want = O.cache_rows(x[b], w[:512], w[512:], np.array([p]), 10000.0)
        mass = np.abs(x[b]).astype(np.float64) @ np.abs(w).astype(np.float64).T
        mass[:, 512:] = np.repeat(mass[:, 512::2] + mass[:, 513::2], 2, 1)
        got = host(pool[order[b, p // 64], p % 64])[None]
        within(got, want, (sh["d_model"] * 2.0 ** -24 + 4e-6) * mass + 2.0 ** -8 * 1.01 * np.abs(want), "appended rows")
