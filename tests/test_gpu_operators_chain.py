"""The tree and block-selection calls together, as a serving step uses them:
a prompt is cached and its blocks summarised, a tree is drafted behind it and
verified, the accepted branch kept and its blocks summarised again, and a
decode step attends selected blocks only.  Every result is compared with the
float64 oracle started from the same hidden states."""

import numpy as np
import pytest
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from tests.gpu_harness import compare
from tests.operators_harness import LITE, TINY, V2, dev, handle, host, ints, ok, shape, stored, torch_type, words
from workloads import WORKLOADS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from head_latent_attention_09_b200 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("sh,page", [(shape(LITE), 64), (shape(LITE), 0), (shape(V2, n_h=128), 64), (shape(TINY), 0)])
def test_draft_verify_accept_then_sparse_decode(sh, page):
    wl = WORKLOADS["tiny_fp32" if sh["dtype"] == "fp32" else "v2lite_b32_ctx4k"]     # compare()'s tolerances
    rng = np.random.default_rng(5)
    n_h, d_h, d_c, d_r, d = (sh[k] for k in ("n_h", "d_h", "d_c", "d_r", "d_model"))
    D, B, T, k = d_c + d_r, 3, 6, 4
    ctx = [450, 65, 256]
    kw = dict(n_h=n_h, d_h=d_h, d_r=d_r, base=10000.0)
    w = {n: stored(sh, rng.standard_normal(s) * s[1] ** -0.5)
         for n, s in (("dkv", (d_c, d)), ("kr", (d_r, d)), ("uk", (n_h * d_h, d_c)), ("uv", (n_h * d_h, d_c)))}
    w["uk"] = stored(sh, rng.standard_normal((n_h * d_h, d_c)) * d_h ** -0.5 * (d_h / d_c) ** 0.5)
    wd = {n: dev(sh, x) for n, x in w.items()}
    hid = [stored(sh, rng.standard_normal((n, d))) for n in ctx]
    h_tree = stored(sh, rng.standard_normal((B, T, d)))
    parents = [-1, 0, 0, 1, 3, 2]
    bits, depth = O.tree_bits(parents), O.tree_depths(parents)
    paths = [[0, 1, 3], [], [0, 2, 5]]
    qn = stored(sh, rng.standard_normal((B, T, n_h, d_h)))
    qr = stored(sh, rng.standard_normal((B, T, n_h, d_r)))
    h_new, qn1, qr1 = (stored(sh, rng.standard_normal((B, *s))) for s in ((1, d), (n_h, d_h), (n_h, d_r)))
    slots, dt = max(ctx) + T + 1, torch_type(sh)
    blocks = -(-slots // 64)
    h = handle(sh, page)

    if page:
        order = rng.permutation(B * blocks)
        pool = torch.full((B * blocks, 64, D), float("nan"), dtype=dt, device="cuda")
        table = ints(order.reshape(B, blocks))
        cache = (pool, B * blocks, table, blocks)
    else:
        cache = (torch.full((B, slots, D), float("nan"), dtype=dt, device="cuda"), slots, None, 0)
    for b in range(B):       # the prompts, one sequence at a time
        if page:
            one = (cache[0], cache[1], table[b:b + 1].contiguous(), blocks)
        else:
            one = (cache[0][b], slots, None, 0)
        M.mla_cache_append(h, dev(sh, hid[b]), 1, ctx[b], ints([0]), wd["dkv"], wd["kr"], *one)
    lens = ints(ctx)
    keys = torch.zeros(B, blocks, D, dtype=dt, device="cuda")
    M.mla_block_keys(h, *cache, None, lens, B, max(ctx), keys, blocks)

    # draft and verify
    M.mla_cache_append_tree(h, dev(sh, h_tree), B, T, lens, ints([depth] * B), wd["dkv"], wd["kr"], *cache)
    pos = ints([[n + t for t in depth] for n in ctx])
    q_abs = torch.empty(B, T, n_h, D, dtype=dt, device="cuda")
    M.mla_absorb_q(h, dev(sh, qn), dev(sh, qr), pos, wd["uk"], q_abs, B * T)
    out = torch.empty(B, T, n_h, d_c, dtype=dt, device="cuda")
    lse = torch.empty(B, T, n_h, device="cuda")
    ws = torch.empty(M.mla_tree_workspace_size(h, B, T), dtype=torch.uint8, device="cuda")
    M.mla_tree_attn(h, q_abs, *cache, lens, words([bits] * B), B, T, 0, out, lse, ws, ws.numel())
    o = torch.empty(B, T, n_h, d_h, dtype=dt, device="cuda")
    M.mla_out_proj(h, out, wd["uv"], None, o, None, B * T)

    # keep the accepted branch, and decode the next token over selected blocks
    path = np.zeros((B, T))
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    before = lens.clone()
    M.mla_tree_accept(h, *cache, lens, ints(path), ints([len(p) for p in paths]), B, T, lens)
    M.mla_cache_append(h, dev(sh, h_new), B, 1, lens, wd["dkv"], wd["kr"], *cache)
    lens += 1
    M.mla_block_keys(h, *cache, before, lens, B, T + 1, keys, blocks)
    q1 = torch.empty(B, n_h, D, dtype=dt, device="cuda")
    M.mla_absorb_q(h, dev(sh, qn1), dev(sh, qr1), lens - 1, wd["uk"], q1, B)
    scores = torch.empty(B, blocks, device="cuda")
    sws = torch.empty(M.mla_block_scores_workspace_size(h, B, blocks), dtype=torch.uint8, device="cuda")
    M.mla_block_scores(h, q1, keys, blocks, lens, B, scores, sws, sws.numel())
    sel, n_sel = torch.empty(B, k, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    M.mla_block_select(h, scores, blocks, lens, B, k, 1, 1, sel, n_sel)
    dws = torch.empty(M.mla_decode_workspace_size(h, B), dtype=torch.uint8, device="cuda")
    M.mla_decode_attn_sparse(h, q1, *cache, lens, sel, n_sel, k, B, 0, dws, dws.numel())
    o1 = torch.empty(B, n_h, d_h, dtype=dt, device="cuda")
    ctx1, lse1 = torch.empty(B, n_h, d_c, dtype=dt, device="cuda"), torch.empty(B, n_h, device="cuda")
    M.mla_combine_out_proj(h, dws, dws.numel(), B, 0, wd["uv"], None, o1, None, ctx1, lse1)
    ok(h)
    M.mla_destroy(h)

    scale = O.softmax_scale(d_h, d_r)
    want = {n: {} for n in ("tree_ctx", "tree_lse", "tree_o", "ctx", "lse", "o", "scores")}
    for b, n in enumerate(ctx):
        rows = O.cache_rows(hid[b], w["dkv"], w["kr"], np.arange(n), 10000.0)
        drafted = O.cache_rows(h_tree[b], w["dkv"], w["kr"], n + np.array(depth), 10000.0)
        q = np.stack([O.absorb_query(qn[b, t], qr[b, t], n + depth[t], w["uk"], **kw) for t in range(T)])
        want["tree_ctx"][b], want["tree_lse"][b] = O.tree_attention(q, rows, drafted, bits, d_c=d_c, scale=scale)
        want["tree_o"][b] = np.stack([O.out_project(want["tree_ctx"][b][t], w["uv"], n_h=n_h, d_h=d_h)[0]
                                      for t in range(T)])
        kept = O.tree_accept(np.concatenate([rows, drafted]), n, paths[b])[:n + len(paths[b])]
        m = len(kept)
        kept = np.concatenate([kept, O.cache_rows(h_new[b], w["dkv"], w["kr"], np.array([m]), 10000.0)])
        assert lens[b].item() == m + 1
        q = O.absorb_query(qn1[b], qr1[b], m, w["uk"], **kw)
        nb = -(-(m + 1) // 64)
        want["scores"][b] = O.block_scores(q, O.block_means(kept), m + 1, scale=scale)
        got = host(scores)[b]
        assert (got[nb:] == 0).all()
        mine = O.block_select(got[:nb].tolist(), k, 1, 1)      # of the call's own scores: exact
        assert sel[b].tolist() == mine + [-1] * (k - len(mine)) and n_sel[b].item() == len(mine)
        taken = np.concatenate([kept[64 * j:64 * j + 64] for j in mine])
        want["ctx"][b], want["lse"][b] = O.latent_attention(q, taken, d_c=d_c, scale=scale)
        want["o"][b] = O.out_project(want["ctx"][b], w["uv"], n_h=n_h, d_h=d_h)[0]
        # shares of attention: means and queries rounded to the cache's type
        # move a score by at most a few percent of itself
        assert np.abs(got[:nb] - want["scores"][b]).max() <= (5e-2 if sh["dtype"] == "bf16" else 1e-4) * n_h
    compare(host(out), want["tree_ctx"], wl, "ctx_lat of the tree")
    compare(host(lse), want["tree_lse"], wl, "lse of the tree")
    compare(host(o), want["tree_o"], wl, "o of the tree")
    compare(host(ctx1), want["ctx"], wl, "ctx_lat over selected blocks")
    compare(host(lse1), want["lse"], wl, "lse over selected blocks")
    compare(host(o1), want["o"], wl, "o over selected blocks")


@pytest.mark.parametrize("sh", [shape(LITE), shape(V2)])
def test_calls_at_the_same_time_on_two_streams(sh):
    """One handle, two streams, workspaces of their own: every run of either call
    gives what it gives alone, bit for bit; a block listed twice counts twice."""
    rng = np.random.default_rng(11)
    B, T, n, k, D, n_h, dt = 5, 7, 900, 6, 576, sh["n_h"], torch_type(sh)
    h = handle(sh)
    cache = dev(sh, rng.standard_normal((B, n + T, D)))
    ctx, q = ints([n, 65, 448, 0, 701]), dev(sh, rng.standard_normal((B, T, n_h, D)) * 0.7)
    mask = words([O.tree_bits([-1, 0, 0, 1, 3, 2, 4])] * B)
    sel = ints([[0, 3, 3, 9, 13, 14], [0, 1, -1, -1, -1, -1], [6, 2, 5, 0, 1, 4], [-1] * k, [1, 2, 3, 4, 5, 10]])
    n_sel = ints([6, 2, 6, 0, 6])
    out = torch.empty(B, T, n_h, 512, dtype=dt, device="cuda")
    out1, lse1 = torch.empty(B, n_h, 512, dtype=dt, device="cuda"), torch.empty(B, n_h, device="cuda")
    ws = torch.empty(M.mla_tree_workspace_size(h, B, T), dtype=torch.uint8, device="cuda")
    ws1 = torch.empty(M.mla_decode_workspace_size(h, B), dtype=torch.uint8, device="cuda")

    def tree(st):
        M.mla_tree_attn(h, q, cache, n + T, None, 0, ctx, mask, B, T, 0, out, None, ws, ws.numel(), st)

    def sparse(st):
        M.mla_decode_attn_sparse(h, q, cache, n + T, None, 0, ctx, sel, n_sel, k, B, 0, ws1, ws1.numel(), st)
        M.mla_combine_splits(h, ws1, ws1.numel(), B, 0, out1, lse1, st)

    tree(None)
    sparse(None)
    torch.cuda.synchronize()
    alone, alone1, alone_lse = out.clone(), out1.clone(), lse1.clone()
    rows = host(cache)[0].reshape(-1, D)[:960]
    twice = np.concatenate([rows[64 * j:min(64 * j + 64, n)] for j in (0, 3, 3, 9, 13, 14)])
    want, _ = O.latent_attention(host(q).reshape(-1, n_h, D)[0], twice, d_c=512,
                                   scale=O.softmax_scale(sh["d_h"], sh["d_r"]))
    wl = WORKLOADS["v2lite_b32_ctx4k"]
    compare(host(alone1)[:1], {0: want}, wl, "ctx_lat with a block listed twice")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        out.fill_(0)
        out1.fill_(0)
        torch.cuda.synchronize()
        for _ in range(3):
            tree(a)
            sparse(b)
        torch.cuda.synchronize()
        assert torch.equal(out, alone) and torch.equal(out1, alone1) and torch.equal(lse1, alone_lse)
    ok(h)
    M.mla_destroy(h)
