"""Scores that are NaN or overflow float32 on the GPU: they reach the rows that
attend them, whatever kernel, split or merge computes the row, and no others."""

import numpy as np
import pytest
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from tests.operators_harness import (LITE, ODD, TINY, V2, Cache, attention_bounds, dev, handle, host, ints, ok, shape,
                                     stored, torch_type, within)
from tests.test_gpu_blocks import Sparse, compare_scores, scores_of
from tests.test_gpu_tree import Tree

pytestmark = pytest.mark.gpu

# 16, 32 and 128 heads on the tensor cores, 40 heads and float32 on the CUDA cores
SHAPES = [(shape(LITE), 64), (shape(LITE, n_h=32), 0), (shape(V2), 64), (shape(V2), 0), (shape(V2, n_h=40), 64),
          (shape(TINY), 0)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from head_latent_attention_09_b200 import build
    build.build()
    assert torch.cuda.is_available()


BIG = float(stored(shape(LITE), np.array([1e20]))[0])     # BIG * BIG overflows float32


@pytest.mark.parametrize("parts", [1, 0])       # every row in one piece, or in several
@pytest.mark.parametrize("sh,page", SHAPES)
def test_sparse_attention_keeps_a_nan(sh, page, parts):
    """A NaN in a selected row reaches every head of its sequence, one in a query
    that head alone; a score of +inf makes its row NaN."""
    s = Sparse(sh, (1601, 700, 1601, 60, 130), 26, 3, page)
    s.sel = [list(range(26)), [0, 2, 3, 10], list(range(25)), [0], [1, 2]]
    s.rows[0][70, 3] = np.nan
    s.rows[3][10, -1] = np.nan
    s.q[1, 2, 7] = np.nan
    s.run(parts)


@pytest.mark.parametrize("parts", [1, 0])
@pytest.mark.parametrize("sh,page", SHAPES)
def test_sparse_attention_of_a_score_of_plus_infinity(sh, page, parts):
    s = Sparse(sh, (1601, 700), 26, 3, page)
    s.sel = [list(range(26)), list(range(11))]
    for r in s.rows:
        r[:, -1] = 0
    s.q[:, :, -1] = BIG
    clean = s.run(parts)
    s.rows[0][1000, -1] = BIG
    got = attend(s, parts)
    assert np.isnan(got[0][0]).all() and np.isnan(got[1][0]).all()
    assert np.array_equal(got[0][1], clean[0][1]) and np.array_equal(got[1][1], clean[1][1])


def attend(s, parts):
    """ctx_lat and lse of a sparse call, without a comparison."""
    sh, B, k = s.sh, len(s.ctx), s.k
    h = handle(sh, s.page)
    cache = Cache(sh, s.rows, max(s.ctx) + 5, s.page, np.random.default_rng(1))
    sel = np.full((B, k), -1)
    for b, x in enumerate(s.sel):
        sel[b, :len(x)] = x
    size = M.mla_decode_workspace_size(h, B, parts)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.empty(B, sh["n_h"], sh["d_c"], dtype=torch_type(sh), device="cuda")
    lse = torch.empty(B, sh["n_h"], device="cuda")
    M.mla_decode_attn_sparse(h, dev(sh, s.q), *cache.args, ints(s.ctx), ints(sel), ints([len(x) for x in s.sel]), k, B,
                             parts, ws, size)
    M.mla_combine_splits(h, ws, size, B, parts, out, lse)
    ok(h)
    M.mla_destroy(h)
    return host(out), host(lse)


@pytest.mark.parametrize("parts", [1, 0])
@pytest.mark.parametrize("finish", ["splits", "f32", "out_proj", "ranges"])
@pytest.mark.parametrize("sh,page", SHAPES)
def test_every_merge_keeps_a_nan(sh, page, finish, parts):
    """Decode attention ends in the same pieces and merges; the sequences and
    heads without a NaN keep their results bit for bit."""
    rng = np.random.default_rng(7)
    n_h, d_h, d_c = (sh[k] for k in ("n_h", "d_h", "d_c"))
    D, ctx = d_c + sh["d_r"], [1500, 64, 900, 0]
    B = len(ctx)
    rows = [stored(sh, rng.standard_normal((n, D))) for n in ctx]
    q = stored(sh, rng.standard_normal((B, n_h, D)) * 0.7)
    w_uv = dev(sh, rng.standard_normal((n_h * d_h, d_c)) * d_c ** -0.5)
    h = handle(sh, page, strict=False)
    ws = torch.empty(M.mla_decode_workspace_size(h, B, parts), dtype=torch.uint8, device="cuda")
    lens = ints(ctx)

    def results(rows, q):
        cache = Cache(sh, rows, max(ctx), page, np.random.default_rng(1))
        M.mla_decode_attn(h, dev(sh, q), *cache.args, lens, B, parts, ws, ws.numel())
        out = torch.empty(B, n_h, d_c, dtype=torch_type(sh), device="cuda")
        lse = torch.empty(B, n_h, device="cuda")
        if finish == "splits":
            M.mla_combine_splits(h, ws, ws.numel(), B, parts, out, lse)
        elif finish == "out_proj":
            o = torch.empty(B, n_h, d_h, dtype=torch_type(sh), device="cuda")
            M.mla_combine_out_proj(h, ws, ws.numel(), B, parts, w_uv, None, o, None, out, lse)
            ok(h)
            return host(out), host(lse), host(o)
        else:
            one = torch.empty(2, B, n_h, d_c, device="cuda"), torch.empty(2, B, n_h, device="cuda")
            M.mla_combine_splits_f32(h, ws, ws.numel(), B, parts, one[0][0], one[1][0])
            if finish == "f32":
                out, lse = one[0][0], one[1][0]
            else:      # the other range holds no tokens
                one[0][1].zero_()
                one[1][1].fill_(-np.inf)
                M.mla_merge_ranges(h, *one, 2, B, out, lse)
        ok(h)
        return host(out), host(lse)

    clean = results(rows, q)
    bad, badq = [r.copy() for r in rows], q.copy()
    bad[0][130, 5] = np.nan
    badq[1, 1, 3] = np.nan
    got = results(bad, badq)
    M.mla_destroy(h)
    lost = np.zeros((B, n_h), bool)
    lost[0] = True
    lost[1, 1] = True
    for g, c in zip(got, clean):
        assert np.isfinite(c).all() or np.isneginf(c[3]).all()
        assert np.isnan(g[lost]).all()
        assert np.array_equal(g[~lost], c[~lost])
    assert (got[0][3] == 0).all() and np.isneginf(got[1][3]).all()


@pytest.mark.parametrize("parts", [1, 0])
@pytest.mark.parametrize("n_h", [16, 32, 128])
def test_fp8_attention_keeps_a_nan(n_h, parts):
    """The code 0x7f is E4M3's NaN."""
    sh = shape(LITE, n_h=n_h)
    rng = np.random.default_rng(1)
    ctx, n = [700, 100], 700
    h = handle(sh, strict=False)
    rows = dev(sh, rng.standard_normal((2, n, 576)))
    codes = torch.empty(2, n, 576, dtype=torch.uint8, device="cuda")
    scale = torch.empty(2, n, M.mla_fp8_scale_groups(h), device="cuda")
    M.mla_quantize_rows_fp8(h, rows, 2 * n, codes, scale)
    q = dev(sh, rng.standard_normal((2, n_h, 576)) * 0.7)
    ws = torch.empty(M.mla_decode_workspace_size(h, 2, parts), dtype=torch.uint8, device="cuda")
    res = []
    for _ in range(2):
        out, lse = torch.empty(2, n_h, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, n_h, device="cuda")
        M.mla_decode_attn_fp8(h, q, codes, scale, n, None, 0, ints(ctx), 2, parts, ws, ws.numel())
        M.mla_combine_splits(h, ws, ws.numel(), 2, parts, out, lse)
        ok(h)
        res.append((host(out), host(lse)))
        codes[0, 300, 17] = 0x7f
    M.mla_destroy(h)
    for g, c in zip(res[1], res[0]):
        assert np.isfinite(c).all() and np.isnan(g[0]).all() and np.array_equal(g[1], c[1])


@pytest.mark.parametrize("parts", [1, 0])
@pytest.mark.parametrize("first", [1, 64, 256, 300, 700])
@pytest.mark.parametrize("sh,page", SHAPES)
def test_sparse_scores_that_overflow_to_minus_infinity(sh, page, first, parts):
    """Tokens whose scores overflow to -inf draw nothing, whole tiles and pieces
    of them at the front included; where no other token is left the row is
    empty."""
    s = Sparse(sh, (700, 1000, 1), 16, first, page)
    s.sel = [list(range(11)), list(range(16)), [0]]
    s.q[..., -1] = BIG
    for r in s.rows:
        r[:, -1] = 0
    given = [r.copy() for r in s.rows]
    for r in given:
        r[:first, -1] = -BIG
    kept, s.rows = s.rows, given
    got = attend(s, parts)
    scale = O.softmax_scale(sh["d_h"], sh["d_r"])
    for b, r in enumerate(kept):
        rest, q = r[first:].astype(np.float64), s.q[b].astype(np.float64)
        want, lse = O.latent_attention(q, rest, d_c=sh["d_c"], scale=scale)
        bo, bl = attention_bounds(sh, q, rest, scale, want, lse)
        within(got[0][b], want, bo, f"ctx_lat of sequence {b}")
        within(got[1][b], lse, bl, f"lse of sequence {b}")


@pytest.mark.parametrize("blocks", [1, 5, 300, 1100])
@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(V2, n_h=200), shape(TINY), shape(ODD)])
def test_block_scores_of_a_head_with_nothing_but_minus_infinity(sh, blocks):
    """Such a head adds nothing to any block; where every head is one the scores
    are zero."""
    rng = np.random.default_rng(blocks)
    ctx, n_h = [64 * blocks, 64 * blocks - 9], sh["n_h"]
    keys = stored(sh, rng.standard_normal((2, blocks, sh["d_c"] + sh["d_r"])))
    q = stored(sh, rng.standard_normal((2, n_h, sh["d_c"] + sh["d_r"])) * 0.7)
    keys[:, :, 0], q[:, :, 0] = -BIG, 0
    q[0, n_h - 2, 0] = BIG
    q[1, :, 0] = BIG
    h = handle(sh)
    got = scores_of(sh, h, q, keys, ctx, blocks)
    ok(h)
    M.mla_destroy(h)
    keys[:, :, 0] = 0
    others = np.delete(q[0], n_h - 2, axis=0)
    compare_scores({**sh, "n_h": n_h - 1}, got[:1], others[None], keys[:1], ctx[:1])
    assert (got[1] == 0).all()


@pytest.mark.parametrize("bad", [np.inf, -np.inf])
@pytest.mark.parametrize("parts", [0, 3])
@pytest.mark.parametrize("sh,page", [(shape(LITE), 0), (shape(LITE), 64), (shape(LITE), 32), (shape(TINY), 0),
                                     (shape(ODD), 48)])
def test_drafted_infinity_that_meets_minus_infinity(sh, page, parts, bad):
    """An infinity of a drafted row's latent part whose scores are -inf counts as
    zero for the tokens that attend it: theirs are the results without the row."""
    t = Tree(sh, (60, 128, 300), 4, 8, page, [[1, 2, 5, 10]] * 3)
    t.q[..., 0] = stored(sh, -np.sign(bad) * (np.abs(t.q[..., 0]) + 0.25))
    rows = [r.copy() for r in t.rows]
    for r, n in zip(rows, t.ctx):
        r[n + 1, 0] = bad
    got = t.run(parts, rows=rows)
    t.bits = [[1, 0, 5, 8]] * 3
    t.check(got)
