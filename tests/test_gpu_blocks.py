"""Sparse decode attention on the GPU: block means, block scores, selection
and attention over the selected blocks, against the float64 oracle."""

import numpy as np
import pytest
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from tests.operators_harness import (LITE, ODD, TINY, V2, Cache, attention_bounds, dev, handle, host, ints, ok, score_error,
                                     shape, stored, torch_type, within)

pytestmark = pytest.mark.gpu

SHAPES = [(shape(LITE), 0), (shape(LITE), 64), (shape(V2), 64), (shape(V2, n_h=40), 0), (shape(TINY), 0),
          (shape(TINY), 16), (shape(ODD), 48)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from head_latent_attention_09_b200 import build
    build.build()
    assert torch.cuda.is_available()


def half_step(sh):
    return 2.0 ** -8 if sh["dtype"] == "bf16" else 2.0 ** -24


def status(fn, *a):
    try:
        fn(*a)
    except M.MlaError as e:
        return e.status
    return M.MLA_OK


@pytest.mark.parametrize("sh,page", SHAPES)
def test_block_keys(sh, page):
    rng = np.random.default_rng(page)
    D = sh["d_c"] + sh["d_r"]
    ctx = [0, 1, 63, 64, 65, 129, 700, 300]
    begin = [0, 0, 62, 0, 64, 128, 0, 300]
    rows = [stored(sh, rng.standard_normal((n, D)) + 0.3) for n in ctx]
    h = handle(sh, page)
    cache = Cache(sh, rows, 701, page, rng)
    blocks = 12
    for beg, hint in ((None, 700), (begin, 700), (begin, 1)):
        keys = torch.full((len(ctx), blocks, D), 9.0, dtype=torch_type(sh), device="cuda")
        M.mla_block_keys(h, *cache.args, None if beg is None else ints(beg), ints(ctx), len(ctx), hint, keys, blocks)
        ok(h)
        got = host(keys)
        for b, n in enumerate(ctx):
            want = O.block_means(rows[b])
            first = 0 if beg is None else (beg[b] // 64 if beg[b] < n else len(want))
            assert (got[b, :first] == 9.0).all() and (got[b, len(want):] == 9.0).all()
            # 63 additions and a division in float32, one rounding
            mass = O.block_means(np.abs(rows[b]))
            within(got[b, first:len(want)], want[first:], (half_step(sh) * 1.01 * np.abs(want) + 65 * 2.0 ** -24 * mass)[first:],
                   f"means of sequence {b}")
    M.mla_destroy(h)


@pytest.mark.parametrize("sh,page", SHAPES[:1] + SHAPES[4:5])
def test_block_keys_bounds(sh, page):
    rng = np.random.default_rng(0)
    D = sh["d_c"] + sh["d_r"]
    rows = [stored(sh, rng.standard_normal((130, D)))] * 2
    h = handle(sh, page)
    cache = Cache(sh, rows, 130, page, rng)
    keys = torch.full((2, 2, D), 9.0, dtype=torch_type(sh), device="cuda")
    for beg, ctx in (((0, 0), (130, 64)), ((0, 0), (131, 64)), ((-1, 0), (64, 64)), ((0, 0), (-1, 64))):
        M.mla_block_keys(h, *cache.args, ints(beg), ints(ctx), 2, 130, keys, 2)
        assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
        want = O.block_means(rows[1][:64])
        within(host(keys)[1, :1], want, half_step(sh) * 1.01 * np.abs(want) + 2.0 ** -16, "the other sequence")
    M.mla_destroy(h)


def scores_of(sh, h, q, keys, ctx, blocks):
    B = len(ctx)
    size = M.mla_block_scores_workspace_size(h, B, blocks)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((B, blocks), float("nan"), device="cuda")
    M.mla_block_scores(h, dev(sh, q), dev(sh, keys), blocks, ints(ctx), B, out, ws, size)
    return host(out)


@pytest.mark.parametrize("blocks", [1, 5, 127, 128, 129, 300, 520, 1100, 2049, 3900])
@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(V2, n_h=200), shape(TINY), shape(ODD)])
def test_block_scores(sh, blocks):
    rng = np.random.default_rng(blocks)
    D = sh["d_c"] + sh["d_r"]
    ctx = [64 * blocks, max(0, 64 * blocks - 63), 0, 1, min(64, 64 * blocks), 64 * (blocks // 2) + 5]
    B = len(ctx)
    keys = stored(sh, rng.standard_normal((B, blocks, D)))
    q = stored(sh, rng.standard_normal((B, sh["n_h"], D)) * 0.7)
    given = keys.copy()
    for b, n in enumerate(ctx):
        given[b, -(-n // 64):] = np.nan          # keys of blocks that are not there
    h = handle(sh)
    got = scores_of(sh, h, q, given, ctx, blocks)
    ok(h)
    M.mla_destroy(h)
    compare_scores(sh, got, q, keys, ctx)


def test_block_scores_beyond_the_tensor_core_kernel():
    """More than 4096 blocks run on the CUDA cores (strict mode refuses)."""
    sh = shape(LITE)
    rng = np.random.default_rng(0)
    ctx = [64 * 4100 - 5, 70]
    keys = stored(sh, rng.standard_normal((2, 4100, 576)))
    q = stored(sh, rng.standard_normal((2, 16, 576)) * 0.7)
    h = handle(sh, strict=True)
    with pytest.raises(M.MlaError) as e:
        scores_of(sh, h, q, keys, ctx, 4100)
    assert e.value.status == M.MLA_ERR_UNSUPPORTED
    M.mla_set_strict(h, 0)
    got = scores_of(sh, h, q, keys, ctx, 4100)
    ok(h)
    M.mla_destroy(h)
    compare_scores(sh, got, q, keys, ctx)


def compare_scores(sh, got, q, keys, ctx):
    scale = O.softmax_scale(sh["d_h"], sh["d_r"])
    for b, n in enumerate(ctx):
        nb = -(-n // 64)
        assert (got[b, nb:] == 0).all()
        if nb == 0:
            continue
        k = keys[b, :nb].astype(np.float64)
        want = O.block_scores(q[b], k, n, scale=scale)
        # a share is off by twice its head's largest score error, and by a few
        # steps per exponential and per term of the two sums
        e = score_error(q[b].astype(np.float64), k, scale).max() + 2.0 ** -23 * 8
        within(got[b, :nb], want, want * (2 * e + (nb + sh["n_h"] + 32) * 2.0 ** -23), f"scores of sequence {b}")
        assert abs(got[b].sum() - sh["n_h"]) < 1e-3 * sh["n_h"]


def test_block_scores_more_blocks_than_keys():
    sh = shape(LITE)
    rng = np.random.default_rng(0)
    keys = stored(sh, rng.standard_normal((2, 3, 576)))
    q = stored(sh, rng.standard_normal((2, 16, 576)))
    h = handle(sh)
    got = scores_of(sh, h, q, keys, [64 * 3 + 1, 100], 3)
    assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    assert abs(got.sum(1) - 16).max() < 1e-3
    M.mla_destroy(h)


@pytest.mark.parametrize("blocks,k", [(1, 1), (2, 1), (40, 7), (40, 40), (40, 64), (129, 16), (500, 33), (2048, 64),
                                      (5000, 1), (49152, 100)])
@pytest.mark.parametrize("first,last", [(0, 0), (1, 2), (3, 0), (100, 100)])
def test_block_select(blocks, k, first, last):
    rng = np.random.default_rng(blocks + k)
    ctx = [64 * blocks, 64 * blocks - 63, 0, 1, 64 * (blocks // 2), 64 * blocks, 64 * blocks, 64 * blocks]
    B = len(ctx)
    x = rng.standard_normal((B, blocks)).astype(np.float32)
    x[1] = np.exp(3 * x[1]) / np.exp(3 * x[1]).sum()
    x[5] = np.round(x[5])                        # many equal values, zeros of both signs
    x[6] = 0.25                                  # all equal
    x[7, ::3] = np.nan
    x[7, 1::7] = np.inf
    x[7, 2::7] = -np.inf
    h = handle(shape(LITE))
    sel = torch.full((B, k), -7, dtype=torch.int32, device="cuda")
    n_sel = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    M.mla_block_select(h, torch.from_numpy(x).cuda(), blocks, ints(ctx), B, k, first, last, sel, n_sel)
    ok(h)
    for b, n in enumerate(ctx):
        nb = -(-n // 64)
        want = O.block_select(x[b, :nb].tolist(), k, first, last)
        assert n_sel[b].item() == len(want)
        assert sel[b].tolist() == want + [-1] * (k - len(want)), b
    M.mla_destroy(h)


def test_block_select_bounds_and_refusals():
    h = handle(shape(LITE))
    x = torch.arange(8, dtype=torch.float32, device="cuda").reshape(2, 4)
    sel, n_sel = ints([[0, 0]] * 2), ints([0, 0])
    M.mla_block_select(h, x, 4, ints([64 * 5, 65]), 2, 2, 0, 0, sel, n_sel)
    assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    assert sel.tolist() == [[2, 3], [0, 1]] and n_sel.tolist() == [2, 2]
    good = [h, x, 4, n_sel, 2, 2, 0, 0, sel, n_sel]
    for at, bad in ((1, None), (3, None), (8, None), (9, None), (2, -1), (4, -1), (5, -1), (6, -1), (7, -1),
                    (5, (1 << 20) + 1)):
        a = list(good)
        a[at] = bad
        assert status(M.mla_block_select, *a) == M.MLA_ERR_INVALID_ARG, at
    a = list(good)
    a[2] = 49153
    assert status(M.mla_block_select, *a) == M.MLA_ERR_UNSUPPORTED
    assert status(M.mla_block_keys, h, x, 1, None, 0, None, None, 1, 1, x, 1) == M.MLA_ERR_INVALID_ARG
    assert status(M.mla_block_keys, h, x, 1, n_sel, 0, None, n_sel, 1, 1, x, 1) == M.MLA_ERR_INVALID_ARG
    assert status(M.mla_block_keys, h, x, 1, None, 0, None, n_sel, 1, 1, None, 1) == M.MLA_ERR_INVALID_ARG
    assert status(M.mla_block_keys, h, x, 1, None, 0, None, n_sel, 1, -1, x, 1) == M.MLA_ERR_INVALID_ARG
    assert status(M.mla_block_scores, h, None, x, 1, n_sel, 1, x, x, 1 << 20) == M.MLA_ERR_INVALID_ARG
    assert status(M.mla_block_scores, h, x, x, 1, n_sel, 1, x, None, 1 << 20) == M.MLA_ERR_WORKSPACE
    assert status(M.mla_block_scores, h, x, x, 1, n_sel, 1, x, x, 1) == M.MLA_ERR_WORKSPACE
    sp = [h, x, x, 1, None, 0, n_sel, sel, n_sel, 2, 2, 0, None, 0]
    assert status(M.mla_decode_attn_sparse, *sp) == M.MLA_ERR_WORKSPACE
    for at, bad in ((1, None), (2, None), (6, None), (7, None), (8, None), (9, 0), (9, -1), (10, -1), (4, n_sel)):
        a = list(sp)
        a[at] = bad
        assert status(M.mla_decode_attn_sparse, *a) == M.MLA_ERR_INVALID_ARG, at
    ok(h)
    M.mla_destroy(h)
    h = handle(shape(TINY), 16)
    sp[0], sp[4], sp[5] = h, n_sel, 1
    assert status(M.mla_decode_attn_sparse, *sp) == M.MLA_ERR_UNSUPPORTED
    M.mla_destroy(h)


class Sparse:
    def __init__(self, sh, ctx, k, seed, page):
        rng = np.random.default_rng(seed)
        D = sh["d_c"] + sh["d_r"]
        self.sh, self.ctx, self.k, self.page, self.rng = sh, list(ctx), k, page, rng
        self.rows = [stored(sh, rng.standard_normal((n, D))) for n in ctx]
        self.q = stored(sh, rng.standard_normal((len(ctx), sh["n_h"], D)) * 0.7)
        self.sel = []
        for n in ctx:
            nb = -(-n // 64)
            take = sorted(rng.choice(nb, min(nb, int(rng.integers(1, k + 1))), replace=False).tolist()) if nb else []
            self.sel.append(take)

    def run(self, parts=0):
        sh, B, k = self.sh, len(self.ctx), self.k
        h = handle(sh, self.page)
        cache = Cache(sh, self.rows, max(self.ctx) + 5, self.page, np.random.default_rng(1))
        sel = np.full((B, k), -1)
        for b, s in enumerate(self.sel):
            sel[b, :len(s)] = s
        size = M.mla_decode_workspace_size(h, B, parts)
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((B, sh["n_h"], sh["d_c"]), float("nan"), dtype=torch_type(sh), device="cuda")
        lse = torch.full((B, sh["n_h"]), float("nan"), device="cuda")
        M.mla_decode_attn_sparse(h, dev(sh, self.q), *cache.args, ints(self.ctx), ints(sel),
                                 ints([len(s) for s in self.sel]), k, B, parts, ws, size)
        M.mla_combine_splits(h, ws, size, B, parts, out, lse)
        ok(h)
        M.mla_destroy(h)
        sc = O.softmax_scale(sh["d_h"], sh["d_r"])
        got = host(out), host(lse)
        for b, n in enumerate(self.ctx):
            parts_ = [self.rows[b][64 * j:64 * j + 64] for j in self.sel[b]]
            rows = np.concatenate(parts_).astype(np.float64) if parts_ else np.zeros((0, self.q.shape[-1]))
            q = self.q[b].astype(np.float64)
            want, z = O.latent_attention(q, rows, d_c=sh["d_c"], scale=sc)
            bo, bl = attention_bounds(sh, q, rows, sc, want, z)
            within(got[0][b], want, bo, f"ctx_lat of sequence {b}")
            within(got[1][b], z, bl, f"lse of sequence {b}")
        return got


@pytest.mark.parametrize("k", [1, 5, 20])
@pytest.mark.parametrize("sh,page", [(shape(LITE), 0), (shape(LITE), 64), (shape(LITE, n_h=32), 64), (shape(V2), 0),
                                     (shape(V2), 64), (shape(TINY), 0), (shape(TINY), 64), (shape(ODD), 128)])
def test_sparse_attention(sh, page, k):
    Sparse(sh, (0, 1, 64, 65, 640, 1000, 1601), k, k + page, page).run()


@pytest.mark.parametrize("parts", [1, 3, 50, 500])
@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(TINY)])
def test_sparse_split_counts(sh, parts):
    Sparse(sh, (1601, 700), 16, parts, 0).run(parts)


@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(V2, n_h=40)])
@pytest.mark.parametrize("B", [90, 300])
def test_many_short_sequences(sh, B):
    """Several ragged sequences to a share, so that one partial last block
    follows another; more of them than plan sequences that are planned in line."""
    rng = np.random.default_rng(B)
    Sparse(sh, [int(n) for n in rng.integers(0, 700, B)], 6, B, 64).run()


def test_every_block_selected_is_dense_attention():
    sh = shape(LITE)
    s = Sparse(sh, (640, 333), 10, 1, 64)
    s.sel = [list(range(10)), list(range(6))]
    got = s.run()
    h = handle(sh, 64)
    cache = Cache(sh, s.rows, 645, 64, np.random.default_rng(1))
    size = M.mla_decode_workspace_size(h, 2, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda")
    M.mla_decode_attn(h, dev(sh, s.q), *cache.args, ints(s.ctx), 2, 0, ws, size)
    M.mla_combine_splits(h, ws, size, 2, 0, out)
    ok(h)
    assert np.array_equal(host(out), got[0])
    M.mla_destroy(h)


def test_blocks_in_any_order_and_twice():
    s = Sparse(shape(LITE), (640, 700), 8, 1, 64)
    s.sel = [[7, 2, 2, 0], [5, 1, 5, 3, 10]]     # 10 is the partial one
    s.run()


@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(TINY)])
def test_wrong_blocks_are_flagged_and_not_read(sh):
    ctx = (640, 700)
    s = Sparse(sh, ctx, 4, 1, 64)
    h = handle(sh, 64)
    cache = Cache(sh, s.rows, 700, 64, s.rng)
    size = M.mla_decode_workspace_size(h, 2, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for sel, n in (([0, -1, 2, 3], 4), ([0, 11, 2, 3], 4), ([10, 1, 2, 3], 4), ([0, 1 << 30, 2, 3], 4),
                   ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -1), ([0, 1, 2, -1], 4), ([0, 1, 2, 2 ** 31 - 1], 4)):
        M.mla_decode_attn_sparse(h, dev(sh, s.q), *cache.args, ints(ctx), ints([[0, 1, 2, 3], sel]), ints([4, n]), 4,
                                 2, 0, ws, size)
        assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS, (sel, n)
    M.mla_destroy(h)


@pytest.mark.parametrize("sh,page", [(shape(LITE), 64), (shape(V2), 0), (shape(TINY), 16)])
def test_guard_bands_streams_and_graphs(sh, page):
    """Nothing is written outside the outputs; the calls are the same on another
    stream, and captured and replayed on other inputs."""
    rng = np.random.default_rng(3)
    D, B, k, blocks = sh["d_c"] + sh["d_r"], 3, 4, 12
    ctx, ctx2 = [700, 63, 321], [128, 700, 1]
    h = handle(sh, page)
    caches = [Cache(sh, [stored(sh, rng.standard_normal((n, D))) for n in c], 700, page, np.random.default_rng(1))
              for c in (ctx, ctx2)]
    dt, raws = torch_type(sh), []

    def buffer(shape_, dtype):
        n = int(np.prod(shape_)) * torch.empty((), dtype=dtype).element_size()
        raws.append(torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda"))
        return raws[-1][4096:-4096].view(dtype).view(shape_)

    keys, scores = buffer((B, blocks, D), dt), buffer((B, blocks), torch.float32)
    sel, n_sel = buffer((B, k), torch.int32), buffer((B,), torch.int32)
    sws = buffer((M.mla_block_scores_workspace_size(h, B, blocks),), torch.uint8)
    sparse = page % 64 == 0
    ws = buffer((M.mla_decode_workspace_size(h, B, 0),), torch.uint8)
    out = buffer((B, sh["n_h"], sh["d_c"]), dt)
    q = dev(sh, rng.standard_normal((B, sh["n_h"], D)) * 0.7)
    data, lens = caches[0].data.clone(), ints(ctx)
    args = (data, caches[0].len, caches[0].table, caches[0].max_blk)

    def call(st):
        M.mla_block_keys(h, *args, None, lens, B, 700, keys, blocks, st)
        M.mla_block_scores(h, q, keys, blocks, lens, B, scores, sws, sws.numel(), st)
        M.mla_block_select(h, scores, blocks, lens, B, k, 1, 1, sel, n_sel, st)
        if sparse:
            M.mla_decode_attn_sparse(h, q, *args, lens, sel, n_sel, k, B, 0, ws, ws.numel(), st)
            M.mla_combine_splits(h, ws, ws.numel(), B, 0, out, None, st)

    def results():
        torch.cuda.synchronize()
        valid = [-(-n // 64) for n in lens.tolist()]
        return [host(keys)[b, :v] for b, v in enumerate(valid)] + [host(x) for x in (scores, sel, n_sel, *((out,) if sparse else ()))]

    want = []
    for c, cache in ((ctx, caches[0]), (ctx2, caches[1])):
        data.copy_(cache.data)
        lens.copy_(ints(c))
        call(None)
        want.append(results())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(torch.cuda.current_stream())
    data.copy_(caches[0].data)
    lens.copy_(ints(ctx))
    torch.cuda.synchronize()
    call(s)
    assert all(np.array_equal(a, b) for a, b in zip(results(), want[0]))
    data.copy_(caches[1].data)
    lens.copy_(ints(ctx2))
    for _ in range(2):
        out.fill_(0)
        g.replay()
    assert all(np.array_equal(a, b) for a, b in zip(results(), want[1]))
    ok(h)
    for r in raws:
        assert (r[:4096] == 0x5A).all() and (r[-4096:] == 0x5A).all()
    M.mla_destroy(h)


@pytest.mark.parametrize("at", [[0], list(range(32)), list(range(32, 64)), list(range(128)), list(range(128, 256)), [299]])
@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(TINY)])
def test_block_scores_of_nan_and_of_minus_infinity(sh, at):
    """A mean row with a NaN makes every share of the sequence NaN, wherever it
    stands; a block whose scores overflow to -inf draws nothing and changes no
    other block."""
    rng = np.random.default_rng(at[0])
    blocks, D = 300, sh["d_c"] + sh["d_r"]
    ctx = [64 * blocks, 64 * blocks - 9]
    keys = stored(sh, rng.standard_normal((2, blocks, D)))
    q = stored(sh, rng.standard_normal((2, sh["n_h"], D)) * 0.7)
    h = handle(sh)
    bad = keys.copy()
    bad[0, at, 5] = np.nan
    got = scores_of(sh, h, q, bad, ctx, blocks)
    assert np.isnan(got[0]).all()
    compare_scores(sh, got[1:], q[1:], keys[1:], ctx[1:])
    keys[:, :, 0] = 0
    q[:, :, 0] = stored(sh, np.array([1e20]))
    bad = keys.copy()
    bad[0, at, 0] = stored(sh, np.array([-1e20]))      # q . key = -1e40
    got = scores_of(sh, h, q, bad, ctx, blocks)
    ok(h)
    M.mla_destroy(h)
    rest = [j for j in range(blocks) if j not in at]
    assert (got[0, at] == 0).all()
    compare_scores(sh, got[:1, rest], q[:1], keys[:1, rest], [64 * len(rest)])
    compare_scores(sh, got[1:], q[1:], keys[1:], ctx[1:])


@pytest.mark.parametrize("sh", [shape(LITE), shape(V2)])
@pytest.mark.parametrize("B,k", [(256, 3), (257, 3), (33, 1)])
def test_sparse_plan_in_line_and_by_its_own_kernel(sh, B, k):
    """Up to 256 sequences the attention kernel makes the plan itself."""
    rng = np.random.default_rng(B)
    D, n_h = sh["d_c"] + sh["d_r"], sh["n_h"]
    ctx = [int(c) for c in rng.integers(0, 400, B)]
    ctx[5], ctx[6] = 0, 64
    rows = [stored(sh, rng.standard_normal((n, D))) for n in ctx]
    h = handle(sh)
    cache = Cache(sh, rows, 400, 0, rng)
    sel, n_sel = np.full((B, k), -1), np.zeros(B)
    for b, n in enumerate(ctx):
        blocks = -(-n // 64)
        take = sorted(rng.permutation(blocks)[:k])
        sel[b, :len(take)], n_sel[b] = take, len(take)
    q = stored(sh, rng.standard_normal((B, n_h, D)) * 0.7)
    for parts in (0, 7):
        ws = torch.empty(M.mla_decode_workspace_size(h, B, parts), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty(B, n_h, sh["d_c"], dtype=torch_type(sh), device="cuda"), torch.empty(B, n_h, device="cuda")
        M.mla_decode_attn_sparse(h, dev(sh, q), *cache.args, ints(ctx), ints(sel), ints(n_sel), k, B, parts, ws, ws.numel())
        M.mla_combine_splits(h, ws, ws.numel(), B, parts, out, lse)
        ok(h)
        got, got_lse = host(out), host(lse)
        for b in range(B):
            mine = [rows[b][64 * j:64 * j + 64] for j in sel[b] if j >= 0]
            if not mine:
                assert (got[b] == 0).all() and np.isneginf(got_lse[b]).all()
                continue
            mine, qb = np.concatenate(mine).astype(np.float64), q[b].astype(np.float64)
            scale = O.softmax_scale(sh["d_h"], sh["d_r"])
            want, wl = O.latent_attention(qb, mine, d_c=sh["d_c"], scale=scale)
            bo, bl = attention_bounds(sh, qb, mine, scale, want, wl)
            within(got[b], want, bo, f"ctx_lat of sequence {b}")
            within(got_lse[b], wl, bl, f"lse of sequence {b}")
    M.mla_destroy(h)


@pytest.mark.parametrize("sh,page", SHAPES)
def test_block_keys_of_many_blocks(sh, page):
    """More blocks than the GPU has SMs: the form with fewer threads a block."""
    rng = np.random.default_rng(page + 1)
    D = sh["d_c"] + sh["d_r"]
    ctx = [64 * 60, 64 * 59 + 1, 64 * 31 - 1, 200]
    rows = [stored(sh, rng.standard_normal((n, D)) + 0.3) for n in ctx]
    h = handle(sh, page)
    cache = Cache(sh, rows, 64 * 60, page, rng)
    keys = torch.full((4, 60, D), 9.0, dtype=torch_type(sh), device="cuda")
    M.mla_block_keys(h, *cache.args, None, ints(ctx), 4, 64 * 60, keys, 60)
    ok(h)
    M.mla_destroy(h)
    got = host(keys)
    for b in range(4):
        want, mass = O.block_means(rows[b]), O.block_means(np.abs(rows[b]))
        assert (got[b, len(want):] == 9.0).all()
        within(got[b, :len(want)], want, half_step(sh) * 1.01 * np.abs(want) + 65 * 2.0 ** -24 * mass,
               f"means of sequence {b}")


@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(TINY)])
@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 63, 2 ** 31 - 64, -1, -2 ** 31])
def test_lengths_at_the_ends_of_the_integers(sh, n):
    """Scores and selection of a length that no cache holds: flagged, and taken
    over the blocks there are (none of a negative length); nothing is written
    outside the outputs."""
    rng = np.random.default_rng(0)
    blocks, k, D = 5, 3, sh["d_c"] + sh["d_r"]
    keys = stored(sh, rng.standard_normal((2, blocks, D)))
    q = stored(sh, rng.standard_normal((2, sh["n_h"], D)) * 0.7)
    ctx = [n, 64 * 4]
    h = handle(sh)
    got = scores_of(sh, h, q, keys, ctx, blocks)
    assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    compare_scores(sh, got, q, keys, [64 * blocks if n > 0 else 0, ctx[1]])
    guard = torch.full((2 * k + 4096,), 77, dtype=torch.int32, device="cuda")
    sel, n_sel = guard[2048:2048 + 2 * k], ints([9, 9])
    M.mla_block_select(h, torch.from_numpy(got.astype(np.float32)).cuda(), blocks, ints(ctx), 2, k, 0, 1, sel, n_sel)
    assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    M.mla_destroy(h)
    want = [O.block_select(got[0].tolist(), k, 0, 1) if n > 0 else [], O.block_select(got[1, :4].tolist(), k, 0, 1)]
    assert n_sel.tolist() == [len(w) for w in want]
    assert sel.tolist() == want[0] + [-1] * (k - len(want[0])) + want[1]
    assert (guard[:2048] == 77).all() and (guard[2048 + 2 * k:] == 77).all()


@pytest.mark.parametrize("page", [0, 64])
def test_an_odd_latent_width(page):
    sh = shape((3, 24, 41, 6, 128, "bf16"))
    test_block_keys(sh, page)
    test_block_scores(sh, 130)
    Sparse(sh, (0, 1, 64, 65, 640, 1000, 1601), 5, 1, page).run()
