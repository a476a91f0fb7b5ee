"""Tree of drafted tokens on the GPU: the append at tree positions, attention
under the tree's masks and the accepted path, against the float64 oracle."""

import numpy as np
import pytest
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from tests.operators_harness import (LITE, ODD, TINY, V2, Cache, attention_bounds, dev, handle, host, ints, ok,
                                     random_parents, shape, stored, torch_type, within, words)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from head_latent_attention_09_b200 import build
    build.build()
    assert torch.cuda.is_available()


class Tree:
    def __init__(self, sh, ctx, T, seed, page=0, bits=None, slots=None, gap=3):
        rng = np.random.default_rng(seed)
        self.sh, self.ctx, self.T, self.B = sh, list(ctx), T, len(ctx)
        D = sh["d_c"] + sh["d_r"]
        self.rows = [stored(sh, rng.standard_normal((n + T, D))) for n in ctx]
        self.bits = bits or [O.tree_bits(random_parents(rng, T)) for _ in ctx]
        self.q = stored(sh, rng.standard_normal((self.B, T, sh["n_h"], D)) * 0.7)
        self.slots = slots or max(ctx) + T + gap
        self.page, self.rng = page, rng

    def run(self, parts=0, h=None, stream=None, rows=None):
        sh, B, T = self.sh, self.B, self.T
        own = h is None
        h = h or handle(sh, self.page)
        cache = Cache(sh, rows or self.rows, self.slots, self.page, np.random.default_rng(1))
        out = torch.full((B, T, sh["n_h"], sh["d_c"]), float("nan"), dtype=torch_type(sh), device="cuda")
        lse = torch.full((B, T, sh["n_h"]), float("nan"), device="cuda")
        size = M.mla_tree_workspace_size(h, B, T, parts)
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
        M.mla_tree_attn(h, dev(sh, self.q), *cache.args, ints(self.ctx), words(self.bits), B, T, parts, out, lse, ws,
                        size, stream)
        ok(h)
        if own:
            M.mla_destroy(h)
        return host(out), host(lse)

    def check(self, got, scale=None):
        sh = self.sh
        scale = scale or O.softmax_scale(sh["d_h"], sh["d_r"])
        for b, n in enumerate(self.ctx):
            r = self.rows[b].astype(np.float64)
            q = self.q[b].astype(np.float64)
            want, lse = O.tree_attention(q, r[:n], r[n:], self.bits[b], d_c=sh["d_c"], scale=scale)
            for t in range(self.T):
                mine = np.concatenate([r[:n], r[n:][[j for j in range(self.T) if self.bits[b][t] >> j & 1]]])
                bo, bl = attention_bounds(sh, q[t], mine, scale, want[t], lse[t])
                within(got[0][b, t], want[t], bo, f"ctx_lat of sequence {b}, token {t}")
                within(got[1][b, t], lse[t], bl, f"lse of sequence {b}, token {t}")


LENGTHS = (0, 1, 63, 64, 65, 200, 255, 256, 257, 511, 700)


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("T", [1, 2, 13, 64])
def test_lite_lengths_and_sizes(T, page):
    t = Tree(shape(LITE), LENGTHS, T, 10 * T + page, page)
    t.check(t.run())


@pytest.mark.parametrize("B", [100, 300])
def test_many_short_sequences(B):
    """Several trees to a share; more of them than are planned in line."""
    rng = np.random.default_rng(B)
    t = Tree(shape(LITE), [int(n) for n in rng.integers(0, 500, B)], 3, B, 64)
    t.check(t.run())


@pytest.mark.parametrize("n_h,T", [(128, 1), (128, 3), (32, 5), (1, 7), (33, 4), (200, 2)])
def test_head_counts(n_h, T):
    t = Tree(shape(V2, n_h=n_h), (130, 0, 300), T, n_h, 0)
    t.check(t.run())


@pytest.mark.parametrize("parts", [1, 2, 5, 37, 1000])
def test_split_counts(parts):
    t = Tree(shape(LITE), (1500, 3, 900), 20, parts, 64)
    t.check(t.run(parts))


@pytest.mark.parametrize("sh,page", [(shape(TINY), 0), (shape(TINY), 16), (shape(ODD), 0), (shape(ODD), 48),
                                     (shape(LITE), 32)])
@pytest.mark.parametrize("parts", [0, 3])
def test_cuda_core_shapes(sh, page, parts):
    t = Tree(sh, (0, 1, 64, 130, 65), 6, page + parts, page)
    t.check(t.run(parts))


@pytest.mark.parametrize("sh", [shape(LITE), shape(TINY)])
def test_masks_that_leave_nothing_and_ignored_bits(sh):
    """A padding token (mask 0) attends the cached tokens only, and nothing
    where there are none; bits from T on are ignored."""
    T = 5
    bits = [[0b1, 0, 0b101, 0b1010, 0], [0, 0, 0, 0, 0], [0b11111] * 5]
    t = Tree(sh, (0, 70, 256), T, 3, 0, bits)
    want = t.run()
    t.check(want)
    t.bits = [[w | (2 ** 64 - 2 ** T) for w in row] for row in bits]
    again = t.run()
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(want, again))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("sh", [shape(LITE), shape(TINY)])
def test_masked_rows_may_hold_anything(sh, page, bad):
    """A drafted row that some tokens do not attend: theirs are the results of
    the row without it, bit for bit."""
    T = 4
    t = Tree(sh, (60, 128), T, 8, page, [[1, 2, 5, 10]] * 2)
    clean = t.run()
    rows = [r.copy() for r in t.rows]
    for b, n in enumerate(t.ctx):
        rows[b][n + 1] = bad
    got = t.run(rows=rows)
    for t_ in (0, 2):
        assert np.array_equal(got[0][:, t_], clean[0][:, t_]) and np.array_equal(got[1][:, t_], clean[1][:, t_])
    if np.isnan(bad):
        assert np.isnan(got[0][:, [1, 3]]).all() and np.isnan(got[1][:, [1, 3]]).all()


def test_full_cache_and_lengths_it_cannot_hold():
    sh = shape(LITE)
    t = Tree(sh, (100, 61), 3, 4, 0, slots=103)
    t.check(t.run())
    h = handle(sh)
    cache = Cache(sh, t.rows, 103, 0, t.rng)
    out = torch.zeros(2, 3, 16, 512, dtype=torch.bfloat16, device="cuda")
    size = M.mla_tree_workspace_size(h, 2, 3)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for ctx in ((101, 61), (100, -1), (2 ** 31 - 1, 61)):
        M.mla_tree_attn(h, dev(sh, t.q), *cache.args, ints(ctx), words(t.bits), 2, 3, 0, out, None, ws, size)
        assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    ok(h)
    M.mla_destroy(h)


def test_unmapped_page_is_flagged():
    sh = shape(LITE)
    t = Tree(sh, (200, 100), 3, 4, 64)
    h = handle(sh, 64)
    cache = Cache(sh, t.rows, t.slots, 64, t.rng)
    out = torch.zeros(2, 3, 16, 512, dtype=torch.bfloat16, device="cuda")
    size = M.mla_tree_workspace_size(h, 2, 3)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for bad in (-1, cache.len):
        table = cache.table.clone()
        table[0, 1] = bad
        M.mla_tree_attn(h, dev(sh, t.q), cache.data, cache.len, table, cache.max_blk, ints(t.ctx), words(t.bits), 2,
                        3, 0, out, None, ws, size)
        assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    M.mla_destroy(h)


def test_empty_capacity_gives_zero_rows():
    sh = shape(LITE)
    h = handle(sh, 64)
    out = torch.full((1, 2, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 2, 16), 7.0, device="cuda")
    q = torch.ones(1, 2, 16, 576, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    size = M.mla_tree_workspace_size(h, 1, 2)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    M.mla_tree_attn(h, q, pool, 1, ints([[0]]), 1, ints([0]), words([[0, 0]]), 1, 2, 0, out, lse, ws, size)
    ok(h)
    assert (out == 0).all() and torch.isneginf(lse).all()
    M.mla_destroy(h)


def test_scaled_rope_temperature_is_applied():
    sh = shape(LITE)
    t = Tree(sh, (90,), 3, 6)
    h = handle(sh)
    M.mla_set_rope_scaling(h, 40.0, 4096, 1.0, 32.0, 0.0707)
    got = t.run(h=h)
    M.mla_destroy(h)
    t.check(got, O.softmax_scale(sh["d_h"], sh["d_r"]) * (0.0707 * np.log(40.0) + 1.0) ** 2)


def test_late_dominant_token_and_large_scores():
    """The running maximum rises by far more than the rescale threshold."""
    sh = shape(LITE)
    t = Tree(sh, (700, 40), 8, 2, 64)
    t.q = stored(sh, t.q * 6)
    t.rows[0][600] *= 8
    t.rows[1][45] *= 8
    t.rows = [stored(sh, r) for r in t.rows]
    t.check(t.run())
    t.check(t.run(3))


def test_guard_bands_second_stream_graph_and_repeat():
    """Nothing is written outside the outputs and the workspace; the call is
    the same on another stream and when captured and replayed on new inputs."""
    sh, T = shape(LITE), 9
    t, u = Tree(sh, (300, 64, 1000), T, 1), Tree(sh, (299, 0, 1000), T, 2, slots=1000 + T + 3)
    want, want2 = t.run(), u.run()
    h = handle(sh)
    size = M.mla_tree_workspace_size(h, 3, T)
    raw = [torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
           for n in (3 * T * 16 * 512 * 2, 3 * T * 16 * 4, size)]
    out = raw[0][4096:-4096].view(torch.bfloat16).view(3, T, 16, 512)
    lse = raw[1][4096:-4096].view(torch.float32).view(3, T, 16)
    ws = raw[2][4096:-4096]
    cache = Cache(sh, t.rows, t.slots, 0, t.rng)
    q, ctx, mask = dev(sh, t.q), ints(t.ctx), words(t.bits)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def call(st):
        M.mla_tree_attn(h, q, *cache.args, ctx, mask, 3, T, 0, out, lse, ws, size, st)

    call(s)
    s.synchronize()
    assert np.array_equal(host(out), want[0]) and np.array_equal(host(lse), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(torch.cuda.current_stream())
    q.copy_(dev(sh, u.q))
    cache.data.copy_(Cache(sh, u.rows, u.slots, 0, u.rng).data)
    ctx.copy_(ints(u.ctx))
    mask.copy_(words(u.bits))
    for _ in range(2):
        out.fill_(0)
        g.replay()
    ok(h)
    assert np.array_equal(host(out), want2[0]) and np.array_equal(host(lse), want2[1])
    for r in raw:
        assert (r[:4096] == 0x5A).all() and (r[-4096:] == 0x5A).all()
    M.mla_destroy(h)


def test_strict_mode_refuses_what_the_tensor_cores_cannot_take():
    sh = shape(LITE)
    t = Tree(sh, (70,), 2, 1)
    h = handle(sh, strict=True)
    cache = Cache(sh, t.rows, t.slots, 0, t.rng)
    size = M.mla_tree_workspace_size(h, 1, 2)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    raw = torch.zeros(2 * 16 * 576 + 1, dtype=torch.bfloat16, device="cuda")
    q = raw[1:].view(1, 2, 16, 576)
    q.copy_(dev(sh, t.q))
    out = torch.zeros(1, 2, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 2, 16, device="cuda")
    args = (h, q, *cache.args, ints(t.ctx), words(t.bits), 1, 2, 0, out, lse, ws, size)
    with pytest.raises(M.MlaError) as e:
        M.mla_tree_attn(*args)
    assert e.value.status == M.MLA_ERR_UNSUPPORTED
    M.mla_set_strict(h, 0)
    M.mla_tree_attn(*args)
    ok(h)
    t.check((host(out), host(lse)))
    M.mla_destroy(h)


def test_refusals():
    sh = shape(LITE)
    h = handle(sh)
    x = torch.zeros(256 * 64, device="cuda")
    i = ints([0])
    big = torch.empty(M.mla_tree_workspace_size(h, 1, 1), dtype=torch.uint8, device="cuda")

    def status(fn, *a):
        try:
            fn(*a)
        except M.MlaError as e:
            return e.status
        return M.MLA_OK

    good = [h, x, x, 1, None, 0, i, x, 1, 1, 0, x, None, big, big.numel()]
    for at, bad in ((1, None), (2, None), (6, None), (7, None), (11, None), (8, -1), (9, 65), (9, -1), (10, -1),
                    (3, -1), (4, i)):
        a = list(good)
        a[at] = bad
        assert status(M.mla_tree_attn, *a) == M.MLA_ERR_INVALID_ARG, at
    for at, bad in ((13, None), (13, big[1:]), (14, big.numel() - 1)):
        a = list(good)
        a[at] = bad
        assert status(M.mla_tree_attn, *a) == M.MLA_ERR_WORKSPACE, at
    for at, none in ((8, 0), (9, 0)):      # nothing to do
        a = [h, None, None, 1, None, 0, None, None, 1, 1, 0, None, None, None, 0]
        a[at] = none
        assert status(M.mla_tree_attn, *a) == M.MLA_OK
    assert status(M.mla_tree_workspace_size, h, 1, 65) == M.MLA_ERR_INVALID_ARG
    assert status(M.mla_tree_workspace_size, h, 1 << 30, 64) == M.MLA_ERR_UNSUPPORTED
    acc = [h, x, 1, None, 0, i, i, i, 1, 1, None]
    for at, bad in ((1, None), (5, None), (6, None), (7, None), (8, -1), (9, 65), (2, -1), (3, i)):
        a = list(acc)
        a[at] = bad
        assert status(M.mla_tree_accept, *a) == M.MLA_ERR_INVALID_ARG, at
    app = [h, x, 1, 1, i, i, x, x, x, 1]
    for at, bad in ((1, None), (5, None), (4, None), (3, 65), (2, -1)):
        a = list(app)
        a[at] = bad
        assert status(M.mla_cache_append_tree, *a) == M.MLA_ERR_INVALID_ARG, at
    ok(h)
    M.mla_destroy(h)


# ------------------------------------------------------------------- cache


@pytest.mark.parametrize("sh,page", [(shape(LITE), 0), (shape(LITE), 64), (shape(V2), 64), (shape(TINY), 0),
                                     (shape(TINY), 16), (shape(ODD), 0)])
@pytest.mark.parametrize("T", [1, 7, 64])
def test_append_at_tree_positions(sh, page, T):
    rng = np.random.default_rng(T)
    ctx = (0, 63, 5000)
    D, d = sh["d_c"] + sh["d_r"], sh["d_model"]
    parents = [random_parents(rng, T) for _ in ctx]
    depth = [O.tree_depths(p) for p in parents]
    x = stored(sh, rng.standard_normal((3, T, d)))
    w = stored(sh, rng.standard_normal((D, d)) * d ** -0.5)
    h = handle(sh, page)
    cache = Cache(sh, [np.zeros((0, D))] * 3, 5000 + T + 2, page, rng)
    M.mla_cache_append_tree(h, dev(sh, x), 3, T, ints(ctx), ints(depth), dev(sh, w[:sh["d_c"]]), dev(sh, w[sh["d_c"]:]),
                            *cache.args)
    ok(h)
    M.mla_destroy(h)
    for b, n in enumerate(ctx):
        rows = cache.rows(b, n + T + 2)
        assert np.isnan(rows[:n]).all() and np.isnan(rows[n + T:]).all()
        want = O.cache_rows(x[b], w[:sh["d_c"]], w[sh["d_c"]:], n + np.array(depth[b]), 10000.0)
        # sums of d products in float32, two of them in a rotated value (with
        # the angle's error, 2^-20 of the pair), and one rounding
        mass = np.abs(x[b]).astype(np.float64) @ np.abs(w).astype(np.float64).T
        mass[:, sh["d_c"]:] = np.repeat(mass[:, sh["d_c"]::2] + mass[:, sh["d_c"] + 1::2], 2, 1)
        half = 2.0 ** -8 if sh["dtype"] == "bf16" else 2.0 ** -24
        within(rows[n:n + T], want, (d + 4) * 2.0 ** -24 * mass + 2.0 ** -20 * np.abs(want).max() + half * 1.01 * np.abs(want),
               f"rows of sequence {b}")


@pytest.mark.parametrize("sh,page", [(shape(LITE), 0), (shape(LITE), 64), (shape(TINY), 16), (shape(ODD), 0),
                                     (shape(ODD), 48)])
@pytest.mark.parametrize("T", [1, 9, 64])
def test_accept_moves_the_path(sh, page, T):
    rng = np.random.default_rng(T)
    ctx = [0, 1, 63, 130, 64, 7]
    D = sh["d_c"] + sh["d_r"]
    rows = [stored(sh, rng.standard_normal((n + T, D))) for n in ctx]
    paths = [sorted(rng.choice(T, int(rng.integers(0, T + 1)), replace=False).tolist()) for _ in ctx]
    paths[1] = list(range(T))
    paths[2] = []
    paths[3] = [T - 1]
    path = np.full((len(ctx), T), 1 << 30)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    h = handle(sh, page)
    cache = Cache(sh, rows, max(ctx) + T, page, rng)
    lens = ints(ctx)
    new = ints([-5] * len(ctx))
    before = cache.data.clone()
    M.mla_tree_accept(h, *cache.args, lens, ints(path), ints([len(p) for p in paths]), len(ctx), T, new)
    ok(h)
    assert new.tolist() == [n + len(p) for n, p in zip(ctx, paths)] and lens.tolist() == ctx
    for b, n in enumerate(ctx):
        assert np.array_equal(cache.rows(b, n + T), O.tree_accept(rows[b], n, paths[b]))
    # without new_len, and with new_len written over ctx_len
    cache.data.copy_(before)
    M.mla_tree_accept(h, *cache.args, lens, ints(path), ints([len(p) for p in paths]), len(ctx), T, lens)
    ok(h)
    assert lens.tolist() == new.tolist()
    M.mla_destroy(h)


def test_accept_leaves_a_sequence_with_a_wrong_path():
    sh, T = shape(LITE), 4
    rng = np.random.default_rng(0)
    ctx = [10] * 7
    rows = [stored(sh, rng.standard_normal((14, 576))) for _ in ctx]
    path = [[1, 3, 0, 0], [3, 1, 0, 0], [2, 2, 0, 0], [-1, 0, 0, 0], [4, 0, 0, 0], [0, 0, 0, 0], [1, 2, 3, 0]]
    n_path = [2, 2, 2, 2, 1, 5, -1]
    h = handle(sh)
    cache = Cache(sh, rows, 14, 0, rng)
    new = ints([0] * 7)
    M.mla_tree_accept(h, *cache.args, ints(ctx), ints(path), ints(n_path), 7, T, new)
    assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS
    assert new.tolist() == [12] + [10] * 6
    for b in range(7):
        want = O.tree_accept(rows[b], 10, [1, 3]) if b == 0 else rows[b]
        assert np.array_equal(cache.rows(b, 14), want)
    # a path that ends outside the cache
    M.mla_tree_accept(h, *cache.args, ints([12] * 7), ints([[0, 2, 0, 0]] * 7), ints([2] * 7), 7, T, new)
    assert M.mla_get_device_status(h) == M.MLA_ERR_DEVICE_BOUNDS and new.tolist() == [12] * 7
    M.mla_destroy(h)


@pytest.mark.parametrize("ctx", [(0, 70), (300, 64)])
@pytest.mark.parametrize("sh", [shape(LITE), shape(TINY)])
def test_scores_that_overflow_to_minus_infinity(sh, ctx):
    """A token whose score overflows to -inf draws nothing, the first one too."""
    t = Tree(sh, ctx, 4, 9)
    t.q[..., -1] = stored(sh, np.array([1e20]))
    for r in t.rows:
        r[:, -1] = 0
    given = [r.copy() for r in t.rows]
    for r in given:
        r[0, -1] = stored(sh, np.array([-1e20]))       # q . row = -1e40
    got = t.run(rows=given)
    scale = O.softmax_scale(sh["d_h"], sh["d_r"])
    for b, n in enumerate(ctx):
        r = t.rows[b].astype(np.float64)
        for k in range(t.T):
            mine = np.concatenate([r[:n], r[n:][[j for j in range(t.T) if t.bits[b][k] >> j & 1]]])
            mine = mine[1:] if n or t.bits[b][k] & 1 else mine
            q = t.q[b, k].astype(np.float64)
            if len(mine) == 0:
                assert (got[0][b, k] == 0).all() and np.isneginf(got[1][b, k]).all()
                continue
            want, lse = O.latent_attention(q, mine, d_c=sh["d_c"], scale=scale)
            bo, bl = attention_bounds(sh, q, mine, scale, want, lse)
            within(got[0][b, k], want, bo, f"ctx_lat of sequence {b}, token {k}")
            within(got[1][b, k], lse, bl, f"lse of sequence {b}, token {k}")


@pytest.mark.parametrize("ctx,T,parts", [((12000,), 3, 0), ((9600, 9500), 64, 600), ((2600,), 5, 45)])
def test_rows_cut_into_more_pieces_than_a_warp_has_lanes(ctx, T, parts):
    sh = shape(LITE) if ctx != (2600,) else shape(TINY)
    t = Tree(sh, ctx, T, 4)
    t.check(t.run(parts))


@pytest.mark.parametrize("n,fits", [(3, True), (4, False)])
def test_accept_at_the_largest_length(n, fits):
    """A table may address 2^31 tokens and more (here one page, again and again);
    a length that an integer cannot hold is flagged and the sequence left."""
    sh = shape((1, 8, 2, 2, 64, "fp32"))
    h, T, ctx = handle(sh, 64), 4, 2 ** 31 - 4
    blocks = 2 ** 25 + 1
    table = torch.zeros(1, blocks, dtype=torch.int32, device="cuda")
    pool = torch.arange(64 * 4, dtype=torch.float32, device="cuda").reshape(1, 64, 4)
    before, new = pool.clone(), ints([0])
    M.mla_tree_accept(h, pool, 1, table, blocks, ints([ctx]), ints([[0, 1, 2, 3]]), ints([n]), 1, T, new)
    assert M.mla_get_device_status(h) == (M.MLA_OK if fits else M.MLA_ERR_DEVICE_BOUNDS)
    assert new.tolist() == [ctx + n if fits else ctx]
    assert torch.equal(pool, before)
    M.mla_destroy(h)


@pytest.mark.parametrize("page", [0, 16])
def test_an_odd_latent_width(page):
    sh = shape((3, 24, 41, 6, 128, "bf16"))
    t = Tree(sh, (0, 1, 64, 130, 65), 6, 5, page)
    t.check(t.run())
    h = handle(sh, page)
    cache = Cache(sh, t.rows, t.slots, page, t.rng)
    new = ints([0] * 5)
    M.mla_tree_accept(h, *cache.args, ints(t.ctx), ints([[1, 2, 5, 0, 0, 0]] * 5), ints([3] * 5), 5, 6, new)
    ok(h)
    M.mla_destroy(h)
    for b, n in enumerate(t.ctx):
        assert new[b].item() == n + 3 and np.array_equal(cache.rows(b, n + 6), O.tree_accept(t.rows[b], n, [1, 2, 5]))
