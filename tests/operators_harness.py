"""Caches, queries and bounds for the tests of tree attention and of attention
over selected blocks.  Rows are drawn directly; every slot that a call must
not depend on holds NaN."""

import numpy as np
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from workloads import bf16_bits, bf16_round

# (n_h, d_h, d_c, d_r, d_model, dtype)
V2 = (128, 128, 512, 64, 5120, "bf16")
LITE = (16, 128, 512, 64, 2048, "bf16")
TINY = (4, 32, 128, 16, 256, "fp32")
ODD = (3, 24, 40, 6, 128, "bf16")        # CUDA cores, rows of 92 bytes


def shape(base, **kw):
    names = ("n_h", "d_h", "d_c", "d_r", "d_model", "dtype")
    return {**dict(zip(names, base)), **kw}


def torch_type(sh):
    return torch.bfloat16 if sh["dtype"] == "bf16" else torch.float32


def stored(sh, x):
    """x as the type holds it, float32."""
    x = np.asarray(x, np.float32)
    return bf16_round(x) if sh["dtype"] == "bf16" else x


def dev(sh, x):
    x = np.ascontiguousarray(x, np.float32)
    if sh["dtype"] == "bf16":
        return torch.from_numpy(bf16_bits(x).view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(x).cuda()


def ints(x):
    return torch.tensor(np.asarray(x, np.int64).astype(np.int32), dtype=torch.int32, device="cuda")


def words(bits):
    """Masks (Python integers, [B][T]) as the device's 64-bit words."""
    return torch.from_numpy(np.array(bits, dtype=np.uint64).view(np.int64)).cuda()


def handle(sh, page=0, strict=None):
    h = M.mla_create(M.mla_config(n_h=sh["n_h"], d_h=sh["d_h"], d_c=sh["d_c"], d_r=sh["d_r"], d_model=sh["d_model"],
                                  page_size=page, rope_base=10000.0,
                                  dtype=M.MLA_BF16 if sh["dtype"] == "bf16" else M.MLA_FP32))
    M.mla_set_strict(h, sh["dtype"] == "bf16" and sh["d_c"] == 512 if strict is None else strict)
    return h


class Cache:
    """Rows of sequences (list of [n, D] arrays) in a contiguous or paged cache
    with NaN in every other slot; `slots` token slots per sequence."""

    def __init__(self, sh, rows, slots, page, rng, extra=2):
        D = sh["d_c"] + sh["d_r"]
        self.B, self.page, self.D, self.sh = len(rows), page, D, sh
        if page:
            self.max_blk = -(-slots // page)
            pool = self.B * self.max_blk + extra
            host = np.full((pool, page, D), np.nan, np.float32)
            self.table_np = rng.permutation(pool)[: self.B * self.max_blk].reshape(self.B, self.max_blk)
            for b, r in enumerate(rows):
                for p in range(len(r)):
                    host[self.table_np[b, p // page], p % page] = r[p]
            self.len, self.table = pool, ints(self.table_np)
        else:
            host = np.full((self.B, slots, D), np.nan, np.float32)
            for b, r in enumerate(rows):
                host[b, : len(r)] = r
            self.len, self.max_blk, self.table = slots, 0, None
        self.data = dev(sh, host)

    def rows(self, b, n):
        host = self.data.float().cpu().numpy()
        if not self.page:
            return host[b, :n]
        return np.stack([host[self.table_np[b, p // self.page], p % self.page] for p in range(n)]).reshape(n, self.D)

    @property
    def args(self):
        return self.data, self.len, self.table, self.max_blk


def score_error(q, k, scale):
    """Bound on a score's error [rows, tokens]: a product of D terms summed in
    float32 in any order is off by at most D half steps (2^-24) of the sum of
    the terms' magnitudes; two more for the scale and the change of base."""
    D = q.shape[-1]
    return (D + 2) * 2.0 ** -24 * (np.abs(q) @ np.abs(k).T) * scale


def attention_bounds(sh, q, rows, scale, out, lse):
    """Bounds on ctx_lat [h, d_c] and lse [h] of one query token's attention.
    Scores are off by e (score_error), so weights by 2 e relative (weight and
    sum); the exponential and the float32 sums of n weights add n + 16 steps
    of 2^-23 (a generous count: sums, merge of splits, reciprocal).  The
    tensor cores take the weights in bf16, half a step of 2^-8 each, and the
    result is rounded once to its type."""
    half = 2.0 ** -8 if sh["dtype"] == "bf16" else 2.0 ** -24
    if len(rows) == 0:
        return np.zeros_like(out), np.zeros_like(lse)
    e = score_error(q, rows, scale).max(axis=1)
    x = q @ rows.T * scale
    p = np.exp(x - lse[:, None])
    mass = p @ np.abs(rows[:, : sh["d_c"]])
    rel = 2 * e + (len(rows) + 16) * 2.0 ** -23
    bound = (rel[:, None] + (half if sh["dtype"] == "bf16" else 0.0)) * mass * 1.01 + half * np.abs(out) * 1.01
    return bound, e + (len(rows) + 16) * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse)


def within(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), f"{what}: infinities differ"
    over = np.abs(got[fin] - want[fin]) - np.broadcast_to(bound, want.shape)[fin]
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over its bound"


def random_parents(rng, T):
    return [int(rng.integers(-1, t)) if t else -1 for t in range(T)]


def host(t):
    return t.detach().double().cpu().numpy()


def ok(h):
    st = M.mla_get_device_status(h)
    assert st == M.MLA_OK, M.mla_status_string(st)
