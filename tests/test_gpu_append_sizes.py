"""Cache append over every tile and K split it chooses: the token counts where
the choice changes, and their neighbours, against float64 rows."""

import numpy as np
import pytest
import torch

import head_latent_attention_09_b200 as M
from oracle import mla_oracle as O
from tests.operators_harness import LITE, V2, dev, handle, host, ints, ok, shape, stored, torch_type, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from head_latent_attention_09_b200 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("n", [1, 16, 17, 33, 64, 65, 100, 128, 129, 250, 256, 257, 500, 513, 768, 1000, 1025, 2049])
@pytest.mark.parametrize("sh", [shape(LITE), shape(V2), shape(LITE, d_model=256), shape(LITE, d_model=832)])
def test_append_of_many_tokens(sh, n):
    rng = np.random.default_rng(n)
    d, D = sh["d_model"], sh["d_c"] + sh["d_r"]
    x = stored(sh, rng.standard_normal((n, d)))
    w = {k: stored(sh, rng.standard_normal((m, d)) * d ** -0.5) for k, m in (("dkv", sh["d_c"]), ("kr", sh["d_r"]))}
    h = handle(sh)
    cache = torch.full((n + 2, D), float("nan"), dtype=torch_type(sh), device="cuda")
    M.mla_cache_append(h, dev(sh, x), 1, n, ints([1]), dev(sh, w["dkv"]), dev(sh, w["kr"]), cache, n + 2)
    ok(h)
    M.mla_destroy(h)
    got = host(cache)
    assert np.isnan(got[[0, n + 1]]).all()
    want = O.cache_rows(x, w["dkv"], w["kr"], np.arange(1, n + 1), 10000.0)
    # a product of d terms: float32 sums (d steps of 2^-24 of the terms' total),
    # the rotation (angles to 1e-6, pairs of products), one rounding to bf16
    total = np.abs(x.astype(np.float64)) @ np.abs(np.concatenate([w["dkv"], w["kr"]]).astype(np.float64)).T
    total[:, sh["d_c"]:] = np.repeat(total[:, sh["d_c"]::2] + total[:, sh["d_c"] + 1::2], 2, axis=1)
    within(got[1:n + 1], want, (d * 2.0 ** -24 + 4e-6) * total + 2.0 ** -8 * np.abs(want) * 1.01, "rows")


@pytest.mark.parametrize("n", [3000, 4097, 7500])
@pytest.mark.parametrize("sh", [shape(LITE), shape(LITE, d_model=192), shape(LITE, d_model=256)])
def test_append_of_a_long_prompt(sh, n):
    """Tiles of 256 columns, with and without a K split."""
    test_append_of_many_tokens(sh, n)


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("sh", [shape(LITE, d_c=41, d_r=6, d_model=128), shape(LITE, d_c=1, d_r=2, d_model=64),
                                shape((4, 32, 127, 16, 256, "fp32"))])
def test_append_of_an_odd_latent_width(sh, n):
    test_append_of_many_tokens(sh, n)
