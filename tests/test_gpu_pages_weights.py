"""The decode over chosen pages keeps small softmax weights: heavy first tokens in front of long tails, blocks of
latent dims under scales far apart, and the ordinary inputs, all within half a step of a 16-bit weight."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
from oracle import pages as ref
from tests import serving_data as D
from tests import test_gpu_pages as pg

pytestmark = pytest.mark.gpu
P = D.PAGE
KINDS = ["bf16", "fp8_e4m3", "fp8_e4m3_b128"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


class Given:
    """A generator whose normal draws are rows that were made before."""

    def __init__(self, rng, rows):
        self.permutation, self.rows = rng.permutation, list(rows)

    def standard_normal(self, shape):
        x = self.rows.pop(0)
        assert x.shape == tuple(shape)
        return x


def cache_of(rng, kind, H, rows, **kw):
    return D.Cache(Given(rng, rows), kind, D.dims("v2", H), [len(x) for x in rows], **kw)


# log2 units of a score per product q k of a rotary element
UNIT = oracle.softmax_scale(128, 64) * np.log2(np.e)


def rope_query(B, H, sink, spread):
    """Queries of which only two rotary elements count: k[512] is the sink's, k[513] noise. `sink` [H] and
    `spread` in log2 units for keys of 1."""
    q = np.zeros((B, 1, H, 576), np.float32)
    q[..., 512] = np.asarray(sink) / UNIT
    q[..., 513] = spread / UNIT
    return D.W.round_bf16(q)


def check(c, q_lat, pages, got, lse, monkeypatch):
    """The bound of bf16 weights (2^-8 of sum p |c|) without an allowance for each token; an output of zeros has to
    fail it."""
    monkeypatch.setattr(pg, "low_weights", lambda *a: 0.0)
    pg.check_attend(c, q_lat, pages, got, lse)
    with pytest.raises(AssertionError):
        pg.check_attend(c, q_lat, pages, np.zeros_like(got), lse)


def every_page(c):
    n = [-(-x // P) for x in c.lens]
    return np.stack([np.where(np.arange(max(n)) < k, np.arange(max(n)), -1) for k in n])[:, None].astype(np.int32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,n", [(128, 6144), (16, 8192), (80, 4100)])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_a_heavy_first_token_before_a_long_tail(kind, H, n, spread, monkeypatch):
    """A first token with a latent of 0 that is 8 to 17 log2 units (from head to head) above thousands of others,
    whose latents share a mean."""
    rng = np.random.default_rng(H)
    x = rng.standard_normal((n, 576)) * 0.5
    x[:, :512] += 0.5
    x[0, :512] = 0.0
    x[:, 512:] = 0.0
    x[0, 512] = 1.0
    x[:, 513] = rng.standard_normal(n)
    c = cache_of(rng, kind, H, [x, x[:, :].copy()])
    q_lat = rope_query(2, H, np.linspace(8, 17, H), spread)
    pages = every_page(c)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check(c, q_lat, pages, got, lse, monkeypatch)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rising", [False, True])
def test_scores_of_a_wide_spread(kind, rising, monkeypatch):
    """4096 tokens, scores spread by 2 nats; latents of nonzero mean. Rising: 60 log2 units from first to last."""
    rng = np.random.default_rng(5)
    n, H = 4096, 128
    x = rng.standard_normal((n, 576)) * 0.5
    x[:, :512] += 0.3
    x[:, 512:] = 0.0
    x[:, 512] = np.linspace(0, 1, n) if rising else 0.0
    x[:, 513] = rng.standard_normal(n)
    c = cache_of(rng, kind, H, [x])
    q_lat = rope_query(1, H, 60.0, 2.9)
    pages = every_page(c)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check(c, q_lat, pages, got, lse, monkeypatch)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("how", ["rising", "jump", "falling", "far"])
def test_scores_hundreds_of_octaves_apart(kind, how, monkeypatch):
    """Running maxima that leave the range of a scale's 8 bits and of fp32 itself within one item: 500 log2 units
    up over the list, 300 up at once in the middle of a tile, 300 down; and scores of 10^7, which have no fractions.
    Keys of 0, 0.125 .. 1 are exact in every format, and so are the products."""
    rng = np.random.default_rng(9)
    n, H = 3000, 128
    x = rng.standard_normal((n, 576)) * 0.5
    x[:, :512] += 0.3
    x[:, 512:] = 0.0
    at = np.arange(n)
    x[:, 512] = {"rising": at * 8 // n / 8, "jump": at >= 1500, "falling": at < 1501, "far": at * 8 // n / 8}[how]
    c = cache_of(rng, kind, H, [x], scale=2.0 ** -7)
    q_lat = rope_query(1, H, np.linspace(1, 1.2, H) * {"rising": 500.0, "far": 1.0e7}.get(how, 300.0), 0.0)
    pages = every_page(c)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    # the weights are 0 or equal: the outputs are means of the heaviest tokens' latents, whatever the scores' size
    top = c.values[0][:, 512] == c.values[0][:, 512].max()
    want = c.values[0][top][:, :512].mean(0)
    tol = D.EPS["bf16"] * np.abs(want) * 1.01 + 2.0 ** -8 * np.abs(c.values[0][top][:, :512]).mean(0)
    if how == "far":
        # A list's pieces (ranges of tiles of 128 tokens) are weighed by their LSEs, fp32 numbers near 8e6: rounded to a
        # whole log2 unit (0.35 nat) and then to half a nat (0.25), so that two weights are off by up to e^1.2.
        tiles = [(v[m], m.sum()) for k in range(0, n, 128)
                 for v, m in [(c.values[0][k: k + 128, :512], top[k: k + 128])] if m.any()]
        tol = tol + (np.exp(1.2) - 1) * sum(k * np.abs(v.mean(0) - want) for v, k in tiles) / top.sum()
    D.assert_within(got[0, 0], np.broadcast_to(want, (H, 512)), np.broadcast_to(tol, (H, 512)), how)
    z = oracle.softmax_scale(128, 64) * q_lat[0, 0, :, 512].astype(np.float64) * c.values[0][:, 512].max()
    D.assert_within(lse[0, 0], z + np.log(top.sum()), 2.0 ** -20 * np.abs(z) + 1e-3, how)


@pytest.mark.parametrize("scales", [(1, 1 / 64, 1, 1 / 64), (1, 2.0 ** -8, 2.0 ** -10, 2.0 ** -13), (2.0 ** -30, 1, 2.0 ** 40, 1)])
@pytest.mark.parametrize("spread", [0.0, 2.9])
def test_blocks_of_dims_under_scales_far_apart(scales, spread, monkeypatch):
    rng = np.random.default_rng(6)
    n, H = 4096, 128
    x = rng.standard_normal((n, 576)) * 0.5
    x[:, :512] += 0.3
    x[:, :512] *= np.repeat(scales, 128)
    x[:, 512:] = 0.0
    x[:, 513] = rng.standard_normal(n)
    x[0, 512] = 1.0
    c = cache_of(rng, "fp8_e4m3_b128", H, [x])
    q_lat = rope_query(1, H, np.linspace(0, 14, H), spread)
    pages = every_page(c)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check(c, q_lat, pages, got, lse, monkeypatch)


@pytest.mark.parametrize("octaves", [4, 8])
def test_tokens_under_scales_far_apart(octaves, monkeypatch):
    """Block scales that differ from token to token by up to 2^octaves, the heavy token's among the smallest."""
    rng = np.random.default_rng(7)
    n, H = 3000, 64
    x = rng.standard_normal((n, 576)) * 0.5
    x[:, :512] += 0.3
    x[:, :512] *= np.exp2(-octaves * rng.random((n, 1)))
    x[0, :512] = 0.3 * 2.0 ** -octaves
    x[:, 512:] = 0.0
    x[0, 512] = 1.0
    c = cache_of(rng, "fp8_e4m3_b128", H, [x])
    q_lat = rope_query(1, H, np.linspace(0, 12, H), 0.0)
    pages = every_page(c)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check(c, q_lat, pages, got, lse, monkeypatch)


@pytest.mark.parametrize("kind", ["fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("B,n,budget,H", [(1, 6000, 64, 128), (3, 9000, 141, 128), (40, 1500, 24, 128), (7, 4096, 33, 64),
                                          (200, 300, 5, 128), (5, 700, 11, 16)])
def test_ordinary_inputs_within_the_weights_own_rounding(kind, B, n, budget, H, monkeypatch):
    rng = np.random.default_rng(B)
    c = D.Cache(rng, kind, D.dims("v2", H), [n - 27 * (b % 11) for b in range(B)])
    q_lat, pages = pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, budget, "own")
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check(c, q_lat, pages, got, lse, monkeypatch)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("std", [6.0, 0.0])
def test_far_and_equal_scores_within_the_weights_own_rounding(kind, std, monkeypatch):
    rng = np.random.default_rng(7)
    c = D.Cache(rng, kind, D.dims("v2", 128), (2000, 640))
    q_lat = pg.draw_query(rng, c, 1, std)
    pages = pg.lists(rng, c, 1, 32, "random")
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check(c, q_lat, pages, got, lse, monkeypatch)


def test_the_references_of_these_tests():
    """A sink's share as the formula has it (the figures above are what they say)."""
    q = rope_query(1, 2, [10.0, 14.0], 0.0)[0, 0]
    x = np.zeros((2049, 576))
    x[0, 512] = 1.0
    x[1:, :512] = 1.0
    o, lse, _, _ = ref.attend_pages(q, x, range(33), 2049, P, 512, oracle.softmax_scale(128, 64))
    for h, bits in enumerate((10, 14)):
        assert abs(o[h, 0] - 2048 / (2048 + 2.0 ** bits)) < 0.02
