"""Infinities and NaN in live inputs of the page scores, the decode over chosen pages and the 4-bit product: they
show in the results that they belong to, and nowhere else."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
from tests import serving_data as D
from tests import test_gpu_mx4 as mx4
from tests import test_gpu_pages as pg

pytestmark = pytest.mark.gpu
P = D.PAGE
CASES = [("bf16", "v2", 128), ("fp8_e4m3", "v2", 64), ("fp8_e4m3_b128", "v2", 80), ("f32", "tiny", 16), ("bf16", "tiny", 16)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


def put(c, b, j, k, value):
    """Element k of token j of request b: the cached bytes (e4m3 has only NaN)."""
    slot = c.slots(b, j + 1)[j]
    row, dc = c.bytes[slot], c.d.d_latent
    if c.kind == "f32":
        row[4 * k: 4 * k + 4] = np.array([value], np.float32).view(np.uint8)
    elif c.kind == "bf16" or k >= dc and c.kind == "fp8_e4m3_b128":
        at = 2 * k if c.kind == "bf16" else dc + dc // 32 + 2 * (k - dc)
        row[at: at + 2] = D.bf16_bytes(np.array([[value]], np.float32))[0]
    else:
        row[k] = 0x7F
    c.values[b][j, k] = value


# ----------------------------------------------------------------------------- page scores

@pytest.mark.parametrize("kind,shape,H", [("bf16", "v2", 128), ("bf16", "v2", 40), ("f32", "tiny", 16)])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_scores_of_nan_and_infinite_queries_and_keys(kind, shape, H, value):
    rng = np.random.default_rng(1)
    c = pg.Tables(rng, kind, D.dims(shape, H), (300 * P, 200, 140 * P + 3), 300)
    q_lat, keys = pg.draw_query(rng, c, 1), pg.draw_keys(rng, c)
    good = pg.score(c, q_lat, keys)
    bad = q_lat.copy()
    bad[0, 0, 3, 7] = value                        # one head's sum over the pages is NaN: so is every score
    got = pg.score(c, bad, keys)
    assert np.isnan(got[0, 0]).all() and np.array_equal(got[1:], good[1:])
    bad = keys.copy()
    bad[c.table[2, 77], 7] = value
    got = pg.score(c, q_lat, bad)
    assert np.isnan(got[2, 0, :141]).all() and np.array_equal(got[:2], good[:2])


# ----------------------------------------------------------------------------- decode over pages

def inputs(kind, shape, H, lens=(900, 300, 3000)):
    rng = np.random.default_rng(2)
    c = D.Cache(rng, kind, D.dims(shape, H), lens)
    return c, pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, 40, "random")


@pytest.mark.parametrize("kind,shape,H", CASES)
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_query_element(kind, shape, H, value):
    c, q_lat, pages = inputs(kind, shape, H)
    good = pg.attend(c, q_lat, pages)
    pg.check_attend(c, q_lat, pages, *good[:2])
    for b in (0, 2):
        q = q_lat.copy()
        q[b, 0, 5, 9] = value
        got, lse, st = pg.attend(c, q, pages)
        assert st == M.MLA_OK
        assert np.isnan(got[b, 0, 5]).all() and not np.isfinite(lse[b, 0, 5])
        others = [i for i in range(3) if i != b]
        assert np.array_equal(got[others], good[0][others]) and np.array_equal(lse[others], good[1][others])
        # the query's other heads (their running maxima may be renewed at other places)
        got[b, 0, 5], lse[b, 0, 5] = good[0][b, 0, 5], good[1][b, 0, 5]
        pg.check_attend(c, q_lat, pages, got, lse)


@pytest.mark.parametrize("kind,shape,H", CASES)
@pytest.mark.parametrize("b,j", [(0, 0), (1, 299), (2, 1500)])
def test_a_nan_in_a_row(kind, shape, H, b, j):
    c, q_lat, pages = inputs(kind, shape, H)
    pages[b, 0, : min(40, -(-c.lens[b] // P))] = np.arange(-(-c.lens[b] // P))[:40]
    good = pg.attend(c, q_lat, pages)
    put(c, b, j, 11, np.nan)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK and np.isnan(got[b]).all() and not np.isfinite(lse[b]).any()
    rest = [i for i in range(3) if i != b]
    assert np.array_equal(got[rest], good[0][rest]) and np.array_equal(lse[rest], good[1][rest])


@pytest.mark.parametrize("kind,shape,H", [x for x in CASES if x[0] != "fp8_e4m3"])
@pytest.mark.parametrize("pages_out", [1, 2, 5])
def test_rotary_keys_of_minus_infinity_weigh_nothing(kind, shape, H, pages_out):
    """The first pages' scores are -infinity for every head (half a tile, a tile, and more): the result is that of
    the other pages."""
    c, q_lat, pages = inputs(kind, shape, H, (900, 3000))
    k = c.d.d_latent + 1
    q_lat[..., k] = 0.5
    for b in range(2):
        pages[b, 0, : min(40, -(-c.lens[b] // P))] = np.arange(-(-c.lens[b] // P))[:40]
        for j in range(pages_out * P):
            put(c, b, j, k, -np.inf)
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    pg.check_attend(c, q_lat, np.where(pages < pages_out, -1, pages), got, lse)


def test_nothing_but_minus_infinity():
    """Scores that are all -infinity: no weight at all, so the result of an empty list or NaN, never a number."""
    for kind, shape, H in (("bf16", "v2", 128), ("fp8_e4m3_b128", "v2", 128), ("f32", "tiny", 16)):
        c, q_lat, pages = inputs(kind, shape, H, (100, 900))
        dc = c.d.d_latent
        q_lat[..., dc + 1] = 1.0
        pages[0, 0, :2] = (0, 1)
        for j in range(100):
            put(c, 0, j, dc + 1, -np.inf)
        got, lse, st = pg.attend(c, q_lat, pages)
        assert st == M.MLA_OK
        assert (np.isnan(got[0]) | (got[0] == 0)).all() and (np.isnan(lse[0]) | np.isneginf(lse[0])).all()
        assert np.isfinite(got[1]).all()


# ----------------------------------------------------------------------------- 4-bit product, many rows

FORM8 = [(70, 256, 256), (41, 1024, 160), (300, 128, 70)]


@pytest.mark.parametrize("rows,K,N", FORM8)
def test_product_of_many_rows_with_infinities_and_nan(rows, K, N):
    rng = np.random.default_rng(rows)
    codes, scales, w = mx4.draw_weight(rng, K, N)
    x = D.draw(rng, (rows, K), "bf16")
    good = mx4.project(x, codes, scales, "bf16", N)
    mx4.check(good, x, w, "bf16")
    x[1, 5], x[2, 7], x[rows - 1, K - 1] = np.nan, np.inf, -np.inf
    s = scales.cpu().numpy()
    s[0, 0, 3, 0, 0] = 255                         # column 3, first block
    got = mx4.project(x, codes, D.dev(s), "bf16", N)
    assert not np.isfinite(got[[1, 2, rows - 1]]).any() and np.isnan(got[:, 3]).all()
    rest = [r for r in range(rows) if r not in (1, 2, rows - 1)]
    cols = [n for n in range(N) if n != 3]
    assert np.array_equal(got[np.ix_(rest, cols)], good[np.ix_(rest, cols)])


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("log2", [90, 120, -90, -100])
def test_product_of_extreme_magnitudes(rows, log2):
    rng = np.random.default_rng(8)
    codes, scales, w = mx4.draw_weight(rng, 256, 130)
    x = (D.draw(rng, (rows, 256), "bf16").astype(np.float64) * 2.0 ** log2).astype(np.float32)
    mx4.check(mx4.project(x, codes, scales, "bf16", 130), x, w, "bf16")


@pytest.mark.parametrize("rows", [3, 70])
def test_product_of_the_smallest_magnitudes(rows):
    """Below 2^-111 the scales of the activations end: elements are off by at most 2^-128 (2^-17 of 2^-111)."""
    rng = np.random.default_rng(9)
    codes, scales, w = mx4.draw_weight(rng, 256, 130)
    for log2 in (-112, -118, -125):
        x = (D.draw(rng, (rows, 256), "bf16").astype(np.float64) * 2.0 ** log2).astype(np.float32)
        x = D.W.round_bf16(x)
        got = mx4.project(x, codes, scales, "bf16", 130)
        want, mag = x.astype(np.float64) @ w, np.abs(x).astype(np.float64) @ np.abs(w)
        # the product's own rounding: bf16 subnormals are 2^-133 apart
        tol = D.EPS["bf16"] * np.abs(want) * 1.01 + 512 * 2.0 ** -24 * mag + 2.0 ** -128 * np.abs(w).sum(0) + 2.0 ** -133
        D.assert_within(got, want, tol, f"product at 2^{log2}")


@pytest.mark.parametrize("rows,K,N", [(70, 256, 256), (129, 384, 130)])
def test_product_of_many_rows_with_codes_off_32_bytes(rows, K, N):
    """Codes at a multiple of 16 but not of 32 bytes (the form of six columns, in several row tiles)."""
    rng = np.random.default_rng(rows)
    codes, scales, w = mx4.draw_weight(rng, K, N)
    x = D.draw(rng, (rows, K), "bf16")
    flat = torch.zeros(codes.numel() + 64, dtype=torch.uint8, device="cuda")
    at = 16 if flat.data_ptr() % 32 == 0 else 0
    view = flat[at: at + codes.numel()].view(codes.shape)
    view.copy_(codes)
    assert view.data_ptr() % 32 == 16
    mx4.check(mx4.project(x, view, scales, "bf16", N), x, w, "bf16")
