"""Lists of pages that a decode over chosen pages must not take: each sets the guard, wherever its end is, and leaves
the other queries alone."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
from tests import serving_data as D
from tests import test_gpu_pages as pg

pytestmark = pytest.mark.gpu
BAD = [(-1, 0, 1, -1), (-1, -1, -1, 2), (0, -1, 2, -1), (0, -1, 1, 2), (2, -1, -1, 1), (0, 1, -1, 1), (1, 0, -1, -1), (0, 4, -1, -1),
       (-1, 9, -1, -1)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


@pytest.mark.parametrize("kind,shape,H", [("f32", "tiny", 16), ("bf16", "v2", 128), ("fp8_e4m3", "v2", 16),
                                          ("fp8_e4m3_b128", "v2", 64)])
def test_lists_with_an_entry_out_of_place(kind, shape, H):
    rng = np.random.default_rng(1)
    c = D.Cache(rng, kind, D.dims(shape, H), (300, 200, 150), max_pages=8)
    q_lat, pages = pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, 4, "own")
    for bad in BAD:
        p = pages.copy()
        p[1, 0] = bad
        got, lse, st = pg.attend(c, q_lat, p)
        assert st == M.MLA_ERR_DEVICE_GUARD, bad
        pg.check_attend(c, q_lat, pages, got, lse, skip=(1,))
    # a request without tokens has no pages to see: its list is not looked at
    p = pages.copy()
    p[1, 0] = (5, 3, -1, 2)
    got, lse, st = pg.attend(c, q_lat, p, lens=(300, 0, 150))
    assert st == M.MLA_OK and (got[1] == 0).all() and np.isneginf(lse[1]).all()
    pg.check_attend(c, q_lat, pages, got, lse, skip=(1,))


@pytest.mark.parametrize("kind,shape,H", [("f32", "tiny", 16), ("bf16", "v2", 128), ("fp8_e4m3", "v2", 16)])
@pytest.mark.parametrize("bad", [{32: 5}, {9: 5, 10: 6}, {0: -1, 1: -1, 20: 3}, {63: 7}, {0: -1, 1: -1, 41: 0}])
def test_long_lists_with_an_entry_far_behind_their_end(kind, shape, H, bad):
    rng = np.random.default_rng(2)
    c = D.Cache(rng, kind, D.dims(shape, H), (3000, 900, 700))
    q_lat, pages = pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, 64, "short")
    p = pages.copy()
    p[1, 0, 2:] = -1
    p[1, 0, :2] = (0, 1)
    for k, page in bad.items():
        p[1, 0, k] = page
    got, lse, st = pg.attend(c, q_lat, p)
    assert st == M.MLA_ERR_DEVICE_GUARD
    pg.check_attend(c, q_lat, pages, got, lse, skip=(1,))
