"""A wait of the page scores that runs out (a copied chunk is never handed over, under a short limit): none of the
query's scores is written by any CTA of its cluster, the status says so, and other queries have theirs."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
from tests import serving_data as D
from tests import test_gpu_pages as pg

pytestmark = pytest.mark.gpu
P = D.PAGE


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


@pytest.mark.parametrize("pages,H,withhold", [(100, 128, 1), (300, 128, 1), (1024, 128, 5), (600, 48, 9), (4100, 128, 2)])
def test_a_withheld_chunk(pages, H, withhold):
    rng = np.random.default_rng(pages)
    c = pg.Tables(rng, "bf16", D.dims("v2", H), (pages * P, 200, pages * P - 70), pages)
    q_lat, keys = pg.draw_query(rng, c, 1), pg.draw_keys(rng, c)
    good = pg.score(c, q_lat, keys)
    pg.check_scores(c, q_lat, keys, good)
    st = pg.status()
    try:
        M.mla_testing_waits(wait_limit_us=200, withhold=withhold)
        got = pg.score(c, q_lat, keys, st=st)
    finally:
        M.mla_testing_waits()
    assert M.mla_read_device_status(st) == M.MLA_ERR_TIMEOUT
    assert (got[0] == 7.0).all() and np.array_equal(got[1:], good[1:])
    assert np.array_equal(pg.score(c, q_lat, keys, st=st), good) and M.mla_read_device_status(st) == M.MLA_OK
