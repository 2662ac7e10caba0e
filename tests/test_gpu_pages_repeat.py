"""The decode over chosen pages gives the same bits in every call: hundreds of short requests (an item ends every tile
or two), long lists, and scores whose maxima keep moving the references."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
from tests import serving_data as D
from tests import test_gpu_pages as pg

pytestmark = pytest.mark.gpu
REPEATS = 1000


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("H,lens,budget,std", [(128, [1 + (37 * b) % 400 for b in range(300)], 6, 0.6), (16, [5000] * 10, 64, 0.6),
                                               (80, [3000 + 7 * b for b in range(20)], 40, 20.0)])
def test_calls_repeat_bit_for_bit(kind, H, lens, budget, std):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    rng = np.random.default_rng(H)
    c = D.Cache(rng, kind, D.dims("v2", H), lens)
    q_lat, pages = pg.draw_query(rng, c, 1, std), pg.i32(pg.lists(rng, c, 1, budget, "own"))
    cfg, B = c.config(), len(lens)
    q, pool, table, n = D.dev(q_lat, "bf16"), c.device(), pg.i32(c.table), pg.i32(lens)
    ws = torch.zeros(M.mla_decode_pages_workspace_size(cfg, B, 1, budget), dtype=torch.uint8, device="cuda")

    def call():
        o = torch.empty(B, 1, H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, 1, H, device="cuda")
        M.mla_decode_pages(cfg, q, pool, table, n, pages, o, lse, ws)
        return o.view(torch.int16), lse
    first = call()
    assert M.mla_read_device_status(ws) == M.MLA_OK
    assert torch.isfinite(first[1]).all()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(REPEATS):
        again = call()
        differ += (again[0] != first[0]).any() | (again[1] != first[1]).any()
    assert int(differ) == 0 and M.mla_read_device_status(ws) == M.MLA_OK
