"""A wait of the 4-bit product that runs out (its first copy is withheld, under a short limit): the status word says
so, and no output is anything but the right value or what was there before."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
from tests import serving_data as D
from tests import test_gpu_mx4 as mx4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


def call(x, codes, scales, N, ws):
    out = torch.full((x.shape[0], N), 7.0, dtype=torch.bfloat16, device="cuda")
    M.mla_mx4_project(mx4.config("bf16"), D.dev(x, "bf16"), codes, scales, out, ws)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), M.mla_read_device_status(ws)


@pytest.mark.parametrize("rows,K,N,withhold", [(4, 8192, 256, 1), (4, 8192, 256, 2), (20, 1024, 20000, 1), (70, 4096, 384, 2),
                                               (300, 2048, 140, 1)])
def test_a_withheld_copy(rows, K, N, withhold):
    rng = np.random.default_rng(rows)
    code = rng.integers(0, 16, (K, N)).astype(np.uint8)
    e = rng.integers(-9, -3, (K // 32, N))
    codes, scales = mx4.arrays("bf16", K, N)
    c = np.ascontiguousarray(code.T)
    codes.copy_(torch.from_numpy((c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1)))
    byte = np.full((-(-N // 128) * 128, -(-K // 128) * 4), 127, np.uint8)
    byte[:N, : K // 32] = (e + 127).T
    byte = byte.reshape(-1, 4, 32, byte.shape[1] // 4, 4).transpose(0, 3, 2, 1, 4)
    scales.copy_(torch.from_numpy(np.ascontiguousarray(byte).reshape(-1)))
    w = mx4.ref.mx4_values(code, e)
    x = D.draw(rng, (rows, K), "bf16")
    n = M.mla_mx4_project_workspace_size(mx4.config("bf16"), K, N, rows)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    good, st = call(x, codes, scales, N, ws)
    assert st == M.MLA_OK
    mx4.check(good, x, w, "bf16")
    try:
        M.mla_testing_waits(wait_limit_us=200, withhold=withhold)
        got, st = call(x, codes, scales, N, ws)
    finally:
        M.mla_testing_waits()
    assert st == M.MLA_ERR_TIMEOUT
    left = got == 7.0
    assert left.any() and np.array_equal(got[~left], good[~left])
    # the next call is whole again, with the same workspace
    again, st = call(x, codes, scales, N, ws)
    assert st == M.MLA_OK and np.array_equal(again, good)


def test_a_product_on_the_simt_kernel_clears_the_word_too():
    rng = np.random.default_rng(1)
    codes, scales, w = mx4.draw_weight(rng, 256, 64)
    x = D.draw(rng, (3, 256), "bf16")
    ws = torch.full((M.mla_mx4_project_workspace_size(mx4.config("bf16"), 256, 64, 3),), 255, dtype=torch.uint8, device="cuda")
    out = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    M.mla_mx4_project(mx4.config("bf16"), D.shifted(D.dev(x, "bf16")), codes, scales, out, ws)
    torch.cuda.synchronize()
    assert M.mla_read_device_status(ws) == M.MLA_OK
    mx4.check(out.double().cpu().numpy(), x, w, "bf16")
