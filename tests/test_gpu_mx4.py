"""4-bit weights: codes, scales and values bit for bit, products against fp64 references."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import workloads as W
from oracle import pages as ref
from tests import serving_data as D

pytestmark = pytest.mark.gpu
assert_within = D.assert_within


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


def config(act):
    return M.make_config(W.V2, act, act)


def arrays(act, K, N):
    c, s = M.mla_mx4_bytes(config(act), K, N)
    return (torch.full((c,), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((s,), 0x5A, dtype=torch.uint8, device="cuda"))


def quantize(x, act, shift=0):
    K, N = x.shape
    codes, scales = arrays(act, K, N)
    w = D.dev(x, act)
    M.mla_mx4_quantize(config(act), D.shifted(w, shift) if shift else w, codes, scales)
    back = torch.full((K, N), 7.0, dtype=D.torch_type(act), device="cuda")
    back = D.shifted(back, shift) if shift else back
    M.mla_mx4_dequantize(config(act), codes, scales, back)
    torch.cuda.synchronize()
    return codes, scales, back


SHAPES = [(32, 1), (64, 3), (96, 130), (128, 128), (256, 64), (288, 257), (1024, 33), (2080, 70)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_quantize(act, K, N, shift):
    rng = np.random.default_rng(K + N)
    x = D.draw(rng, (K, N), act) * np.exp2(rng.integers(-20, 20, (K // 32, 1, N)).repeat(32, 1).reshape(K, N)).astype(np.float32)
    x[rng.random((K, N)) < 0.1] = 0.0
    x[:32, 0] = 0.0                                # a block of zeros
    near = np.repeat(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32), 4)   # half-way values
    x[-32:, N - 1] = near * np.where(np.arange(32) % 2, -1, 1)
    codes, scales, back = quantize(x, act, shift)
    code, e = ref.mx4_quantize(x)
    want_codes, want_scales = ref.mx4_pack(code, e)
    assert np.array_equal(scales.cpu().numpy(), want_scales.reshape(-1))
    assert np.array_equal(codes.cpu().numpy(), want_codes.reshape(-1))
    assert np.array_equal(back.double().cpu().numpy(), ref.mx4_values(code, e))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_quantize_at_the_ends_of_the_range(act):
    """The largest and smallest magnitudes, infinities and NaN."""
    big = float(torch.finfo(D.torch_type(act)).max)
    tiny = float(torch.finfo(D.torch_type(act)).tiny)
    x = np.zeros((32, 8), np.float32)
    x[:2, 0] = (big, -1.0)
    x[:2, 1] = (tiny, -tiny / 2)
    x[:2, 2] = (np.inf, 1.0)
    x[:2, 3] = (np.nan, 1.0)
    x[:2, 4] = (2.0 ** 127, -(2.0 ** 126))
    x[:2, 5] = (2.0 ** -126 * 6, 2.0 ** -126)
    _, scales, back = quantize(x, act)
    got = back.double().cpu().numpy()
    code, e = ref.mx4_quantize(np.where(np.isfinite(x), x, 0.0))
    want = ref.mx4_values(code, e)
    assert np.array_equal(got[:, [0, 1, 4, 5, 6, 7]], want[:, [0, 1, 4, 5, 6, 7]]) and np.isfinite(want).all()
    assert np.isnan(got[:, 2:4]).all()
    s = scales.cpu().numpy().reshape(1, 1, 32, 4, 4)
    assert s[0, 0, 2, 0, 0] == 255 and s[0, 0, 3, 0, 0] == 255 and (s[0, 0, 8:] == 127).all()


def project(x, codes, scales, act, N, ws_fill=255, shift=()):
    rows, K = x.shape
    cfg = config(act)
    n = M.mla_mx4_project_workspace_size(cfg, K, N, rows)
    ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((rows, N), 7.0, dtype=D.torch_type(act), device="cuda")
    xd = D.dev(x, act)
    xd, out = (D.shifted(xd) if "x" in shift else xd), (D.shifted(out) if "out" in shift else out)
    M.mla_mx4_project(cfg, xd, codes, scales, out, ws)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def draw_weight(rng, K, N):
    """Random codes under exponents of a spread, as device arrays, and their values."""
    code = rng.integers(0, 16, (K, N)).astype(np.uint8)
    e = rng.integers(-9, -3, (K // 32, N))
    packed, scales = ref.mx4_pack(code, e)
    return D.dev(packed), D.dev(scales), ref.mx4_values(code, e)


def check(got, x, w, act):
    K = x.shape[1]
    want, mag = x.astype(np.float64) @ w, np.abs(x).astype(np.float64) @ np.abs(w)
    # fp32 sums of K products; six base-8 digits leave at most 0.5 * 8^-5 * 2^(E - 1) = 2^-17 2^E of an
    # element, E the exponent of its block's largest magnitude
    blocks = np.abs(x).reshape(x.shape[0], K // 32, 32).max(2).astype(np.float64)
    low = 2.0 ** -17 * (blocks @ np.abs(w).reshape(K // 32, 32, -1).sum(1)) if act == "bf16" else 0.0
    assert_within(got, want, D.EPS[act] * np.abs(want) * 1.01 + 2 * K * 2.0 ** -24 * mag + low, "product")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,N", [(1, 32, 1), (3, 96, 130), (1, 128, 128), (2, 128, 5), (5, 256, 257), (17, 1024, 256),
                                      (33, 640, 300), (64, 2176, 129), (65, 384, 1000), (100, 512, 576), (128, 256, 128),
                                      (129, 1536, 70), (200, 384, 260), (300, 128, 129), (513, 256, 140)])
def test_project(act, rows, K, N):
    rng = np.random.default_rng(rows + K)
    codes, scales, w = draw_weight(rng, K, N)
    x = D.draw(rng, (rows, K), act)
    x[0, : K // 2] *= 2.0 ** -12                   # elements far below their block's largest
    x[0, :K:7] = 0.0
    got = project(x, codes, scales, act, N)
    check(got, x, w, act)
    assert np.array_equal(got, project(x, codes, scales, act, N, ws_fill=0))     # the same bits every time


@pytest.mark.parametrize("rows,K,N", [(1, 5120, 576), (32, 16384, 640), (40, 5120, 8192), (150, 16384, 384), (512, 4096, 640)])
def test_project_sizes_of_the_layer(rows, K, N):
    rng = np.random.default_rng(rows)
    codes, scales, w = draw_weight(rng, K, N)
    x = D.draw(rng, (rows, K), "bf16", 0.05)
    check(project(x, codes, scales, "bf16", N), x, w, "bf16")


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("shift", [("x",), ("out",), ("x", "out")])
def test_project_off_16_bytes(rows, shift):
    rng = np.random.default_rng(rows)
    codes, scales, w = draw_weight(rng, 256, 192)
    x = D.draw(rng, (rows, 256), "bf16")
    check(project(x, codes, scales, "bf16", 192, shift=shift), x, w, "bf16")


@pytest.mark.parametrize("rows,K,N", [(4, 256, 256), (20, 1024, 160), (9, 96, 70)])
def test_project_of_infinities_and_nan(rows, K, N):
    """A row's infinities and NaN stay in that row; a column of NaN scales in that column."""
    rng = np.random.default_rng(rows)
    codes, scales, w = draw_weight(rng, K, N)
    x = D.draw(rng, (rows, K), "bf16")
    good = project(x, codes, scales, "bf16", N)
    x[1, 5], x[2, 7] = np.nan, np.inf
    s = scales.cpu().numpy()
    s[0, 0, 3, 0, 0] = 255                         # column 3, first block
    got = project(x, codes, D.dev(s), "bf16", N)
    assert np.isnan(got[1]).all() and not np.isfinite(got[2]).any() and np.isnan(got[:, 3]).all()
    rest = [r for r in range(rows) if r not in (1, 2)]
    cols = [n for n in range(N) if n != 3]
    assert np.array_equal(got[np.ix_(rest, cols)], good[np.ix_(rest, cols)])


def test_project_of_extreme_magnitudes():
    """Rows of very large and very small elements keep their relative precision."""
    rng = np.random.default_rng(8)
    codes, scales, w = draw_weight(rng, 256, 130)
    for s in (2.0 ** 90, 2.0 ** -90):
        x = (D.draw(rng, (3, 256), "bf16").astype(np.float64) * s).astype(np.float32)
        check(project(x, codes, scales, "bf16", 130), x, w, "bf16")
    z = np.zeros((2, 256), np.float32)
    assert (project(z, codes, scales, "bf16", 130) == 0).all()


def test_quantised_output_projection_follows_the_folded_one():
    """W_comb quantised, then the product with the decode's output: the values of the 4-bit weight in
    mla_output_proj give the same result up to rounding."""
    rng = np.random.default_rng(12)
    d = D.dims("v2", 4)
    d.d_model = 264
    K, N, rows = 4 * 512, 264, 9
    cfg = M.make_config(d, "bf16", "bf16")
    w = D.draw(rng, (K, N), "bf16", K ** -0.5)
    codes, scales = arrays("bf16", K, N)
    W_dev = D.dev(w, "bf16")
    M.mla_mx4_quantize(cfg, W_dev, codes, scales)
    M.mla_mx4_dequantize(cfg, codes, scales, W_dev)
    x = D.draw(rng, (rows, K), "bf16")
    ws = torch.zeros(M.mla_output_proj_workspace_size(cfg, rows), dtype=torch.uint8, device="cuda")
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    M.mla_output_proj(cfg, D.dev(x, "bf16"), W_dev, out, ws)
    torch.cuda.synchronize()
    code, e = ref.mx4_quantize(w)
    check(project(x, codes, scales, "bf16", N), x, ref.mx4_values(code, e), "bf16")
    check(out.double().cpu().numpy(), x, ref.mx4_values(code, e), "bf16")


def test_project_captured_and_on_another_stream():
    rng = np.random.default_rng(13)
    codes, scales, w = draw_weight(rng, 1024, 300)
    x1, x2 = D.draw(rng, (20, 1024), "bf16"), D.draw(rng, (20, 1024), "bf16")
    cfg = config("bf16")
    x, out = D.dev(x1, "bf16"), torch.zeros(20, 300, dtype=torch.bfloat16, device="cuda")
    n = M.mla_mx4_project_workspace_size(cfg, 1024, 300, 20)
    ws = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        M.mla_mx4_project(cfg, x, codes, scales, out, ws)
    s.synchronize()
    check(out.double().cpu().numpy(), x1, w, "bf16")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        M.mla_mx4_project(cfg, x, codes, scales, out, ws)
    for v in (x2, x1):
        x.copy_(D.dev(v, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        check(out.double().cpu().numpy(), v, w, "bf16")
