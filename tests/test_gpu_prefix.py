"""The shared-prefix calls (expand, attend, joined projection) against fp64 references.

Bounds, from the arithmetic alone. Half a step of bf16 is 2^-8 of the value, of fp32 2^-24. A
sum of n products in fp32 is off by at most n 2^-24 of the sum of their magnitudes (2^-23 where
the tensor cores may truncate); every bound below doubles its small fp32 terms for exp2, log2
and the order of sums.
"""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
import workloads as W
from oracle import serving as ref
from tests import serving_data as D

pytestmark = pytest.mark.gpu
assert_within = D.assert_within


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


# ----------------------------------------------------------------------------- expansion

def expand(cache, cfg, W_UK, W_UV, L, table=None, status=None):
    d, act = cache.d, D.act_of(cache.kind)
    t, H = D.torch_type(act), d.num_heads
    keys = torch.full((H, L, d.d_nope), 7.0, dtype=t, device="cuda")
    values = torch.full((H, L, d.d_v), 7.0, dtype=t, device="cuda")
    k_pe = torch.full((L, d.d_rope), 7.0, dtype=t, device="cuda")
    M.mla_prefix_expand(cfg, D.dev(W_UK, act), D.dev(W_UV, act), cache.device(),
                        D.dev(cache.table[0] if table is None else table), L, keys, values, k_pe,
                        dev_status=status)
    torch.cuda.synchronize()
    return keys, values, k_pe


def expand_bound(mag, x, act, cache_kind, d_c):
    tol = 4 * d_c * 2.0 ** -24 * mag + D.EPS[act] * np.abs(x)
    if cache_kind == "fp8_e4m3_b128":
        tol = tol + 2.0 ** -8 * mag                     # code * scale rounded to bf16
    return tol * 1.01


@pytest.mark.parametrize("cache,shape,H", [("f32", "tiny", 16), ("bf16", "tiny", 16), ("bf16", "v2", 128),
                                           ("bf16", "v2", 16), ("fp8_e4m3", "v2", 32),
                                           ("fp8_e4m3_b128", "v2", 32), ("f32", "odd", 3), ("fp8_e4m3_b128", "odd128", 3)])
@pytest.mark.parametrize("L", [1, 63, 64, 129, 400, 700, 1800])
def test_expand(cache, shape, H, L):
    rng = np.random.default_rng(L)
    d = D.dims(shape, H)
    c = D.Cache(rng, cache, d, [L])
    act = D.act_of(cache)
    W_UK = D.draw(rng, (d.d_latent, H * d.d_nope), act, d.d_latent ** -0.5)
    W_UV = D.draw(rng, (d.d_latent, H * d.d_v), act, d.d_latent ** -0.5)
    keys, values, k_pe = expand(c, c.config(), W_UK, W_UV, L)
    rows = c.values[0]
    K, V, aK, aV = ref.expand_prefix(rows[:, : d.d_latent], W_UK, W_UV, H)
    assert_within(keys.double().cpu().numpy(), K, expand_bound(aK, K, act, cache, d.d_latent), "keys")
    assert_within(values.double().cpu().numpy(), V, expand_bound(aV, V, act, cache, d.d_latent), "values")
    pe = rows[:, d.d_latent:]
    assert_within(k_pe.double().cpu().numpy(), pe, D.EPS[act] * np.abs(pe) * 1.01, "k_pe")


@pytest.mark.parametrize("cache", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
def test_expand_bad_page_gives_zero_rows(cache):
    rng = np.random.default_rng(5)
    d = D.dims("v2", 16)
    c = D.Cache(rng, cache, d, [200])
    W_UK = D.draw(rng, (512, 16 * 128), "bf16", 512 ** -0.5)
    W_UV = D.draw(rng, (512, 16 * 128), "bf16", 512 ** -0.5)
    good = [x.clone() for x in expand(c, c.config(), W_UK, W_UV, 200)]
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        table = c.table[0].copy()
        table[1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = expand(c, c.config(), W_UK, W_UV, 200, table=table, status=status)
        assert M.mla_read_device_status(status) == M.MLA_ERR_DEVICE_GUARD
        keep = np.r_[0:64, 128:200]
        for g, w in zip(got[:2], good[:2]):
            assert torch.equal(g[:, keep], w[:, keep]) and not g[:, 64:128].any()
        assert torch.equal(got[2][keep], good[2][keep]) and not got[2][64:128].any()


# ----------------------------------------------------------------------------- attention

def attend_inputs(rng, d, B, q, L, act, lens):
    H = d.num_heads
    x = dict(q_nope=D.draw(rng, (B, q, H, d.d_nope), act), q_pe=D.draw(rng, (B, q, H, d.d_rope), act),
             keys=D.draw(rng, (H, L, d.d_nope), act), values=D.draw(rng, (H, L, d.d_v), act),
             k_pe=D.draw(rng, (L, d.d_rope), act))
    return x, np.asarray(lens, np.int32)


def attend(cfg, x, lens, act, status=None, stream=None):
    B, q, H, _ = x["q_nope"].shape
    t = {k: D.dev(v, act) for k, v in x.items()}
    u = torch.full((B, q, H, x["values"].shape[2]), float("nan"), dtype=D.torch_type(act), device="cuda")
    lse = torch.full((B, q, H), float("nan"), device="cuda")
    n = M.mla_prefix_attend_workspace_size(cfg, B, q, x["k_pe"].shape[0])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    M.mla_prefix_attend(cfg, t["q_nope"], t["q_pe"], t["keys"], t["values"], t["k_pe"], D.dev(lens), u, lse,
                        ws, dev_status=status, stream=stream)
    torch.cuda.synchronize()
    return u.double().cpu().numpy(), lse.double().cpu().numpy()


def check_attend(d, x, lens, act, u, lse):
    scale = oracle.softmax_scale(d.d_nope, d.d_rope)
    ru, rl, mag_s, mag_v = ref.attend_prefix(x["q_nope"], x["q_pe"], x["keys"], x["values"], x["k_pe"],
                                             lens, scale)
    L, n = x["k_pe"].shape[0], d.d_nope + d.d_rope
    # scores: fp32 products and sums, sine and cosine off by 2^-20 (fp32: 2^-22), and in bf16 the
    # rotated query as two bf16 terms (2^-16)
    ds = mag_s * (4 * n * 2.0 ** -24 + (2.0 ** -16 + 2.0 ** -20 if act == "bf16" else 2.0 ** -21)) + 2.0 ** -21
    dl = 2 * ds + 4 * (L + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(rl), rl, 0))
    assert_within(lse, rl, dl, "lse")
    # weights: relative 2 ds, their rounding for the product with the values, the fp32 sums
    dw = 2 * ds + (D.EPS["bf16"] if act == "bf16" else 0) + 4 * (L + 64) * 2.0 ** -24
    assert_within(u, ru, dw[..., None] * mag_v * 1.05 + D.EPS[act] * np.abs(ru) * 1.01 + 1e-30, "u")


@pytest.mark.parametrize("act,shape,H", [("f32", "tiny", 16), ("bf16", "tiny", 16), ("bf16", "v2", 16),
                                         ("bf16", "v2", 3), ("f32", "odd", 3)])
@pytest.mark.parametrize("B,q,L", [(1, 1, 1), (7, 2, 2), (1, 3, 3), (2, 1, 4), (130, 1, 1), (3, 1, 64), (2, 3, 127), (5, 1, 128), (4, 2, 129), (3, 4, 700),
                                   (128, 1, 257), (65, 2, 300), (43, 6, 200),
                                   (260, 1, 700), (300, 2, 130)])
def test_attend(act, shape, H, B, q, L):
    rng = np.random.default_rng(B * 1000 + L)
    d = D.dims(shape, H)
    lens = rng.integers(q, 5000, B)
    lens[0] = q                                    # every own token is new
    x, lens = attend_inputs(rng, d, B, q, L, act, lens)
    u, lse = attend(M.make_config(d, act, act), x, lens, act)
    check_attend(d, x, lens, act, u, lse)


@pytest.mark.parametrize("L", [5000])
def test_attend_all_heads_and_long_prefix(L):
    rng = np.random.default_rng(11)
    d = D.dims("v2", 128)
    x, lens = attend_inputs(rng, d, 3, 1, L, "bf16", [1, 100000, 77])
    u, lse = attend(M.make_config(d, "bf16", "bf16"), x, lens, "bf16")
    check_attend(d, x, lens, "bf16", u, lse)


@pytest.mark.parametrize("act,shape,H", [("f32", "tiny", 16), ("bf16", "v2", 16)])
@pytest.mark.parametrize("L", [150, 2])
def test_attend_empty_and_bad_lengths(act, shape, H, L):
    rng = np.random.default_rng(3)
    d = D.dims(shape, H)
    x, lens = attend_inputs(rng, d, 6, 2, L, act, [0, 2, 1, 9, 0, -5])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    u, lse = attend(M.make_config(d, act, act), x, lens, act, status=status)
    assert M.mla_read_device_status(status) == M.MLA_ERR_DEVICE_GUARD
    for b in (0, 2, 4, 5):
        assert not u[b].any() and np.isneginf(lse[b]).all()
    check_attend(d, x, np.where(lens < 2, 0, lens), act, u, lse)
    # no prefix at all: every request is empty, and good lengths raise no flag
    x0, _ = attend_inputs(rng, d, 6, 2, 0, act, lens)
    u, lse = attend(M.make_config(d, act, act), x0, np.array([0, 2, 2, 9, 0, 5], np.int32), act, status=status)
    assert not u.any() and np.isneginf(lse).all()
    assert M.mla_read_device_status(status) == M.MLA_OK


@pytest.mark.parametrize("act,shape,H", [("f32", "tiny", 16), ("bf16", "v2", 16)])
def test_attend_growing_and_large_scores(act, shape, H):
    """Scores that grow along the prefix by hundreds: the running maximum moves at every step, and
    earlier sums vanish."""
    rng = np.random.default_rng(8)
    d = D.dims(shape, H)
    x, lens = attend_inputs(rng, d, 4, 1, 700, act, [1, 2, 3, 4])
    unit = np.ones(d.d_nope, np.float32)
    x["q_nope"][:] = unit
    ramp = np.linspace(-8, 24, 700, dtype=np.float32)[None, :, None]
    x["keys"] = (W.round_bf16(ramp * unit) if act == "bf16" else ramp * unit) * np.ones((H, 1, 1), np.float32)
    u, lse = attend(M.make_config(d, act, act), x, lens, act)
    check_attend(d, x, lens, act, u, lse)
    x["keys"] = x["keys"][:, ::-1].copy()          # and falling
    u, lse = attend(M.make_config(d, act, act), x, lens, act)
    check_attend(d, x, lens, act, u, lse)


@pytest.mark.parametrize("act,shape,H,B,L", [("f32", "tiny", 16, 4, 300), ("bf16", "tiny", 16, 4, 300),
                                             ("f32", "tiny", 16, 4, 1), ("bf16", "v2", 16, 4, 3),
                                             ("bf16", "v2", 16, 4, 90), ("bf16", "v2", 16, 4, 2100),
                                             ("bf16", "v2", 16, 140, 2100)])
def test_attend_nan_shows_in_output_and_lse(act, shape, H, B, L):
    """A NaN query makes its own row NaN, a NaN key its head's rows, and nothing else; neither may
    pass for an empty key set (lse -inf), which the joined projection would leave out."""
    rng = np.random.default_rng(B + L)
    d = D.dims(shape, H)
    x, lens = attend_inputs(rng, d, B, 1, L, act, rng.integers(1, 90, B))
    cfg = M.make_config(d, act, act)
    bad = {k: v.copy() for k, v in x.items()}
    bad["q_nope"][2, 0, 0, 5] = np.nan
    bad["q_pe"][3, 0, 1, 1] = np.nan
    bad["keys"][2, L - 1, 0] = np.nan
    u, lse = attend(cfg, bad, lens, act)
    hit = np.zeros((B, 1, H), bool)
    hit[2, 0, 0] = hit[3, 0, 1] = hit[:, 0, 2] = True
    assert np.isnan(u[hit]).all() and np.isnan(lse[hit]).all()
    good_u, good_lse = attend(cfg, x, lens, act)
    assert np.array_equal(u[~hit], good_u[~hit]) and np.array_equal(lse[~hit], good_lse[~hit])


def test_attend_same_bits_every_time_on_two_streams_and_captured():
    rng = np.random.default_rng(21)
    d = D.dims("v2", 16)
    x, lens = attend_inputs(rng, d, 20, 2, 900, "bf16", rng.integers(2, 90, 20))
    cfg = M.make_config(d, "bf16", "bf16")
    t = {k: D.dev(v, "bf16") for k, v in x.items()}
    ln = D.dev(lens)
    n = max(256, M.mla_prefix_attend_workspace_size(cfg, 20, 2, 900))

    def outs():
        return (torch.zeros(20, 2, 16, 128, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(20, 2, 16, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda"))

    def call(o, stream=None):
        M.mla_prefix_attend(cfg, t["q_nope"], t["q_pe"], t["keys"], t["values"], t["k_pe"], ln, o[0], o[1],
                            o[2], stream=stream)
    first = outs()
    call(first)
    torch.cuda.synchronize()
    check_attend(d, x, lens, "bf16", first[0].double().cpu().numpy(), first[1].double().cpu().numpy())
    a, b, s1, s2 = outs(), outs(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        call(a, s1)
        call(b, s2)
    torch.cuda.synchronize()
    g, c = torch.cuda.CUDAGraph(), outs()
    with torch.cuda.graph(g):
        call(c)
    for _ in range(2):
        c[0].zero_()
        g.replay()
    torch.cuda.synchronize()
    for o in (a, b, c):
        assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])


def shifted(t, elements=1):
    """The same values at an address that is no multiple of 16 bytes."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    view = flat[elements: elements + t.numel()].view(t.shape)
    view.copy_(t)
    return view


def test_unaligned_views():
    rng = np.random.default_rng(41)
    d = D.dims("v2", 16)
    x, lens = attend_inputs(rng, d, 5, 1, 130, "bf16", rng.integers(1, 90, 5))
    cfg = M.make_config(d, "bf16", "bf16")
    t = {k: shifted(D.dev(v, "bf16")) for k, v in x.items()}
    u = shifted(torch.zeros(5, 1, 16, 128, dtype=torch.bfloat16, device="cuda"))
    lse = shifted(torch.zeros(5, 1, 16, device="cuda"))
    ws = torch.empty(max(256, M.mla_prefix_attend_workspace_size(cfg, 5, 1, 130)), dtype=torch.uint8, device="cuda")
    M.mla_prefix_attend(cfg, t["q_nope"], t["q_pe"], t["keys"], t["values"], t["k_pe"], D.dev(lens), u, lse, ws)
    torch.cuda.synchronize()
    check_attend(d, x, lens, "bf16", u.double().cpu().numpy(), lse.double().cpu().numpy())
    c = D.Cache(rng, "bf16", d, [130])
    W_UK = D.draw(rng, (512, 16 * 128), "bf16", 512 ** -0.5)
    W_UV = D.draw(rng, (512, 16 * 128), "bf16", 512 ** -0.5)
    want = expand(c, cfg, W_UK, W_UV, 130)
    got = [shifted(torch.zeros_like(y)) for y in want]
    M.mla_prefix_expand(cfg, D.dev(W_UK, "bf16"), D.dev(W_UV, "bf16"), shifted(c.device(), 2), D.dev(c.table[0]), 130,
                        *got)
    torch.cuda.synchronize()
    for g, y in zip(got, want):
        assert (g.double() - y.double()).abs().max() <= 2.0 ** -7 * y.double().abs().max()


# ----------------------------------------------------------------------------- joined projection

@pytest.mark.parametrize("act,shape,H", [("f32", "tiny", 16), ("bf16", "tiny", 16), ("bf16", "v2", 16),
                                         ("bf16", "v2", 128), ("f32", "odd", 5), ("f32", "v2", 5),
                                         ("bf16", "value64", 5), ("bf16", "value128", 5)])
@pytest.mark.parametrize("rows", [1, 33, 130, 300])
def test_output_proj_prefix(act, shape, H, rows):
    rng = np.random.default_rng(rows)
    d = D.dims(shape, H)
    o_lat = D.draw(rng, (rows, H, d.d_latent), act, 0.1)
    up = D.draw(rng, (rows, H, d.d_v), act, 0.1)
    lse = rng.standard_normal((rows, H)).astype(np.float32) * 3 + 6
    lsep = rng.standard_normal((rows, H)).astype(np.float32) * 3 + 6
    # no own tokens, no prefix, neither, and far apart
    lse[0, 0], lsep[0, 1] = -np.inf, -np.inf
    lse[0, 2] = lsep[0, 2] = -np.inf
    lse[0, 3], lsep[0, 4] = 300.0, 300.0
    o_lat[0, 0], up[0, 1] = np.nan, np.nan             # parts of weight 0 may hold anything
    W_UV = D.draw(rng, (d.d_latent, H * d.d_v), act, d.d_latent ** -0.5)
    W_O = D.draw(rng, (H * d.d_v, d.d_model), act, (H * d.d_v) ** -0.5)
    cfg = M.make_config(d, act, act)
    out = torch.full((rows, d.d_model), float("nan"), dtype=D.torch_type(act), device="cuda")
    ws = torch.full((M.mla_output_proj_prefix_workspace_size(cfg, rows),), 0xFF, dtype=torch.uint8, device="cuda")
    M.mla_output_proj_prefix(cfg, D.dev(o_lat, act), D.dev(lse), D.dev(up, act), D.dev(lsep),
                             D.dev(W_UV, act), D.dev(W_O, act), out, ws)
    torch.cuda.synchronize()
    o0, u0 = o_lat.copy(), up.copy()
    o0[0, 0], u0[0, 1] = 0, 0
    u = ref.join_prefix(o0, lse.astype(np.float64), u0.astype(np.float64), lsep.astype(np.float64), W_UV, H)
    mag_u = ref.join_prefix(np.abs(o0), lse.astype(np.float64), np.abs(u0).astype(np.float64),
                            lsep.astype(np.float64), np.abs(W_UV), H)
    want = u.reshape(rows, -1) @ W_O.astype(np.float64)
    mag = np.abs(u).reshape(rows, -1) @ np.abs(W_O).astype(np.float64)
    # u's rounding, its fp32 sums (weights to 2^-20), the projection's sums, the result's rounding
    du = D.EPS[act] * np.abs(u) + (4 * d.d_latent * 2.0 ** -24 + 2.0 ** -19) * mag_u
    tol = du.reshape(rows, -1) @ np.abs(W_O).astype(np.float64) + 4 * H * d.d_v * 2.0 ** -24 * mag + \
        D.EPS[act] * np.abs(want)
    assert_within(out.double().cpu().numpy(), want, tol * 1.01, "out")
    again = torch.empty_like(out)
    M.mla_output_proj_prefix(cfg, D.dev(o_lat, act), D.dev(lse), D.dev(up, act), D.dev(lsep),
                             D.dev(W_UV, act), D.dev(W_O, act), again, ws)
    assert torch.equal(out, again)                     # same bits


@pytest.mark.parametrize("act,shape", [("f32", "tiny"), ("bf16", "tiny"), ("bf16", "v2"), ("bf16", "value64")])
@pytest.mark.parametrize("rows", [3, 150])
def test_output_proj_prefix_nan_lse(act, shape, rows):
    """A NaN LSE, beside an empty key set or another, makes its row NaN and no other."""
    rng = np.random.default_rng(rows)
    d = D.dims(shape, 16)
    o_lat = D.draw(rng, (rows, 16, d.d_latent), act, 0.1)
    up = D.draw(rng, (rows, 16, d.d_v), act, 0.1)
    lse, lsep = np.zeros((2, rows, 16), np.float32)
    lse[0, 0], lsep[0, 0] = -np.inf, np.nan
    lse[1, 3] = np.nan
    cfg = M.make_config(d, act, act)
    out = torch.zeros((rows, d.d_model), dtype=D.torch_type(act), device="cuda")
    ws = torch.empty(M.mla_output_proj_prefix_workspace_size(cfg, rows), dtype=torch.uint8, device="cuda")
    M.mla_output_proj_prefix(cfg, D.dev(o_lat, act), D.dev(lse), D.dev(up, act), D.dev(lsep),
                             D.dev(D.draw(rng, (d.d_latent, 16 * d.d_v), act), act),
                             D.dev(D.draw(rng, (16 * d.d_v, d.d_model), act), act), out, ws)
    torch.cuda.synchronize()
    assert out[:2].isnan().all() and out[2:].isfinite().all()


# ----------------------------------------------------------------------------- the three together

@pytest.mark.parametrize("cache", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
def test_prefix_step_equals_attention_over_both_key_sets(cache):
    """One step behind a shared prefix: append of the own tokens, expand, attend, decode, joined
    projection, against the decompressed attention over prefix and own tokens at once."""
    rng = np.random.default_rng(77)
    H, L, q, own = 128, 200, 2, [2, 70, 131, 0]
    d = D.dims("v2", H)
    c = D.Cache(rng, cache, d, [L] + own)
    cfg = c.config()
    B = len(own)
    W_UK = D.draw(rng, (512, H * 128), "bf16", 512 ** -0.5)
    W_UV = D.draw(rng, (512, H * 128), "bf16", 512 ** -0.5)
    W_O = D.draw(rng, (H * 128, d.d_model), "bf16", (H * 128) ** -0.5)
    qn, qp = D.draw(rng, (B, q, H, 128), "bf16"), D.draw(rng, (B, q, H, 64), "bf16")
    keys, values, k_pe = expand(c, cfg, W_UK, W_UV, L)
    pool, lens = c.device(), D.dev(np.array(own, np.int32))
    tab = D.dev(c.table[1:].copy())
    u = torch.empty(B, q, H, 128, dtype=torch.bfloat16, device="cuda")
    lse_p, lse = torch.empty(B, q, H, device="cuda"), torch.empty(B, q, H, device="cuda")
    ws = torch.empty(max(M.mla_prefix_attend_workspace_size(cfg, B, q, L), M.mla_decode_workspace_size(cfg, B, q),
                         M.mla_output_proj_prefix_workspace_size(cfg, B * q)), dtype=torch.uint8, device="cuda")
    q_d, qp_d = D.dev(qn, "bf16"), D.dev(qp, "bf16")
    M.mla_prefix_attend(cfg, q_d, qp_d, keys, values, k_pe, lens, u, lse_p, ws)
    W_abs = torch.empty(H * 128 * 512, dtype=torch.bfloat16, device="cuda")
    W_comb = torch.empty(H * 512 * d.d_model, dtype=torch.bfloat16, device="cuda")
    M.mla_absorb_weights(cfg, D.dev(W_UK, "bf16"), D.dev(W_UV, "bf16"), D.dev(W_O, "bf16"), W_abs, W_comb)
    o = torch.empty(B, q, H, 512, dtype=torch.bfloat16, device="cuda")
    M.mla_decode(cfg, q_d, qp_d, W_abs, pool, tab, lens, o, lse, ws)
    out = torch.empty(B * q, d.d_model, dtype=torch.bfloat16, device="cuda")
    M.mla_output_proj_prefix(cfg, o, lse, u, lse_p, D.dev(W_UV, "bf16"), D.dev(W_O, "bf16"), out, ws)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy().reshape(B, q, -1)
    scale = oracle.softmax_scale(128, 64)
    for b, n in enumerate(own):
        if n == 0:
            assert not got[b].any()
            continue
        # own keys were stored as rotated at their own index; at L + index they turn by L more
        rows = c.values[1 + b]
        k = oracle.rope(rows[:, 512:], np.full(n, L))
        both = np.concatenate([c.values[0], np.concatenate([rows[:, :512], k], 1)])
        e = oracle.decode_decompressed(both[:, :512], both[:, 512:], qn[b], qp[b], W_UK, W_UV, scale,
                                       10000.0, heads=list(range(H)))
        want = oracle.mha_output(e["u"], W_O)
        tol = 1e-2 * np.abs(want).max() + 1e-3        # the decode's own tolerance
        assert np.abs(got[b] - want).max() <= tol
