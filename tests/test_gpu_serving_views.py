"""The serving calls on tensors that start off a 16-byte boundary, on head shapes that no tensor map
takes, and at the edges of their kernels' limits."""
import threading

import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
from oracle import serving as ref
from tests import serving_data as D
from tests import test_gpu_evict as evict
from tests import test_gpu_prefix as prefix

pytestmark = pytest.mark.gpu
assert_within = D.assert_within


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


# ----------------------------------------------------------------------------- absorbed query

@pytest.mark.parametrize("shape,H,shift", [("v2", 16, ("q_pe",)), ("v2", 16, ("q_lat",)), ("v2", 16, ("q_nope",)),
                                           ("v2", 16, ("W",)), ("v2", 3, ("q_nope", "q_pe", "W", "q_lat")),
                                           ("tiny", 16, ("q_pe", "q_lat")), ("odd", 3, ()), ("odd128", 3, ()),
                                           ("odd", 3, ("q_nope", "q_pe", "W", "q_lat"))])
def test_absorb_query_off_the_tensor_map(shape, H, shift):
    """bf16 queries at any address and of any head shape: each tensor by itself and all of them two
    bytes off a 16-byte boundary; widths whose rows are no multiple of 16 bytes."""
    rng = np.random.default_rng(len(shift) + H)
    d = D.dims(shape, H)
    B, q, lens = 3, 2, np.array([2, 900, 65], np.int32)
    qn, qp = D.draw(rng, (B, q, H, d.d_nope), "bf16"), D.draw(rng, (B, q, H, d.d_rope), "bf16")
    W_abs = D.draw(rng, (H, d.d_nope, d.d_latent), "bf16", d.d_latent ** -0.5)
    t = {"q_nope": D.dev(qn, "bf16"), "q_pe": D.dev(qp, "bf16"), "W": D.dev(W_abs, "bf16"),
         "q_lat": torch.full((B, q, H, d.d_latent + d.d_rope), 7.0, dtype=torch.bfloat16, device="cuda")}
    for name in shift:
        t[name] = D.shifted(t[name])
    M.mla_absorb_query(M.make_config(d, "bf16", "bf16"), t["q_nope"], t["q_pe"], t["W"], D.dev(lens), t["q_lat"])
    torch.cuda.synchronize()
    pos = lens[:, None] - q + np.arange(q)
    lat = np.einsum("bthn,hnc->bthc", qn.astype(np.float64), W_abs.astype(np.float64))
    mag = np.einsum("bthn,hnc->bthc", np.abs(qn), np.abs(W_abs))
    pe = oracle.rope(qp, np.repeat(pos[:, :, None], H, 2))
    want = np.concatenate([lat, pe], -1)
    # fp32 sums of d_n products, sine and cosine to 2^-20 of values below 6, one rounding
    tol = D.EPS["bf16"] * np.abs(want) * 1.01 + np.concatenate(
        [4 * d.d_nope * 2.0 ** -24 * mag, np.full(pe.shape, 6 * 2.0 ** -20)], -1)
    assert_within(t["q_lat"].double().cpu().numpy(), want, tol, "q_lat")


# ----------------------------------------------------------------------------- several host threads

def _evict_call(rng, keys):
    """An eviction of two requests on tables of `keys` tokens: the call, and its outputs."""
    d = D.dims("tiny", 16)
    c = D.Cache(rng, "f32", d, (300, 200), max_pages=-(-keys // 64))
    w, tab, ln = D.dev(D.draw(rng, (2, c.max_pages * 64), "f32")), D.dev(c.table), D.dev(np.array([300, 200], np.int32))
    pool, cfg = c.device(), c.config()
    new = D.dev(c.spare.reshape(2, 2).copy())          # into new pages: every call does the same
    outs = torch.empty(2, 100, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    return lambda s: M.mla_evict_cache(cfg, w, ln, tab, pool, 100, *outs, new_block_table=new, sinks=2, recent=5,
                                       stream=s), outs


def _attend_call(rng, d_n):
    d = D.dims("tiny", 16)
    d.d_nope = d_n
    x = [D.dev(D.draw(rng, s, "f32")) for s in ((80, 1, 16, d_n), (80, 1, 16, d.d_rope), (16, 9, d_n), (16, 9, d.d_v),
                                                (9, d.d_rope))]
    outs = torch.empty(80, 1, 16, d.d_v, device="cuda"), torch.empty(80, 1, 16, device="cuda")
    ln, cfg = D.dev(np.full(80, 3, np.int32)), M.make_config(d, "f32", "f32")
    return lambda s: M.mla_prefix_attend(cfg, *x, ln, *outs, stream=s), outs


def _weigh_call(rng, d_c):
    d = D.dims("tiny", 16)
    d.d_latent = d_c
    c = D.Cache(rng, "f32", d, (100,))
    q, lse = D.dev(D.draw(rng, (1, 1, 16, d_c + d.d_rope), "f32", 0.1)), torch.zeros(1, 1, 16, device="cuda")
    w, pool, cfg = torch.zeros(1, c.max_pages * 64, device="cuda"), c.device(), c.config()
    tab, ln = D.dev(c.table), D.dev(np.array([100], np.int32))
    return lambda s: M.mla_key_weights(cfg, q, lse, pool, tab, ln, w, decay=0.0, stream=s), (w,)


@pytest.mark.parametrize("make,sizes", [(_evict_call, (640, 150000)), (_attend_call, (1600, 3200)),
                                        (_weigh_call, (256, 512))], ids=["evict", "attend", "weigh"])
def test_host_threads_with_other_sizes(make, sizes):
    """Host threads whose calls need different amounts of shared memory of one kernel, on streams of
    their own: no call fails, and all give what they give alone."""
    calls = [make(np.random.default_rng(i), n) for i, n in enumerate(3 * sizes)]
    streams = [torch.cuda.Stream() for _ in calls]
    want = []
    for call, outs in calls:
        call(None)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    gate, errors = threading.Barrier(len(calls)), []

    def loop(i):
        try:
            gate.wait()
            for _ in range(5000):
                calls[i][0](streams[i])
        except Exception as e:                       # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, outs), w in zip(calls, want):
        assert all(torch.equal(o, y) for o, y in zip(outs, w))


@pytest.mark.parametrize("B,d_n", [(80, 1390), (80, 1400), (80, 1472), (80, 1488), (3, 1488), (80, 7000),
                                   (80, 7200), (80, 14300), (80, 20000), (2, 50001)])
def test_attend_widths_up_to_the_shared_memory(B, d_n):
    """Head widths whose query rows and outputs are just within 48 KB of dynamic shared memory, beside
    the kernel's static arrays (d_n + d_r + d_v up to 1536 at 8 rows a block), and just above; widths
    of which 8 rows, or 4, no longer fit a block."""
    rng = np.random.default_rng(d_n)
    d = D.dims("tiny", 16)
    d.d_nope = d_n
    x = dict(q_nope=D.draw(rng, (B, 1, 16, d_n), "f32"), q_pe=D.draw(rng, (B, 1, 16, d.d_rope), "f32"),
             keys=D.draw(rng, (16, 70, d_n), "f32"), values=D.draw(rng, (16, 70, d.d_v), "f32"),
             k_pe=D.draw(rng, (70, d.d_rope), "f32"))
    lens = rng.integers(1, 50, B).astype(np.int32)
    u, lse = prefix.attend(M.make_config(d, "f32", "f32"), x, lens, "f32")
    prefix.check_attend(d, x, lens, "f32", u, lse)


@pytest.mark.parametrize("pages", [100, 112, 128, 140])
def test_evict_many_requests_of_wide_tables(pages):
    """More requests than SMs, with tables of 6400 to 8960 tokens: the selection's weights take about
    48 KB beside its static arrays."""
    rng = np.random.default_rng(pages)
    c = D.Cache(rng, "f32", D.dims("tiny", 16), list(rng.integers(0, 200, 160)), max_pages=pages)
    w = evict.draw_weights(rng, 160, pages * 64, "plain")
    res = evict.run_evict(c, w, 70, 2, 8)
    evict.check_evict(c, w, 70, 2, 8, res)


# ----------------------------------------------------------------------------- rows inside a warp

@pytest.mark.parametrize("shape,H", [("v2", 16), ("v2", 64), ("value64", 5), ("value128", 5)])
@pytest.mark.parametrize("some,all_", [(131, 160), (129, 256), (283, 288), (33, 64), (5, 32)])
def test_rows_that_end_inside_a_warp_have_the_bits_of_whole_ones(shape, H, some, all_):
    """The joined projection of a batch whose last warp has few live rows equals, bit by bit, the same
    rows of a batch that fills its warps (both cut the product alike)."""
    rng = np.random.default_rng(some)
    d = D.dims(shape, H)
    cfg = M.make_config(d, "bf16", "bf16")
    o, up = (D.dev(D.draw(rng, (all_, H, w), "bf16", 0.1), "bf16") for w in (d.d_latent, d.d_v))
    lse, lsep = (D.dev((rng.standard_normal((all_, H)) * 3).astype(np.float32)) for _ in range(2))
    W_UV = D.dev(D.draw(rng, (d.d_latent, H * d.d_v), "bf16", d.d_latent ** -0.5), "bf16")
    W_O = D.dev(D.draw(rng, (H * d.d_v, d.d_model), "bf16", (H * d.d_v) ** -0.5), "bf16")

    def project(n):
        out = torch.full((n, d.d_model), float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(M.mla_output_proj_prefix_workspace_size(cfg, n), dtype=torch.uint8, device="cuda")
        M.mla_output_proj_prefix(cfg, o[:n], lse[:n], up[:n], lsep[:n], W_UV, W_O, out, ws)
        return out
    got, want = project(some), project(all_)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and torch.equal(got, want[:some])


@pytest.mark.parametrize("some,all_,L", [(131, 160, 1500), (129, 256, 300), (33, 64, 5000), (5, 32, 260)])
def test_attention_rows_that_end_inside_a_warp(some, all_, L):
    rng = np.random.default_rng(some)
    d = D.dims("v2", 16)
    x, lens = prefix.attend_inputs(rng, d, all_, 1, L, "bf16", rng.integers(1, 900, all_))
    cfg = M.make_config(d, "bf16", "bf16")
    u, lse = prefix.attend(cfg, x, lens, "bf16")
    x["q_nope"], x["q_pe"] = x["q_nope"][:some], x["q_pe"][:some]
    su, slse = prefix.attend(cfg, x, lens[:some], "bf16")
    assert np.array_equal(su, u[:some]) and np.array_equal(slse, lse[:some])


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
def test_expansion_of_bad_pages_between_good_ones(kind):
    """Bad pages in every place of a 256-token tile: their rows are zeros, the others' bits stay."""
    rng = np.random.default_rng(7)
    d = D.dims("v2", 16)
    c = D.Cache(rng, kind, d, [600])
    W_UK, W_UV = (D.draw(rng, (512, 16 * 128), "bf16", 512 ** -0.5) for _ in range(2))
    good = prefix.expand(c, c.config(), W_UK, W_UV, 600)
    for bad in ([0], [3], [1, 2, 6], [0, 1, 2, 3], [9]):
        table = c.table[0].copy()
        table[bad] = -1
        gone = np.isin(np.arange(600) // 64, bad)
        got = prefix.expand(c, c.config(), W_UK, W_UV, 600, table=table)
        for g, w in zip(got[:2], good[:2]):
            assert torch.equal(g[:, ~gone], w[:, ~gone]) and not g[:, gone].any()


# ----------------------------------------------------------------------------- wide rows

@pytest.mark.parametrize("kind,d_c,H", [("f32", 768, 16), ("f32", 828, 3), ("bf16", 1400, 16), ("bf16", 1692, 3),
                                        ("fp8_e4m3", 3348, 3), ("fp8_e4m3_b128", 2944, 3), ("f32", 704, 16)])
def test_key_weights_of_rows_up_to_the_shared_memory(kind, d_c, H):
    """Latents so wide that a page leaves room for 8 warps of one query, or for fewer."""
    rng = np.random.default_rng(d_c)
    d = D.dims("tiny", H)
    d.d_latent, d.d_rope = d_c, 64
    c = D.Cache(rng, kind, d, (70, 0, 5))
    q_lat, lse, scale = evict.weigh_inputs(rng, c, 2)
    q_lat, lse = q_lat * np.float32(0.25), np.zeros_like(lse)   # moderate scores; any LSE serves
    old = rng.random((3, c.max_pages * 64)).astype(np.float32)
    got = evict.weigh(c, 2, q_lat, lse, old, 0.5)
    evict.check_weights(c, 2, q_lat, lse, scale, old, 0.5, got)


# ----------------------------------------------------------------------------- many rows

@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_output_proj_prefix_of_a_million_rows(act):
    """More rows than 65535 blocks of 16, at a small shape; every row equals that of a small batch."""
    rng = np.random.default_rng(3)
    d = D.dims("tiny", 2)
    d.d_latent, d.d_nope, d.d_v, d.d_model = 8, 4, 4, 12
    cfg, rows, few = M.make_config(d, act, act), 16 * 65535 + 21, 1000
    o, up = (D.dev(D.draw(rng, (few, 2, w), act, 0.1), act) for w in (8, 4))
    lse, lsep = (D.dev(rng.standard_normal((few, 2)).astype(np.float32)) for _ in range(2))
    W_UV, W_O = D.dev(D.draw(rng, (8, 8), act), act), D.dev(D.draw(rng, (8, 12), act), act)

    def project(at):
        out = torch.full((len(at), 12), float("nan"), dtype=D.torch_type(act), device="cuda")
        ws = torch.empty(M.mla_output_proj_prefix_workspace_size(cfg, len(at)), dtype=torch.uint8, device="cuda")
        M.mla_output_proj_prefix(cfg, o[at], lse[at], up[at], lsep[at], W_UV, W_O, out, ws)
        return out
    want = project(torch.arange(few, device="cuda"))
    at = torch.arange(rows, device="cuda") % few
    got = project(at)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and torch.equal(got, want[at])


# ----------------------------------------------------------------------------- other start addresses

@pytest.mark.parametrize("which", ["W_UK", "W_UV", "cache", "keys", "values", "k_pe", "all"])
def test_expand_off_16_bytes(which):
    """Each tensor of an expansion off a 16-byte boundary, element by element against fp64."""
    rng = np.random.default_rng(50)
    d = D.dims("v2", 3)
    c = D.Cache(rng, "bf16", d, [130])
    W_UK, W_UV = (D.draw(rng, (512, 3 * 128), "bf16", 512 ** -0.5) for _ in range(2))
    t = dict(W_UK=D.dev(W_UK, "bf16"), W_UV=D.dev(W_UV, "bf16"), cache=c.device(),
             keys=torch.full((3, 130, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
             values=torch.full((3, 130, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
             k_pe=torch.full((130, 64), 7.0, dtype=torch.bfloat16, device="cuda"))
    for name in t:
        if which in (name, "all"):
            t[name] = D.shifted(t[name], 2 if name == "cache" else 1)    # (a cache starts on 4 bytes)
    M.mla_prefix_expand(c.config(), t["W_UK"], t["W_UV"], t["cache"], D.dev(c.table[0]), 130, t["keys"], t["values"],
                        t["k_pe"])
    torch.cuda.synchronize()
    rows = c.values[0]
    K, V, aK, aV = ref.expand_prefix(rows[:, :512], W_UK, W_UV, 3)
    assert_within(t["keys"].double().cpu().numpy(), K, prefix.expand_bound(aK, K, "bf16", "bf16", 512), "keys")
    assert_within(t["values"].double().cpu().numpy(), V, prefix.expand_bound(aV, V, "bf16", "bf16", 512), "values")
    assert np.array_equal(t["k_pe"].double().cpu().numpy(), rows[:, 512:])


@pytest.mark.parametrize("rows", [5, 150])
@pytest.mark.parametrize("which", ["o", "lse", "up", "lsep", "W_UV", "W_O", "out", "all"])
def test_output_proj_prefix_off_16_bytes(which, rows):
    """The joined projection at the tensor cores' shape with each tensor off a 16-byte boundary."""
    rng = np.random.default_rng(rows)
    H = 3
    d = D.dims("v2", H)
    cfg = M.make_config(d, "bf16", "bf16")
    h = dict(o=D.draw(rng, (rows, H, 512), "bf16", 0.1), up=D.draw(rng, (rows, H, 128), "bf16", 0.1),
             lse=(rng.standard_normal((rows, H)) * 3).astype(np.float32),
             lsep=(rng.standard_normal((rows, H)) * 3).astype(np.float32),
             W_UV=D.draw(rng, (512, H * 128), "bf16", 512 ** -0.5),
             W_O=D.draw(rng, (H * 128, d.d_model), "bf16", (H * 128) ** -0.5))
    t = {k: D.dev(v, None if k.startswith("lse") else "bf16") for k, v in h.items()}
    t["out"] = torch.full((rows, d.d_model), float("nan"), dtype=torch.bfloat16, device="cuda")
    for name in t:
        if which in (name, "all"):
            t[name] = D.shifted(t[name])
    ws = torch.full((M.mla_output_proj_prefix_workspace_size(cfg, rows),), 0xFF, dtype=torch.uint8, device="cuda")
    M.mla_output_proj_prefix(cfg, t["o"], t["lse"], t["up"], t["lsep"], t["W_UV"], t["W_O"], t["out"], ws)
    torch.cuda.synchronize()
    lse, lsep, W_O = h["lse"].astype(np.float64), h["lsep"].astype(np.float64), h["W_O"].astype(np.float64)
    u = ref.join_prefix(h["o"], lse, h["up"], lsep, h["W_UV"], H)
    mag_u = ref.join_prefix(np.abs(h["o"]), lse, np.abs(h["up"]), lsep, np.abs(h["W_UV"]), H)
    want, mag = u.reshape(rows, -1) @ W_O, np.abs(u).reshape(rows, -1) @ np.abs(W_O)
    # u's rounding, its fp32 sums (weights to 2^-20), the projection's sums, the result's rounding
    du = 2.0 ** -8 * np.abs(u) + (4 * 512 * 2.0 ** -24 + 2.0 ** -19) * mag_u
    tol = du.reshape(rows, -1) @ np.abs(W_O) + 4 * H * 128 * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(want)
    assert_within(t["out"].double().cpu().numpy(), want, tol * 1.01, "out")


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("which", ["q_lat", "lse", "cache", "weights", "all"])
def test_key_weights_off_16_bytes(kind, which):
    """Key weights at the tensor cores' shape with each tensor off a 16-byte boundary (the cache by 4
    bytes, its own alignment)."""
    rng = np.random.default_rng(61)
    c = D.Cache(rng, kind, D.dims("v2", 16), (130, 0, 65, 2), max_pages=3)
    q_lat, lse, scale = evict.weigh_inputs(rng, c, 2)
    old = rng.random((4, 192)).astype(np.float32)
    t = dict(q_lat=D.dev(q_lat, "bf16"), lse=D.dev(lse), cache=c.device(), weights=D.dev(old))
    for name in t:
        if which in (name, "all"):
            t[name] = D.shifted(t[name], 4 // c.device().element_size() if name == "cache" else 1)
    M.mla_key_weights(c.config(), t["q_lat"], t["lse"], t["cache"], D.dev(c.table), D.dev(np.array(c.lens, np.int32)),
                      t["weights"], decay=0.9)
    torch.cuda.synchronize()
    evict.check_weights(c, 2, q_lat, lse, scale, old, 0.9, t["weights"].cpu().numpy())


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "new_pages"])
def test_evict_off_16_bytes(kind, in_place, monkeypatch):
    """Rows that could move 16 bytes at a time, in a cache that starts 4 bytes off: 4 at a time."""
    rng = np.random.default_rng(62)
    c = D.Cache(rng, kind, D.dims("v2", 16), evict.EVICT_LENS, max_pages=13, spare=40)
    aligned = c.device
    monkeypatch.setattr(c, "device", lambda: D.shifted(aligned(), 4 // aligned().element_size()))
    assert c.device().data_ptr() % 16 == 4
    w = evict.draw_weights(rng, len(c.lens), 13 * 64, "plain")
    table = None if in_place else evict.fresh_table(c, c.lens, 130)
    # (the helper reads the pool back through a byte view, which needs no alignment of its own)
    res = evict.run_evict(c, w, 130, 4, 20, in_place=in_place, new_table=table)
    evict.check_evict(c, w, 130, 4, 20, res)
