"""Page-sparse decoding and 4-bit weights at the edges of their documentation: many short requests, calls
at once, pools and weights past 2^31, graphs, whole steps."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
import workloads as W
from oracle import pages as ref
from tests import serving_data as D
from tests import test_gpu_mx4 as mx4
from tests import test_gpu_pages as pg

pytestmark = pytest.mark.gpu
assert_within = D.assert_within
P = D.PAGE


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


# ----------------------------------------------------------------------------- decode over pages

@pytest.mark.parametrize("kind,H", [("bf16", 16), ("fp8_e4m3", 16), ("fp8_e4m3_b128", 32)])
def test_hundreds_of_short_requests(kind, H):
    """1 to 4 pages each: dozens of items a worker, tiles with one page, lists that end anywhere."""
    rng = np.random.default_rng(H)
    c = D.Cache(rng, kind, D.dims("v2", H), [1 + (37 * b) % 256 for b in range(900)])
    q_lat, pages = pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, 4, "own")
    got, lse, st = pg.attend(c, q_lat, pages)
    assert st == M.MLA_OK
    pg.check_attend(c, q_lat, pages, got, lse)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_as_many_queries_as_are_allowed(kind):
    rng = np.random.default_rng(1)
    c = D.Cache(rng, kind, D.dims("v2" if kind == "bf16" else "tiny", 16), [70] * 8)
    B, q = 8192, 1
    big = D.Cache.__new__(D.Cache)
    big.__dict__.update(c.__dict__, lens=[70 - b % 3 for b in range(B)], table=np.tile(c.table, (B // 8, 1)),
                        values=[c.values[b % 8] for b in range(B)])
    q_lat = np.tile(pg.draw_query(rng, c, q), (B // 8, 1, 1, 1))
    pages = np.tile(np.array([[[0, 1]], [[1, -1]], [[0, -1]], [[-1, -1]]], np.int32), (B // 4, 1, 1))
    got, lse, st = pg.attend(big, q_lat, pages)
    assert st == M.MLA_OK
    some = [*range(16), *range(B - 16, B)]
    few = D.Cache.__new__(D.Cache)
    few.__dict__.update(big.__dict__, lens=[big.lens[b] for b in some], values=[big.values[b] for b in some])
    pg.check_attend(few, q_lat[some], pages[some], got[some], lse[some])


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3_b128"])
def test_calls_at_once_and_graphs_in_turn(kind):
    """Two streams with workspaces of their own; then both calls captured and replayed in turn."""
    rng = np.random.default_rng(2)
    c = D.Cache(rng, kind, D.dims("v2", 128), (5000, 3000, 700, 64))
    pool, cfg, table, lens = c.device(), c.config(), pg.i32(c.table), pg.i32(c.lens)
    calls = []
    for k, budget in enumerate((20, 7)):
        q_lat, pages = pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, budget, "own")
        n = M.mla_decode_pages_workspace_size(cfg, 4, 1, budget)
        t = dict(q=D.dev(q_lat, "bf16"), pages=pg.i32(pages), ws=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 o=torch.zeros(4, 1, 128, 512, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros(4, 1, 128, device="cuda"))
        calls.append((q_lat, pages, t))

    def run(t):
        M.mla_decode_pages(cfg, t["q"], pool, table, lens, t["pages"], t["o"], t["lse"], t["ws"])

    def check():
        torch.cuda.synchronize()
        for q_lat, pages, t in calls:
            assert M.mla_read_device_status(t["ws"]) == M.MLA_OK
            pg.check_attend(c, q_lat, pages, t["o"].double().cpu().numpy(), t["lse"].cpu().numpy())
            t["o"].zero_(), t["lse"].zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (_, _, t) in zip(streams, calls):
            with torch.cuda.stream(s):
                run(t)
    check()
    torch.cuda.synchronize()
    graphs = []
    for s, (_, _, t) in zip(streams, calls):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(t)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    check()


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
def test_pools_past_2_31_bytes(kind):
    """The pages in use at the end of a pool of more than 4 GB."""
    rng = np.random.default_rng(3)
    c = D.Cache(rng, kind, D.dims("v2", 16), (300, 129), max_pages=6)
    page = P * c.row
    shift = (1 << 32) // page + 5
    pool = torch.empty((shift + c.num_pages) * page, dtype=torch.uint8, device="cuda")
    pool[shift * page:] = torch.from_numpy(c.bytes.reshape(-1).copy()).cuda()
    c.table[c.table >= 0] += shift
    c.num_pages += shift
    view = pool.view(torch.bfloat16) if kind == "bf16" else pool
    q_lat, pages = pg.draw_query(rng, c, 2), pg.lists(rng, c, 2, 4, "own")
    got, lse, st = pg.attend(c, q_lat, pages, pool=view)
    assert st == M.MLA_OK
    pg.check_attend(c, q_lat, pages, got, lse)
    keys = torch.full((c.num_pages, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    M.mla_page_keys(c.config(), view, pg.i32(c.table), pg.i32(c.lens), keys)
    torch.cuda.synchronize()
    for b, n in enumerate(c.lens):
        want, mag = ref.page_keys(c.values[b], P)
        at = c.table[b, : len(want)]
        assert_within(keys[at.tolist()].double().cpu().numpy(), want, 2.0 ** -8 * np.abs(want) * 1.01 + 70 * 2.0 ** -24 * mag, "keys")


@pytest.mark.parametrize("pages", [4096, 8192])
def test_scores_of_the_longest_requests_that_the_tensor_cores_take(pages):
    """8192 and 4096 pages (clusters of sixteen or eight, four tiles a CTA), and lengths that leave CTAs without a
    tile."""
    rng = np.random.default_rng(4)
    most = pages
    c = pg.Tables(rng, "bf16", D.dims("v2", 128), (most * P, (most - 1) * P + 1, 128 * P, 129 * P + 7, 0, 1), most)
    q_lat, keys = pg.draw_query(rng, c, 1, 1.0), pg.draw_keys(rng, c)
    got = pg.score(c, q_lat, keys)
    pg.check_scores(c, q_lat, keys, got)
    assert np.array_equal(got, pg.score(c, q_lat, keys))


@pytest.mark.parametrize("page_size", [1, 16, 63])
def test_other_page_sizes(page_size, monkeypatch):
    """Pages of other sizes take the SIMT kernels."""
    rng = np.random.default_rng(page_size)
    monkeypatch.setattr(D, "PAGE", page_size)
    monkeypatch.setattr(pg, "P", page_size)
    for kind, shape in (("bf16", "v2"), ("f32", "tiny"), ("fp8_e4m3", "v2")):
        c = D.Cache(rng, kind, D.dims(shape, 16), (130, 63, 1, 64))
        assert c.config().page_size == page_size
        q_lat, pages = pg.draw_query(rng, c, 1), pg.lists(rng, c, 1, 5, "own")
        got, lse, st = pg.attend(c, q_lat, pages)
        assert st == M.MLA_OK
        pg.check_attend(c, q_lat, pages, got, lse)
        pg.check_keys(c, pg.make_keys(c))
        keys = pg.draw_keys(rng, c)
        pg.check_scores(c, q_lat, keys, pg.score(c, q_lat, keys))


# ----------------------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_more_rows_than_a_grid_has(act):
    rng = np.random.default_rng(5)
    codes, scales, w = mx4.draw_weight(rng, 64, 9)
    x = D.draw(rng, (140000, 64), act)
    mx4.check(mx4.project(x, codes, scales, act, 9), x, w, act)


def test_weights_past_2_31_elements():
    """Quantised, read back and multiplied: the last columns of a weight of 2.3e9 elements."""
    K, N = 32768, 70016
    cfg = mx4.config("bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(K, N, dtype=torch.bfloat16, device="cuda")
    for k in range(0, K, 2048):
        w[k: k + 2048] = torch.randn(2048, N, generator=g, device="cuda")
    codes, scales = mx4.arrays("bf16", K, N)
    M.mla_mx4_quantize(cfg, w, codes, scales)
    last = w[:, -40:].float().cpu().numpy()
    del w
    code, e = ref.mx4_quantize(last)
    packed, _ = ref.mx4_pack(code, e)
    assert np.array_equal(codes.view(N, K // 2)[-40:].cpu().numpy(), packed)
    values = ref.mx4_values(code, e)
    for rows in (3, 50):
        x = torch.randn(rows, K, generator=g, device="cuda").to(torch.bfloat16)
        got = mx4.project(x.float().cpu().numpy(), codes, scales, "bf16", N)
        mx4.check(got[:, -40:], x.double().cpu().numpy(), values, "bf16")
    back = torch.empty(K, N, dtype=torch.bfloat16, device="cuda")
    M.mla_mx4_dequantize(cfg, codes, scales, back)
    torch.cuda.synchronize()
    assert np.array_equal(back[:, -40:].double().cpu().numpy(), values)


# ----------------------------------------------------------------------------- a whole step

@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3"])
def test_step_of_sparse_attention_and_4_bit_projection(kind):
    """From hidden states to the layer's output: append, page keys, queries, page scores, selection, attention
    over the chosen pages, projection through 4-bit folded weights; every stage against the references on
    what the stage before gave."""
    rng = np.random.default_rng(6)
    H, d_model = 16, 256
    d = D.dims("v2", H)
    d.d_model = d_model
    c = D.Cache(rng, kind, d, (900, 333), max_pages=16)
    B, budget = 2, 5
    for b in range(B):
        c.table[b, -(-c.lens[b] // P)] = c.spare[b]
    cfg, pool, table = c.config(), c.device(), pg.i32(c.table)
    bf = torch.bfloat16

    def dev(*shape, std=1.0):
        return D.dev(D.draw(rng, shape, "bf16", std), "bf16")
    h, W_kv = dev(B, d_model), dev(d_model, 576, std=d_model ** -0.5)
    W_UK, W_UV = dev(512, H * 128, std=512 ** -0.5), dev(512, H * 128, std=512 ** -0.5)
    W_O = dev(H * 128, d_model, std=(H * 128) ** -0.5)
    W_abs = torch.empty(H, 128, 512, dtype=bf, device="cuda")
    W_comb = torch.empty(H * 512, d_model, dtype=bf, device="cuda")
    M.mla_absorb_weights(cfg, W_UK, W_UV, W_O, W_abs, W_comb)
    codes, scales = mx4.arrays("bf16", H * 512, d_model)
    M.mla_mx4_quantize(cfg, W_comb, codes, scales)
    lens = pg.i32(c.lens)
    keys = torch.zeros(c.num_pages, 576, dtype=bf, device="cuda")
    M.mla_page_keys(cfg, pool, table, lens, keys)                         # the prompts
    M.mla_append_cache(cfg, h, W_kv, pg.i32(range(B)), lens, table, pool)
    lens = lens + 1
    M.mla_page_keys(cfg, pool, table, lens, keys, new_tokens=1)
    qn, qp = dev(B, 1, H, 128, std=0.6), dev(B, 1, H, 64, std=0.6)
    q_lat = torch.empty(B, 1, H, 576, dtype=bf, device="cuda")
    M.mla_absorb_query(cfg, qn, qp, W_abs, lens, q_lat)
    scores = torch.full((B, 1, 16), 7.0, device="cuda")
    ws = torch.zeros(max(1, M.mla_page_scores_workspace_size(cfg, B, 1, 16)), dtype=torch.uint8, device="cuda")
    M.mla_page_scores(cfg, q_lat, keys, table, lens, scores, ws)
    pages = torch.empty(B, 1, budget, dtype=torch.int32, device="cuda")
    M.mla_select_pages(cfg, scores, lens, pages, sinks=1, recent=2)
    o, lse = torch.empty(B, 1, H, 512, dtype=bf, device="cuda"), torch.empty(B, 1, H, device="cuda")
    wd = torch.zeros(M.mla_decode_pages_workspace_size(cfg, B, 1, budget), dtype=torch.uint8, device="cuda")
    M.mla_decode_pages(cfg, q_lat, pool, table, lens, pages, o, lse, wd)
    out = torch.empty(B, d_model, dtype=bf, device="cuda")
    wp = torch.zeros(M.mla_mx4_project_workspace_size(cfg, H * 512, d_model, B), dtype=torch.uint8, device="cuda")
    M.mla_mx4_project(cfg, o.view(B, H * 512), codes, scales, out, wp)
    torch.cuda.synchronize()
    assert M.mla_read_device_status(wd) == M.MLA_OK
    now = [n + 1 for n in c.lens]
    raw = c.back(pool)
    view = D.Cache.__new__(D.Cache)
    view.__dict__.update(c.__dict__, lens=now, values=[pg.decode_rows(c, raw[c.slots(b, now[b])]) for b in range(B)])
    q = q_lat.double().cpu().numpy()
    pg.check_scores(view, q, keys.double().cpu().numpy(), scores.cpu().numpy())
    sel = pages.cpu().numpy()
    for b in range(B):
        assert np.array_equal(sel[b, 0], ref.select_pages(scores[b, 0].cpu().numpy(), -(-now[b] // P), budget, 1, 2))
    pg.check_attend(view, q, sel, o.double().cpu().numpy(), lse.cpu().numpy())
    code, e = ref.mx4_quantize(W_comb.float().cpu().numpy())
    mx4.check(out.double().cpu().numpy(), o.double().cpu().numpy().reshape(B, -1), ref.mx4_values(code, e), "bf16")
    # a list of every page is the decode over all of them
    every = pg.i32(np.tile(np.arange(16, dtype=np.int32), (B, 1, 1)))
    every[0, 0, 15:] = -1
    every[1, 0, 6:] = -1
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    wd = torch.zeros(M.mla_decode_pages_workspace_size(cfg, B, 1, 16), dtype=torch.uint8, device="cuda")
    M.mla_decode_pages(cfg, q_lat, pool, table, lens, every, o2, lse2, wd)
    wa = torch.zeros(M.mla_decode_workspace_size(cfg, B, 1), dtype=torch.uint8, device="cuda")
    M.mla_decode(cfg, qn, qp, W_abs, pool, table, lens, o, lse, wa)
    torch.cuda.synchronize()
    assert float((lse2 - lse).abs().max()) < 1e-3 and float((o2.float() - o.float()).abs().max()) < 2e-2
