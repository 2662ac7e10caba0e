"""The serving calls where their documentation goes further than ordinary use: page sizes, softmax scales
and rotary bases of their own, widths that are no multiple of four, one head and many, offsets past 32
bits, shared pages, whole loops captured and replayed."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
import workloads as W
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


def ragged(H):
    """Widths of which only those that have to be are multiples of four."""
    return D.Dims(H, W.Dims(num_heads=H, d_model=37, d_latent=60, d_rope=4, d_nope=17, d_v=13))


# ----------------------------------------------------------------------------- page sizes

@pytest.mark.parametrize("page", [1, 16, 48, 63])
@pytest.mark.parametrize("kind,shape", [("f32", "tiny"), ("bf16", "v2"), ("fp8_e4m3", "odd"), ("fp8_e4m3_b128", "odd128")])
def test_other_page_sizes(page, kind, shape, monkeypatch):
    """Expansion, key weights and eviction of pages of 1 to 63 tokens."""
    monkeypatch.setattr(D, "PAGE", page)
    rng = np.random.default_rng(page)
    d, lens = D.dims(shape, 16), (130, 1, 0, 97)
    act = D.act_of(kind)
    c = D.Cache(rng, kind, d, lens, spare=200)
    W_UK, W_UV = (D.draw(rng, (d.d_latent, 16 * n), act, d.d_latent ** -0.5) for n in (d.d_nope, d.d_v))
    keys, values, k_pe = prefix.expand(c, c.config(), W_UK, W_UV, 130)
    rows = c.values[0]
    K, V, aK, aV = ref.expand_prefix(rows[:, : d.d_latent], W_UK, W_UV, 16)
    assert_within(keys.double().cpu().numpy(), K, prefix.expand_bound(aK, K, act, kind, d.d_latent), "keys")
    assert_within(values.double().cpu().numpy(), V, prefix.expand_bound(aV, V, act, kind, d.d_latent), "values")
    pe = rows[:, d.d_latent:]
    assert_within(k_pe.double().cpu().numpy(), pe, D.EPS[act] * np.abs(pe) * 1.01, "k_pe")
    q_lat, lse, scale = evict.weigh_inputs(rng, c, 1)
    old = rng.random((4, c.max_pages * page)).astype(np.float32)
    evict.check_weights(c, 1, q_lat, lse, scale, old, 0.5, evict.weigh(c, 1, q_lat, lse, old, 0.5))
    w = evict.draw_weights(rng, 4, c.max_pages * page, "plain")
    for in_place in (True, False):
        ntab = c.table if in_place else evict_table(c, 50, page)
        pool, kept, nl = c.device(), torch.empty(4, 50, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
        before, tab = c.back(pool).copy(), D.dev(c.table)
        M.mla_evict_cache(c.config(), D.dev(w), D.dev(np.array(lens, np.int32)), tab, pool, 50, kept, nl,
                          new_block_table=tab if in_place else D.dev(ntab), sinks=2, recent=9, rotate=False)
        after = c.back(pool)
        for b, S in enumerate(lens):
            keep = ref.evict_order(w[b], S, 50, 2, 9)
            n = len(keep)
            assert int(nl[b]) == n and np.array_equal(kept[b, :n].cpu().numpy(), keep)
            assert np.array_equal(after[c.slots(b, n, ntab)], before[c.slots(b, S)[keep]])


def evict_table(c, budget, page):
    need = [-(-min(n, budget) // page) for n in c.lens]
    t, at = np.full((len(need), max(need)), -1, np.int32), 0
    for b, n in enumerate(need):
        t[b, :n] = c.spare[at: at + n]
        at += n
    return t


# ----------------------------------------------------------------------------- widths and heads

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("L", [2, 150])
def test_widths_that_are_no_multiple_of_four(act, L):
    """Expansion, attention, joined projection and absorbed query at d_n 17, d_v 13, d 37."""
    rng = np.random.default_rng(L)
    H, B, d = 5, 3, ragged(5)
    c = D.Cache(rng, act, d, [L])
    cfg = c.config()
    W_UK, W_UV = (D.draw(rng, (60, H * n), act, 60 ** -0.5) for n in (17, 13))
    keys, values, _ = prefix.expand(c, cfg, W_UK, W_UV, L)
    K, V, aK, aV = ref.expand_prefix(c.values[0][:, :60], W_UK, W_UV, H)
    assert_within(keys.double().cpu().numpy(), K, prefix.expand_bound(aK, K, act, act, 60), "keys")
    assert_within(values.double().cpu().numpy(), V, prefix.expand_bound(aV, V, act, act, 60), "values")
    x, lens = prefix.attend_inputs(rng, d, B, 2, L, act, [2, 40, 0])
    u, lse = prefix.attend(cfg, x, lens, act)
    prefix.check_attend(d, x, lens, act, u, lse)
    W_abs = D.draw(rng, (H, 17, 60), act, 60 ** -0.5)
    q_lat = torch.empty(B, 2, H, 64, dtype=D.torch_type(act), device="cuda")
    M.mla_absorb_query(cfg, D.dev(x["q_nope"], act), D.dev(x["q_pe"], act), D.dev(W_abs, act), D.dev(lens), q_lat)
    lat = np.einsum("bthn,hnc->bthc", x["q_nope"].astype(np.float64), W_abs.astype(np.float64))
    mag = np.einsum("bthn,hnc->bthc", np.abs(x["q_nope"]), np.abs(W_abs))
    assert_within(q_lat[:2, ..., :60].double().cpu().numpy(), lat[:2],
                  (D.EPS[act] * np.abs(lat) * 1.01 + 4 * 17 * 2.0 ** -24 * mag)[:2], "q_lat")
    o = D.draw(rng, (6, H, 60), act, 0.1)
    up = D.draw(rng, (6, H, 13), act, 0.1)
    la, lb = (rng.standard_normal((6, H)).astype(np.float32) for _ in range(2))
    W_O = D.draw(rng, (H * 13, 37), act, (H * 13) ** -0.5)
    out = torch.empty(6, 37, dtype=D.torch_type(act), device="cuda")
    ws = torch.empty(M.mla_output_proj_prefix_workspace_size(cfg, 6), dtype=torch.uint8, device="cuda")
    M.mla_output_proj_prefix(cfg, D.dev(o, act), D.dev(la), D.dev(up, act), D.dev(lb), D.dev(W_UV, act), D.dev(W_O, act), out, ws)
    a64, b64, O64 = la.astype(np.float64), lb.astype(np.float64), W_O.astype(np.float64)
    uj = ref.join_prefix(o, a64, up, b64, W_UV, H)
    mu = ref.join_prefix(np.abs(o), a64, np.abs(up), b64, np.abs(W_UV), H)
    want = uj.reshape(6, -1) @ O64
    du = D.EPS[act] * np.abs(uj) + (4 * 60 * 2.0 ** -24 + 2.0 ** -19) * mu
    tol = du.reshape(6, -1) @ np.abs(O64) + 4 * H * 13 * 2.0 ** -24 * (np.abs(uj).reshape(6, -1) @ np.abs(O64)) + \
        D.EPS[act] * np.abs(want)
    assert_within(out.double().cpu().numpy(), want, tol * 1.01, "out")


@pytest.mark.parametrize("H", [1, 2, 130, 200])
def test_one_head_and_many(H):
    """The tensor cores' prefix kernels with one head, two, and more than a cluster's or an SM count's."""
    rng = np.random.default_rng(H)
    d, L = D.dims("v2", H), 300
    c = D.Cache(rng, "bf16", d, [L])
    W_UK, W_UV = (D.draw(rng, (512, H * 128), "bf16", 512 ** -0.5) for _ in range(2))
    keys, values, _ = prefix.expand(c, c.config(), W_UK, W_UV, L)
    K, V, aK, aV = ref.expand_prefix(c.values[0][:, :512], W_UK, W_UV, H)
    assert_within(keys.double().cpu().numpy(), K, prefix.expand_bound(aK, K, "bf16", "bf16", 512), "keys")
    assert_within(values.double().cpu().numpy(), V, prefix.expand_bound(aV, V, "bf16", "bf16", 512), "values")
    for B in (3, 140):
        x, lens = prefix.attend_inputs(rng, d, B, 1, L, "bf16", rng.integers(1, 99, B))
        u, lse = prefix.attend(c.config(), x, lens, "bf16")
        prefix.check_attend(d, x, lens, "bf16", u, lse)
    k = D.Cache(rng, "bf16", d, (70, 3))
    q_lat, lse, scale = evict.weigh_inputs(rng, k, 2)
    old = rng.random((2, k.max_pages * 64)).astype(np.float32)
    evict.check_weights(k, 2, q_lat, lse, scale, old, 0.5, evict.weigh(k, 2, q_lat, lse, old, 0.5))


# ----------------------------------------------------------------------------- scale and rotary base

@pytest.mark.parametrize("act,shape", [("f32", "tiny"), ("bf16", "v2")])
def test_softmax_scale_and_rotary_base_of_their_own(act, shape):
    """Calls whose configurations differ in scale, base and rotary width, in turn: each call goes by its
    own (the rotary table is kept between calls)."""
    rng = np.random.default_rng(17)
    H, L = 16, 90
    cases = []
    for dr, theta, scale in ((64, 500000.0, 0.02), (64, 10000.0, 0.0), (32, 500000.0, 0.3), (64, 500000.0, 0.02), (64, 0.0, -1.0)):
        d = D.dims(shape, H)
        if shape == "tiny":
            d.d_rope = dr // 4
        elif dr != 64:
            continue
        cases.append((d, theta, scale))
    for d, theta, scale in cases:
        cfg = M.make_config(d, act, act, softmax_scale=scale, rope_theta=theta)
        base, sc = theta or 10000.0, scale if scale > 0 else oracle.softmax_scale(d.d_nope, d.d_rope)
        x, lens = prefix.attend_inputs(rng, d, 4, 1, L, act, [1, 77, 3000, 9])
        u, lse = prefix.attend(cfg, x, lens, act)
        ru, rl, mag_s, mag_v = ref.attend_prefix(x["q_nope"], x["q_pe"], x["keys"], x["values"], x["k_pe"], lens,
                                                 float(np.float32(sc)), base)
        n = d.d_nope + d.d_rope
        ds = mag_s * (4 * n * 2.0 ** -24 + (2.0 ** -16 + 2.0 ** -20 if act == "bf16" else 2.0 ** -21)) + 2.0 ** -21
        assert_within(lse, rl, 2 * ds + 4 * (L + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(rl), "lse")
        dw = 2 * ds + (D.EPS["bf16"] if act == "bf16" else 0) + 4 * (L + 64) * 2.0 ** -24
        assert_within(u, ru, dw[..., None] * mag_v * 1.05 + D.EPS[act] * np.abs(ru) * 1.01 + 1e-30, "u")
        c = D.Cache(rng, act, d, (90, 64), spare=8)
        w = evict.draw_weights(rng, 2, c.max_pages * 64, "plain")
        pool, kept, nl = c.device(), torch.empty(2, 30, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
        before = c.back(pool).copy()
        M.mla_evict_cache(cfg, D.dev(w), D.dev(np.array([90, 64], np.int32)), D.dev(c.table), pool, 30, kept, nl, recent=5)
        after, size = c.back(pool), 4 if act == "f32" else 2
        for b, S in enumerate((90, 64)):
            keep = ref.evict_order(w[b], S, 30, 0, 5)
            pe = [np.ascontiguousarray(y[:, size * d.d_latent:]) for y in (after[c.slots(b, 30)], before[c.slots(b, S)[keep]])]
            got, o = ((y.view(np.float32) if act == "f32" else (y.view(np.uint16).astype(np.uint32) << 16).view(np.float32))
                      for y in pe)
            want = ref.turn_rows(o.astype(np.float64), np.arange(30) - keep, base)
            tol = D.EPS[act] * np.abs(want) * 1.01 + 4 * np.abs(o).max() * (2.0 ** -22 if act == "f32" else 2.0 ** -20)
            assert_within(got, want, tol, "rotary keys")
        k = D.Cache(rng, act, d, (70,))
        q_lat = D.draw(rng, (1, 1, H, d.d_latent + d.d_rope), act, 0.3)
        zero = np.zeros((1, 1, H), np.float32)
        wd = torch.zeros(1, k.max_pages * 64, device="cuda")
        M.mla_key_weights(cfg, D.dev(q_lat, act), D.dev(zero), k.device(), D.dev(k.table), D.dev(np.array([70], np.int32)), wd)
        evict.check_weights(k, 1, q_lat, zero, float(np.float32(sc)), np.zeros((1, k.max_pages * 64), np.float32), 1.0, wd.cpu().numpy())


# ----------------------------------------------------------------------------- past 32 bits

def test_prefix_of_more_than_2_to_the_31_elements():
    """Keys and values of 140000 tokens x 128 heads (2.3e9 elements each): expansion and attention at
    their far ends, against fp64 on the device."""
    rng = np.random.default_rng(70)
    H, L, B = 128, 140000, 2
    d = D.dims("v2", H)
    cfg = M.make_config(d, "bf16", "bf16")
    g = torch.Generator(device="cuda").manual_seed(5)
    pages = -(-L // 64)
    pool = torch.randn(pages, 64, 576, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    W_UK, W_UV = (torch.randn(512, H * 128, generator=g, device="cuda").mul_(512 ** -0.5).to(torch.bfloat16) for _ in range(2))
    keys, values = (torch.empty(H, L, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k_pe = torch.empty(L, 64, dtype=torch.bfloat16, device="cuda")
    M.mla_prefix_expand(cfg, W_UK, W_UV, pool, table, L, keys, values, k_pe)
    rows = pool[table.long()].view(-1, 576)[:L]
    assert torch.equal(k_pe, rows[:, 512:])
    at = torch.tensor([0, 1, 65535, L // 2, L - 130, L - 1], device="cuda")
    for h in (0, 64, 119, 127):
        for out, w in ((keys, W_UK), (values, W_UV)):
            c, wh = rows[at, :512].double(), w[:, 128 * h: 128 * h + 128].double()
            want, mag = c @ wh, c.abs() @ wh.abs()
            assert_within(out[h, at].double().cpu().numpy(), want.cpu().numpy(),
                          prefix.expand_bound(mag.cpu().numpy(), want.cpu().numpy(), "bf16", "bf16", 512), "expansion")
    qn, qp = D.draw(rng, (B, 1, H, 128), "bf16"), D.draw(rng, (B, 1, H, 64), "bf16")
    lens = np.array([1, 2 ** 31 - 1 - L], np.int32)
    u, lse = torch.empty(B, 1, H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, H, device="cuda")
    ws = torch.empty(max(256, M.mla_prefix_attend_workspace_size(cfg, B, 1, L)), dtype=torch.uint8, device="cuda")
    M.mla_prefix_attend(cfg, D.dev(qn, "bf16"), D.dev(qp, "bf16"), keys, values, k_pe, D.dev(lens), u, lse, ws)
    scale = oracle.softmax_scale(128, 64)
    for h in (0, 64, 119, 127):
        k, v, pe = keys[h].double(), values[h].double(), k_pe.double()
        for b in range(B):
            pos = L + int(lens[b]) - 1
            qr = torch.from_numpy(oracle.rope(qp[b, 0, h: h + 1].astype(np.float64), np.array([pos]))[0]).cuda()
            q = torch.from_numpy(qn[b, 0, h].astype(np.float64)).cuda()
            s = scale * (k @ q + pe @ qr)
            mag = float((scale * (k.abs() @ q.abs() + pe.abs() @ qr.abs())).max())
            want_l = torch.logsumexp(s, 0)
            p = torch.exp(s - want_l)
            want, mag_v = p @ v, p @ v.abs()
            # as for the other prefixes; at the far position the table's angle is off by 2^-24 turn more
            ds = mag * (4 * 192 * 2.0 ** -24 + 2.0 ** -16 + 2.0 ** -20 + (2.0 ** -21 if b else 0)) + 2.0 ** -21
            dl = 2 * ds + 4 * (L + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(float(want_l))
            assert abs(float(lse[b, 0, h]) - float(want_l)) <= dl
            dw = 2 * ds + 2.0 ** -8 + 4 * (L + 64) * 2.0 ** -24
            tol = dw * mag_v * 1.05 + 2.0 ** -8 * want.abs() * 1.01
            assert ((u[b, 0, h].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind,shape,pages", [("bf16", "v2", 66000), ("fp8_e4m3", "v2", 66000),
                                              ("fp8_e4m3_b128", "v2", 66000), ("f32", "tiny", 110000)])
def test_cache_pools_past_32_bits(kind, shape, pages):
    """Key weights and eviction on the last pages of a pool of more than 2^31 bytes."""
    rng = np.random.default_rng(8)
    c = D.Cache(rng, kind, D.dims(shape, 16), (300, 65), max_pages=6)
    shift = pages - c.num_pages
    table = np.where(c.table >= 0, c.table + shift, -1).astype(np.int32)
    pool = torch.zeros(pages * 64 * c.row, dtype=torch.uint8, device="cuda")
    tail = pool[shift * 64 * c.row:]
    tail.copy_(torch.from_numpy(c.bytes.reshape(-1)))
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}.get(kind, torch.uint8)
    q_lat, lse, scale = evict.weigh_inputs(rng, c, 1)
    old = rng.random((2, 6 * 64)).astype(np.float32)
    w, lens, tab = D.dev(old), D.dev(np.array(c.lens, np.int32)), D.dev(table)
    M.mla_key_weights(c.config(), D.dev(q_lat, D.act_of(kind)), D.dev(lse), pool.view(dt), tab, lens, w, decay=0.5)
    evict.check_weights(c, 1, q_lat, lse, scale, old, 0.5, w.cpu().numpy())
    for in_place in (True, False):
        tail.copy_(torch.from_numpy(c.bytes.reshape(-1)))
        before = c.back(tail).copy()
        ntab = c.table if in_place else evict.fresh_table(c, c.lens, 70)
        kept, nl = torch.full((2, 70), 99, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
        nw = torch.full((2, ntab.shape[1] * 64), -3.0, device="cuda")
        M.mla_evict_cache(c.config(), D.dev(old), lens, tab, pool.view(dt), 70, kept, nl, new_weights=nw, sinks=2, recent=9,
                          new_block_table=tab if in_place else D.dev(np.where(ntab >= 0, ntab + shift, -1).astype(np.int32)))
        res = before, c.back(tail), kept.cpu().numpy(), nl.cpu().numpy(), nw.cpu().numpy(), ntab
        evict.check_evict(c, old, 70, 2, 9, res)
        assert not pool[: 64 * c.row].any()


# ----------------------------------------------------------------------------- shared pages, optional outputs

@pytest.mark.parametrize("kind,shape", [("bf16", "v2"), ("f32", "tiny"), ("fp8_e4m3_b128", "v2")])
def test_requests_that_share_old_pages(kind, shape):
    """Two requests on the same old pages (a prompt sampled twice): key weights of both, and an eviction
    into new pages of their own; without new_weights."""
    rng = np.random.default_rng(23)
    c = D.Cache(rng, kind, D.dims(shape, 16), (300, 0), spare=12)
    c.lens, c.values = [300, 300], [c.values[0]] * 2
    c.table[1] = c.table[0]
    q_lat, lse, scale = evict.weigh_inputs(rng, c, 1)
    old = rng.random((2, c.max_pages * 64)).astype(np.float32)
    evict.check_weights(c, 1, q_lat, lse, scale, old, 0.5, evict.weigh(c, 1, q_lat, lse, old, 0.5))
    new = evict.fresh_table(c, c.lens, 90)
    pool, kept, nl = c.device(), torch.empty(2, 90, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    before = c.back(pool).copy()
    M.mla_evict_cache(c.config(), D.dev(old), D.dev(np.array(c.lens, np.int32)), D.dev(c.table), pool, 90, kept, nl,
                      new_block_table=D.dev(new), sinks=4, recent=20, rotate=False)
    after = c.back(pool)
    for b in range(2):
        keep = ref.evict_order(old[b], 300, 90, 4, 20)
        assert np.array_equal(kept[b].cpu().numpy(), keep)
        assert np.array_equal(after[c.slots(b, 90, new)], before[c.slots(b, 300)[keep]])


# ----------------------------------------------------------------------------- captured loops

@pytest.mark.parametrize("cache,act,shape,H", [("bf16", "bf16", "v2", 16), ("fp8_e4m3", "bf16", "v2", 16),
                                               ("fp8_e4m3_b128", "bf16", "v2", 16), ("f32", "f32", "tiny", 16)])
def test_whole_step_captured_and_replayed(cache, act, shape, H):
    """Expand, attend, decode, join, absorb, weigh and evict captured as one graph: its replays give the
    bits of the same calls one by one, on restored inputs."""
    rng = np.random.default_rng(19)
    d, L, own = D.dims(shape, H), 200, [70, 131, 0]
    c = D.Cache(rng, cache, d, [L] + own)
    cfg, B, t = c.config(), 3, D.torch_type(act)
    dc, dr, dn, dv = d.d_latent, d.d_rope, d.d_nope, d.d_v
    W_UK, W_UV = (D.dev(D.draw(rng, (dc, H * n), act, dc ** -0.5), act) for n in (dn, dv))
    W_O = D.dev(D.draw(rng, (H * dv, d.d_model), act, (H * dv) ** -0.5), act)
    W_abs, W_comb = torch.empty(H * dn * dc, dtype=t, device="cuda"), torch.empty(H * dc * d.d_model, dtype=t, device="cuda")
    M.mla_absorb_weights(cfg, W_UK, W_UV, W_O, W_abs, W_comb)
    qn, qp = D.dev(D.draw(rng, (B, 1, H, dn), act), act), D.dev(D.draw(rng, (B, 1, H, dr), act), act)
    pages, tab = D.dev(c.table[0].copy()), D.dev(c.table[1:].copy())
    start = dict(pool=c.device(), lens=D.dev(np.array(own, np.int32)), w=torch.zeros(B, c.max_pages * 64, device="cuda"))
    s = {k: v.clone() for k, v in start.items()}

    def empty(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device="cuda")
    o = dict(keys=empty(H, L, dn), values=empty(H, L, dv), pe=empty(L, dr), u=empty(B, 1, H, dv),
             lse_p=empty(B, 1, H, dtype=torch.float32), o=empty(B, 1, H, dc), lse=empty(B, 1, H, dtype=torch.float32),
             out=empty(B, d.d_model), q_lat=empty(B, 1, H, dc + dr), kept=empty(B, 100, dtype=torch.int32))
    ws = torch.empty(max(M.mla_prefix_attend_workspace_size(cfg, B, 1, L), M.mla_decode_workspace_size(cfg, B, 1),
                         M.mla_output_proj_prefix_workspace_size(cfg, B)), dtype=torch.uint8, device="cuda")

    def step():
        M.mla_prefix_expand(cfg, W_UK, W_UV, s["pool"], pages, L, o["keys"], o["values"], o["pe"])
        M.mla_prefix_attend(cfg, qn, qp, o["keys"], o["values"], o["pe"], s["lens"], o["u"], o["lse_p"], ws)
        M.mla_decode(cfg, qn, qp, W_abs, s["pool"], tab, s["lens"], o["o"], o["lse"], ws)
        M.mla_output_proj_prefix(cfg, o["o"], o["lse"], o["u"], o["lse_p"], W_UV, W_O, o["out"], ws)
        M.mla_absorb_query(cfg, qn, qp, W_abs, s["lens"], o["q_lat"])
        M.mla_key_weights(cfg, o["q_lat"], o["lse"], s["pool"], tab, s["lens"], s["w"], decay=0.9)
        M.mla_evict_cache(cfg, s["w"], s["lens"], tab, s["pool"], 100, o["kept"], s["lens"], new_weights=s["w"], sinks=4,
                          recent=16)

    def restore():
        for k in s:
            s[k].copy_(start[k])
        for k in o:
            o[k].zero_()

    def results():
        torch.cuda.synchronize()
        return {k: v.clone().view(torch.uint8) for k, v in {**o, **s}.items()}

    def same(a, b):
        for k in a:                                # (rows of the empty request's q_lat are not defined)
            x, y = (r[k] if k != "q_lat" else r[k].view(B, -1)[:2] for r in (a, b))
            assert torch.equal(x, y), k
    restore()
    step()
    want = results()
    assert s["lens"].tolist() == [70, 100, 0]
    g = torch.cuda.CUDAGraph()
    restore()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        restore()
        g.replay()
        same(results(), want)
    restore()
    step()
    same(results(), want)


# ----------------------------------------------------------------------------- the largest batches

@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3"])
def test_key_weights_of_more_requests_than_the_cost_table_holds(kind):
    """Above 8192 requests the ranges are cut by tiles alone."""
    rng = np.random.default_rng(1)
    c = D.Cache(rng, kind, D.dims("v2", 16), list(rng.integers(0, 4, 8300)), max_pages=1)
    q_lat = D.draw(rng, (8300, 1, 16, 576), "bf16", 0.6)
    lse = rng.standard_normal((8300, 1, 16)).astype(np.float32)
    old = rng.random((8300, 64)).astype(np.float32)
    got = evict.weigh(c, 1, q_lat, lse, old, 0.5)
    evict.check_weights(c, 1, q_lat, lse, oracle.softmax_scale(128, 64), old, 0.5, got)


@pytest.mark.parametrize("B,q,L", [(32768, 1, 2), (32768, 1, 10), (8192, 4, 10)])
@pytest.mark.parametrize("act,shape", [("bf16", "v2"), ("f32", "tiny")])
def test_attend_of_the_largest_batch(act, shape, B, q, L):
    rng = np.random.default_rng(L)
    d = D.dims(shape, 1)
    x, lens = prefix.attend_inputs(rng, d, B, q, L, act, rng.integers(q, 3000, B))
    u, lse = prefix.attend(M.make_config(d, act, act), x, lens, act)
    prefix.check_attend(d, x, lens, act, u, lse)


@pytest.mark.parametrize("act,shape", [("bf16", "v2"), ("f32", "tiny"), ("bf16", "odd")])
def test_absorb_query_of_the_largest_batch(act, shape):
    rng = np.random.default_rng(2)
    d, B = D.dims(shape, 2), 32768
    qn, qp = D.draw(rng, (B, 1, 2, d.d_nope), act), D.draw(rng, (B, 1, 2, d.d_rope), act)
    W_abs = D.draw(rng, (2, d.d_nope, d.d_latent), act, d.d_latent ** -0.5)
    lens = rng.integers(1, 5000, B).astype(np.int32)
    out = torch.empty(B, 1, 2, d.d_latent + d.d_rope, dtype=D.torch_type(act), device="cuda")
    M.mla_absorb_query(M.make_config(d, act, act), D.dev(qn, act), D.dev(qp, act), D.dev(W_abs, act), D.dev(lens), out)
    lat = np.einsum("bthn,hnc->bthc", qn.astype(np.float64), W_abs.astype(np.float64))
    mag = np.einsum("bthn,hnc->bthc", np.abs(qn), np.abs(W_abs))
    pe = oracle.rope(qp.astype(np.float64), np.repeat(lens.astype(np.int64)[:, None, None] - 1, 2, 2))
    want = np.concatenate([lat, pe], -1)
    # fp32 sums of d_n products; sine and cosine to 2^-20 of values below 7; one rounding
    tol = D.EPS[act] * np.abs(want) * 1.01 + np.concatenate(
        [4 * d.d_nope * 2.0 ** -24 * mag, np.full(pe.shape, 7 * 2.0 ** -20)], -1)
    assert_within(out.double().cpu().numpy(), want, tol, "q_lat")


def test_output_proj_prefix_of_many_rows():
    """40000 rows on the tensor cores, against fp64 on the device."""
    H, rows = 2, 40000
    d = D.dims("v2", H)
    cfg, g = M.make_config(d, "bf16", "bf16"), torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    o, up, W_UV, W_O = rand(rows, H, 512, std=0.1), rand(rows, H, 128, std=0.1), rand(512, H * 128, std=512 ** -0.5), rand(H * 128, 5120, std=1 / 16)
    lse, lsep = rand(rows, H, std=3, dtype=torch.float32), rand(rows, H, std=3, dtype=torch.float32)
    out = torch.full((rows, 5120), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(M.mla_output_proj_prefix_workspace_size(cfg, rows), dtype=torch.uint8, device="cuda")
    M.mla_output_proj_prefix(cfg, o, lse, up, lsep, W_UV, W_O, out, ws)
    a = torch.sigmoid(lse.double() - lsep.double())[..., None]
    W = W_UV.double().view(512, H, 128)

    def joined(x, y, w):
        return a * torch.einsum("rhc,chv->rhv", x, w) + (1 - a) * y
    u = joined(o.double(), up.double(), W).view(rows, -1)
    mag_u = joined(o.double().abs(), up.double().abs(), W.abs()).view(rows, -1)
    O64 = W_O.double()
    want = u @ O64
    # u's rounding, its fp32 sums (weights to 2^-20), the projection's sums, the result's rounding
    tol = (2.0 ** -8 * u.abs() + (4 * 512 * 2.0 ** -24 + 2.0 ** -19) * mag_u) @ O64.abs() + \
        4 * H * 128 * 2.0 ** -24 * (u.abs() @ O64.abs()) + 2.0 ** -8 * want.abs()
    assert ((out.double() - want).abs() <= tol * 1.01).all()


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "new_pages"])
def test_evict_of_the_largest_batch(in_place):
    """32768 requests of three tokens down to two, pages of four tokens."""
    B, dims = 32768, D.dims("tiny", 16)
    dims.page_size = 4
    cfg, row = M.make_config(dims, "f32", "f32"), 80
    g = torch.Generator(device="cuda").manual_seed(4)
    pool = torch.randn(2 * B, 4, row, generator=g, device="cuda")
    perm = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32)
    table, new = perm[:B].view(B, 1).contiguous(), perm[B:].view(B, 1).contiguous()
    w = torch.rand(B, 4, generator=g, device="cuda")
    lens = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    kept, nl, before = torch.empty(B, 2, dtype=torch.int32, device="cuda"), torch.empty_like(lens), pool.clone()
    M.mla_evict_cache(cfg, w, lens, table, pool, 2, kept, nl, new_block_table=table if in_place else new, rotate=False)
    want = torch.sort(torch.topk(w[:, :3], 2).indices, 1).values
    assert (nl == 2).all() and torch.equal(kept, want.int())
    src = before[table[:, 0].long()[:, None], want]
    assert torch.equal(pool[(table if in_place else new)[:, 0].long(), :2], src)
