"""Key weights and cache eviction against fp64 references; rows that move are compared bit for
bit, turned rotary keys within their rounding."""
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


# ----------------------------------------------------------------------------- key weights

FORMATS = [("f32", "tiny", 16), ("bf16", "tiny", 16), ("bf16", "v2", 128), ("bf16", "v2", 16),
           ("fp8_e4m3", "v2", 128), ("fp8_e4m3_b128", "v2", 128), ("fp8_e4m3_b128", "v2", 32),
           ("f32", "v2", 4), ("bf16", "v2", 32), ("bf16", "v2", 48), ("fp8_e4m3", "v2", 32), ("fp8_e4m3", "v2", 64),
           ("bf16", "v2", 10), ("f32", "odd", 3), ("fp8_e4m3", "odd", 3), ("fp8_e4m3_b128", "odd128", 3)]
LENS = {1: (1, 63, 64, 65, 130, 700, 0), 2: (2, 3, 64, 129, 0, 517), 4: (4, 5, 127, 128, 300)}


def weigh(c, q_len, q_lat, lse, old, decay, status=None, table=None, lens=None):
    w = torch.from_numpy(old.copy()).cuda()
    M.mla_key_weights(c.config(), D.dev(q_lat, D.act_of(c.kind)), D.dev(lse), c.device(),
                      D.dev(c.table if table is None else table),
                      D.dev(np.asarray(c.lens if lens is None else lens, np.int32)), w, decay=decay,
                      dev_status=status)
    torch.cuda.synchronize()
    return w.cpu().numpy()


def weigh_inputs(rng, c, q_len):
    B, H, Dm = len(c.lens), c.d.num_heads, c.d.d_latent + c.d.d_rope
    q_lat = D.draw(rng, (B, q_len, H, Dm), D.act_of(c.kind), 0.6)
    scale = oracle.softmax_scale(c.d.d_nope, c.d.d_rope)
    lse = np.full((B, q_len, H), -np.inf, np.float32)
    for b, n in enumerate(c.lens):
        for t in range(q_len):
            if n:
                z = scale * (q_lat[b, t].astype(np.float64) @ c.values[b][: n - q_len + t + 1].T)
                lse[b, t] = np.log(np.exp(z).sum(1))
    return q_lat, lse, scale


def check_weights(c, q_len, q_lat, lse, scale, old, decay, got, skip=()):
    for b, n in enumerate(c.lens):
        if n == 0 or b in skip:
            assert np.array_equal(got[b], old[b], equal_nan=True)
            continue
        want, mag = ref.key_weights(q_lat[b], lse[b], c.values[b], old[b], q_len, scale, decay)
        # fp32 scores (sums of 576 products, and for block scales two terms of 2^-17), exponent
        # arithmetic to 2^-21 of its magnitude, then sums of H q_len terms
        Dm, H = c.d.d_latent + c.d.d_rope, c.d.num_heads
        rel = 2 * mag * (4 * Dm * 2.0 ** -24 + 2.0 ** -16 * (c.kind == "fp8_e4m3_b128")) + \
            2.0 ** -20 * (4 + np.abs(lse[b]).max()) + 4 * H * q_len * 2.0 ** -24
        assert_within(got[b, :n], want, rel * np.abs(want), f"weights of request {b}")
        assert np.array_equal(got[b, n:], old[b, n:], equal_nan=True), "entries behind the request"


@pytest.mark.parametrize("kind,shape,H", FORMATS)
@pytest.mark.parametrize("q_len,decay", [(1, 0.0), (2, 1.0), (4, 0.9)])
def test_key_weights(kind, shape, H, q_len, decay):
    rng = np.random.default_rng(q_len + H)
    c = D.Cache(rng, kind, D.dims(shape, H), LENS[q_len], max_pages=12)
    q_lat, lse, scale = weigh_inputs(rng, c, q_len)
    old = rng.random((len(c.lens), 12 * 64)).astype(np.float32)
    for b, n in enumerate(c.lens):                 # tokens never cached before hold garbage
        old[b, max(0, n - q_len):] = np.nan
        if decay == 0:
            old[b] = np.nan
    got = weigh(c, q_len, q_lat, lse, old, decay)
    check_weights(c, q_len, q_lat, lse, scale, old, decay, got)
    if decay == 0:                                 # the weights of a request share out H * q_len
        for b, n in enumerate(c.lens):
            if n:
                assert abs(got[b, :n].sum() - H * q_len) < 1e-3 * H * q_len
    assert np.array_equal(got, weigh(c, q_len, q_lat, lse, old, decay), equal_nan=True)   # same bits


@pytest.mark.parametrize("kind,shape,H", [("bf16", "tiny", 16), ("bf16", "v2", 128), ("fp8_e4m3", "v2", 128),
                                          ("fp8_e4m3_b128", "v2", 128)])
def test_key_weights_guards(kind, shape, H):
    rng = np.random.default_rng(2)
    c = D.Cache(rng, kind, D.dims(shape, H), (300, 200, 150, 90), max_pages=5)
    q_lat, lse, scale = weigh_inputs(rng, c, 1)
    old = rng.random((4, 320)).astype(np.float32)
    table = c.table.copy()
    table[0, 2], table[1, 0] = c.num_pages, -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # lengths: past the table's row, and negative
    got = weigh(c, 1, q_lat, lse, old, 1.0, status=status, table=table, lens=(300, 200, 321, -2))
    assert M.mla_read_device_status(status) == M.MLA_ERR_DEVICE_GUARD
    good = weigh(c, 1, q_lat, lse, old, 1.0, status=status)
    assert M.mla_read_device_status(status) == M.MLA_OK
    assert np.array_equal(got[0, :128], good[0, :128]) and np.array_equal(got[0, 192:], good[0, 192:])
    assert np.array_equal(got[0, 128:192], old[0, 128:192])
    assert np.array_equal(got[1, :64], old[1, :64]) and np.array_equal(got[1, 64:], good[1, 64:])
    assert np.array_equal(got[2:], old[2:])


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("lens", ["many", "few", "equal"])
def test_key_weights_shares_of_the_work(kind, lens):
    """More requests than SMs, few long ones, and equal ones (CTAs of their own)."""
    rng = np.random.default_rng(9)
    lens = {"many": [9000] + list(rng.integers(1, 140, 300)), "few": [9000, 130, 4100],
            "equal": [1500] * 20}[lens]
    c = D.Cache(rng, kind, D.dims("v2", 16), lens)
    q_lat, lse, scale = weigh_inputs(rng, c, 1)
    old = rng.random((len(lens), c.max_pages * 64)).astype(np.float32)
    got = weigh(c, 1, q_lat, lse, old, 0.5)
    check_weights(c, 1, q_lat, lse, scale, old, 0.5, got)


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("H,q_len", [(16, 4), (48, 4), (64, 3), (32, 6)])
def test_key_weights_several_tokens_over_long_runs(kind, H, q_len):
    """Several query tokens of requests longer than a run, which is passed over several times where
    their heads do not fit one product (one, two or three tokens a pass)."""
    rng = np.random.default_rng(12)
    c = D.Cache(rng, kind, D.dims("v2", H), [12000, 5001])
    q_lat, lse, scale = weigh_inputs(rng, c, q_len)
    old = rng.random((2, c.max_pages * 64)).astype(np.float32)
    got = weigh(c, q_len, q_lat, lse, old, 1.0)
    check_weights(c, q_len, q_lat, lse, scale, old, 1.0, got)


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
def test_key_weights_queries_of_any_magnitude(kind):
    """Heads of zeros, of tiny and of large values, and heads whose elements span 2^30."""
    rng = np.random.default_rng(15)
    c = D.Cache(rng, kind, D.dims("v2", 16), [200, 70])
    q_lat, lse, scale = weigh_inputs(rng, c, 1)
    size = np.ones((16, 1), np.float32)
    size[0], size[1], size[2], size[3] = 0.0, 2.0 ** -100, 2.0 ** 7, 2.0 ** -126
    q_lat = W.round_bf16(q_lat * size)
    spread = np.float32(2.0) ** -rng.integers(0, 30, q_lat[:, :, 4:8].shape)
    q_lat[:, :, 4:8] = W.round_bf16(q_lat[:, :, 4:8] * spread)
    for b, n in enumerate(c.lens):                 # the LSE of these scores, so that none overflows
        z = scale * (q_lat[b, 0].astype(np.float64) @ c.values[b].T)
        m = z.max(1)
        lse[b, 0] = m + np.log(np.exp(z - m[:, None]).sum(1))
    old = np.full((2, c.max_pages * 64), np.nan, np.float32)
    got = weigh(c, 1, q_lat, lse, old, 0.0)
    check_weights(c, 1, q_lat, lse, scale, old, 0.0, got)


@pytest.mark.parametrize("act,shape,H", [("f32", "tiny", 16), ("bf16", "v2", 128), ("bf16", "tiny", 16)])
def test_absorb_query(act, shape, H):
    rng = np.random.default_rng(4)
    d = D.dims(shape, H)
    B, q, lens = 3, 2, np.array([2, 900, 65], np.int32)
    qn, qp = D.draw(rng, (B, q, H, d.d_nope), act), D.draw(rng, (B, q, H, d.d_rope), act)
    W_UK = D.draw(rng, (d.d_latent, H * d.d_nope), act, d.d_latent ** -0.5)
    W_abs = np.stack([W_UK[:, h * d.d_nope: (h + 1) * d.d_nope].T for h in range(H)])
    out = torch.empty(B, q, H, d.d_latent + d.d_rope, dtype=D.torch_type(act), device="cuda")
    M.mla_absorb_query(M.make_config(d, act, act), D.dev(qn, act), D.dev(qp, act), D.dev(W_abs, act),
                       D.dev(lens), out)
    torch.cuda.synchronize()
    pos = lens[:, None] - q + np.arange(q)
    lat = np.einsum("bthn,hnc->bthc", qn.astype(np.float64), W_abs.astype(np.float64))
    mag = np.einsum("bthn,hnc->bthc", np.abs(qn), np.abs(W_abs))
    pe = oracle.rope(qp, np.repeat(pos[:, :, None], H, 2))
    want = np.concatenate([lat, pe], -1)
    tol = D.EPS[act] * np.abs(want) * 1.01 + np.concatenate(
        [4 * d.d_nope * 2.0 ** -24 * mag, np.full(pe.shape, 6 * 2.0 ** -20)], -1)
    assert_within(out.double().cpu().numpy(), want, tol, "q_lat")


# ----------------------------------------------------------------------------- eviction

def run_evict(c, weights, budget, sinks, recent, in_place=True, rotate=True, alias=False, new_pages=None,
              status=None, lens=None, table=None, new_table=None):
    """Returns the pool's bytes before and after, kept, the new lengths and weights, the new table."""
    table = c.table if table is None else table
    pool, B = c.device(), len(c.lens)
    before = c.back(pool).copy()
    w, ln, tab = torch.from_numpy(weights.copy()).cuda(), D.dev(np.asarray(lens if lens is not None else c.lens, np.int32)), D.dev(table)
    if in_place:
        new_table, ntab = table, tab
    else:
        ntab = D.dev(new_table)
    kept = torch.full((B, budget), 99, dtype=torch.int32, device="cuda")
    nw = w if alias else torch.full((B, new_table.shape[1] * 64), -3.0, device="cuda")
    nl = ln if alias else torch.full((B,), 99, dtype=torch.int32, device="cuda")
    M.mla_evict_cache(c.config(), w, ln, tab, pool, budget, kept, nl, new_block_table=ntab, new_weights=nw,
                      sinks=sinks, recent=recent, rotate=rotate, dev_status=status)
    torch.cuda.synchronize()
    return before, c.back(pool), kept.cpu().numpy(), nl.cpu().numpy(), nw.cpu().numpy(), new_table


def check_evict(c, weights, budget, sinks, recent, res, rotate=True, alias=False):
    before, after, kept, nl, nw, new_table = res
    dc, dr, kind = c.d.d_latent, c.d.d_rope, c.kind
    untouched = np.ones(before.shape[0], bool)
    pe0 = c.row - dr * {"f32": 4, "bf16": 2, "fp8_e4m3": 1, "fp8_e4m3_b128": 2}[kind]
    for b, S in enumerate(c.lens):
        keep = ref.evict_order(weights[b], S, budget, sinks, recent)
        n = len(keep)
        assert nl[b] == n and np.array_equal(kept[b, :n], keep) and (kept[b, n:] == -1).all()
        old_w = weights[b] if alias else np.full(nw.shape[1], -3.0, np.float32)
        assert np.array_equal(nw[b, :n], weights[b, keep], equal_nan=True)
        assert np.array_equal(nw[b, n:], old_w[n: nw.shape[1]], equal_nan=True)
        src, dst = c.slots(b, S)[keep], c.slots(b, n, new_table)
        untouched[dst] = False
        assert np.array_equal(after[dst, :pe0], before[src, :pe0]), f"latents of request {b}"
        delta = np.arange(n) - keep
        still = delta == 0 if rotate else np.ones(n, bool)
        assert np.array_equal(after[dst][still, pe0:], before[src][still, pe0:])
        a, o = (np.ascontiguousarray(x[~still][:, pe0:]) for x in (after[dst], before[src]))
        if kind == "fp8_e4m3":
            y, codes = ref.turn_codes(o, delta[~still])
            got = oracle.e4m3_decode(a)
            # the nearest code, or its neighbour where the turned value is within the arithmetic's
            # 2^-18 of the middle between two
            near = np.abs(oracle.e4m3_decode(codes) - np.clip(y, -448, 448))
            assert (np.abs(got - np.clip(y, -448, 448)) <= near + 448 * 2.0 ** -18).all()
        else:
            f32 = kind == "f32"
            o, a = ((x.view(np.float32) if f32 else
                     (x.view(np.uint16).astype(np.uint32) << 16).view(np.float32)) for x in (o, a))
            y = ref.turn_rows(o.astype(np.float64), delta[~still])
            size = np.abs(o).max() if o.size else 0.0
            # sine and cosine to 2^-20 (fp32: the angle's 2^-23 and sincosf), then one rounding
            tol = D.EPS[D.act_of(kind)] * np.abs(y) * 1.01 + 4 * size * (2.0 ** -22 if f32 else 2.0 ** -20)
            assert_within(a, y, tol, f"rotary keys of request {b}")
    assert np.array_equal(after[untouched], before[untouched]), "rows that no request owns"


def fresh_table(c, lens, budget):
    """New pages for every request out of the pool's spare ones."""
    need = [-(-min(n, budget) // 64) for n in lens]
    t = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = c.spare[at: at + n]
        at += n
    return t


KINDS = [("f32", "tiny"), ("bf16", "tiny"), ("bf16", "v2"), ("fp8_e4m3", "tiny"), ("fp8_e4m3", "v2"),
         ("fp8_e4m3_b128", "v2"), ("f32", "odd"), ("bf16", "odd"), ("fp8_e4m3", "odd"), ("fp8_e4m3_b128", "odd128")]
EVICT_LENS = (700, 1, 65, 0, 200, 333, 64, 129)


def draw_weights(rng, B, width, how):
    w = np.exp(1.5 * rng.standard_normal((B, width))).astype(np.float32)
    if how == "ties":
        w = np.round(w).astype(np.float32)         # a handful of values, many zeros
    if how == "equal":
        w[:] = 1.25
    if how == "odd":                               # NaN, infinities, both zeros, negatives
        w[:, ::7], w[:, 1::7], w[:, 2::7] = np.nan, np.inf, -np.inf
        w[:, 3::7], w[:, 4::7], w[:, 5::7] = 0.0, -0.0, -w[:, 5::7]
    return w


@pytest.mark.parametrize("kind,shape", KINDS)
@pytest.mark.parametrize("how,budget,sinks,recent", [("plain", 130, 4, 20), ("ties", 65, 0, 0), ("odd", 100, 1, 7),
                                                     ("equal", 64, 3, 61), ("plain", 1, 0, 0), ("ties", 700, 4, 9)])
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "new_pages"])
def test_evict(kind, shape, how, budget, sinks, recent, in_place):
    rng = np.random.default_rng(budget + sinks)
    c = D.Cache(rng, kind, D.dims(shape, 16), EVICT_LENS, max_pages=13, spare=40)
    w = draw_weights(rng, len(c.lens), 13 * 64, how)
    table = None if in_place else fresh_table(c, c.lens, budget)
    res = run_evict(c, w, budget, sinks, recent, in_place=in_place, new_table=table)
    check_evict(c, w, budget, sinks, recent, res)


@pytest.mark.parametrize("kind,shape", [("bf16", "v2"), ("fp8_e4m3_b128", "v2"), ("f32", "tiny")])
def test_evict_in_its_own_arrays_without_turning(kind, shape):
    rng = np.random.default_rng(6)
    c = D.Cache(rng, kind, D.dims(shape, 16), (900, 500, 40, 0))
    w = draw_weights(rng, 4, c.max_pages * 64, "plain")
    res = run_evict(c, w, 300, 4, 250, alias=True, rotate=False)
    check_evict(c, w, 300, 4, 250, res, rotate=False, alias=True)


@pytest.mark.parametrize("S", [20000, 70000, 140001])
@pytest.mark.parametrize("how", ["plain", "ties"])
def test_evict_long_requests(S, how):
    rng = np.random.default_rng(S)
    c = D.Cache(rng, "bf16", D.dims("tiny", 16), (S, 300, S // 3))
    w = draw_weights(rng, 3, c.max_pages * 64, how)
    for budget, sinks, recent in ((S // 2, 4, 5000), (777, 0, 0)):
        res = run_evict(c, w, budget, sinks, recent, alias=True)
        check_evict(c, w, budget, sinks, recent, res, alias=True)


@pytest.mark.parametrize("kind,shape", [("bf16", "v2"), ("f32", "tiny")])
def test_evict_guards(kind, shape):
    rng = np.random.default_rng(13)
    c = D.Cache(rng, kind, D.dims(shape, 16), (300, 300, 300, 300), spare=20)
    w = draw_weights(rng, 4, c.max_pages * 64, "plain")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cap = c.max_pages * 64
    before, after, kept, nl, nw, _ = run_evict(c, w, 100, 2, 5, status=status, lens=(300, cap + 1, -1, 0))
    assert M.mla_read_device_status(status) == M.MLA_ERR_DEVICE_GUARD
    assert list(nl) == [100, cap + 1, -1, 0] and (kept[1:] == -1).all()
    assert np.array_equal(after[c.slots(1, 300)], before[c.slots(1, 300)])
    keep = ref.evict_order(w[0], 300, 100, 2, 5)
    assert np.array_equal(kept[0], keep)
    # new pages too few for the kept tokens: the request is left alone
    new = c.spare[:4].reshape(4, 1).astype(np.int32)
    before, after, kept, nl, nw, _ = run_evict(c, w, 100, 2, 5, status=status, in_place=False, new_table=new)
    assert M.mla_read_device_status(status) == M.MLA_ERR_DEVICE_GUARD
    assert np.array_equal(after, before) and (kept == -1).all() and list(nl) == [300] * 4
    # a bad old page and a bad new page: their rows stay, the rest moves
    new = fresh_table(c, c.lens, 100)
    table = c.table.copy()
    table[0, 1], new[1, 0] = c.num_pages + 5, -1
    before, after, kept, nl, nw, _ = run_evict(c, w, 100, 2, 5, status=status, in_place=False, table=table,
                                               new_table=new, rotate=False)
    assert M.mla_read_device_status(status) == M.MLA_ERR_DEVICE_GUARD
    same = np.ones(before.shape[0], bool)
    for b in range(4):
        keep = ref.evict_order(w[b], 300, 100, 2, 5)
        i = np.arange(100)
        ok = ~((b == 0) & (keep // 64 == 1)) & ~((b == 1) & (i // 64 == 0))
        src, dst = c.slots(b, 300)[keep][ok], new[b][i // 64].astype(np.int64)[ok] * 64 + (i % 64)[ok]
        assert np.array_equal(after[dst], before[src])
        same[dst] = False
    assert np.array_equal(after[same], before[same])


# ----------------------------------------------------------------------------- the calls together

@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3_b128"])
def test_decode_weigh_evict_decode(kind):
    """A serving loop over its budget: decode, accumulate weights, evict, append, decode again; the
    second decode equals the attention over the kept rows, turned to their new places."""
    rng = np.random.default_rng(31)
    H, lens, budget = 128, [300, 64, 130], 100
    d = D.dims("v2", H)
    c = D.Cache(rng, kind, d, lens)
    cfg, B = c.config(), 3
    W_abs = D.draw(rng, (H, 128, 512), "bf16", 512 ** -0.5)
    qn, qp = D.draw(rng, (B, 1, H, 128), "bf16"), D.draw(rng, (B, 1, H, 64), "bf16")
    pool, tab, ln = c.device(), D.dev(c.table), D.dev(np.array(lens, np.int32))
    qd, qpd, wd = D.dev(qn, "bf16"), D.dev(qp, "bf16"), D.dev(W_abs, "bf16")
    ws = torch.empty(M.mla_decode_workspace_size(cfg, B, 1), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(B, 1, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, H, device="cuda")
    q_lat = torch.empty(B, 1, H, 576, dtype=torch.bfloat16, device="cuda")
    w = torch.full((B, c.max_pages * 64), float("nan"), device="cuda")
    M.mla_decode(cfg, qd, qpd, wd, pool, tab, ln, o, lse, ws)
    M.mla_absorb_query(cfg, qd, qpd, wd, ln, q_lat)
    M.mla_key_weights(cfg, q_lat, lse, pool, tab, ln, w, decay=0.0)
    got = w.cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):                   # the decode's own LSE: the weights share out H
        assert abs(got[b, :n].sum() / H - 1) < 1e-2
    kept = torch.empty(B, budget, dtype=torch.int32, device="cuda")
    M.mla_evict_cache(cfg, w, ln, tab, pool, budget, kept, ln, new_weights=w, sinks=4, recent=16)
    nl = ln.cpu().numpy()
    assert list(nl) == [100, 64, 100]
    M.mla_decode(cfg, qd, qpd, wd, pool, tab, ln, o, lse, ws)
    torch.cuda.synchronize()
    out, k = o.double().cpu().numpy(), kept.cpu().numpy()
    scale = oracle.softmax_scale(128, 64)
    for b in range(B):
        keep = k[b, : nl[b]]
        assert np.array_equal(keep, ref.evict_order(got[b].astype(np.float32), lens[b], budget, 4, 16))
        rows = c.values[b][keep]
        pe = oracle.rope(rows[:, 512:], np.arange(nl[b]) - keep)
        want, wl = oracle.decode_absorbed(rows[:, :512], pe, qn[b], qp[b], W_abs.astype(np.float64), scale)
        assert np.abs(out[b] - want).max() <= 1e-2 * np.abs(want).max() + 1e-3
        assert np.abs(lse[b].double().cpu().numpy() - wl).max() <= 1e-2 * np.abs(wl).max() + 1e-3
