"""Page keys, page scores, page selection and the decode over chosen pages against fp64 references."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
from oracle import pages as ref
from tests import serving_data as D

pytestmark = pytest.mark.gpu
assert_within = D.assert_within
P = D.PAGE


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M.lib()


def i32(x):
    return D.dev(np.asarray(x, np.int32))


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


FORMATS = [("f32", "tiny", 16), ("bf16", "tiny", 16), ("bf16", "v2", 128), ("bf16", "v2", 16), ("bf16", "v2", 48),
           ("bf16", "v2", 96), ("fp8_e4m3", "v2", 128), ("fp8_e4m3", "v2", 32), ("fp8_e4m3_b128", "v2", 128),
           ("fp8_e4m3_b128", "v2", 80), ("f32", "v2", 4), ("bf16", "v2", 10), ("f32", "odd", 3),
           ("fp8_e4m3", "odd", 3), ("fp8_e4m3_b128", "odd128", 3)]
LENS = {1: (1, 63, 64, 65, 130, 700, 0), 2: (2, 3, 64, 129, 0, 517), 4: (4, 5, 127, 128, 300)}


# ----------------------------------------------------------------------------- page keys

def make_keys(c, lens=None, new=None, table=None, st=None, pool=None, before=None):
    Dm = c.d.d_latent + c.d.d_rope
    if before is None:
        before = np.full((c.num_pages, Dm), 7.0, np.float32)
    k = D.dev(before, D.act_of(c.kind))
    M.mla_page_keys(c.config(), c.device() if pool is None else pool, i32(c.table if table is None else table),
                    i32(c.lens if lens is None else lens), k, new_tokens=new, dev_status=st)
    torch.cuda.synchronize()
    return k.double().cpu().numpy()


def check_keys(c, got, new=None, skip=()):
    touched = set()
    for b, n in enumerate(c.lens):
        if n == 0 or b in skip:
            continue
        want, mag = ref.page_keys(c.values[b], P)
        first = 0 if new is None else max(0, n - new) // P
        ids = c.table[b, first: -(-n // P)]
        # fp32 sums of up to 64 values, the scales' products and the division, one rounding
        tol = D.EPS[D.act_of(c.kind)] * np.abs(want) * 1.01 + 70 * 2.0 ** -24 * mag
        assert_within(got[ids], want[first:], tol[first:], f"page keys of request {b}")
        touched.update(ids.tolist())
    rest = [p for p in range(c.num_pages) if p not in touched]
    assert (got[rest] == 7.0).all(), "pages that were not to be written"


@pytest.mark.parametrize("kind,shape,H", [f for f in FORMATS if f[2] in (16, 128, 3, 4, 10, 32)])
@pytest.mark.parametrize("new", [None, 1, 2, 65])
def test_page_keys(kind, shape, H, new):
    rng = np.random.default_rng(H)
    c = D.Cache(rng, kind, D.dims(shape, H), LENS[1], max_pages=12)
    check_keys(c, make_keys(c, new=new), new)


def test_page_keys_guards_and_addresses():
    rng = np.random.default_rng(5)
    for kind, shape in (("bf16", "v2"), ("fp8_e4m3_b128", "v2"), ("f32", "tiny")):
        c = D.Cache(rng, kind, D.dims(shape, 16), (300, 200, 150, 90), max_pages=5)
        table, st = c.table.copy(), status()
        table[0, 2], table[1, 0] = c.num_pages, -7
        got = make_keys(c, lens=(300, 200, 321, -2), table=table, st=st)
        assert M.mla_read_device_status(st) == M.MLA_ERR_DEVICE_GUARD
        good = make_keys(c, st=st)
        assert M.mla_read_device_status(st) == M.MLA_OK
        check_keys(c, good)
        left = [c.table[0, 2], c.table[1, 0], *c.table[2, :3], *c.table[3, :2]]
        assert (got[left] == 7.0).all()
        same = [p for p in range(c.num_pages) if p not in left]
        assert np.array_equal(got[same], good[same])
        # a cache four bytes behind a 16-byte boundary (read by words: rows are summed in another order)
        pool = c.device()
        check_keys(c, make_keys(c, pool=D.shifted(pool, 4 // pool.element_size())))


# ----------------------------------------------------------------------------- page scores

def draw_query(rng, c, q_len, std=0.6):
    return D.draw(rng, (len(c.lens), q_len, c.d.num_heads, c.d.d_latent + c.d.d_rope), D.act_of(c.kind), std)


def draw_keys(rng, c):
    return D.draw(rng, (c.num_pages, c.d.d_latent + c.d.d_rope), D.act_of(c.kind), 0.4)


def score(c, q_lat, keys, lens=None, table=None, st=None, shift=()):
    B, q_len = q_lat.shape[:2]
    cfg, act = c.config(), D.act_of(c.kind)
    out = torch.full((B, q_len, c.max_pages), 7.0, device="cuda")
    n = M.mla_page_scores_workspace_size(cfg, B, q_len, c.max_pages)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
    q, k = D.dev(q_lat, act), D.dev(keys, act)
    q, k = (D.shifted(q) if "q" in shift else q), (D.shifted(k) if "k" in shift else k)
    M.mla_page_scores(cfg, q, k, i32(c.table if table is None else table), i32(c.lens if lens is None else lens), out,
                      ws if n else None, dev_status=st)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def check_scores(c, q_lat, keys, got, skip=()):
    q_len, H = q_lat.shape[1], c.d.num_heads
    scale = oracle.softmax_scale(c.d.d_nope, c.d.d_rope)
    Dm = c.d.d_latent + c.d.d_rope
    for b, n in enumerate(c.lens):
        for t in range(q_len):
            if n == 0 or b in skip:
                assert (got[b, t] == 7.0).all()
                continue
            see = n - q_len + t + 1
            pages = -(-see // P)
            want, lse, mag = ref.page_scores(q_lat[b, t], keys[c.table[b, :pages]], see, P, scale)
            # fp32 scores (sums of D products), exponents' arithmetic to 2^-21 of their magnitude, sums of
            # pages and of heads
            rel = 2 * mag * 4 * Dm * 2.0 ** -24 + 2.0 ** -20 * (4 + np.abs(lse).max()) + (4 * H + pages) * 2.0 ** -24
            assert_within(got[b, t, :pages], want, rel * np.abs(want), f"scores of request {b}, token {t}")
            assert (got[b, t, pages:] == 7.0).all(), "entries behind the query's pages"


@pytest.mark.parametrize("kind,shape,H", [f for f in FORMATS if not f[0].startswith("fp8") or f[1] == "odd"])
@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_page_scores(kind, shape, H, q_len):
    rng = np.random.default_rng(q_len + H)
    c = D.Cache(rng, kind, D.dims(shape, H), LENS[q_len], max_pages=12)
    q_lat, keys = draw_query(rng, c, q_len), draw_keys(rng, c)
    got = score(c, q_lat, keys)
    check_scores(c, q_lat, keys, got)
    assert np.array_equal(got, score(c, q_lat, keys))              # the same bits every time


class Tables:
    """What the scores and the selection read of a cache: long requests without the rows."""

    def __init__(self, rng, kind, d, lens, max_pages):
        self.kind, self.d, self.lens, self.max_pages = kind, d, list(lens), max_pages
        pages = [-(-n // P) for n in lens]
        self.num_pages = sum(pages) + 2
        perm = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at: at + n]
            at += n

    def config(self):
        return M.make_config(self.d, D.act_of(self.kind), self.kind)


@pytest.mark.parametrize("H,q_len,pages", [(128, 1, 129), (128, 1, 1025), (64, 2, 2500), (128, 1, 4100), (16, 1, 9000)])
def test_page_scores_of_long_requests(H, q_len, pages):
    """One tile of pages and one page more, several tiles of a block, and more than a cluster holds."""
    rng = np.random.default_rng(pages)
    lens = (pages * P, pages * P // 3 + 5, 70)
    c = Tables(rng, "bf16", D.dims("v2", H), lens, pages + 3)
    q_lat, keys = draw_query(rng, c, q_len, 1.2), draw_keys(rng, c)
    check_scores(c, q_lat, keys, score(c, q_lat, keys))


@pytest.mark.parametrize("kind,shape,H", [("bf16", "v2", 128), ("f32", "tiny", 16)])
def test_page_scores_guards_infinities_and_addresses(kind, shape, H):
    rng = np.random.default_rng(9)
    c = D.Cache(rng, kind, D.dims(shape, H), (300, 200, 150, 90), max_pages=5)
    q_lat, keys = draw_query(rng, c, 1), draw_keys(rng, c)
    good = score(c, q_lat, keys)
    check_scores(c, q_lat, keys, good)
    table, st = c.table.copy(), status()
    table[0, 2] = c.num_pages
    got = score(c, q_lat, keys, lens=(300, 200, 321, -2), table=table, st=st)
    assert M.mla_read_device_status(st) == M.MLA_ERR_DEVICE_GUARD
    assert (got[2:] == 7.0).all() and np.array_equal(got[1], good[1])
    assert got[0, 0, 2] == 0.0 and abs(got[0, 0, :5].sum() - H) < 1e-3 * H
    for shift in (("q",), ("k",), ("q", "k")):
        check_scores(c, q_lat, keys, score(c, q_lat, keys, shift=shift))
    # pages that no request names may hold anything; scores far apart
    bad = keys.copy()
    used = set(c.table[c.table >= 0].tolist())
    bad[[p for p in range(c.num_pages) if p not in used]] = np.nan
    assert np.array_equal(good, score(c, q_lat, bad))
    far = q_lat * 64
    check_scores(c, far, keys, score(c, far, keys))


# ----------------------------------------------------------------------------- selection

def select(c, scores, lens, q_len, budget, sinks, recent, st=None):
    pages = torch.full((scores.shape[0], q_len, budget), 99, dtype=torch.int32, device="cuda")
    M.mla_select_pages(c.config(), D.dev(scores), i32(lens), pages, sinks=sinks, recent=recent, dev_status=st)
    torch.cuda.synchronize()
    return pages.cpu().numpy()


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 1), (1, 0, 0), (5, 1, 2), (8, 8, 0), (16, 4, 4), (64, 1, 2),
                                                 (700, 2, 3), (2100, 0, 1)])
@pytest.mark.parametrize("what", ["normal", "ties", "nan"])
def test_select_pages(q_len, budget, sinks, recent, what):
    rng = np.random.default_rng(budget)
    pages = 2048
    c = Tables(rng, "bf16", D.dims("v2", 16), (1,), pages)
    lens = (0, 3, 64, 65, 130, 5 * P, 64 * P, 64 * P + 1, 777 * P - 9, 2048 * P)
    s = rng.standard_normal((len(lens), q_len, pages)).astype(np.float32)
    if what == "ties":
        s = np.round(s).astype(np.float32) * np.where(rng.random(s.shape) < 0.3, -0.0, 1.0).astype(np.float32)
    if what == "nan":
        s = np.where(rng.random(s.shape) < 0.4, rng.choice([np.nan, -np.nan, np.inf, -np.inf], s.shape), s).astype(np.float32)
    st = status()
    got = select(c, s, lens, q_len, budget, sinks, recent, st)
    assert M.mla_read_device_status(st) == M.MLA_OK
    for b, n in enumerate(lens):
        for t in range(q_len):
            see = n - q_len + t + 1 if n else 0
            want = ref.select_pages(s[b, t], -(-see // P), budget, sinks, recent)
            assert np.array_equal(got[b, t], want), (b, t)


def test_select_pages_of_the_longest_rows_and_guards():
    rng = np.random.default_rng(4)
    c = Tables(rng, "bf16", D.dims("v2", 16), (1,), 49152)
    s = rng.random((2, 1, 49152)).astype(np.float32)
    s[1] = 0.5
    got = select(c, s, (49152 * P, 49152 * P - 64), 1, 3000, 5, 7)
    for b, n in enumerate((49152, 49151)):
        assert np.array_equal(got[b, 0], ref.select_pages(s[b, 0], n, 3000, 5, 7))
    st = status()
    got = select(c, s, (-1, 49152 * P + 1), 1, 10, 1, 1, st)
    assert M.mla_read_device_status(st) == M.MLA_ERR_DEVICE_GUARD and (got == -1).all()
    got = select(c, s.repeat(2, 1), (1, 5), 2, 10, 1, 1, st)
    assert M.mla_read_device_status(st) == M.MLA_ERR_DEVICE_GUARD and (got[0] == -1).all() and got[1, 1, 0] == 0


# ----------------------------------------------------------------------------- decode over pages

def lists(rng, c, q_len, budget, how="random"):
    out = np.full((len(c.lens), q_len, budget), -1, np.int32)
    for b, n in enumerate(c.lens):
        for t in range(q_len):
            seen = -(-(n - q_len + t + 1) // P) if n else 0
            if how == "empty" and (b + t) % 2:
                continue
            k = min(budget, seen) if how != "short" else min(budget, seen, 1 + (b + t) % 3)
            keep = rng.choice(seen, k, replace=False) if seen else []
            if how == "own" and seen and seen - 1 not in keep:
                keep[0] = seen - 1
            out[b, t, :k] = np.sort(keep)
    return out


def attend(c, q_lat, pages, lens=None, table=None, pool=None, shift=(), ws=None):
    B, q_len, H = q_lat.shape[:3]
    cfg, act = c.config(), D.act_of(c.kind)
    o = torch.full((B, q_len, H, c.d.d_latent), 7.0, dtype=D.torch_type(act), device="cuda")
    o = D.shifted(o) if "o" in shift else o
    lse = torch.full((B, q_len, H), 7.0, device="cuda")
    n = M.mla_decode_pages_workspace_size(cfg, B, q_len, pages.shape[2])
    if ws is None:
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    q, pool = D.dev(q_lat, act), c.device() if pool is None else pool
    q = D.shifted(q) if "q" in shift else q
    pool = D.shifted(pool, 4 // pool.element_size()) if "cache" in shift else pool
    M.mla_decode_pages(cfg, q, pool, i32(c.table if table is None else table), i32(c.lens if lens is None else lens),
                       i32(pages), o, lse, ws)
    torch.cuda.synchronize()
    return o.double().cpu().numpy(), lse.cpu().numpy(), M.mla_read_device_status(ws)


def check_attend(c, q_lat, pages, got, lse, skip=()):
    q_len, dc, H = q_lat.shape[1], c.d.d_latent, c.d.num_heads
    scale = oracle.softmax_scale(c.d.d_nope, c.d.d_rope)
    Dm = dc + c.d.d_rope
    act = D.act_of(c.kind)
    for b, n in enumerate(c.lens):
        for t in range(q_len):
            if b in skip:
                continue
            see = n - q_len + t + 1 if n else 0
            want, wl, mag, wmag = ref.attend_pages(q_lat[b, t], c.values[b], pages[b, t], see, P, dc, scale)
            if not np.isfinite(wl).any():
                assert (got[b, t] == 0).all() and np.isneginf(lse[b, t]).all()
                continue
            # fp32 scores: sums of D products, and an fp8 query's two terms (2^-19); exponents to 2^-21
            dz = mag * (4 * Dm * 2.0 ** -24 + 2.0 ** -18 * c.kind.startswith("fp8"))
            tok = P * pages.shape[2]
            assert_within(lse[b, t], wl, dz + 2.0 ** -20 * (4 + np.abs(wl)) + tok * 2.0 ** -24, f"lse {b} {t}")
            # the softmax's weights in 16 bits (bf16; fp8: two e4m3 terms, at most that), then sums of fp32
            soft = (2.0 ** -8 if act == "bf16" else 0.0) + 2 * dz + 2.0 ** -19 * (4 + np.abs(wl).max()) + 2 * tok * 2.0 ** -24
            assert_within(got[b, t], want, D.EPS[act] * np.abs(want) * 1.01 + soft * wmag + low_weights(c, b, pages[b, t], see),
                          f"output {b} {t}")


def low_weights(c, b, pages, see):
    """Of an fp8 cache the weights P are two e4m3 terms, off by up to 2^-10 where that exceeds 2^-8 P, and
    the largest P is at least 16: 2^-14 of the sum's total for each token (block scales: P times the scale,
    at least 16 for the largest scale)."""
    if not c.kind.startswith("fp8"):
        return 0.0
    at = np.concatenate([np.arange(p * P, min(see, p * P + P)) for p in pages if p >= 0])
    x = np.abs(c.values[b][at][:, : c.d.d_latent])
    if c.kind == "fp8_e4m3_b128":
        s = x.reshape(len(at), -1, 128).max(2)
        x = x * np.repeat(np.where(s > 0, s.max() / np.where(s > 0, s, 1.0), 0.0), 128, 1)
    return 2.0 ** -14 * x.sum(0)


@pytest.mark.parametrize("kind,shape,H", FORMATS)
@pytest.mark.parametrize("q_len,budget,how", [(1, 4, "random"), (1, 1, "own"), (2, 12, "own"), (4, 3, "short"),
                                              (2, 5, "empty")])
def test_decode_pages(kind, shape, H, q_len, budget, how):
    rng = np.random.default_rng(q_len + H + budget)
    c = D.Cache(rng, kind, D.dims(shape, H), LENS[q_len], max_pages=12)
    q_lat, pages = draw_query(rng, c, q_len), lists(rng, c, q_len, budget, how)
    got, lse, st = attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check_attend(c, q_lat, pages, got, lse)
    again = attend(c, q_lat, pages)
    assert np.array_equal(got, again[0]) and np.array_equal(lse, again[1])


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("B,n,budget,H", [(1, 6000, 64, 128), (3, 9000, 141, 128), (40, 1500, 24, 128), (7, 4096, 33, 64),
                                          (200, 300, 5, 128)])
def test_decode_pages_split_over_workers(kind, B, n, budget, H):
    rng = np.random.default_rng(B)
    c = D.Cache(rng, kind, D.dims("v2", H), [n - 27 * (b % 11) for b in range(B)])
    q_lat, pages = draw_query(rng, c, 1), lists(rng, c, 1, budget, "own")
    got, lse, st = attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check_attend(c, q_lat, pages, got, lse)


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("std", [6.0, 0.0])
def test_decode_pages_of_far_and_of_equal_scores(kind, std):
    """Scores that grow along the request, so that the running maximum keeps rising, and no scores."""
    rng = np.random.default_rng(7)
    c = D.Cache(rng, kind, D.dims("v2", 128), (2000, 640))
    q_lat = draw_query(rng, c, 1, std)
    pages = lists(rng, c, 1, 32, "random")
    got, lse, st = attend(c, q_lat, pages)
    assert st == M.MLA_OK
    check_attend(c, q_lat, pages, got, lse)


@pytest.mark.parametrize("kind,shape,H", [("f32", "tiny", 16), ("bf16", "v2", 128), ("fp8_e4m3", "v2", 128),
                                          ("fp8_e4m3_b128", "v2", 128)])
def test_decode_pages_guards(kind, shape, H):
    rng = np.random.default_rng(3)
    c = D.Cache(rng, kind, D.dims(shape, H), (300, 200, 150, 90, 400), max_pages=8)
    q_lat, pages = draw_query(rng, c, 1), lists(rng, c, 1, 4, "own")
    good = attend(c, q_lat, pages)
    check_attend(c, q_lat, pages, *good[:2])
    for what in ("page", "order", "twice", "behind", "length"):
        table, lens, bad = c.table.copy(), list(c.lens), pages.copy()
        if what == "page":
            table[1, bad[1, 0, 0]] = c.num_pages + 3
        elif what == "order":
            bad[1, 0, :2] = (2, 1)
        elif what == "twice":
            bad[1, 0, :2] = (1, 1)
        elif what == "behind":
            bad[1, 0] = (0, 1, 4, -1)
        else:
            lens[1] = 8 * P + 1
        got, lse, st = attend(c, q_lat, bad, table=table, lens=lens)
        assert st == M.MLA_ERR_DEVICE_GUARD, what
        rest = [0, 2, 3, 4]
        check_attend(c, q_lat, pages, got, lse, skip=(1,))
        assert np.array_equal(lse[rest], good[1][rest]) or kind != "f32"
        if what == "length":
            assert (got[1] == 0).all() and np.isneginf(lse[1]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8_e4m3", "fp8_e4m3_b128"])
@pytest.mark.parametrize("shift", [("q",), ("cache",), ("o",), ("q", "cache", "o")])
def test_decode_pages_off_16_bytes(kind, shift):
    rng = np.random.default_rng(11)
    c = D.Cache(rng, kind, D.dims("v2", 16), (300, 70))
    q_lat, pages = draw_query(rng, c, 1), lists(rng, c, 1, 3, "own")
    got, lse, st = attend(c, q_lat, pages, shift=shift)
    assert st == M.MLA_OK
    check_attend(c, q_lat, pages, got, lse)


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("kind,H", [("bf16", 128), ("fp8_e4m3_b128", 128), ("fp8_e4m3", 64)])
def test_sparse_steps_captured(kind, H):
    """Append, summarise, score, select and attend as steps would, in one graph replayed over two
    steps: each step against the references on what was cached by then."""
    rng = np.random.default_rng(21)
    d = D.dims("v2", H)
    c = D.Cache(rng, kind, d, (700, 64, 1000, 127), max_pages=20)
    B, budget, dc, dr = 4, 6, 512, 64
    cfg, pool, lens = c.config(), c.device(), i32(c.lens)
    for b in range(B):                              # pages for the tokens to come
        n = -(-c.lens[b] // P)
        c.table[b, n] = c.spare[b]
    table = i32(c.table)
    act = torch.bfloat16
    keys = torch.zeros(c.num_pages, dc + dr, dtype=act, device="cuda")
    M.mla_page_keys(cfg, pool, table, lens, keys)
    W_abs = D.dev(D.draw(rng, (H, d.d_nope, dc), "bf16", dc ** -0.5), "bf16")
    new_c, new_k = torch.zeros(B, dc, dtype=act, device="cuda"), torch.zeros(B, dr, dtype=act, device="cuda")
    qn = torch.zeros(B, 1, H, d.d_nope, dtype=act, device="cuda")
    qp = torch.zeros(B, 1, H, dr, dtype=act, device="cuda")
    q_lat = torch.zeros(B, 1, H, dc + dr, dtype=act, device="cuda")
    scores = torch.zeros(B, 1, 20, device="cuda")
    pages = torch.zeros(B, 1, budget, dtype=torch.int32, device="cuda")
    o, lse = torch.zeros(B, 1, H, dc, dtype=act, device="cuda"), torch.zeros(B, 1, H, device="cuda")
    req, pos = i32(range(B)), torch.zeros(B, dtype=torch.int32, device="cuda")
    ws_s = torch.zeros(max(1, M.mla_page_scores_workspace_size(cfg, B, 1, 20)), dtype=torch.uint8, device="cuda")
    ws_d = torch.zeros(M.mla_decode_pages_workspace_size(cfg, B, 1, budget), dtype=torch.uint8, device="cuda")
    st = status()

    def step():
        pos.copy_(lens)
        lens.add_(1)
        M.mla_append_cache_latent(cfg, new_c, new_k, req, pos, table, pool, dev_status=st)
        M.mla_page_keys(cfg, pool, table, lens, keys, new_tokens=1, dev_status=st)
        M.mla_absorb_query(cfg, qn, qp, W_abs, lens, q_lat)
        M.mla_page_scores(cfg, q_lat, keys, table, lens, scores, ws_s, dev_status=st)
        M.mla_select_pages(cfg, scores, lens, pages, sinks=1, recent=2, dev_status=st)
        M.mla_decode_pages(cfg, q_lat, pool, table, lens, pages, o, lse, ws_d)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = pool.clone(), lens.clone(), keys.clone()
    with torch.cuda.stream(s):
        step()                                      # warm-up
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    pool.copy_(keep[0]), lens.copy_(keep[1]), keys.copy_(keep[2])
    for k in range(2):
        for x, std in ((new_c, 1.0), (new_k, 1.0), (qn, 0.6), (qp, 0.6)):
            x.copy_(D.dev(D.draw(rng, tuple(x.shape), "bf16", std), "bf16"))
        g.replay()
        torch.cuda.synchronize()
        assert M.mla_read_device_status(st) == M.MLA_OK and M.mla_read_device_status(ws_d) == M.MLA_OK
        now = [n + k + 1 for n in c.lens]
        raw = c.back(pool)
        q, sc, pg = (x.double().cpu().numpy() for x in (q_lat, scores, pages))
        kk = keys.double().cpu().numpy()
        view = D.Cache.__new__(D.Cache)
        view.__dict__.update(c.__dict__, lens=now, values=[])
        for b in range(B):                          # the rows as they are cached now
            rows = raw[c.slots(b, now[b])]
            view.values.append(decode_rows(c, rows))
            want, mag = ref.page_keys(view.values[b], P)
            assert_within(kk[c.table[b, : len(want)]], want, 2.0 ** -8 * np.abs(want) * 1.01 + 70 * 2.0 ** -24 * mag, "keys")
            assert np.array_equal(pg[b, 0], ref.select_pages(sc[b, 0], -(-now[b] // P), budget, 1, 2))
        check = sc.copy()
        for b in range(B):
            check[b, 0, -(-now[b] // P):] = 7.0     # (entries behind the pages are the caller's)
        check_scores(view, q, kk, check)
        check_attend(view, q, pg.astype(np.int32), o.double().cpu().numpy(), lse.cpu().numpy())


def decode_rows(c, raw):
    dc, dr = 512, 64
    if c.kind == "bf16":
        return torch.from_numpy(raw.copy()).view(torch.bfloat16).double().numpy()
    if c.kind == "fp8_e4m3":
        return oracle.e4m3_decode(raw) * float(np.float32(c.scale))
    sc = raw[:, dc: dc + 16].copy().view(np.float32).astype(np.float64)
    k = torch.from_numpy(raw[:, dc + 16:].copy()).view(torch.bfloat16).double().numpy()
    return np.concatenate([oracle.e4m3_decode(raw[:, :dc]) * np.repeat(sc, 128, 1), k], 1)
