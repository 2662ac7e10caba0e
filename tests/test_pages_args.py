"""Host-side checks of page-sparse decoding and 4-bit weights, and pins of their fp64 references.
No test here needs a GPU or runs a kernel."""
import ctypes
import itertools
import math

import numpy as np
import pytest

import mla_latent_kv_04_gb300 as M
import workloads as W
from oracle import pages as ref
from tests.test_serving_args import FAKE, ODD_ADDRESS, call, cfg, lib  # noqa: F401 (lib is a fixture)
from tests.test_serving_limits import Elsewhere

GOOD = {
    "mla_page_keys": dict(cache=FAKE, num_pages=4, table=FAKE, max_pages=2, seq_lens=FAKE, batch=4, new_tokens=1,
                          page_keys=FAKE, status=None, stream=None),
    "mla_page_scores": dict(q_lat=FAKE, page_keys=FAKE, num_pages=4, table=FAKE, max_pages=2, seq_lens=FAKE,
                            batch=4, q_len=1, scores=FAKE, workspace=FAKE, bytes=1 << 40, status=None, stream=None),
    "mla_select_pages": dict(scores=FAKE, max_pages=8, seq_lens=FAKE, batch=4, q_len=1, budget=5, sinks=1, recent=2,
                             pages=FAKE, status=None, stream=None),
    "mla_decode_pages": dict(q_lat=FAKE, cache=FAKE, num_pages=4, table=FAKE, max_pages=8, seq_lens=FAKE, batch=4,
                             q_len=1, pages=FAKE, budget=5, out=FAKE, lse=FAKE, workspace=FAKE, bytes=1 << 40,
                             stream=None),
    "mla_mx4_quantize": dict(W=FAKE, K=64, N=10, codes=FAKE, scales=FAKE, stream=None),
    "mla_mx4_dequantize": dict(codes=FAKE, scales=FAKE, K=64, N=10, W=FAKE, stream=None),
    "mla_mx4_project": dict(x=FAKE, codes=FAKE, scales=FAKE, K=64, N=10, rows=3, out=FAKE, workspace=FAKE,
                            bytes=1 << 40, stream=None),
}
I, U, Ws = M.MLA_ERR_INVALID, M.MLA_ERR_UNSUPPORTED, M.MLA_ERR_WORKSPACE
REFUSED = [
    ("mla_page_keys", dict(batch=0), I), ("mla_page_keys", dict(batch=32769), I),
    ("mla_page_keys", dict(new_tokens=-1), I), ("mla_page_keys", dict(max_pages=0), I),
    ("mla_page_keys", dict(num_pages=0), I), ("mla_page_keys", dict(cache=ODD_ADDRESS), I),
    ("mla_page_keys", dict(max_pages=1 << 26), U),
    ("mla_page_scores", dict(batch=0), I), ("mla_page_scores", dict(q_len=0), I),
    ("mla_page_scores", dict(batch=40000), U), ("mla_page_scores", dict(max_pages=0), I),
    ("mla_page_scores", dict(num_pages=-1), I), ("mla_page_scores", dict(max_pages=1 << 26), U),
    ("mla_select_pages", dict(budget=0), I), ("mla_select_pages", dict(budget=2), I),
    ("mla_select_pages", dict(sinks=-1), I), ("mla_select_pages", dict(recent=-1), I),
    ("mla_select_pages", dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), I), ("mla_select_pages", dict(batch=0), I),
    ("mla_select_pages", dict(max_pages=49153), U), ("mla_select_pages", dict(batch=32768, q_len=2), U),
    ("mla_select_pages", dict(budget=1 << 26), U),
    ("mla_decode_pages", dict(budget=0), I), ("mla_decode_pages", dict(batch=8193), U),
    ("mla_decode_pages", dict(budget=1 << 26), U), ("mla_decode_pages", dict(cache=ODD_ADDRESS), I),
    ("mla_decode_pages", dict(workspace=None), Ws), ("mla_decode_pages", dict(bytes=100), Ws),
    ("mla_decode_pages", dict(workspace=ODD_ADDRESS), I), ("mla_decode_pages", dict(q_len=-1), I),
    ("mla_decode_pages", dict(num_pages=0), I),
    ("mla_mx4_quantize", dict(K=0), I), ("mla_mx4_quantize", dict(K=33), I), ("mla_mx4_quantize", dict(N=0), I),
    ("mla_mx4_quantize", dict(K=1 << 24), U), ("mla_mx4_quantize", dict(codes=ODD_ADDRESS), I),
    ("mla_mx4_quantize", dict(scales=ODD_ADDRESS), I), ("mla_mx4_dequantize", dict(K=48), I),
    ("mla_mx4_dequantize", dict(N=(1 << 23) + 1), U), ("mla_mx4_dequantize", dict(codes=ODD_ADDRESS), I),
    ("mla_mx4_project", dict(rows=-1), I), ("mla_mx4_project", dict(K=16), I),
    ("mla_mx4_project", dict(codes=ODD_ADDRESS), I), ("mla_mx4_project", dict(scales=ODD_ADDRESS), I),
]
OPTIONAL = {"status", "stream", "workspace"}


@pytest.mark.parametrize("name,change,code", REFUSED)
def test_refused(lib, name, change, code):  # noqa: F811
    assert call(getattr(lib, name), cfg(), {**GOOD[name], **change}.values()) == code
    assert M.mla_last_error()


@pytest.mark.parametrize("name", GOOD)
def test_null_pointers_and_configs_refused(lib, name):  # noqa: F811
    for arg, v in GOOD[name].items():
        if v is FAKE and arg not in OPTIONAL:
            assert call(getattr(lib, name), cfg(), {**GOOD[name], arg: None}.values()) == I, arg
    for bad, code in ((dict(page_size=65), U), (dict(d_rope=3), I), (dict(act_dtype=7), I)):
        assert call(getattr(lib, name), cfg(**bad), GOOD[name].values()) == code
    assert getattr(lib, name)(None, *GOOD[name].values()) == I


def test_latents_that_the_attention_cannot_hold_are_refused(lib):  # noqa: F811
    assert call(lib.mla_decode_pages, cfg(d_latent=516), GOOD["mla_decode_pages"].values()) == U
    assert call(lib.mla_page_keys, cfg(d_latent=58100, d_rope=64), GOOD["mla_page_keys"].values()) == U


def test_empty_calls_do_nothing(lib):  # noqa: F811
    assert call(lib.mla_mx4_project, cfg(), {**GOOD["mla_mx4_project"], "rows": 0}.values()) == M.MLA_OK
    assert call(lib.mla_page_keys, cfg(), {**GOOD["mla_page_keys"], "new_tokens": 0}.values()) == M.MLA_OK


def test_workspace_sizes(lib):  # noqa: F811
    n, m = ctypes.c_size_t(7), ctypes.c_size_t(7)
    c = ctypes.byref(cfg())
    assert lib.mla_decode_pages_workspace_size(c, 4, 2, 9, ctypes.byref(n)) == M.MLA_OK and n.value % 256 == 0
    assert lib.mla_decode_pages_workspace_size(c, 4, 2, 9000, ctypes.byref(m)) == M.MLA_OK
    assert m.value >= n.value + 8 * 8991 * 4 - 256
    assert lib.mla_page_scores_workspace_size(c, 4, 2, 9, ctypes.byref(n)) == M.MLA_OK
    assert lib.mla_mx4_project_workspace_size(c, 64, 9, 0, ctypes.byref(n)) == M.MLA_OK
    assert lib.mla_mx4_bytes(c, 96, 130, ctypes.byref(n), ctypes.byref(m)) == M.MLA_OK
    assert (n.value, m.value) == (130 * 48, 2 * 1 * 512)
    for f, a in ((lib.mla_decode_pages_workspace_size, (4, 1, 9)), (lib.mla_page_scores_workspace_size, (4, 1, 9)),
                 (lib.mla_mx4_project_workspace_size, (64, 9, 3))):
        assert f(c, *a, None) == I
        assert f(c, -1, *a[1:], ctypes.byref(n)) == I
    assert lib.mla_mx4_bytes(c, 96, 130, None, ctypes.byref(m)) == I


def test_binding_refuses_other_devices_and_sizes(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(M, "_device_query", lambda: 0)
    c = M.make_config(W.V2, "bf16", "bf16")
    bf16, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8

    def calls(device, table_width=4, n=256):
        def t(*shape, dtype=bf16):
            return Elsewhere(*shape, dtype=dtype, device=device)
        cache, table, lens = t(4, 64, 576), t(1, table_width, dtype=i32), t(1, dtype=i32)
        q, pk, sc, pg = t(1, 1, 128, 576), t(4, 576), t(1, 1, 4, dtype=f32), t(1, 1, 3, dtype=i32)
        ws, codes, scales = t(1 << 30, dtype=u8), t(n * 32, dtype=u8), t(2 * 512, dtype=u8)
        return [lambda: M.mla_page_keys(c, cache, table, lens, pk, stream=0),
                lambda: M.mla_page_scores(c, q, pk, table, lens, sc, ws, stream=0),
                lambda: M.mla_select_pages(c, sc, lens, pg, stream=0),
                lambda: M.mla_decode_pages(c, q, cache, table, lens, pg, t(1, 1, 128, 512), t(1, 1, 128, dtype=f32), ws,
                                           stream=0),
                lambda: M.mla_mx4_quantize(c, t(64, 256), codes, scales, stream=0),
                lambda: M.mla_mx4_dequantize(c, codes, scales, t(64, 256), stream=0),
                lambda: M.mla_mx4_project(c, t(3, 64), codes, scales, t(3, 256), ws, stream=0)]

    for f in calls(1):
        with pytest.raises(ValueError, match="not the current device"):
            f()
    for f in calls(-1):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f()
    for f in calls(0, n=255)[4:]:
        with pytest.raises(ValueError, match="elements, expected"):
            f()


# ----------------------------------------------------------------------------- the references

def test_page_scores_share_out_the_heads_and_equal_token_softmax():
    """With every token's key equal to its page's, the scores are the pages' sums of softmax weights."""
    rng = np.random.default_rng(1)
    P, see, H, D = 4, 11, 3, 6
    q, keys = rng.standard_normal((H, D)), rng.standard_normal((3, D))
    got, lse, _ = ref.page_scores(q, keys, see, P, 0.7)
    want = np.zeros(3)
    for h in range(H):
        e = [math.exp(0.7 * float(q[h] @ keys[j // P])) for j in range(see)]
        for j in range(see):
            want[j // P] += e[j] / sum(e)
        assert abs(lse[h] - math.log(sum(e))) < 1e-12
    assert np.allclose(got, want, rtol=1e-12) and abs(got.sum() - H) < 1e-12


def test_page_keys_are_means():
    rows = np.arange(30.0).reshape(10, 3)
    k, _ = ref.page_keys(rows, 4)
    assert np.array_equal(k, np.array([[4.5, 5.5, 6.5], [16.5, 17.5, 18.5], [25.5, 26.5, 27.5]]))


def test_attend_all_pages_is_softmax_attention():
    rng = np.random.default_rng(2)
    q, x = rng.standard_normal((2, 5)), rng.standard_normal((9, 5))
    o, lse, _, _ = ref.attend_pages(q, x, [0, 1, 2], 9, 4, 3, 0.5)
    for h in range(2):
        e = [math.exp(0.5 * sum(a * b for a, b in zip(q[h], x[j]))) for j in range(9)]
        assert abs(lse[h] - math.log(sum(e))) < 1e-12
        for k in range(3):
            assert abs(o[h, k] - sum(e[j] * x[j, k] for j in range(9)) / sum(e)) < 1e-12
    o2, _, _, _ = ref.attend_pages(q, x, [0, 2], 9, 4, 3, 0.5)
    o3, _, _, _ = ref.attend_pages(q, np.delete(x, range(4, 8), 0), [0, 1], 5, 4, 3, 0.5)
    assert np.allclose(o2, o3)


def test_selection_of_small_cases_by_trying_all():
    s = np.array([1.0, 5.0, 2.0, 5.0, np.nan, 0.5, -np.inf, 3.0])
    assert list(ref.select_pages(s, 8, 4, 1, 1)) == [0, 1, 3, 7]
    assert list(ref.select_pages(s, 8, 7, 0, 1)) == [0, 1, 2, 3, 5, 6, 7]
    assert list(ref.select_pages(s, 3, 5, 1, 1)) == [0, 1, 2, -1, -1]
    for budget in range(2, 6):                     # the largest sum of all choices
        got = ref.select_pages(np.abs(np.nan_to_num(s, neginf=0)), 8, budget, 0, 1)
        v = np.abs(np.nan_to_num(s, neginf=0))
        best = max(sum(v[list(c)]) for c in itertools.combinations(range(7), budget - 1))
        assert v[got].sum() == best + v[7]


def test_mx4_codes_and_scales_by_hand():
    W = np.zeros((64, 3))
    W[:8, 0] = [6.0, -5.0, 0.25, 0.75, 1.25, 2.5, -3.5, 0.26]    # ties go to even codes
    W[:3, 1] = [7.0, 1.0, -0.5]                                  # 7 rounds up to 8: scale 2
    W[32:35, 0] = [6.99, 3.49, -0.1]                             # 6.99 saturates at 6
    c, e = ref.mx4_quantize(W)
    assert list(ref.mx4_values(c, e)[:8, 0]) == [6.0, -4.0, 0.0, 1.0, 1.0, 2.0, -4.0, 0.5] and e[0, 0] == 0
    assert e[0, 1] == 1 and list(ref.mx4_values(c, e)[:3, 1]) == [8.0, 1.0, -0.0]
    assert e[1, 0] == 0 and list(ref.mx4_values(c, e)[32:35, 0]) == [6.0, 3.0, -0.0]
    assert e[0, 2] == -127 and (ref.mx4_values(c, e)[:, 2] == 0).all()
    p, s = ref.mx4_pack(c, e)
    assert p.shape == (3, 32) and p[0, 0] == (c[0, 0] | c[1, 0] << 4) and s[0, 0, 1, 0, 0] == 128
    assert s[0, 0, 3, 0, 0] == 127 and s[0, 0, 0, 0, 2] == 127   # behind N, behind K


def test_mx4_error_is_within_half_a_step():
    rng = np.random.default_rng(3)
    W = rng.standard_normal((128, 40)) * np.exp(rng.standard_normal((128, 40)))
    c, e = ref.mx4_quantize(W)
    y = np.abs(W).reshape(4, 32, 40) / np.exp2(e)[:, None]
    step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    err = np.abs(ref.mx4_values(c, e) - W).reshape(4, 32, 40) / np.exp2(e)[:, None]
    assert (err <= step / 2 + 1e-12).all() and (y.max(1) < 7).all() and (y.max(1) >= 3.5).all()
