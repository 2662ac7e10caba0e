"""Host-side checks of the shared-prefix and eviction calls, and pins of their fp64 references.
No test here needs a GPU or runs a kernel."""
import ctypes

import numpy as np
import pytest

import mla_latent_kv_04_gb300 as M
import oracle
import workloads as W
from oracle import serving as ref

FAKE = ctypes.c_void_p(1 << 20)
ODD_ADDRESS = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(M.LIB_PATH):
        from mla_latent_kv_04_gb300 import build
        build.build()
    return M.lib()


def cfg(act="bf16", cache="bf16", dims=W.V2, **kw):
    c = M.make_config(dims, act, cache)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def call(f, c, args):
    return f(ctypes.byref(c), *args)


# every argument of a call with a good value, by name
GOOD = {
    "mla_prefix_expand": dict(W_UK=FAKE, W_UV=FAKE, cache=FAKE, num_pages=4, pages=FAKE, prefix_len=100,
                              keys=FAKE, values=FAKE, k_pe=FAKE, status=None, stream=None),
    "mla_prefix_attend": dict(q_nope=FAKE, q_pe=FAKE, keys=FAKE, values=FAKE, k_pe=FAKE, prefix_len=100,
                              seq_lens=FAKE, batch=4, q_len=1, u=FAKE, lse=FAKE, workspace=FAKE,
                              bytes=1 << 40, status=None, stream=None),
    "mla_output_proj_prefix": dict(o=FAKE, lse=FAKE, up=FAKE, lse_p=FAKE, W_UV=FAKE, W_O=FAKE, rows=3,
                                   out=FAKE, workspace=FAKE, bytes=1 << 40, stream=None),
    "mla_absorb_query": dict(q_nope=FAKE, q_pe=FAKE, W=FAKE, seq_lens=FAKE, batch=4, q_len=1, q_lat=FAKE,
                             stream=None),
    "mla_key_weights": dict(q_lat=FAKE, lse=FAKE, cache=FAKE, num_pages=4, table=FAKE, max_pages=2,
                            seq_lens=FAKE, batch=4, q_len=1, decay=ctypes.c_float(1.0), weights=FAKE,
                            status=None, stream=None),
    "mla_evict_cache": dict(weights=FAKE, seq_lens=FAKE, table=FAKE, max_pages=2, batch=4, budget=10, sinks=1,
                            recent=2, rotate=1, cache=FAKE, num_pages=4, new_table=FAKE, new_max_pages=2,
                            new_weights=None, kept=FAKE, new_lens=FAKE, status=None, stream=None),
}
OTHER = ctypes.c_void_p(1 << 21)
I, U, Ws = M.MLA_ERR_INVALID, M.MLA_ERR_UNSUPPORTED, M.MLA_ERR_WORKSPACE
REFUSED = [
    ("mla_prefix_expand", dict(prefix_len=-1), I), ("mla_prefix_expand", dict(prefix_len=(1 << 22) + 1), U),
    ("mla_prefix_expand", dict(num_pages=0), I), ("mla_prefix_expand", dict(cache=ODD_ADDRESS), I),
    ("mla_key_weights", dict(cache=ODD_ADDRESS), I),
    ("mla_prefix_attend", dict(prefix_len=-1), I), ("mla_prefix_attend", dict(batch=0), I),
    ("mla_prefix_attend", dict(q_len=0), I), ("mla_prefix_attend", dict(batch=40000), U),
    ("mla_output_proj_prefix", dict(rows=-1), I), ("mla_output_proj_prefix", dict(bytes=100), Ws),
    ("mla_output_proj_prefix", dict(workspace=None), Ws), ("mla_output_proj_prefix", dict(workspace=ODD_ADDRESS), I),
    ("mla_absorb_query", dict(batch=0), I), ("mla_absorb_query", dict(q_len=-3), I),
    ("mla_key_weights", dict(decay=ctypes.c_float(-0.1)), I), ("mla_key_weights", dict(decay=ctypes.c_float(1.5)), I),
    ("mla_key_weights", dict(decay=ctypes.c_float(float("nan"))), I), ("mla_key_weights", dict(max_pages=0), I),
    ("mla_key_weights", dict(num_pages=-1), I), ("mla_key_weights", dict(batch=32768, max_pages=1 << 17), U),
    ("mla_evict_cache", dict(budget=0), I), ("mla_evict_cache", dict(budget=2), I),
    ("mla_evict_cache", dict(sinks=-1), I), ("mla_evict_cache", dict(recent=-1), I),
    ("mla_evict_cache", dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), I), ("mla_evict_cache", dict(batch=0), I),
    ("mla_evict_cache", dict(batch=32769), I), ("mla_evict_cache", dict(max_pages=7000, new_table=OTHER), U),
    ("mla_evict_cache", dict(new_max_pages=3), I), ("mla_evict_cache", dict(new_table=OTHER, new_max_pages=0), I),
    ("mla_evict_cache", dict(new_table=OTHER, new_max_pages=3, new_weights=FAKE), I),
    ("mla_evict_cache", dict(budget=(1 << 30) + 1), U),
    ("mla_evict_cache", dict(num_pages=1 << 26), U), ("mla_evict_cache", dict(cache=ODD_ADDRESS), I),
]
OPTIONAL = {"status", "stream", "new_weights", "workspace"}


@pytest.mark.parametrize("name,change,code", REFUSED)
def test_refusals(lib, name, change, code):
    args = {**GOOD[name], **change}
    assert call(getattr(lib, name), cfg(), args.values()) == code
    assert M.mla_last_error()


@pytest.mark.parametrize("name,arg", [(n, a) for n, d in GOOD.items() for a, v in d.items()
                                      if v is FAKE and a not in OPTIONAL])
def test_null_pointers(lib, name, arg):
    args = {**GOOD[name], arg: None}
    assert call(getattr(lib, name), cfg(), args.values()) == I


@pytest.mark.parametrize("name", GOOD)
def test_bad_config(lib, name):
    assert call(getattr(lib, name), cfg(num_heads=0), GOOD[name].values()) == I
    assert call(getattr(lib, name), cfg(cache_dtype=M.MLA_F32), GOOD[name].values()) == U


def test_empty_calls_touch_nothing(lib):
    assert call(lib.mla_prefix_expand, cfg(), {**GOOD["mla_prefix_expand"], "prefix_len": 0, "keys": None,
                                               "cache": None}.values()) == M.MLA_OK
    assert call(lib.mla_output_proj_prefix, cfg(), {**GOOD["mla_output_proj_prefix"], "rows": 0, "o": None,
                                                    "workspace": None}.values()) == M.MLA_OK


def test_fp32_cache_alignment(lib):
    c = cfg("f32", "f32", W.TINY)
    args = {**GOOD["mla_evict_cache"], "cache": ctypes.c_void_p((1 << 20) + 4)}
    assert call(lib.mla_evict_cache, c, args.values()) == I


def test_workspace_sizes(lib):
    for rows in (1, 32, 128):
        assert M.mla_output_proj_prefix_workspace_size(cfg(), rows) == \
            M.mla_output_proj_unfolded_workspace_size(cfg(), rows)
    # more rows: fp32 pieces of the product with W_O
    assert M.mla_output_proj_prefix_workspace_size(cfg(), 129) > M.mla_output_proj_unfolded_workspace_size(cfg(), 129)
    n = ctypes.c_size_t(0)
    assert lib.mla_prefix_attend_workspace_size(ctypes.byref(cfg()), 4, 1, -1, ctypes.byref(n)) == I
    assert lib.mla_prefix_attend_workspace_size(ctypes.byref(cfg()), 4, 1, 10, None) == I


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    class OnDevice:
        def __init__(self, device):
            self.device, self.is_cuda = device, device >= 0

        def get_device(self):
            return self.device

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 4096

    monkeypatch.setattr(M, "_device_query", lambda: 0)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        M._ptr(OnDevice(-1), "x")
    assert M._ptr(OnDevice(0), "x") == 4096
    with pytest.raises(ValueError, match="not the current device"):
        M._ptr(OnDevice(1), "x")


# ----------------------------------------------------------------------------- reference pins

def test_reference_attention_is_the_decompressed_decode():
    """Expansion, attention and joining over a split key set = the decompressed attention of the
    oracle over all keys (keys numbered from 0)."""
    rng = np.random.default_rng(0)
    H, dc, dr, dn, L, n = 3, 8, 4, 6, 5, 4
    c, k = rng.standard_normal((L + n, dc)), rng.standard_normal((L + n, dr))
    k_rot = oracle.rope(k, np.arange(L + n))
    W_UK, W_UV = rng.standard_normal((dc, H * dn)), rng.standard_normal((dc, H * dn))
    qn, qp = rng.standard_normal((2, H, dn)), rng.standard_normal((2, H, dr))
    scale = 0.3
    full = oracle.decode_decompressed(c, k_rot, qn, qp, W_UK, W_UV, scale)
    K, V, _, _ = ref.expand_prefix(c[:L], W_UK, W_UV, H)
    u, lse, _, _ = ref.attend_prefix(qn[None], qp[None], K, V, k_rot[:L], [n], scale)
    W_abs = np.stack([W_UK[:, h * dn:(h + 1) * dn].T for h in range(H)])
    own_pe = oracle.rope(k[L:], np.arange(n))           # own tokens numbered from 0
    o, l = oracle.decode_absorbed(c[L:], own_pe, qn, qp, W_abs, scale)
    joined = ref.join_prefix(o, l, u[0], lse[0], W_UV, H)
    assert np.abs(joined - full["u"]).max() < 1e-12
    assert np.abs(np.logaddexp(l, lse[0]) - full["lse"]).max() < 1e-12


def test_reference_weights_are_the_softmax():
    rng = np.random.default_rng(1)
    q, rows = rng.standard_normal((2, 3, 5)), rng.standard_normal((7, 5))
    mass = np.zeros(7)
    lse = np.zeros((2, 3))
    for t in range(2):
        for h in range(3):
            s = [0.5 * float(q[t, h] @ rows[j]) for j in range(7 - 2 + t + 1)]
            e = np.exp(s)
            lse[t, h] = np.log(e.sum())
            mass[: len(s)] += e / e.sum()
    old = rng.random(9)
    got, _ = ref.key_weights(q, lse, rows, old, 2, 0.5, 0.25)
    want = mass + np.where(np.arange(7) < 5, 0.25 * old[:7], 0)
    assert np.abs(got - want).max() < 1e-12


def test_reference_order():
    w = np.array([9, 1, 5, 5, np.nan, 7, -np.inf, 5, 0, 0], np.float32)
    assert list(ref.evict_order(w, 10, 10, 1, 1)) == list(range(10))
    assert list(ref.evict_order(w, 10, 5, 1, 1)) == [0, 2, 3, 5, 9]
    assert list(ref.evict_order(w, 10, 8, 0, 2)) == [0, 1, 2, 3, 5, 7, 8, 9]
    assert list(ref.evict_order(w, 9, 8, 0, 0)) == [0, 1, 2, 3, 5, 6, 7, 8]


def test_reference_turn():
    k = np.random.default_rng(2).standard_normal((4, 6))
    at = np.array([900, 17, 5, 3])
    to = np.array([3, 2, 1, 0])
    assert np.abs(ref.turn_rows(oracle.rope(k, at), to - at) - oracle.rope(k, to)).max() < 1e-12
