"""Host-side limits of the shared-prefix and eviction calls: what is too large for their kernels is
refused before anything is enqueued. No test here needs a GPU."""
import ctypes

import pytest

import mla_latent_kv_04_gb300 as M
import workloads as W
from tests.test_serving_args import GOOD, call, cfg, lib  # noqa: F401 (lib is a fixture)

U = M.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("widths", [dict(d_nope=57344), dict(d_v=57300), dict(d_nope=2 ** 31 - 1, d_v=2 ** 31 - 1)])
def test_prefix_attend_refuses_heads_wider_than_its_shared_memory(lib, widths):  # noqa: F811
    c = cfg(**widths)
    assert call(lib.mla_prefix_attend, c, GOOD["mla_prefix_attend"].values()) == U
    assert "57344" in M.mla_last_error()
    n = ctypes.c_size_t(0)
    assert lib.mla_prefix_attend_workspace_size(ctypes.byref(c), 4, 1, 10, ctypes.byref(n)) == U


@pytest.mark.parametrize("act,cache,widths", [("f32", "f32", dict(d_latent=832, d_rope=64)), ("f32", "f32", dict(d_latent=2 ** 31 - 4, d_rope=64)),
                                              ("bf16", "bf16", dict(d_latent=1696, d_rope=64)),
                                              ("bf16", "fp8_e4m3", dict(d_latent=3352, d_rope=64)),
                                              ("bf16", "fp8_e4m3_b128", dict(d_latent=3200, d_rope=64))])
def test_key_weights_refuses_rows_wider_than_its_shared_memory(lib, act, cache, widths):  # noqa: F811
    assert call(lib.mla_key_weights, cfg(act, cache, **widths), GOOD["mla_key_weights"].values()) == U
    assert "shared memory" in M.mla_last_error()


def test_decode_refuses_latents_wider_than_its_registers(lib):  # noqa: F811
    """The SIMT kernel's accumulators end at 512 elements: wider outputs were left unwritten."""
    for act in ("f32", "bf16"):
        c, n = cfg(act, act, d_latent=516), ctypes.c_size_t(0)
        assert lib.mla_decode_workspace_size(ctypes.byref(c), 4, 1, None, ctypes.byref(n)) == U
        assert lib.mla_decode(ctypes.byref(c), *[ctypes.c_void_p(1 << 20)] * 4, 4, ctypes.c_void_p(1 << 20), 2,
                              ctypes.c_void_p(1 << 20), 4, 1, *[ctypes.c_void_p(1 << 20)] * 3, 1 << 40, None) == U


# ----------------------------------------------------------------------------- addresses

def at(offset):
    return ctypes.c_void_p((1 << 20) + offset)


@pytest.mark.parametrize("kernel,out,cache,code", [(0, 2, 0, M.MLA_ERR_INVALID), (2, 8, 0, M.MLA_ERR_INVALID),
                                                   (1, 2, 2, M.MLA_ERR_INVALID)])
def test_decode_refuses_addresses_that_its_kernels_cannot_take(lib, kernel, out, cache, code):  # noqa: F811
    """The tensor-core kernel writes out_latent 16 bytes at a time, the SIMT kernel reads the cache by
    32-bit words; elsewhere these were misaligned accesses."""
    opts = M._opts(0, kernel)
    assert lib.mla_decode_ex(ctypes.byref(cfg()), at(0), at(0), at(0), at(cache), 4, at(0), 2, at(0), 4, 1, at(out), at(0),
                             at(0), 1 << 40, ctypes.byref(opts), None) == code
    assert "aligned" in M.mla_last_error()


def test_append_refuses_addresses_that_its_kernels_cannot_take(lib):  # noqa: F811
    c = cfg("bf16", "fp8_e4m3_b128")
    assert lib.mla_append_cache_latent(ctypes.byref(c), at(0), at(0), 3, at(0), at(0), at(0), 1, 2, at(2), 4, 1, None,
                                       None) == M.MLA_ERR_INVALID
    assert lib.mla_append_cache(ctypes.byref(c), at(0), at(0), 3, at(0), at(0), at(0), 1, 2, at(2), 4, None, None, 0,
                                None) == M.MLA_ERR_INVALID
    assert "aligned" in M.mla_last_error()


# ----------------------------------------------------------------------------- devices

class Elsewhere:
    """What the binding reads of a tensor, on a device other than the current one (0)."""

    def __init__(self, *shape, dtype=None, device=1):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, device, device >= 0

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def _calls(bf16, i32, f32, u8, device=1):
    """Calls of the ABI before the serving calls, and the serving calls, on tensors of `device`."""
    c = M.make_config(W.V2, "bf16", "bf16")

    def t(*shape, dtype=bf16):
        return Elsewhere(*shape, dtype=dtype, device=device)
    H, d = 128, W.V2.d_model
    cache, table, lens, ws = t(4, 64, 576), t(1, 4, dtype=i32), t(1, dtype=i32), t(64, dtype=u8)
    qn, qp, o, lse = t(1, 1, H, 128), t(1, 1, H, 64), t(1, 1, H, 512), t(1, 1, H, dtype=f32)
    u, keys, pe = t(1, 1, H, 128), t(H, 2, 128), t(2, 64)
    W_UV, W_O, out = t(512, H * 128), t(H * 128, d), t(1, d)
    q_lat, weights, kept = t(1, 1, H, 576), t(1, 256, dtype=f32), t(1, 9, dtype=i32)
    before = [
        lambda: M.mla_append_cache(c, t(2, d), t(d, 576), t(2, dtype=i32), t(2, dtype=i32), table, cache, stream=0),
        lambda: M.mla_append_cache_latent(c, t(2, 512), t(2, 64), t(2, dtype=i32), t(2, dtype=i32), table, cache, stream=0),
        lambda: M.mla_absorb_weights(c, t(512, H * 128), W_UV, W_O, t(H, 128, 512), t(H * 512, d), stream=0),
        lambda: M.mla_decode(c, qn, qp, t(H, 128, 512), cache, table, lens, o, lse, ws, stream=0),
        lambda: M.mla_decode_noalloc(c, qn, qp, t(H, 128, 512), cache, table, lens, o, lse, stream=0),
        lambda: M.mla_output_proj(c, o, t(H * 512, d), out, ws, stream=0),
        lambda: M.mla_output_proj_unfolded(c, o, W_UV, W_O, out, ws, stream=0),
        lambda: M.mla_query_from_hidden(c, 1536, t(1, d), t(d, 1536), t(1536, H * 128), t(d, H * 64), qn, qp, ws, stream=0),
        lambda: M.mla_read_device_status(lens, stream=0),
    ]
    serving = [
        lambda: M.mla_prefix_expand(c, t(512, H * 128), W_UV, cache, t(1, dtype=i32), 2, keys, keys, pe, stream=0),
        lambda: M.mla_prefix_attend(c, qn, qp, keys, keys, pe, lens, u, lse, ws, stream=0),
        lambda: M.mla_output_proj_prefix(c, o, lse, u, lse, W_UV, W_O, out, ws, stream=0),
        lambda: M.mla_absorb_query(c, qn, qp, t(H, 128, 512), lens, q_lat, stream=0),
        lambda: M.mla_key_weights(c, q_lat, lse, cache, table, lens, weights, stream=0),
        lambda: M.mla_evict_cache(c, weights, lens, table, cache, 9, kept, lens, stream=0),
    ]
    return before, serving


def test_calls_and_the_device_of_their_tensors(monkeypatch):
    """The calls that were there before the serving calls leave a tensor's device to the caller, who may
    have peer access; the serving calls refuse tensors of another device; no call takes host tensors."""
    torch = pytest.importorskip("torch")
    types = torch.bfloat16, torch.int32, torch.float32, torch.uint8
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or M.MLA_OK

    monkeypatch.setattr(M, "_device_query", lambda: 0)
    monkeypatch.setattr(M, "_lib_handle", Library())
    before, serving = _calls(*types)
    for f in before:
        f()
    assert len(seen) == len(before)
    for f in serving:
        with pytest.raises(ValueError, match="not the current device"):
            f()
    for f in _calls(*types, device=0)[1]:
        f()
    assert len(seen) == len(before) + len(serving)
    for f in sum(_calls(*types, device=-1), []):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f()
