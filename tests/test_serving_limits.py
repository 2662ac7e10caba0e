"""Host-side limits of the shared-prefix and eviction calls: what is too large for their kernels is
refused before anything is enqueued. No test here needs a GPU."""
import ctypes

import pytest

import mla_latent_kv_04_gb300 as M
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
