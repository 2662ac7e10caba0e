"""The decode's results are the same bits in every call: partial scores that the CTAs of a pair send each
other must not land in a buffer that a warp of the receiver still reads (thousands of short requests, where
every page or two ends a work item, held warps up long enough for that in about 1 call of 130)."""
import numpy as np
import pytest
import torch

import harness as Hn
import mla_latent_kv_04_gb300 as M
import workloads as W

pytestmark = pytest.mark.gpu


def test_decode_of_thousands_of_short_requests_repeats_bit_for_bit():
    lens = np.random.default_rng(31).integers(1, 257, size=2100)
    wl = W.scaled(W.WORKLOADS["v2_b32_s4096"], tuple(int(x) for x in lens), name="v2_many", spare_pages=3)
    st, q = Hn.build_state(wl, "cuda"), W.queries(wl)
    B, H, d_c = wl.batch, wl.dims.num_heads, wl.dims.d_latent
    q_nope, q_pe = (Hn.to_dev(q[k], torch.bfloat16, "cuda") for k in ("q_nope", "q_pe"))
    ws = torch.empty(M.mla_decode_workspace_size(st["cfg"], B, 1), dtype=torch.uint8, device="cuda")

    def call():
        out = torch.empty(B * H * d_c, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B * H, dtype=torch.float32, device="cuda")
        M.mla_decode(st["cfg"], q_nope, q_pe, st["W_UK_abs"], st["cache"], st["bt_d"], st["seq_lens_d"], out, lse, ws)
        assert M.mla_read_device_status(ws) == M.MLA_OK
        return out.view(torch.int16), lse

    # (a call that a fault hits differs from all the others: the first one has two more to agree with)
    first = call()
    differ = sum(not all(torch.equal(a, b) for a, b in zip(first, call())) for _ in range(1000))
    assert differ == 0
