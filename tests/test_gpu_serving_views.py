"""The serving calls on tensors that start off a 16-byte boundary, on head shapes that no tensor map
takes, and at the edges of their kernels' limits."""
import numpy as np
import pytest
import torch

import mla_latent_kv_04_gb300 as M
import oracle
from tests import serving_data as D

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
