"""Inputs shared by the tests of the shared-prefix and eviction calls: seeded draws, paged
caches in every storage format (unwritten slots hold NaN patterns), and error bounds."""
from __future__ import annotations

import numpy as np
import torch

import mla_latent_kv_04_gb300 as M
import oracle
import workloads as W

PAGE = 64
EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}        # half a step, relative


class Dims:
    def __init__(self, H, base):
        self.num_heads, self.d_model = H, base.d_model
        self.d_latent, self.d_rope, self.d_nope, self.d_v = base.d_latent, base.d_rope, base.d_nope, base.d_v
        self.page_size = PAGE


# rows that are no multiple of 16 bytes
ODD = W.Dims(num_heads=3, d_model=40, d_latent=60, d_rope=8, d_nope=20, d_v=12)
ODD128 = W.Dims(num_heads=3, d_model=40, d_latent=128, d_rope=12, d_nope=20, d_v=12)
# other value and latent widths that the tensor cores take in the joined projection
VALUE64 = W.Dims(num_heads=5, d_model=256, d_latent=192, d_rope=16, d_nope=32, d_v=64)
VALUE128 = W.Dims(num_heads=5, d_model=264, d_latent=192, d_rope=16, d_nope=32, d_v=128)


def dims(shape, H):
    return Dims(H, {"v2": W.V2, "tiny": W.TINY, "odd": ODD, "odd128": ODD128, "value64": VALUE64,
                    "value128": VALUE128}[shape])


def act_of(cache):
    return "f32" if cache == "f32" else "bf16"


def torch_type(act):
    return torch.float32 if act == "f32" else torch.bfloat16


def draw(rng, shape, act, std=1.0):
    """N(0, std^2) values exactly representable in the activation type (float32 array)."""
    x = (rng.standard_normal(shape) * std).astype(np.float32)
    return W.round_bf16(x) if act == "bf16" else x


def dev(x, act=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    if act is not None:
        t = t.to(torch_type(act))
    return t.cuda()


class Cache:
    """A pool of pages with every request's rows in it, and the rows as fp64 values."""

    def __init__(self, rng, kind, d, lens, max_pages=None, spare=4, scale=3.0 / 448):
        self.kind, self.d, self.lens = kind, d, list(lens)
        self.scale = scale if kind == "fp8_e4m3" else 1.0
        pages = [-(-n // PAGE) for n in lens]
        self.max_pages = max_pages or max(1, max(pages))
        perm = rng.permutation(sum(pages) + spare)
        self.num_pages = len(perm)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        dc, dr = d.d_latent, d.d_rope
        if kind == "fp8_e4m3_b128":
            row = dc + dc // 32 + 2 * dr
        else:
            row = (dc + dr) * {"f32": 4, "bf16": 2, "fp8_e4m3": 1}[kind]
        self.row = row
        fill = {"f32": (0xDE, 0xAD, 0xC0, 0x7F), "bf16": (0xC1, 0x7F)}.get(kind, (0x7F,))
        self.bytes = np.resize(np.array(fill, np.uint8), self.num_pages * PAGE * row).reshape(-1, row)
        self.values, at = [], 0
        for b, n in enumerate(lens):
            self.table[b, : pages[b]] = perm[at: at + pages[b]]
            at += pages[b]
            raw, vals = self.encode(rng, n)
            self.bytes[self.slots(b, n)] = raw
            self.values.append(vals)
        self.spare = perm[at:].astype(np.int32)

    def slots(self, b, n, table=None):
        t = (self.table if table is None else table)[b]
        j = np.arange(n)
        return t[j // PAGE].astype(np.int64) * PAGE + j % PAGE

    def encode(self, rng, n):
        dc, dr = self.d.d_latent, self.d.d_rope
        x = draw(rng, (n, dc + dr), act_of(self.kind))
        if self.kind == "f32":
            return x.view(np.uint8).reshape(n, 4 * (dc + dr)), x.astype(np.float64)
        if self.kind == "bf16":
            return bf16_bytes(x), x.astype(np.float64)
        if self.kind == "fp8_e4m3":
            codes = oracle.e4m3_encode(x / np.float32(self.scale))
            return codes, oracle.e4m3_decode(codes) * float(np.float32(self.scale))
        if n == 0:
            return np.zeros((0, self.row), np.uint8), x.astype(np.float64)
        codes, scales = oracle.e4m3_block_quantize(x[:, :dc], 128)
        vals = np.concatenate([oracle.e4m3_block_dequantize(codes, scales, 128), x[:, dc:]], 1)
        raw = np.concatenate([np.asarray(codes, np.uint8).reshape(n, dc),
                              np.ascontiguousarray(scales, np.float32).view(np.uint8).reshape(n, -1),
                              bf16_bytes(x[:, dc:])], 1)
        return raw, vals

    def device(self):
        t = torch.from_numpy(self.bytes.reshape(-1).copy()).cuda()
        if self.kind == "f32":
            return t.view(torch.float32)
        return t.view(torch.bfloat16) if self.kind == "bf16" else t

    def back(self, t):
        """A device pool as bytes [slots][row]."""
        return t.view(torch.uint8).cpu().numpy().reshape(-1, self.row)

    def config(self, **kw):
        return M.make_config(self.d, act_of(self.kind), self.kind, cache_scale=self.scale, **kw)


def bf16_bytes(x):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint8).reshape(x.shape[0], 2 * x.shape[1])


def assert_within(got, ref, tol, what):
    """|got - ref| <= tol element by element; non-finite references match exactly."""
    got, ref, tol = np.broadcast_arrays(np.asarray(got, np.float64), ref, tol)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin], equal_nan=True), f"{what}: non-finite entries differ"
    err = np.abs(got[fin] - ref[fin])
    over = err - tol[fin]
    assert err.size == 0 or not (over > 0).any(), (
        f"{what}: off by {err[over.argmax()]:.3e}, allowed {tol[fin][over.argmax()]:.3e}, "
        f"{(over > 0).sum()} of {err.size} values")
    assert np.isfinite(got[fin]).all(), f"{what}: NaN or infinity"


def shifted(t, elements=1):
    """The same values at an address that is no multiple of 16 bytes."""
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    view = flat[elements: elements + t.numel()].view(t.shape)
    view.copy_(t)
    return view
