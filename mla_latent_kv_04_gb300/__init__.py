"""Python binding of libmla, the C-ABI weight-absorbed MLA decode library for GB300.

Argument marshalling only: each function takes torch tensors that already live on
the GPU, checks their dtype/shape/contiguity, and passes raw pointers and sizes to
the C entry point of the same name declared in include/mla.h. Every step of the
computation runs in the library's CUDA kernels; there is no fallback path. When
libmla.so has not been built the first call raises ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libmla.so")

MLA_OK = 0
MLA_ERR_INVALID = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE = 3
MLA_ERR_CUDA = 4
MLA_ERR_DEVICE_GUARD = 5
MLA_ERR_TIMEOUT = 6

MLA_F32 = 0
MLA_BF16 = 1
MLA_FP8_E4M3 = 2
MLA_FP8_E4M3_B128 = 3

KERNEL_AUTO = 0
KERNEL_SIMT = 1
KERNEL_TC = 2

_DTYPE_CODES = {"f32": MLA_F32, "bf16": MLA_BF16, "fp8_e4m3": MLA_FP8_E4M3,
                "fp8_e4m3_b128": MLA_FP8_E4M3_B128}


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}" + (f" ({detail})" if detail else ""))


class MlaConfig(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int), ("d_model", ctypes.c_int), ("d_latent", ctypes.c_int),
        ("d_rope", ctypes.c_int), ("d_nope", ctypes.c_int), ("d_v", ctypes.c_int),
        ("page_size", ctypes.c_int), ("softmax_scale", ctypes.c_float),
        ("rope_theta", ctypes.c_float), ("rope_interleaved", ctypes.c_int),
        ("act_dtype", ctypes.c_int), ("cache_dtype", ctypes.c_int), ("cache_scale", ctypes.c_float),
    ]


class MlaDecodeOpts(ctypes.Structure):
    _fields_ = [("num_workers", ctypes.c_int), ("kernel", ctypes.c_int),
                ("attn_events", ctypes.c_void_p * 2), ("wait_limit_us", ctypes.c_int),
                ("withhold_page", ctypes.c_int)]


_lib_handle = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_CFG = ctypes.POINTER(MlaConfig)

_SIGNATURES = {
    "mla_absorb_weights": (_I, [_CFG, _P, _P, _P, _P, _P, _P]),
    "mla_append_cache": (_I, [_CFG, _P, _P, _I, _P, _P, _P, _I, _I, _P, _I, _P, _P, _SZ, _P]),
    "mla_append_cache_workspace_size": (_I, [_CFG, _I, ctypes.POINTER(_SZ)]),
    "mla_append_cache_latent": (_I, [_CFG, _P, _P, _I, _P, _P, _P, _I, _I, _P, _I, _I, _P, _P]),
    "mla_decode_workspace_size": (_I, [_CFG, _I, _I, ctypes.POINTER(MlaDecodeOpts),
                                       ctypes.POINTER(_SZ)]),
    "mla_decode": (_I, [_CFG, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "mla_decode_ex": (_I, [_CFG, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P, _SZ,
                           ctypes.POINTER(MlaDecodeOpts), _P]),
    "mla_decode_noalloc": (_I, [_CFG, _P, _P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P]),
    "mla_decode_noalloc_status": (_I, [_P, ctypes.POINTER(_I)]),
    "mla_output_proj_workspace_size": (_I, [_CFG, _I, ctypes.POINTER(_SZ)]),
    "mla_output_proj": (_I, [_CFG, _P, _P, _I, _P, _P, _SZ, _P]),
    "mla_output_proj_unfolded_workspace_size": (_I, [_CFG, _I, ctypes.POINTER(_SZ)]),
    "mla_output_proj_unfolded": (_I, [_CFG, _P, _P, _P, _I, _P, _P, _SZ, _P]),
    "mla_cache_row_bytes": (_I, [_CFG, ctypes.POINTER(_SZ)]),
    "mla_query_workspace_size": (_I, [_CFG, _I, _I, ctypes.POINTER(_SZ)]),
    "mla_query_from_hidden": (_I, [_CFG, _I, _P, _P, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "mla_prefix_expand": (_I, [_CFG, _P, _P, _P, _I, _P, _I, _P, _P, _P, _P, _P]),
    "mla_prefix_attend_workspace_size": (_I, [_CFG, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "mla_prefix_attend": (_I, [_CFG, _P, _P, _P, _P, _P, _I, _P, _I, _I, _P, _P, _P, _SZ, _P, _P]),
    "mla_output_proj_prefix_workspace_size": (_I, [_CFG, _I, ctypes.POINTER(_SZ)]),
    "mla_output_proj_prefix": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _I, _P, _P, _SZ, _P]),
    "mla_absorb_query": (_I, [_CFG, _P, _P, _P, _P, _I, _I, _P, _P]),
    "mla_key_weights": (_I, [_CFG, _P, _P, _P, _I, _P, _I, _P, _I, _I, ctypes.c_float, _P, _P, _P]),
    "mla_evict_cache": (_I, [_CFG, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P,
                             _P, _P]),
    "mla_page_keys": (_I, [_CFG, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P]),
    "mla_page_scores_workspace_size": (_I, [_CFG, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "mla_page_scores": (_I, [_CFG, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _SZ, _P, _P]),
    "mla_select_pages": (_I, [_CFG, _P, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "mla_decode_pages_workspace_size": (_I, [_CFG, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "mla_decode_pages": (_I, [_CFG, _P, _P, _I, _P, _I, _P, _I, _I, _P, _I, _P, _P, _P, _SZ, _P]),
    "mla_mx4_bytes": (_I, [_CFG, _I, _I, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "mla_mx4_quantize": (_I, [_CFG, _P, _I, _I, _P, _P, _P]),
    "mla_mx4_dequantize": (_I, [_CFG, _P, _P, _I, _I, _P, _P]),
    "mla_mx4_project_workspace_size": (_I, [_CFG, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "mla_mx4_project": (_I, [_CFG, _P, _P, _P, _I, _I, _I, _P, _P, _SZ, _P]),
    "mla_read_device_status": (_I, [_P, _P, ctypes.POINTER(_I)]),
    "mla_status_string": (ctypes.c_char_p, [_I]),
    "mla_last_error": (ctypes.c_char_p, []),
    "mla_version": (_I, []),
    "mla_testing_waits": (None, [_I, _I]),
    "mla_kernel_launches": (ctypes.c_uint64, []),
}


def lib():
    """The loaded libmla.so (raises RuntimeError when it has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmla.so is not built ({LIB_PATH}); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib_handle = h
    return _lib_handle


def status_string(status: int) -> str:
    try:
        return lib().mla_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def mla_status_string(status: int) -> str:
    return status_string(status)


def mla_last_error() -> str:
    return lib().mla_last_error().decode()


def mla_version() -> int:
    return lib().mla_version()


def mla_testing_waits(wait_limit_us: int = 0, withhold: int = 0):
    """Testing hook of failure paths, for this thread's calls until it is set again (0, 0: off)."""
    lib().mla_testing_waits(int(wait_limit_us), int(withhold))


def _check(status: int, where: str):
    if status != MLA_OK:
        raise MlaError(status, where, mla_last_error())


def make_config(dims, act: str = "bf16", cache: str = "bf16", cache_scale: float = 1.0,
                softmax_scale: float = 0.0, rope_theta: float = 10000.0) -> MlaConfig:
    """Config from an object with num_heads/d_model/d_latent/d_rope/d_nope/d_v/page_size."""
    return MlaConfig(dims.num_heads, dims.d_model, dims.d_latent, dims.d_rope, dims.d_nope, dims.d_v,
                     dims.page_size, float(softmax_scale), float(rope_theta), 1,
                     _DTYPE_CODES[act], _DTYPE_CODES[cache], float(cache_scale))


# ----------------------------------------------------------------------------- marshalling

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _act_dtype(cfg):
    t = _torch()
    return t.float32 if cfg.act_dtype == MLA_F32 else t.bfloat16


def _cache_dtypes(cfg):
    t = _torch()
    if cfg.cache_dtype == MLA_F32:
        return (t.float32,)
    if cfg.cache_dtype == MLA_BF16:
        return (t.bfloat16,)
    return (t.uint8, t.float8_e4m3fn)


def _cache_row_elems(cfg):
    """Elements of the cache tensor per token row: d_c + d_r, or the row's bytes for the
    block-scaled fp8 cache (a uint8 tensor)."""
    if cfg.cache_dtype == MLA_FP8_E4M3_B128:
        return cfg.d_latent + cfg.d_latent // 32 + 2 * cfg.d_rope
    return cfg.d_latent + cfg.d_rope


_device_query = None


def _current_device() -> int:
    global _device_query
    if _device_query is None:
        _device_query = _torch()._C._cuda_getDevice if _torch().cuda.is_available() else lambda: 0
    return _device_query()


def _ptr(x, name, dtypes=None, numel=None, allow_none=False, peer=False):
    """peer: tensors of a device that the current one can access are let through."""
    if x is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    device = x.get_device()
    if device != (_device_query or _current_device)():
        if not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not peer:
            raise ValueError(f"{name} is on cuda:{device}, which is not the current device")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and x.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {x.dtype}, expected one of {dtypes}")
    if numel is not None and x.numel() != numel:
        raise ValueError(f"{name} has {x.numel()} elements, expected {numel}")
    return x.data_ptr()


# The calls of ABI 1.02 and before leave a tensor's device to the caller.
_peer_ptr = functools.partial(_ptr, peer=True)


def _stream(stream):
    if stream is None:
        # the current stream of the current device, without the Stream object around it (4 us a call)
        return _torch()._C._cuda_getCurrentRawStream(_current_device())
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _opts(num_workers, kernel, attn_events=None, wait_limit_us=0, withhold_page=0):
    o = MlaDecodeOpts(int(num_workers), int(kernel))
    o.wait_limit_us = int(wait_limit_us)
    o.withhold_page = int(withhold_page)
    if attn_events is not None:
        o.attn_events[0] = attn_events[0].cuda_event
        o.attn_events[1] = attn_events[1].cuda_event
    return o


def mla_kernel_launches() -> int:
    return int(lib().mla_kernel_launches())


# ----------------------------------------------------------------------------- entry points

def mla_absorb_weights(cfg, W_UK, W_UV, W_O, W_UK_abs, W_comb, stream=None):
    a = (_act_dtype(cfg),)
    H, d_c, d_n, d_v, d = cfg.num_heads, cfg.d_latent, cfg.d_nope, cfg.d_v, cfg.d_model
    _check(lib().mla_absorb_weights(
        ctypes.byref(cfg), _peer_ptr(W_UK, "W_UK", a, d_c * H * d_n), _peer_ptr(W_UV, "W_UV", a, d_c * H * d_v),
        _peer_ptr(W_O, "W_O", a, H * d_v * d), _peer_ptr(W_UK_abs, "W_UK_abs", a, H * d_n * d_c),
        _peer_ptr(W_comb, "W_comb", a, H * d_c * d), _stream(stream)), "mla_absorb_weights")


_i32_types = None


def _i32(t):
    global _i32_types
    if _i32_types is None:
        _i32_types = (_torch().int32,)
    return _i32_types


def mla_append_cache_workspace_size(cfg, T) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_append_cache_workspace_size(ctypes.byref(cfg), int(T), ctypes.byref(n)),
           "mla_append_cache_workspace_size")
    return int(n.value)


def mla_append_cache(cfg, h, W_DKV_KR, req_ids, positions, block_table, cache, dev_status=None,
                     workspace=None, stream=None):
    """workspace: uint8 device tensor of mla_append_cache_workspace_size bytes (None if 0)."""
    a = (_act_dtype(cfg),)
    T = req_ids.numel()
    D = cfg.d_latent + cfg.d_rope
    batch, max_pages = block_table.shape
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    _check(lib().mla_append_cache(
        ctypes.byref(cfg), _peer_ptr(h, "h", a, T * cfg.d_model), _peer_ptr(W_DKV_KR, "W_DKV_KR", a, cfg.d_model * D),
        T, _peer_ptr(req_ids, "req_ids", _i32(0), T), _peer_ptr(positions, "positions", _i32(0), T),
        _peer_ptr(block_table, "block_table", _i32(0)), batch, max_pages,
        _peer_ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _peer_ptr(dev_status, "dev_status", _i32(0), allow_none=True),
        _peer_ptr(workspace, "workspace", (_torch().uint8,), allow_none=True),
        0 if workspace is None else workspace.numel(), _stream(stream)),
        "mla_append_cache")


def mla_append_cache_latent(cfg, c_kv, k_pe, req_ids, positions, block_table, cache, rotate=True,
                            dev_status=None, stream=None):
    a = (_act_dtype(cfg),)
    T = req_ids.numel()
    D = cfg.d_latent + cfg.d_rope
    batch, max_pages = block_table.shape
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    _check(lib().mla_append_cache_latent(
        ctypes.byref(cfg), _peer_ptr(c_kv, "c_kv", a, T * cfg.d_latent), _peer_ptr(k_pe, "k_pe", a, T * cfg.d_rope),
        T, _peer_ptr(req_ids, "req_ids", _i32(0), T), _peer_ptr(positions, "positions", _i32(0), T),
        _peer_ptr(block_table, "block_table", _i32(0)), batch, max_pages,
        _peer_ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        1 if rotate else 0, _peer_ptr(dev_status, "dev_status", _i32(0), allow_none=True),
        _stream(stream)), "mla_append_cache_latent")


def mla_decode_workspace_size(cfg, batch, q_len, num_workers=0, kernel=KERNEL_AUTO) -> int:
    n = ctypes.c_size_t(0)
    o = _opts(num_workers, kernel)
    _check(lib().mla_decode_workspace_size(ctypes.byref(cfg), int(batch), int(q_len), ctypes.byref(o),
                                           ctypes.byref(n)), "mla_decode_workspace_size")
    return int(n.value)


def mla_decode(cfg, q_nope, q_pe, W_UK_abs, cache, block_table, seq_lens, out_latent, lse,
               workspace, num_workers=0, kernel=KERNEL_AUTO, stream=None, attn_events=None,
               wait_limit_us=0, withhold_page=0):
    """attn_events: optional pair of torch.cuda.Event recorded around the attention kernel.
    wait_limit_us, withhold_page: testing hooks of the tensor-core kernel's failure path
    (see mla_decode_opts in include/mla.h)."""
    a = (_act_dtype(cfg),)
    t = _torch()
    batch, q_len = q_nope.shape[0], q_nope.shape[1]
    H, d_c, d_r, d_n = cfg.num_heads, cfg.d_latent, cfg.d_rope, cfg.d_nope
    D = d_c + d_r
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    max_pages = block_table.shape[1]
    o = _opts(num_workers, kernel, attn_events, wait_limit_us, withhold_page)
    _check(lib().mla_decode_ex(
        ctypes.byref(cfg), _peer_ptr(q_nope, "q_nope", a, batch * q_len * H * d_n),
        _peer_ptr(q_pe, "q_pe", a, batch * q_len * H * d_r),
        _peer_ptr(W_UK_abs, "W_UK_abs", a, H * d_n * d_c),
        _peer_ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _peer_ptr(block_table, "block_table", _i32(0), batch * max_pages), max_pages,
        _peer_ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len,
        _peer_ptr(out_latent, "out_latent", a, batch * q_len * H * d_c),
        _peer_ptr(lse, "lse", (t.float32,), batch * q_len * H),
        _peer_ptr(workspace, "workspace", (t.uint8,)), workspace.numel(), ctypes.byref(o),
        _stream(stream)), "mla_decode")


def mla_decode_noalloc(cfg, q_nope, q_pe, W_UK_abs, cache, block_table, seq_lens, out_latent, lse,
                       stream=None):
    """mla_decode with the library's fixed 64 MiB device scratch array instead of a workspace,
    for callers that cannot allocate device memory at decode time. Calls sharing the array
    must be ordered on the GPU; the first call on a device must come before any capture."""
    a = (_act_dtype(cfg),)
    t = _torch()
    batch, q_len = q_nope.shape[0], q_nope.shape[1]
    H, d_c, d_r, d_n = cfg.num_heads, cfg.d_latent, cfg.d_rope, cfg.d_nope
    D = d_c + d_r
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    max_pages = block_table.shape[1]
    _check(lib().mla_decode_noalloc(
        ctypes.byref(cfg), _peer_ptr(q_nope, "q_nope", a, batch * q_len * H * d_n),
        _peer_ptr(q_pe, "q_pe", a, batch * q_len * H * d_r),
        _peer_ptr(W_UK_abs, "W_UK_abs", a, H * d_n * d_c),
        _peer_ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _peer_ptr(block_table, "block_table", _i32(0), batch * max_pages), max_pages,
        _peer_ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len,
        _peer_ptr(out_latent, "out_latent", a, batch * q_len * H * d_c),
        _peer_ptr(lse, "lse", (t.float32,), batch * q_len * H), _stream(stream)), "mla_decode_noalloc")


def mla_decode_noalloc_status(stream=None) -> int:
    """Synchronises the stream and returns (then clears) the device status of the last
    mla_decode_noalloc on the current device."""
    code = ctypes.c_int(0)
    _check(lib().mla_decode_noalloc_status(_stream(stream), ctypes.byref(code)),
           "mla_decode_noalloc_status")
    return int(code.value)


def mla_output_proj_workspace_size(cfg, rows) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_output_proj_workspace_size(ctypes.byref(cfg), int(rows), ctypes.byref(n)),
           "mla_output_proj_workspace_size")
    return int(n.value)


def mla_output_proj(cfg, out_latent, W_comb, out, workspace, stream=None):
    a = (_act_dtype(cfg),)
    K = cfg.num_heads * cfg.d_latent
    rows = out_latent.numel() // K
    _check(lib().mla_output_proj(
        ctypes.byref(cfg), _peer_ptr(out_latent, "out_latent", a, rows * K),
        _peer_ptr(W_comb, "W_comb", a, K * cfg.d_model), rows, _peer_ptr(out, "out", a, rows * cfg.d_model),
        _peer_ptr(workspace, "workspace", (_torch().uint8,)), workspace.numel(), _stream(stream)),
        "mla_output_proj")


def mla_output_proj_unfolded_workspace_size(cfg, rows) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_output_proj_unfolded_workspace_size(ctypes.byref(cfg), int(rows),
                                                         ctypes.byref(n)),
           "mla_output_proj_unfolded_workspace_size")
    return int(n.value)


def mla_output_proj_unfolded(cfg, out_latent, W_UV, W_O, out, workspace, stream=None):
    a = (_act_dtype(cfg),)
    K = cfg.num_heads * cfg.d_latent
    HV = cfg.num_heads * cfg.d_v
    rows = out_latent.numel() // K
    _check(lib().mla_output_proj_unfolded(
        ctypes.byref(cfg), _peer_ptr(out_latent, "out_latent", a, rows * K),
        _peer_ptr(W_UV, "W_UV", a, cfg.d_latent * HV), _peer_ptr(W_O, "W_O", a, HV * cfg.d_model), rows,
        _peer_ptr(out, "out", a, rows * cfg.d_model),
        _peer_ptr(workspace, "workspace", (_torch().uint8,)), workspace.numel(), _stream(stream)),
        "mla_output_proj_unfolded")


def mla_cache_row_bytes(cfg) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_cache_row_bytes(ctypes.byref(cfg), ctypes.byref(n)), "mla_cache_row_bytes")
    return int(n.value)


def mla_query_workspace_size(cfg, d_q, T) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_query_workspace_size(ctypes.byref(cfg), int(d_q), int(T), ctypes.byref(n)),
           "mla_query_workspace_size")
    return int(n.value)


def mla_query_from_hidden(cfg, d_q, h, W_DQ, W_UQ, W_QR, q_nope, q_pe, workspace, stream=None):
    """h [T][d_model] -> q_nope [T][H][d_n], q_pe [T][H][d_r] (not rotated)."""
    a = (_act_dtype(cfg),)
    d, H = cfg.d_model, cfg.num_heads
    T = h.numel() // d
    _check(lib().mla_query_from_hidden(
        ctypes.byref(cfg), int(d_q), _peer_ptr(h, "h", a, T * d), _peer_ptr(W_DQ, "W_DQ", a, d * d_q),
        _peer_ptr(W_UQ, "W_UQ", a, d_q * H * cfg.d_nope), _peer_ptr(W_QR, "W_QR", a, d * H * cfg.d_rope), T,
        _peer_ptr(q_nope, "q_nope", a, T * H * cfg.d_nope), _peer_ptr(q_pe, "q_pe", a, T * H * cfg.d_rope),
        _peer_ptr(workspace, "workspace", (_torch().uint8,)), workspace.numel(), _stream(stream)),
        "mla_query_from_hidden")


def mla_prefix_expand(cfg, W_UK, W_UV, cache, prefix_pages, prefix_len, keys, values, k_pe,
                      dev_status=None, stream=None):
    """keys [H][L][d_n], values [H][L][d_v], k_pe [L][d_r] of the first L = prefix_len tokens on
    prefix_pages (int32, at least ceil(L / page_size) entries)."""
    a = (_act_dtype(cfg),)
    H, d_c, d_n, d_v, L = cfg.num_heads, cfg.d_latent, cfg.d_nope, cfg.d_v, int(prefix_len)
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    if prefix_pages.numel() * cfg.page_size < L:
        raise ValueError(f"prefix_pages has {prefix_pages.numel()} pages, too few for {L} tokens")
    _check(lib().mla_prefix_expand(
        ctypes.byref(cfg), _ptr(W_UK, "W_UK", a, d_c * H * d_n), _ptr(W_UV, "W_UV", a, d_c * H * d_v),
        _ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _ptr(prefix_pages, "prefix_pages", _i32(0)), L, _ptr(keys, "keys", a, H * L * d_n),
        _ptr(values, "values", a, H * L * d_v), _ptr(k_pe, "k_pe", a, L * cfg.d_rope),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_prefix_expand")


def mla_prefix_attend_workspace_size(cfg, batch, q_len, prefix_len) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_prefix_attend_workspace_size(ctypes.byref(cfg), int(batch), int(q_len),
                                                  int(prefix_len), ctypes.byref(n)),
           "mla_prefix_attend_workspace_size")
    return int(n.value)


def mla_prefix_attend(cfg, q_nope, q_pe, keys, values, k_pe, seq_lens, u, lse, workspace=None,
                      dev_status=None, stream=None):
    """q_nope [B][q_len][H][d_n]; the prefix length is k_pe's. workspace: uint8 device tensor of
    mla_prefix_attend_workspace_size bytes (None if 0)."""
    a = (_act_dtype(cfg),)
    t = _torch()
    batch, q_len = q_nope.shape[0], q_nope.shape[1]
    H, d_n, d_r, d_v = cfg.num_heads, cfg.d_nope, cfg.d_rope, cfg.d_v
    L = k_pe.numel() // d_r
    _check(lib().mla_prefix_attend(
        ctypes.byref(cfg), _ptr(q_nope, "q_nope", a, batch * q_len * H * d_n),
        _ptr(q_pe, "q_pe", a, batch * q_len * H * d_r), _ptr(keys, "keys", a, H * L * d_n),
        _ptr(values, "values", a, H * L * d_v), _ptr(k_pe, "k_pe", a, L * d_r), L,
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len,
        _ptr(u, "u", a, batch * q_len * H * d_v), _ptr(lse, "lse", (t.float32,), batch * q_len * H),
        _ptr(workspace, "workspace", (t.uint8,), allow_none=True),
        0 if workspace is None else workspace.numel(),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_prefix_attend")


def mla_output_proj_prefix_workspace_size(cfg, rows) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_output_proj_prefix_workspace_size(ctypes.byref(cfg), int(rows), ctypes.byref(n)),
           "mla_output_proj_prefix_workspace_size")
    return int(n.value)


def mla_output_proj_prefix(cfg, out_latent, lse, u_prefix, lse_prefix, W_UV, W_O, out, workspace,
                           stream=None):
    a = (_act_dtype(cfg),)
    t = _torch()
    H, d_c, d_v, d = cfg.num_heads, cfg.d_latent, cfg.d_v, cfg.d_model
    rows = out_latent.numel() // (H * d_c)
    _check(lib().mla_output_proj_prefix(
        ctypes.byref(cfg), _ptr(out_latent, "out_latent", a, rows * H * d_c),
        _ptr(lse, "lse", (t.float32,), rows * H), _ptr(u_prefix, "u_prefix", a, rows * H * d_v),
        _ptr(lse_prefix, "lse_prefix", (t.float32,), rows * H), _ptr(W_UV, "W_UV", a, d_c * H * d_v),
        _ptr(W_O, "W_O", a, H * d_v * d), rows, _ptr(out, "out", a, rows * d),
        _ptr(workspace, "workspace", (t.uint8,)), workspace.numel(), _stream(stream)),
        "mla_output_proj_prefix")


def mla_absorb_query(cfg, q_nope, q_pe, W_UK_abs, seq_lens, q_lat, stream=None):
    """q_lat [B][q_len][H][d_c + d_r] from q_nope, q_pe [B][q_len][H][..] (mla_decode's query)."""
    a = (_act_dtype(cfg),)
    batch, q_len = q_nope.shape[0], q_nope.shape[1]
    H, d_c, d_r, d_n = cfg.num_heads, cfg.d_latent, cfg.d_rope, cfg.d_nope
    _check(lib().mla_absorb_query(
        ctypes.byref(cfg), _ptr(q_nope, "q_nope", a, batch * q_len * H * d_n),
        _ptr(q_pe, "q_pe", a, batch * q_len * H * d_r), _ptr(W_UK_abs, "W_UK_abs", a, H * d_n * d_c),
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len,
        _ptr(q_lat, "q_lat", a, batch * q_len * H * (d_c + d_r)), _stream(stream)), "mla_absorb_query")


def mla_key_weights(cfg, q_lat, lse, cache, block_table, seq_lens, weights, decay=1.0, dev_status=None,
                    stream=None):
    """q_lat [B][q_len][H][d_c + d_r]; weights [B][max_pages * page_size] fp32, updated in place."""
    a = (_act_dtype(cfg),)
    t = _torch()
    batch, q_len = q_lat.shape[0], q_lat.shape[1]
    max_pages = block_table.shape[1]
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    _check(lib().mla_key_weights(
        ctypes.byref(cfg), _ptr(q_lat, "q_lat", a, batch * q_len * cfg.num_heads * (cfg.d_latent + cfg.d_rope)),
        _ptr(lse, "lse", (t.float32,), batch * q_len * cfg.num_heads),
        _ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _ptr(block_table, "block_table", _i32(0), batch * max_pages), max_pages,
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len, float(decay),
        _ptr(weights, "weights", (t.float32,), batch * max_pages * cfg.page_size),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_key_weights")


def mla_evict_cache(cfg, weights, seq_lens, block_table, cache, budget, kept, new_seq_lens,
                    new_block_table=None, new_weights=None, sinks=0, recent=0, rotate=True,
                    dev_status=None, stream=None):
    """Cuts every request to at most `budget` tokens; new_block_table None: in place. kept
    [B][budget] and new_seq_lens [B] int32 are outputs; new_weights (optional) gets the kept
    tokens' weights, new_seq_lens may be seq_lens."""
    t = _torch()
    batch, max_pages = block_table.shape
    if new_block_table is None:
        new_block_table = block_table
    new_max = new_block_table.shape[1]
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    _check(lib().mla_evict_cache(
        ctypes.byref(cfg), _ptr(weights, "weights", (t.float32,), batch * max_pages * cfg.page_size),
        _ptr(seq_lens, "seq_lens", _i32(0), batch), _ptr(block_table, "block_table", _i32(0), batch * max_pages),
        max_pages, batch, int(budget), int(sinks), int(recent), 1 if rotate else 0,
        _ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _ptr(new_block_table, "new_block_table", _i32(0), batch * new_max), new_max,
        _ptr(new_weights, "new_weights", (t.float32,), batch * new_max * cfg.page_size, allow_none=True),
        _ptr(kept, "kept", _i32(0), batch * max(int(budget), 0)),
        _ptr(new_seq_lens, "new_seq_lens", _i32(0), batch),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_evict_cache")


def mla_page_keys(cfg, cache, block_table, seq_lens, page_keys, new_tokens=None, dev_status=None,
                  stream=None):
    """page_keys [num_pages][d_c + d_r]: means of the pages that hold any of each request's last
    new_tokens tokens (None: of all its pages)."""
    batch, max_pages = block_table.shape
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    new = max_pages * cfg.page_size if new_tokens is None else new_tokens
    _check(lib().mla_page_keys(
        ctypes.byref(cfg),
        _ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _ptr(block_table, "block_table", _i32(0), batch * max_pages), max_pages,
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, min(int(new), 2 ** 31 - 1),
        _ptr(page_keys, "page_keys", (_act_dtype(cfg),), num_pages * (cfg.d_latent + cfg.d_rope)),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_page_keys")


def mla_page_scores_workspace_size(cfg, batch, q_len, max_pages) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_page_scores_workspace_size(ctypes.byref(cfg), int(batch), int(q_len), int(max_pages),
                                                ctypes.byref(n)), "mla_page_scores_workspace_size")
    return int(n.value)


def mla_page_scores(cfg, q_lat, page_keys, block_table, seq_lens, scores, workspace=None, dev_status=None,
                    stream=None):
    """q_lat [B][q_len][H][d_c + d_r] (mla_absorb_query) -> scores [B][q_len][max_pages] fp32. workspace:
    uint8 device tensor of mla_page_scores_workspace_size bytes."""
    a = (_act_dtype(cfg),)
    t = _torch()
    batch, q_len = q_lat.shape[0], q_lat.shape[1]
    max_pages = block_table.shape[1]
    D = cfg.d_latent + cfg.d_rope
    num_pages = page_keys.numel() // D
    _check(lib().mla_page_scores(
        ctypes.byref(cfg), _ptr(q_lat, "q_lat", a, batch * q_len * cfg.num_heads * D),
        _ptr(page_keys, "page_keys", a, num_pages * D), num_pages,
        _ptr(block_table, "block_table", _i32(0), batch * max_pages), max_pages,
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len,
        _ptr(scores, "scores", (t.float32,), batch * q_len * max_pages),
        _ptr(workspace, "workspace", (t.uint8,), allow_none=True),
        0 if workspace is None else workspace.numel(),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_page_scores")


def mla_select_pages(cfg, scores, seq_lens, pages, sinks=0, recent=1, dev_status=None, stream=None):
    """scores [B][q_len][max_pages] fp32 -> pages [B][q_len][budget] int32, ascending, then -1."""
    t = _torch()
    batch, q_len, max_pages = scores.shape
    budget = pages.shape[2]
    _check(lib().mla_select_pages(
        ctypes.byref(cfg), _ptr(scores, "scores", (t.float32,)), max_pages,
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len, budget, int(sinks), int(recent),
        _ptr(pages, "pages", _i32(0), batch * q_len * budget),
        _ptr(dev_status, "dev_status", _i32(0), allow_none=True), _stream(stream)), "mla_select_pages")


def mla_decode_pages_workspace_size(cfg, batch, q_len, budget) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_decode_pages_workspace_size(ctypes.byref(cfg), int(batch), int(q_len), int(budget),
                                                 ctypes.byref(n)), "mla_decode_pages_workspace_size")
    return int(n.value)


def mla_decode_pages(cfg, q_lat, cache, block_table, seq_lens, pages, out_latent, lse, workspace, stream=None):
    """Attention over the pages [B][q_len][budget] of each query token; q_lat [B][q_len][H][d_c + d_r]
    from mla_absorb_query. workspace: its first int32 is the call's status word, as in mla_decode."""
    a = (_act_dtype(cfg),)
    t = _torch()
    batch, q_len = q_lat.shape[0], q_lat.shape[1]
    H, d_c, D = cfg.num_heads, cfg.d_latent, cfg.d_latent + cfg.d_rope
    budget, max_pages = pages.shape[2], block_table.shape[1]
    num_pages = cache.numel() // (cfg.page_size * _cache_row_elems(cfg))
    _check(lib().mla_decode_pages(
        ctypes.byref(cfg), _ptr(q_lat, "q_lat", a, batch * q_len * H * D),
        _ptr(cache, "cache", _cache_dtypes(cfg), num_pages * cfg.page_size * _cache_row_elems(cfg)), num_pages,
        _ptr(block_table, "block_table", _i32(0), batch * max_pages), max_pages,
        _ptr(seq_lens, "seq_lens", _i32(0), batch), batch, q_len,
        _ptr(pages, "pages", _i32(0), batch * q_len * budget), budget,
        _ptr(out_latent, "out_latent", a, batch * q_len * H * d_c),
        _ptr(lse, "lse", (t.float32,), batch * q_len * H),
        _ptr(workspace, "workspace", (t.uint8,)), workspace.numel(), _stream(stream)), "mla_decode_pages")


def mla_mx4_bytes(cfg, K, N):
    """Bytes of the codes and of the scales of a 4-bit weight [K][N]."""
    c, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().mla_mx4_bytes(ctypes.byref(cfg), int(K), int(N), ctypes.byref(c), ctypes.byref(s)),
           "mla_mx4_bytes")
    return int(c.value), int(s.value)


def _mx4(cfg, K, N, codes, scales):
    # (the sizes of mla_mx4_bytes, without a call; K and N are checked by the call that follows)
    u8 = (_torch().uint8,)
    return (_ptr(codes, "codes", u8, N * (K // 2)),
            _ptr(scales, "scales", u8, -(-N // 128) * -(-K // 128) * 512))


def mla_mx4_quantize(cfg, W, codes, scales, stream=None):
    """W [K][N] -> codes [N][K / 2], scales (uint8 tensors of mla_mx4_bytes bytes)."""
    K, N = W.shape
    c, s = _mx4(cfg, K, N, codes, scales)
    _check(lib().mla_mx4_quantize(ctypes.byref(cfg), _ptr(W, "W", (_act_dtype(cfg),), K * N), K, N, c, s,
                                  _stream(stream)), "mla_mx4_quantize")


def mla_mx4_dequantize(cfg, codes, scales, W, stream=None):
    """codes, scales -> their values W [K][N]."""
    K, N = W.shape
    c, s = _mx4(cfg, K, N, codes, scales)
    _check(lib().mla_mx4_dequantize(ctypes.byref(cfg), c, s, K, N, _ptr(W, "W", (_act_dtype(cfg),), K * N),
                                    _stream(stream)), "mla_mx4_dequantize")


def mla_mx4_project_workspace_size(cfg, K, N, rows) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mla_mx4_project_workspace_size(ctypes.byref(cfg), int(K), int(N), int(rows), ctypes.byref(n)),
           "mla_mx4_project_workspace_size")
    return int(n.value)


def mla_mx4_project(cfg, x, codes, scales, out, workspace=None, stream=None):
    """out [rows][N] = x [rows][K] times the 4-bit weight. workspace: uint8 device tensor of
    mla_mx4_project_workspace_size bytes (None if 0); its first int32 is the call's status word."""
    a = (_act_dtype(cfg),)
    rows, K = x.shape
    N = out.shape[1]
    c, s = _mx4(cfg, K, N, codes, scales)
    _check(lib().mla_mx4_project(
        ctypes.byref(cfg), _ptr(x, "x", a, rows * K), c, s, K, N, rows, _ptr(out, "out", a, rows * N),
        _ptr(workspace, "workspace", (_torch().uint8,), allow_none=True),
        0 if workspace is None else workspace.numel(), _stream(stream)), "mla_mx4_project")


def mla_read_device_status(status_word, stream=None) -> int:
    """Synchronises the stream and returns (then clears) the device status code."""
    code = ctypes.c_int(0)
    _check(lib().mla_read_device_status(_peer_ptr(status_word, "status_word"), _stream(stream),
                                        ctypes.byref(code)), "mla_read_device_status")
    return int(code.value)
