"""Thin ctypes binding over libmla's C ABI (include/mla.h).

Argument marshalling only: tensors are passed as raw device pointers, the
stream as the raw CUDA stream handle.  Every computation runs in libmla's
kernels; importing this module fails loudly when libmla.so is missing.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Dict, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmla.so")

MLA_OK = 0
STATUS = {0: "MLA_OK", -1: "MLA_ERR_INVALID_ARG", -2: "MLA_ERR_UNSUPPORTED", -3: "MLA_ERR_WORKSPACE",
          -4: "MLA_ERR_CUDA", -5: "MLA_ERR_DEVICE_BOUNDS", -6: "MLA_ERR_TIMEOUT"}
F32, BF16 = 0, 1

EXPORTED = [
    "mla_absorbed_weights_bytes", "mla_absorb_weights", "mla_release_weights", "mla_weights_dims",
    "mla_append_workspace_bytes", "mla_append_latent", "mla_decode_workspace_bytes", "mla_decode",
    "mla_prefill_workspace_bytes", "mla_prefill", "mla_get_error", "mla_status_string",
    "mla_last_launch_count", "mla_profile_begin", "mla_profile_end", "mla_append_latent_noalloc",
    "mla_decode_cp_workspace_bytes", "mla_decode_cp_partial", "mla_decode_cp_combine",
    "mla_selftest_wait_timeout", "mla_prefill_materialised_workspace_bytes", "mla_prefill_materialised",
    "mla_decode_step_workspace_bytes", "mla_decode_step", "mla_plan_step", "mla_append_normed",
    "mla_query_norm_rope", "mla_attend_ragged_workspace_bytes", "mla_attend_ragged",
    "mla_ragged_step_workspace_bytes", "mla_ragged_step",
]
APPEND_NOALLOC_MAX_T = 256


class MlaError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str = ""):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}" + (f" ({detail})" if detail else ""))
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("n_h", ctypes.c_int), ("d_h", ctypes.c_int), ("d_v", ctypes.c_int), ("d_c", ctypes.c_int),
                ("d_r", ctypes.c_int), ("d_model", ctypes.c_int), ("d_cq", ctypes.c_int),
                ("rope_base", ctypes.c_float), ("softmax_scale", ctypes.c_float), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int), ("rope_key_per_head", ctypes.c_int)]


def make_dims(n_h, d_h, d_v, d_c, d_r, d_model, d_cq=0, rope_base=10000.0, softmax_scale=0.0,
              page_size=64, dtype=BF16, rope_key_per_head=0) -> Dims:
    return Dims(n_h, d_h, d_v, d_c, d_r, d_model, d_cq, rope_base, softmax_scale, page_size, dtype,
                int(rope_key_per_head))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmla.so not built ({LIB_PATH}); run head_latent_attention_append_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int
    L, F = ctypes.c_int64, ctypes.c_float
    D = ctypes.POINTER(Dims)
    sig = {
        "mla_absorbed_weights_bytes": (Z, [D]),
        "mla_absorb_weights": (S, [D, P, P, P, P, P, P, P, P, Z, ctypes.POINTER(P), P]),
        "mla_release_weights": (None, [P]),
        "mla_weights_dims": (S, [P, D]),
        "mla_append_workspace_bytes": (Z, [D, I]),
        "mla_append_latent": (S, [P, P, P, P, P, I, I, I, P, I, P, Z, P]),
        "mla_decode_workspace_bytes": (Z, [D, I, I, I]),
        "mla_decode": (S, [P, P, P, P, I, I, P, P, I, I, I, P, Z, P]),
        "mla_decode_step_workspace_bytes": (Z, [D, I, I, I]),
        "mla_decode_step": (S, [P, P, P, P, I, I, P, P, I, I, I, P, Z, P]),
        "mla_prefill_workspace_bytes": (Z, [D, I, I]),
        "mla_prefill": (S, [P, P, P, I, I, P, P, I, I, P, Z, P]),
        "mla_get_error": (S, [P, P]),
        "mla_status_string": (ctypes.c_char_p, [S]),
        "mla_last_launch_count": (I, []),
        "mla_profile_begin": (S, [I]),
        "mla_append_latent_noalloc": (S, [P, P, P, P, P, I, I, I, P, I, P, P]),
        "mla_profile_end": (S, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]),
        "mla_decode_cp_workspace_bytes": (Z, [D, I, I]),
        "mla_decode_cp_partial": (S, [P, P, P, P, P, P, I, I, P, P, P, I, I, I, P, Z, P]),
        "mla_decode_cp_combine": (S, [P, I, P, P, P, I, I, P, Z, P]),
        "mla_selftest_wait_timeout": (S, [P, I, P]),
        "mla_prefill_materialised_workspace_bytes": (Z, [D, I, I]),
        "mla_prefill_materialised": (S, [P, P, P, I, I, P, P, I, I, P, Z, P]),
        "mla_plan_step": (S, [P, P, I, P, I, P, I, I, P, P, P, P, P, I, P, P, P]),
        "mla_append_normed": (S, [D, P, L, P, P, L, P, P, L, F, P, P, P, I, I, P, P]),
        "mla_query_norm_rope": (S, [D, P, L, P, F, P, P, L, L, P, L, L, I, P]),
        "mla_attend_ragged_workspace_bytes": (Z, [D, I, I]),
        "mla_ragged_step_workspace_bytes": (Z, [D, I, I]),
        "mla_ragged_step": (S, [P, P, P, P, P, P, P, I, I, P, P, I, I, P, Z, P]),
        "mla_attend_ragged": (S, [D, P, L, L, P, P, P, I, I, P, P, P, I, I, P, Z, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def _check(fn: str, code: int):
    if code != MLA_OK:
        raise MlaError(fn, code)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def absorbed_weights_bytes(dims: Dims) -> int:
    return lib.mla_absorbed_weights_bytes(ctypes.byref(dims))


def append_workspace_bytes(dims: Dims, T: int) -> int:
    return lib.mla_append_workspace_bytes(ctypes.byref(dims), T)


def decode_workspace_bytes(dims: Dims, B: int, n_q: int, max_kv_len: int) -> int:
    return lib.mla_decode_workspace_bytes(ctypes.byref(dims), B, n_q, max_kv_len)


def decode_step_workspace_bytes(dims: Dims, B: int, n_q: int, max_kv_len: int) -> int:
    return lib.mla_decode_step_workspace_bytes(ctypes.byref(dims), B, n_q, max_kv_len)


def prefill_workspace_bytes(dims: Dims, B: int, S: int) -> int:
    return lib.mla_prefill_workspace_bytes(ctypes.byref(dims), B, S)


def last_launch_count() -> int:
    return lib.mla_last_launch_count()


def profile_begin(max_launches: int):
    _check("mla_profile_begin", lib.mla_profile_begin(max_launches))


def profile_end():
    """Returns (summed attention-kernel milliseconds, timed launches)."""
    ms, n = ctypes.c_double(), ctypes.c_int()
    _check("mla_profile_end", lib.mla_profile_end(ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


class Weights:
    """Absorbed weights: a caller-owned device buffer plus libmla's handle."""

    def __init__(self, dims: Dims, W: Dict[str, "torch.Tensor"], stream=None):
        import torch
        self.dims = dims
        nbytes = absorbed_weights_bytes(dims)
        if nbytes == 0:
            raise MlaError("mla_absorbed_weights_bytes", -2)
        dev = W["W_DKV"].device
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        h = ctypes.c_void_p()
        _check("mla_absorb_weights", lib.mla_absorb_weights(
            ctypes.byref(dims), _ptr(W["W_DKV"]), _ptr(W["W_KR"]), _ptr(W.get("W_DQ")), _ptr(W["W_UQ"]),
            _ptr(W["W_QR"]), _ptr(W["W_UK"]), _ptr(W["W_UV"]), self.buffer.data_ptr(), nbytes, ctypes.byref(h),
            _stream(stream)))
        self.handle = h

    def close(self):
        if self.handle:
            lib.mla_release_weights(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def append_latent(w: Weights, h, seq_idx, pos, page_table, num_pages: int, cache, workspace, stream=None):
    T = h.shape[0]
    num_seqs, max_pages = page_table.shape
    _check("mla_append_latent", lib.mla_append_latent(
        w.handle, _ptr(h), _ptr(seq_idx), _ptr(pos), _ptr(page_table), num_seqs, max_pages, num_pages,
        _ptr(cache), T, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def append_latent_noalloc(w: Weights, h, seq_idx, pos, page_table, num_pages: int, cache, device_error=None,
                          stream=None):
    """mla_append_latent without a workspace (scratch inside libmla; T <= 256)."""
    T = h.shape[0]
    num_seqs, max_pages = page_table.shape
    _check("mla_append_latent_noalloc", lib.mla_append_latent_noalloc(
        w.handle, _ptr(h), _ptr(seq_idx), _ptr(pos), _ptr(page_table), num_seqs, max_pages, num_pages,
        _ptr(cache), T, _ptr(device_error), _stream(stream)))


def decode(w: Weights, h_q, kv_len, page_table, num_pages: int, cache, out, max_kv_len: int, workspace,
           stream=None):
    B, n_q = h_q.shape[0], h_q.shape[1]
    _check("mla_decode", lib.mla_decode(
        w.handle, _ptr(h_q), _ptr(kv_len), _ptr(page_table), page_table.shape[1], num_pages, _ptr(cache),
        _ptr(out), B, n_q, max_kv_len, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def decode_step(w: Weights, h, kv_len, page_table, num_pages: int, cache, out, max_kv_len: int, workspace,
                stream=None):
    """Append the new tokens' latent rows, then decode them (one call)."""
    B, n_q = h.shape[0], h.shape[1]
    _check("mla_decode_step", lib.mla_decode_step(
        w.handle, _ptr(h), _ptr(kv_len), _ptr(page_table), page_table.shape[1], num_pages, _ptr(cache),
        _ptr(out), B, n_q, max_kv_len, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def prefill(w: Weights, h, page_table, num_pages: int, cache, out, workspace, stream=None):
    B, S = h.shape[0], h.shape[1]
    _check("mla_prefill", lib.mla_prefill(
        w.handle, _ptr(h), _ptr(page_table), page_table.shape[1], num_pages, _ptr(cache), _ptr(out), B, S,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def prefill_materialised_workspace_bytes(dims: Dims, B: int, S: int) -> int:
    return lib.mla_prefill_materialised_workspace_bytes(ctypes.byref(dims), B, S)


def prefill_materialised(w: Weights, h, page_table, num_pages: int, cache, out, workspace, stream=None):
    """Causal prefill through expanded per-head keys and values (include/mla.h)."""
    B, S = h.shape[0], h.shape[1]
    _check("mla_prefill_materialised", lib.mla_prefill_materialised(
        w.handle, _ptr(h), _ptr(page_table), page_table.shape[1], num_pages, _ptr(cache), _ptr(out), B, S,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def decode_cp_workspace_bytes(dims: Dims, B: int, n_q: int) -> int:
    return lib.mla_decode_cp_workspace_bytes(ctypes.byref(dims), B, n_q)


def decode_cp_partial(w: Weights, h_q, kv_len, window_start, window_count, page_table, num_pages: int, cache,
                      obar_out, lse_out, max_kv_len: int, workspace, stream=None):
    """This rank's share of a context-parallel decode step (include/mla.h)."""
    B, n_q = h_q.shape[0], h_q.shape[1]
    _check("mla_decode_cp_partial", lib.mla_decode_cp_partial(
        w.handle, _ptr(h_q), _ptr(kv_len), _ptr(window_start), _ptr(window_count), _ptr(page_table),
        page_table.shape[1], num_pages, _ptr(cache), _ptr(obar_out), _ptr(lse_out), B, n_q, max_kv_len,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def decode_cp_combine(w: Weights, obar_parts, lse_parts, out, workspace, stream=None):
    """Merges all ranks' partials [n_ranks, B, n_q, ...] into out [B, n_q, n_h, d_v]."""
    n_ranks, B, n_q = obar_parts.shape[0], obar_parts.shape[1], obar_parts.shape[2]
    _check("mla_decode_cp_combine", lib.mla_decode_cp_combine(
        w.handle, n_ranks, _ptr(obar_parts), _ptr(lse_parts), _ptr(out), B, n_q, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


# ---------------------------------------------------------------- ragged step
# These calls go through a compiled module, which checks every tensor's type,
# device, shape and layout (sizes are taken from the shapes) and calls libmla:
# in Python that costs several times what the kernels take at decode sizes.  It
# answers 1, without having called libmla, when a tensor is not the call's; the
# checks below then find the one to name.
_ragged = None


def _module():
    global _ragged
    if _ragged is None:
        import torch  # noqa: F401  (its libraries, which the module is linked to)
        try:
            from . import _ragged as m
        except ImportError as e:
            raise ImportError(f"_ragged.so cannot be loaded ({e}); run head_latent_attention_append_b200/build.py") from e
        _ragged = m
    return _ragged


def _path_dtype(dims: Dims):
    import torch
    return torch.bfloat16 if dims.dtype == BF16 else torch.float32


def _refuse(fn: str, code: int, tensors):
    """Raises for a call that answered `code`.  Each tensor: (name, tensor or None, dtype, shape (None: any size),
    packed: contiguous, else with a contiguous last axis); dtype or shape None: any; the first one on a GPU gives the
    device."""
    import torch
    if code != 1:
        raise MlaError(fn, code)
    devices = [t.device for _, t, *_ in tensors if isinstance(t, torch.Tensor)]
    device = next((d for d in devices if d.type == "cuda"), devices[0])
    for name, t, dtype, shape, packed in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise MlaError(fn, -1, f"{name}: a tensor is expected")
        got = tuple(t.shape)
        if dtype is not None and t.dtype != dtype:
            raise MlaError(fn, -1, f"{name}: {t.dtype}, expected {dtype}")
        if shape is not None and (len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got))):
            raise MlaError(fn, -1, f"{name}: shape {got}, expected {tuple('any' if w is None else w for w in shape)}")
        if t.device != device:
            raise MlaError(fn, -1, f"{name} is on {t.device}, expected {device}")
        if not (t.is_contiguous() if packed else (t.stride(-1) == 1 or got[-1] <= 1)):
            raise MlaError(fn, -1, f"{name}: not contiguous" + ("" if packed else " along the last axis"))
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise MlaError(fn, -1, f"tensors are on {device}, expected the current CUDA device")
    raise MlaError(fn, -1, "an argument is missing or of another kind")


def _sized(fn: str, code: int, name: str, t, dims: int) -> int:
    """The first size of the tensor that gives a call its size, where the call answered `code`."""
    import torch
    if code != 1:
        raise MlaError(fn, code)
    if not isinstance(t, torch.Tensor):
        raise MlaError(fn, -1, f"{name}: a tensor is expected")
    if t.dim() != dims:
        raise MlaError(fn, -1, f"{name}: shape {tuple(t.shape)}, expected {dims} axes")
    return t.shape[0]


def plan_step(new_len, past_len, free_pages, page_table, num_pages: int, q_start, kv_len, seq_idx, pos, slot, counts,
              device_error=None, stream=None):
    """Page-table entries, slots and positions of a ragged step from the requests' lengths (include/mla.h)."""
    s = (_ragged or _module()).plan_step(new_len, past_len, free_pages, page_table, num_pages, q_start, kv_len, seq_idx,
                                         pos, slot, counts, device_error, stream)
    if s:
        import torch
        fn, i32 = "mla_plan_step", torch.int32
        B, rows = _sized(fn, s, "new_len", new_len, 1), _sized(fn, s, "seq_idx", seq_idx, 1)
        _refuse(fn, s, (
            ("new_len", new_len, i32, (B,), True), ("past_len", past_len, i32, (B,), True),
            ("free_pages", free_pages, i32, (None,), True), ("page_table", page_table, i32, (B, None), True),
            ("q_start", q_start, i32, (B + 1,), True), ("kv_len", kv_len, i32, (B,), True),
            ("seq_idx", seq_idx, i32, (rows,), True), ("pos", pos, i32, (rows,), True),
            ("slot", slot, torch.int64, (rows,), True), ("counts", counts, i32, (3,), True),
            ("device_error", device_error, i32, (1,), True)))


def append_normed(dims: Dims, kv, kv_gamma, pos, slot, cache, eps: float = 1e-6, cq=None, cq_gamma=None, cq_out=None,
                  device_error=None, stream=None):
    """RMS norms of the latents, rotation of the position key and the write into the paged cache (include/mla.h)."""
    s = (_ragged or _module()).append_normed(dims, kv, kv_gamma, pos, slot, cache, eps, cq, cq_gamma, cq_out,
                                             device_error, stream)
    if s:
        import torch
        fn, dt = "mla_append_normed", _path_dtype(dims)
        T, row = _sized(fn, s, "kv", kv, 2), dims.d_c + (dims.n_h if dims.rope_key_per_head else 1) * dims.d_r
        if (cq is None) != (cq_out is None):
            raise MlaError(fn, -1, "cq and cq_out go together")
        _refuse(fn, s, (
            ("kv", kv, dt, (T, row), False), ("kv_gamma", kv_gamma, dt, (dims.d_c,), True),
            ("pos", pos, torch.int32, (T,), True), ("slot", slot, torch.int64, (T,), True),
            ("cache", cache, dt, (None, dims.page_size, row), True), ("cq", cq, dt, (T, dims.d_cq), False),
            ("cq_gamma", cq_gamma, dt, (dims.d_cq,), True), ("cq_out", cq_out, dt, (T, dims.d_cq), False),
            ("device_error", device_error, torch.int32, (1,), True)))


def query_norm_rope(dims: Dims, q, gamma, pos, qc_out, qr_out, eps: float = 1e-6, stream=None):
    """RMS norm of every query head's content and rotation of its position part (include/mla.h)."""
    s = (_ragged or _module()).query_norm_rope(dims, q, gamma, pos, qc_out, qr_out, eps, stream)
    if s:
        import torch
        fn, dt, n_h, d_h, d_r = "mla_query_norm_rope", _path_dtype(dims), dims.n_h, dims.d_h, dims.d_r
        T = _sized(fn, s, "q", q, 3)
        if n_h > 1 and q.shape[1:] == (n_h, d_h + d_r) and q.stride(1) != d_h + d_r:
            raise MlaError(fn, -1, "q: a token's heads have to be contiguous")
        _refuse(fn, s, (
            ("q", q, dt, (T, n_h, d_h + d_r), False), ("gamma", gamma, dt, (d_h,), True),
            ("pos", pos, torch.int32, (T,), True), ("qc_out", qc_out, dt, (T, n_h, d_h), False),
            ("qr_out", qr_out, dt, (T, n_h, d_r), False)))


def attend_ragged_workspace_bytes(dims: Dims, B: int, T: int) -> int:
    return lib.mla_attend_ragged_workspace_bytes(ctypes.byref(dims), B, T)


def attend_ragged(dims: Dims, q, q_start, kv_len, page_table, cache, out, lse, workspace, stream=None):
    """Absorbed attention of every request's new tokens over its paged cache (include/mla.h)."""
    s = (_ragged or _module()).attend_ragged(dims, q, q_start, kv_len, page_table, cache, out, lse, workspace, stream)
    if s:
        import torch
        fn, dt, i32, n_h, row = "mla_attend_ragged", _path_dtype(dims), torch.int32, dims.n_h, dims.d_c + dims.d_r
        T, B = _sized(fn, s, "q", q, 3), _sized(fn, s, "kv_len", kv_len, 1)
        _refuse(fn, s, (
            ("q", q, dt, (T, n_h, row), False), ("q_start", q_start, i32, (B + 1,), True),
            ("kv_len", kv_len, i32, (B,), True), ("page_table", page_table, i32, (B, None), True),
            ("cache", cache, dt, (None, dims.page_size, row), True), ("out", out, dt, (T, n_h, dims.d_c), True),
            ("lse", lse, torch.float32, (T, n_h), True),
            ("workspace", workspace, None, None, True)))


def ragged_step_workspace_bytes(dims: Dims, B: int, T: int) -> int:
    return lib.mla_ragged_step_workspace_bytes(ctypes.byref(dims), B, T)


def ragged_step(w: Weights, h, q_start, kv_len, seq_idx, pos, page_table, num_pages: int, cache, out, workspace,
                stream=None):
    """Append and attention of every request's new tokens, from hidden states (include/mla.h).  num_pages: at most the
    cache's."""
    s = (_ragged or _module()).ragged_step(w.handle.value if w.handle else 0, w.buffer, h, q_start, kv_len, seq_idx, pos,
                                           page_table, num_pages, cache, out, workspace, stream)
    if s:
        import torch
        fn, d, dt, i32 = "mla_ragged_step", w.dims, _path_dtype(w.dims), torch.int32
        T, B = _sized(fn, s, "h", h, 2), _sized(fn, s, "kv_len", kv_len, 1)
        if isinstance(num_pages, int) and num_pages > _sized(fn, s, "cache", cache, 3):
            raise MlaError(fn, -1, f"num_pages: {num_pages}, the cache has {cache.shape[0]}")
        _refuse(fn, s, (
            ("h", h, dt, (T, d.d_model), True), ("q_start", q_start, i32, (B + 1,), True),
            ("kv_len", kv_len, i32, (B,), True), ("seq_idx", seq_idx, i32, (T,), True), ("pos", pos, i32, (T,), True),
            ("page_table", page_table, i32, (B, None), True),
            ("cache", cache, dt, (None, d.page_size, d.d_c + (d.n_h if d.rope_key_per_head else 1) * d.d_r), True),
            ("out", out, torch.float32, (T, d.n_h, d.d_v), True), ("weights", w.buffer, None, None, True),
            ("workspace", workspace, None, None, True)))


def selftest_wait_timeout(workspace, limit_us: int, stream=None):
    """Test hook: a bounded wait that nothing satisfies (include/mla.h)."""
    _check("mla_selftest_wait_timeout", lib.mla_selftest_wait_timeout(_ptr(workspace), limit_us, _stream(stream)))


def get_error(workspace, stream=None) -> int:
    return lib.mla_get_error(_ptr(workspace), _stream(stream))


def status_string(code: int) -> str:
    return lib.mla_status_string(code).decode()
