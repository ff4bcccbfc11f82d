"""Python binding of the C ABI in include/kivi.h (ctypes; marshalling only).

The module-level functions carry the C names and take plain integers for
pointers and streams.  ``KiviCache`` wraps one handle with torch tensors for
device memory and the current torch stream.  Every computation runs in the
library's CUDA kernels; importing this module fails loudly when libkivi.so is
missing (build it with ``python -m bit_kivi_kv_gb300.build``).
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkivi.so")

KIVI_OK, KIVI_ERR_INVALID_ARG, KIVI_ERR_UNSUPPORTED, KIVI_ERR_CAPACITY, KIVI_ERR_STATE, KIVI_ERR_CUDA = range(6)
STATUS_NAMES = ["KIVI_OK", "KIVI_ERR_INVALID_ARG", "KIVI_ERR_UNSUPPORTED", "KIVI_ERR_CAPACITY",
                "KIVI_ERR_STATE", "KIVI_ERR_CUDA"]


class kivi_config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("bits", ctypes.c_int), ("group", ctypes.c_int),
                ("residual", ctypes.c_int), ("max_tokens", ctypes.c_longlong)]


class kivi_layout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("blocks_per_slot", ctypes.c_longlong),
                ("tile_bytes", ctypes.c_size_t), ("part_bytes", ctypes.c_size_t),
                ("slot_bytes", ctypes.c_size_t), ("k_resid_offset", ctypes.c_size_t),
                ("v_resid_offset", ctypes.c_size_t), ("resid_slot_bytes", ctypes.c_size_t)]


class kivi_paged_config(ctypes.Structure):
    _fields_ = [("max_seqs", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("bits", ctypes.c_int), ("group", ctypes.c_int),
                ("residual", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int), ("n_pages", ctypes.c_longlong)]


class kivi_paged_layout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("tile_bytes", ctypes.c_size_t),
                ("part_bytes", ctypes.c_size_t), ("page_bytes", ctypes.c_size_t),
                ("k_resid_offset", ctypes.c_size_t), ("v_resid_offset", ctypes.c_size_t),
                ("resid_seq_bytes", ctypes.c_size_t), ("table_offset", ctypes.c_size_t)]


class kivi_qkv(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("n_tokens", ctypes.c_longlong), ("dtype", ctypes.c_int),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3),
                ("v_stride", ctypes.c_longlong * 3), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("cos_sin", ctypes.c_void_p), ("n_positions", ctypes.c_longlong),
                ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("positions", ctypes.c_void_p),
                ("positions_64bit", ctypes.c_int), ("first_position", ctypes.c_longlong),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p)]


_QKV = struct.Struct("@iiiiqiPPPqqqqqqqqqPPfPqiiPiqPPP")   # kivi_qkv, field by field
assert _QKV.size == ctypes.sizeof(kivi_qkv)

KIVI_PAGED_MAX_CALL_SEQS = 512
KIVI_F16, KIVI_BF16, KIVI_F32 = 0, 1, 2


class KiviError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{STATUS_NAMES[status] if 0 <= status < 6 else status}: {message}")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m bit_kivi_kv_gb300.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, SZ, LL, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_int, ctypes.c_float
    cfgp = ctypes.POINTER(kivi_config)
    pcfgp = ctypes.POINTER(kivi_paged_config)
    IP = ctypes.POINTER(ctypes.c_int)
    sigs = {
        "kivi_cache_bytes": (SZ, [cfgp]),
        "kivi_cache_layout": (I, [cfgp, ctypes.POINTER(kivi_layout)]),
        "kivi_cache_create": (I, [cfgp, P, SZ, ctypes.POINTER(P)]),
        "kivi_cache_destroy": (I, [P]),
        "kivi_cache_reset": (I, [P]),
        "kivi_cache_counts": (I, [P, ctypes.POINTER(LL), ctypes.POINTER(LL)]),
        "kivi_prefill": (I, [P, P, P, LL, P]),
        "kivi_append": (I, [P, P, P, P]),
        "kivi_decode_workspace_bytes": (SZ, [cfgp]),
        "kivi_decode_attn": (I, [P, P, P, F, P, SZ, P]),
        "kivi_append_decode": (I, [P, P, P, P, P, F, P, SZ, P]),
        "kivi_last_error_string": (ctypes.c_char_p, []),
        "kivi_launch_count": (ctypes.c_ulonglong, []),
        "kivi_cache_set_decode_kernel": (I, [P, I]),
        "kivi_cache_set_value_residual": (I, [P, I]),
        "kivi_cache_set_fault": (I, [P, I]),
        "kivi_cache_set_max_ctas": (I, [P, I]),
        "kivi_decode_attn_static_ws": (I, [P, P, P, F, P]),
        "kivi_paged_bytes": (SZ, [pcfgp]),
        "kivi_paged_cache_layout": (I, [pcfgp, ctypes.POINTER(kivi_paged_layout)]),
        "kivi_paged_create": (I, [pcfgp, P, SZ, ctypes.POINTER(P)]),
        "kivi_paged_destroy": (I, [P]),
        "kivi_paged_add": (I, [P, P, P, LL, P, IP]),
        "kivi_paged_release": (I, [P, I]),
        "kivi_paged_seq_counts": (I, [P, I, ctypes.POINTER(LL), ctypes.POINTER(LL)]),
        "kivi_paged_seq_pages": (I, [P, I, IP, I, IP]),
        "kivi_paged_free": (I, [P, ctypes.POINTER(LL), IP]),
        "kivi_paged_workspace_bytes": (SZ, [pcfgp, I]),
        "kivi_paged_set_max_ctas": (I, [P, I]),
        "kivi_paged_append_decode": (I, [P, IP, I, P, P, P, P, F, P, SZ, P]),
        "kivi_block_scores": (I, [P, P, F, P, LL, P]),
        "kivi_select_blocks": (I, [P, LL, LL, LL, I, I, P, P]),
        "kivi_decode_blocks": (I, [P, P, P, I, P, F, P]),
        "kivi_paged_block_scores": (I, [P, IP, I, P, F, P, LL, P]),
        "kivi_paged_decode_blocks": (I, [P, IP, I, P, P, I, P, F, P]),
        "kivi_paged_append": (I, [P, IP, I, P, P, P]),
        "kivi_qk_norm_rope": (I, [P, P]),     # a kivi_qkv by reference, or its packed bytes
        "kivi_append_qkv": (I, [P, P, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


lib = _load()


def _check(status: int):
    if status != KIVI_OK:
        raise KiviError(status, lib.kivi_last_error_string().decode())


def make_config(batch, n_q_heads, n_kv_heads, head_dim, bits, group, residual, max_tokens) -> kivi_config:
    return kivi_config(batch, n_q_heads, n_kv_heads, head_dim, bits, group, residual, max_tokens)


# ---- the C calls, same names --------------------------------------------------
def kivi_cache_bytes(cfg: kivi_config) -> int:
    return lib.kivi_cache_bytes(ctypes.byref(cfg))


def kivi_cache_layout(cfg: kivi_config) -> kivi_layout:
    out = kivi_layout()
    _check(lib.kivi_cache_layout(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def kivi_cache_create(cfg: kivi_config, dev_buf: int, nbytes: int) -> int:
    h = ctypes.c_void_p()
    _check(lib.kivi_cache_create(ctypes.byref(cfg), dev_buf, nbytes, ctypes.byref(h)))
    return h.value


def kivi_cache_destroy(h: int):
    _check(lib.kivi_cache_destroy(h))


def kivi_cache_reset(h: int):
    _check(lib.kivi_cache_reset(h))


def kivi_cache_counts(h: int):
    a, b = ctypes.c_longlong(), ctypes.c_longlong()
    _check(lib.kivi_cache_counts(h, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def kivi_prefill(h: int, K: int, V: int, L: int, stream: int):
    _check(lib.kivi_prefill(h, K, V, L, stream))


def kivi_append(h: int, k: int, v: int, stream: int):
    _check(lib.kivi_append(h, k, v, stream))


def kivi_decode_workspace_bytes(cfg: kivi_config) -> int:
    return lib.kivi_decode_workspace_bytes(ctypes.byref(cfg))


def kivi_decode_attn(h: int, q: int, out: int, softmax_scale: float, workspace: int, ws_bytes: int, stream: int):
    _check(lib.kivi_decode_attn(h, q, out, softmax_scale, workspace, ws_bytes, stream))


def kivi_append_decode(h: int, k: int, v: int, q: int, out: int, softmax_scale: float, workspace: int,
                       ws_bytes: int, stream: int):
    _check(lib.kivi_append_decode(h, k, v, q, out, softmax_scale, workspace, ws_bytes, stream))


def kivi_decode_attn_static_ws(h: int, q: int, out: int, softmax_scale: float, stream: int):
    """Decode with the library's static workspace (for callers that cannot allocate)."""
    _check(lib.kivi_decode_attn_static_ws(h, q, out, softmax_scale, stream))


KIVI_DECODE_AUTO, KIVI_DECODE_CUDA_CORE, KIVI_DECODE_TENSOR_CORE = 0, 1, 2


def kivi_cache_set_decode_kernel(h: int, kernel: int):
    _check(lib.kivi_cache_set_decode_kernel(h, kernel))


KIVI_VALUE_FLUSH, KIVI_VALUE_QUEUE = 0, 1
KIVI_FAULT_NONE, KIVI_FAULT_COPY_STALL = 0, 1


def kivi_cache_set_max_ctas(h: int, max_ctas: int):
    _check(lib.kivi_cache_set_max_ctas(h, max_ctas))


def kivi_cache_set_fault(h: int, fault: int):
    """Failure-detection test hook (kivi.h): the next decode call's first copy stage in CTA 0 times out."""
    _check(lib.kivi_cache_set_fault(h, fault))


def kivi_cache_set_value_residual(h: int, mode: int):
    _check(lib.kivi_cache_set_value_residual(h, mode))


# ---- paged cache ----------------------------------------------------------------
def make_paged_config(max_seqs, n_q_heads, n_kv_heads, head_dim, bits, group, residual, max_blocks_per_seq,
                      n_pages) -> kivi_paged_config:
    return kivi_paged_config(max_seqs, n_q_heads, n_kv_heads, head_dim, bits, group, residual,
                             max_blocks_per_seq, n_pages)


def kivi_paged_bytes(cfg: kivi_paged_config) -> int:
    return lib.kivi_paged_bytes(ctypes.byref(cfg))


def kivi_paged_cache_layout(cfg: kivi_paged_config) -> kivi_paged_layout:
    out = kivi_paged_layout()
    _check(lib.kivi_paged_cache_layout(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def kivi_paged_create(cfg: kivi_paged_config, dev_buf: int, nbytes: int) -> int:
    h = ctypes.c_void_p()
    _check(lib.kivi_paged_create(ctypes.byref(cfg), dev_buf, nbytes, ctypes.byref(h)))
    return h.value


def kivi_paged_destroy(h: int):
    _check(lib.kivi_paged_destroy(h))


def kivi_paged_add(h: int, K: int, V: int, L: int, stream: int) -> int:
    s = ctypes.c_int()
    _check(lib.kivi_paged_add(h, K, V, L, stream, ctypes.byref(s)))
    return s.value


def kivi_paged_release(h: int, seq: int):
    _check(lib.kivi_paged_release(h, seq))


def kivi_paged_seq_counts(h: int, seq: int):
    a, b = ctypes.c_longlong(), ctypes.c_longlong()
    _check(lib.kivi_paged_seq_counts(h, seq, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def kivi_paged_seq_pages(h: int, seq: int) -> list:
    n = ctypes.c_int()
    _check(lib.kivi_paged_seq_pages(h, seq, None, 0, ctypes.byref(n)))
    buf = (ctypes.c_int * max(n.value, 1))()
    _check(lib.kivi_paged_seq_pages(h, seq, buf, n.value, ctypes.byref(n)))
    return list(buf[:n.value])


def kivi_paged_free(h: int):
    a, b = ctypes.c_longlong(), ctypes.c_int()
    _check(lib.kivi_paged_free(h, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def kivi_paged_set_max_ctas(h: int, max_ctas: int):
    _check(lib.kivi_paged_set_max_ctas(h, max_ctas))


def kivi_paged_workspace_bytes(cfg: kivi_paged_config, n: int) -> int:
    return lib.kivi_paged_workspace_bytes(ctypes.byref(cfg), n)


def kivi_paged_append_decode(h: int, seqs, k: int, v: int, q: int, out: int, softmax_scale: float,
                             workspace: int, ws_bytes: int, stream: int):
    arr = (ctypes.c_int * max(len(seqs), 1))(*seqs)
    _check(lib.kivi_paged_append_decode(h, arr, len(seqs), k, v, q, out, softmax_scale, workspace, ws_bytes,
                                        stream))


# ---- decode over chosen blocks ------------------------------------------------------
def kivi_block_scores(h: int, q: int, softmax_scale: float, scores: int, ld: int, stream: int):
    _check(lib.kivi_block_scores(h, q, softmax_scale, scores, ld, stream))


def kivi_select_blocks(scores: int, rows: int, cols: int, ld: int, n_keep: int, keep_first: int, blocks: int,
                       stream: int):
    _check(lib.kivi_select_blocks(scores, rows, cols, ld, n_keep, keep_first, blocks, stream))


def kivi_decode_blocks(h: int, q: int, blocks: int, n_list: int, out: int, softmax_scale: float, stream: int):
    _check(lib.kivi_decode_blocks(h, q, blocks, n_list, out, softmax_scale, stream))


def _seq_array(seqs):
    return (ctypes.c_int * max(len(seqs), 1))(*seqs)


def kivi_paged_block_scores(h: int, seqs, q: int, softmax_scale: float, scores: int, ld: int, stream: int):
    _check(lib.kivi_paged_block_scores(h, _seq_array(seqs), len(seqs), q, softmax_scale, scores, ld, stream))


def kivi_paged_decode_blocks(h: int, seqs, q: int, blocks: int, n_list: int, out: int, softmax_scale: float,
                             stream: int):
    _check(lib.kivi_paged_decode_blocks(h, _seq_array(seqs), len(seqs), q, blocks, n_list, out, softmax_scale,
                                        stream))


def kivi_paged_append(h: int, seqs, k: int, v: int, stream: int):
    _check(lib.kivi_paged_append(h, _seq_array(seqs), len(seqs), k, v, stream))


# ---- norm and rotation of queries and keys -----------------------------------------
def kivi_qk_norm_rope(args: kivi_qkv, stream: int):
    _check(lib.kivi_qk_norm_rope(ctypes.byref(args), stream))


def kivi_append_qkv(h: int, args: kivi_qkv, stream: int):
    _check(lib.kivi_append_qkv(h, ctypes.byref(args), stream))


def kivi_last_error_string() -> str:
    return lib.kivi_last_error_string().decode()


def kivi_launch_count() -> int:
    return lib.kivi_launch_count()


# ---- torch convenience wrapper -----------------------------------------------
# torch, and its lookups of the current device and of a device's current stream (what
# torch.cuda.current_device() and current_stream().cuda_stream are, without their set-up
# checks and objects: 0.1 us each against 0.3 and 2.9).  Bound when the first wrapper is
# made, since the C calls need no torch.
_torch = _device = _current_stream = None


def _bind():
    global _torch, _device, _current_stream
    import torch
    _torch = torch
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream)


def _expect(t, what, dtype, shape, device):
    """Raise KIVI_ERR_INVALID_ARG unless t is a dense CUDA tensor of this type and
    shape on the current device (the one the kernels run on)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise KiviError(KIVI_ERR_INVALID_ARG, f"{what} must be a contiguous CUDA {dtype} tensor of shape "
                                              f"{tuple(shape)}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    raise KiviError(KIVI_ERR_INVALID_ARG, f"{what} is on {t.device}, not on the current device")


def _on(cache):
    """The current device, which has to be the one that holds the cache's buffer (the
    kernels run on the current device, whatever the buffer's)."""
    device = _device()
    if device != cache._device:
        raise KiviError(KIVI_ERR_INVALID_ARG, f"the cache is on cuda:{cache._device}, not on the current device")
    return device


def _new(shape, dtype, device, stream):
    """An output of a call that runs on stream: its memory has to come from that
    stream's pool, where no earlier work of another stream may still use it."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def select_blocks(scores, n_keep, keep_first=0, out=None, stream=None):
    """The n_keep best columns of each row of scores (fp32 [..., cols], rows dense or
    evenly strided), as int32 [..., n_keep] in ascending order with -1 behind; the
    first keep_first columns always among them (kivi_select_blocks)."""
    if _torch is None:
        _bind()
    shape, device = scores.shape, _device()
    if scores.dtype is not _torch.float32 or scores.get_device() != device:
        raise KiviError(KIVI_ERR_INVALID_ARG, "scores must be a float32 tensor on the current CUDA device")
    *lead, cols = shape
    ld = cols
    if not scores.is_contiguous():
        if len(lead) != 1 or scores.stride(1) != 1:
            raise KiviError(KIVI_ERR_INVALID_ARG, "scores must be contiguous, or a matrix with dense rows")
        ld = scores.stride(0)
    if out is None:
        out = _new((*lead, max(n_keep, 0)), _torch.int32, scores.device, stream)
    else:
        _expect(out, "out", _torch.int32, (*lead, n_keep), device)
    _check(lib.kivi_select_blocks(scores.data_ptr(), math.prod(lead), cols, ld, n_keep, keep_first, out.data_ptr(),
                                  _current_stream(device) if stream is None else stream.cuda_stream))
    return out


def rope_table(n_positions, rot_dim, base=10000.0, device="cuda"):
    """The cosines and sines of a rotation as QKNormRope takes them: fp32
    [n_positions][rot_dim], pair j at position p turned by p * base^(-2j / rot_dim),
    the angles in fp64 (their error in fp32 grows with the position)."""
    import torch
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


class QKNormRope:
    """The norm of every query and key head, the position rotation and the change to
    the cache's fp16 head-major layout, in one pass (kivi_qk_norm_rope).

    q_weight, k_weight: fp32 [head_dim], None: no norm.  cos_sin: fp32
    [n_positions][rot_dim] (see rope_table), None: no rotation."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim, q_weight=None, k_weight=None, cos_sin=None, eps=1e-6,
                 interleaved=False):
        _bind()
        f32 = _torch.float32
        for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None:
                _expect(w, what, f32, (head_dim,), _device())
        rot_dim = n_positions = table = 0
        if cos_sin is not None:
            if cos_sin.dim() != 2:
                raise KiviError(KIVI_ERR_INVALID_ARG, "cos_sin must be [n_positions, rot_dim]")
            _expect(cos_sin, "cos_sin", f32, cos_sin.shape, _device())
            table, (n_positions, rot_dim) = cos_sin.data_ptr(), cos_sin.shape
        self._keep = (q_weight, k_weight, cos_sin)
        self._device = next((t.get_device() for t in self._keep if t is not None), None)
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self._fixed = (q_weight.data_ptr() if q_weight is not None else 0, k_weight.data_ptr() if k_weight is not None
                       else 0, eps, table, n_positions, rot_dim, bool(interleaved))
        self._dtypes = {_torch.float16: KIVI_F16, _torch.bfloat16: KIVI_BF16, f32: KIVI_F32}
        self._positions = {_torch.int32: 0, _torch.int64: 1}
        self._layouts = {}      # what _layout found out about shapes, strides and types seen before

    def _layout(self, key):
        """Checks the inputs' types, shapes and strides (key); the packed fields that
        follow from them, the leading sizes, and the shapes of the outputs."""
        dtypes, shapes, all_strides = key[:3], key[3:6], key[6:]
        lead = tuple(shapes[0][:-2])
        n = len(lead)
        if n != 1 and n != 2:
            raise KiviError(KIVI_ERR_INVALID_ARG, "q, k and v have 3 or 4 dimensions")
        code = self._dtypes.get(dtypes[0])
        if code is None:
            raise KiviError(KIVI_ERR_INVALID_ARG, f"no input type {dtypes[0]}")
        strides, D = (), self.head_dim
        heads = (self.n_q_heads, self.n_kv_heads, self.n_kv_heads)
        for dtype, shape, s, h, what in zip(dtypes, shapes, all_strides, heads, "qkv"):
            if dtype is not dtypes[0]:
                raise KiviError(KIVI_ERR_INVALID_ARG, f"{what} must be of q's type")
            if tuple(shape) != lead + (h, D) or s[-1] != 1:
                raise KiviError(KIVI_ERR_INVALID_ARG, f"{what} must be [..., {h}, {D}] with dense channels and q's "
                                                      f"leading sizes, got {tuple(shape)}")
            strides += (s[0], 0, s[1]) if n == 1 else s[:3]
        head = (lead[0], self.n_q_heads, self.n_kv_heads, D, 1 if n == 1 else lead[1], code)
        outs = tuple((lead[0], h) + lead[1:] + (D,) for h in heads)
        if len(self._layouts) >= 256:
            self._layouts.clear()
        found = self._layouts[key] = (head, strides, lead, outs)
        return found

    def _inputs(self, q, k, v, positions, device):
        """Checks the inputs [batch, tokens, heads, head_dim] (or [batch, heads,
        head_dim]: one token a row): the packed fields up to the strides, the address and
        width of the positions, and the shapes of the outputs."""
        if q.get_device() != device or k.get_device() != device or v.get_device() != device:
            raise KiviError(KIVI_ERR_INVALID_ARG, "q, k and v must be on the current device")
        if self._device is not None and self._device != device:
            raise KiviError(KIVI_ERR_INVALID_ARG, f"the weights are on cuda:{self._device}, not on the current device")
        key = (q.dtype, k.dtype, v.dtype, q.shape, k.shape, v.shape, q.stride(), k.stride(), v.stride())
        head, strides, lead, shapes = self._layouts.get(key) or self._layout(key)
        wide = pos = 0
        if positions is not None:
            wide = self._positions.get(positions.dtype)
            if wide is None:
                raise KiviError(KIVI_ERR_INVALID_ARG, "positions must be int32 or int64")
            _expect(positions, "positions", positions.dtype, lead, device)
            pos = positions.data_ptr()
        return (*head, q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides, *self._fixed, pos, wide), shapes

    def __call__(self, q, k, v, positions=None, first_position=0, out=None, stream=None):
        """q [B, L, Hq, D], k and v [B, L, Hkv, D] (fp16, bf16 or fp32; any strides with
        dense channels, e.g. parts of one projection's output; without L: one token
        a row), positions [B, L] int32 or int64 (None: first_position + token).
        Returns fp16 (q [B, Hq, L, D], k [B, Hkv, L, D], v), without L where the
        inputs have none."""
        device, f16 = _device(), _torch.float16
        fields, (sq, sk, sv) = self._inputs(q, k, v, positions, device)
        if out is None:
            out = oq, ok, ov = tuple(_new(s, f16, q.device, stream) for s in (sq, sk, sv))
        else:
            oq, ok, ov = out
            _expect(oq, "out[0]", f16, sq, device)
            _expect(ok, "out[1]", f16, sk, device)
            _expect(ov, "out[2]", f16, sv, device)
        # (the fields of kivi_qkv in order, packed at once: a few times faster than one by one)
        _check(lib.kivi_qk_norm_rope(_QKV.pack(*fields, first_position, oq.data_ptr(), ok.data_ptr(), ov.data_ptr()),
                                     _current_stream(device) if stream is None else stream.cuda_stream))
        return out


class KiviCache:
    """One layer's cache: a torch-owned device buffer plus the library handle."""

    def __init__(self, batch, n_q_heads, n_kv_heads, head_dim, bits, group, residual, max_tokens,
                 device="cuda"):
        _bind()
        self.cfg = make_config(batch, n_q_heads, n_kv_heads, head_dim, bits, group, residual, max_tokens)
        nbytes = kivi_cache_bytes(self.cfg)
        if nbytes == 0:
            raise KiviError(KIVI_ERR_INVALID_ARG, kivi_last_error_string())
        self.layout = kivi_cache_layout(self.cfg)
        self.buffer = self._alloc(nbytes, device)
        self.workspace = self._alloc(kivi_decode_workspace_bytes(self.cfg), device)
        self.handle = kivi_cache_create(self.cfg, self.buffer.data_ptr(), nbytes)
        self._q_shape, self._rows = (batch, n_q_heads, head_dim), (batch, n_kv_heads)
        self._device = self.buffer.get_device()

    def _alloc(self, nbytes, device):
        """Device bytes for the cache buffer and the workspace (256-byte aligned);
        a subclass may place them differently (the tests put guard bands around them)."""
        import torch
        return torch.empty(nbytes, dtype=torch.uint8, device=device)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            lib.kivi_cache_destroy(h)
            self.handle = None

    @staticmethod
    def _stream(stream):
        import torch
        return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream

    @staticmethod
    def _ptr(t):
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return t.data_ptr()

    def counts(self):
        return kivi_cache_counts(self.handle)

    def set_decode_kernel(self, kernel: int):
        kivi_cache_set_decode_kernel(self.handle, kernel)

    def set_value_residual(self, mode: int):
        """KIVI_VALUE_FLUSH (default) or KIVI_VALUE_QUEUE; on an empty cache."""
        kivi_cache_set_value_residual(self.handle, mode)

    def reset(self):
        kivi_cache_reset(self.handle)

    def prefill(self, K, V, stream=None):
        kivi_prefill(self.handle, self._ptr(K), self._ptr(V), K.shape[2], self._stream(stream))

    def append(self, k, v, stream=None):
        kivi_append(self.handle, self._ptr(k), self._ptr(v), self._stream(stream))

    def decode_attn(self, q, out=None, softmax_scale=0.0, stream=None):
        import torch
        if out is None:
            out = torch.empty_like(q)
        kivi_decode_attn(self.handle, self._ptr(q), self._ptr(out), softmax_scale,
                         self.workspace.data_ptr(), self.workspace.numel(), self._stream(stream))
        return out

    def append_decode(self, k, v, q, out=None, softmax_scale=0.0, stream=None):
        """append(k, v) then decode_attn(q) in one call (one launch fewer)."""
        import torch
        if out is None:
            out = torch.empty_like(q)
        kivi_append_decode(self.handle, self._ptr(k), self._ptr(v), self._ptr(q), self._ptr(out), softmax_scale,
                           self.workspace.data_ptr(), self.workspace.numel(), self._stream(stream))
        return out


    def append_qkv(self, norm_rope, q, k, v, positions=None, first_position=0, q_out=None, stream=None):
        """Append one token a row from a projection's output: norm and rotation by
        norm_rope (QKNormRope), k and v stored in the cache by the same kernel.
        q [B, Hq, D], k, v [B, Hkv, D]; returns the query, fp16 [B, Hq, D]."""
        device, f16 = _on(self), _torch.float16
        fields, (shape, _, _) = norm_rope._inputs(q, k, v, positions, device)
        if q_out is None:
            q_out = _new(shape, f16, q.device, stream)
        else:
            _expect(q_out, "q_out", f16, shape, device)
        _check(lib.kivi_append_qkv(self.handle, _QKV.pack(*fields, first_position, q_out.data_ptr(), 0, 0),
                                   _current_stream(device) if stream is None else stream.cuda_stream))
        return q_out

    def block_scores(self, q, out=None, softmax_scale=0.0, stream=None):
        """A bound on the logits of each quantized block for q [B, Hq, D]: fp32
        [B, Hkv, blocks] (kivi_block_scores); out may have more columns (-inf there)."""
        device, f32 = _on(self), _torch.float32
        _expect(q, "q", _torch.float16, self._q_shape, device)
        if out is None:
            cols = self.counts()[0] // self.cfg.group
            out = _new((*self._rows, cols), f32, q.device, stream)
        else:
            cols = out.shape[-1]
            _expect(out, "out", f32, (*self._rows, cols), device)
        _check(lib.kivi_block_scores(self.handle, q.data_ptr(), softmax_scale, out.data_ptr(), cols,
                                     _current_stream(device) if stream is None else stream.cuda_stream))
        return out

    def decode_blocks(self, q, blocks, out=None, softmax_scale=0.0, stream=None):
        """Decode attention of q [B, Hq, D] over the listed blocks (int32
        [B, Hkv, n], negative anywhere: none) and the residual (kivi_decode_blocks)."""
        device, f16, n = _on(self), _torch.float16, blocks.shape[-1]
        _expect(q, "q", f16, self._q_shape, device)
        _expect(blocks, "blocks", _torch.int32, (*self._rows, n), device)
        if out is None:
            out = _new(self._q_shape, f16, q.device, stream)
        else:
            _expect(out, "out", f16, self._q_shape, device)
        _check(lib.kivi_decode_blocks(self.handle, q.data_ptr(), blocks.data_ptr(), n, out.data_ptr(), softmax_scale,
                                      _current_stream(device) if stream is None else stream.cuda_stream))
        return out

    def sparse_decode(self, q, n_keep, keep_first=1, out=None, softmax_scale=0.0, stream=None):
        """Decode attention over the n_keep blocks of the largest scores (the first
        keep_first always) and the residual: block_scores, select_blocks and
        decode_blocks in sequence."""
        with _torch.cuda.stream(stream):
            scores = self.block_scores(q, softmax_scale=softmax_scale)
            n_keep = min(n_keep, scores.shape[-1])
            blocks = select_blocks(scores, n_keep, min(keep_first, n_keep))
            return self.decode_blocks(q, blocks, out, softmax_scale)


class KiviPagedCache:
    """A paged cache for ragged sequences: a torch-owned device buffer (page pool,
    residual rows, block table) plus the library handle."""

    def __init__(self, max_seqs, n_q_heads, n_kv_heads, head_dim, bits, group, residual, max_blocks_per_seq,
                 n_pages, device="cuda"):
        _bind()
        self.cfg = make_paged_config(max_seqs, n_q_heads, n_kv_heads, head_dim, bits, group, residual,
                                     max_blocks_per_seq, n_pages)
        nbytes = kivi_paged_bytes(self.cfg)
        if nbytes == 0:
            raise KiviError(KIVI_ERR_INVALID_ARG, kivi_last_error_string())
        self.layout = kivi_paged_cache_layout(self.cfg)
        self.buffer = self._alloc(nbytes, device)
        self.workspace = self._alloc(kivi_paged_workspace_bytes(self.cfg, min(max_seqs, KIVI_PAGED_MAX_CALL_SEQS)),
                                     device)
        self.handle = kivi_paged_create(self.cfg, self.buffer.data_ptr(), nbytes)
        self._heads = (n_q_heads, n_kv_heads, head_dim)
        self._device = self.buffer.get_device()

    def _alloc(self, nbytes, device):
        """Device bytes for the buffer and the workspace (see KiviCache._alloc)."""
        import torch
        return torch.empty(nbytes, dtype=torch.uint8, device=device)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            lib.kivi_paged_destroy(h)
            self.handle = None

    def add(self, K, V, stream=None) -> int:
        """New sequence with prompt K, V [Hkv][L][D] fp16; returns its id."""
        L = K.shape[1]
        return kivi_paged_add(self.handle, KiviCache._ptr(K) if L else 0, KiviCache._ptr(V) if L else 0, L,
                              KiviCache._stream(stream))

    def release(self, seq: int):
        kivi_paged_release(self.handle, seq)

    def counts(self, seq: int):
        return kivi_paged_seq_counts(self.handle, seq)

    def pages(self, seq: int) -> list:
        return kivi_paged_seq_pages(self.handle, seq)

    def free(self):
        return kivi_paged_free(self.handle)

    def append_decode(self, seqs, k, v, q, out=None, softmax_scale=0.0, stream=None):
        """For each listed sequence: append k[i], v[i] ([n][Hkv][D]; both None: no
        append), then decode q[i] ([n][Hq][D]) into out[i]."""
        import torch
        if out is None:
            out = torch.empty_like(q)
        kp = KiviCache._ptr(k) if k is not None else 0
        vp = KiviCache._ptr(v) if v is not None else 0
        kivi_paged_append_decode(self.handle, list(seqs), kp, vp, KiviCache._ptr(q), KiviCache._ptr(out),
                                 softmax_scale, self.workspace.data_ptr(), self.workspace.numel(),
                                 KiviCache._stream(stream))
        return out

    def append(self, seqs, k, v, stream=None):
        """For each listed sequence: append k[i], v[i] ([n][Hkv][D])."""
        n, (_, hkv, d), device = len(seqs), self._heads, _on(self)
        _expect(k, "k", _torch.float16, (n, hkv, d), device)
        _expect(v, "v", _torch.float16, (n, hkv, d), device)
        _check(lib.kivi_paged_append(self.handle, _seq_array(seqs), n, k.data_ptr(), v.data_ptr(),
                                     _current_stream(device) if stream is None else stream.cuda_stream))

    def block_scores(self, seqs, q, out=None, softmax_scale=0.0, stream=None):
        """KiviCache.block_scores for the listed sequences: q [n, Hq, D] -> fp32
        [n, Hkv, the longest sequence's blocks], -inf behind a sequence's last."""
        n, (hq, hkv, d), device = len(seqs), self._heads, _on(self)
        _expect(q, "q", _torch.float16, (n, hq, d), device)
        if out is None:
            cols = max((self.counts(s)[0] // self.cfg.group for s in seqs), default=0)
            out = _new((n, hkv, cols), _torch.float32, q.device, stream)
        else:
            cols = out.shape[-1]
            _expect(out, "out", _torch.float32, (n, hkv, cols), device)
        _check(lib.kivi_paged_block_scores(self.handle, _seq_array(seqs), n, q.data_ptr(), softmax_scale, out.data_ptr(),
                                           cols, _current_stream(device) if stream is None else stream.cuda_stream))
        return out

    def decode_blocks(self, seqs, q, blocks, out=None, softmax_scale=0.0, stream=None):
        """KiviCache.decode_blocks for the listed sequences: blocks int32 [n, Hkv, m]."""
        n, (hq, hkv, d), device, m = len(seqs), self._heads, _on(self), blocks.shape[-1]
        _expect(q, "q", _torch.float16, (n, hq, d), device)
        _expect(blocks, "blocks", _torch.int32, (n, hkv, m), device)
        if out is None:
            out = _new((n, hq, d), _torch.float16, q.device, stream)
        else:
            _expect(out, "out", _torch.float16, (n, hq, d), device)
        _check(lib.kivi_paged_decode_blocks(self.handle, _seq_array(seqs), n, q.data_ptr(), blocks.data_ptr(), m,
                                            out.data_ptr(), softmax_scale,
                                            _current_stream(device) if stream is None else stream.cuda_stream))
        return out

    def sparse_decode(self, seqs, q, n_keep, keep_first=1, out=None, softmax_scale=0.0, stream=None):
        """KiviCache.sparse_decode for the listed sequences."""
        seqs = list(seqs)
        with _torch.cuda.stream(stream):
            scores = self.block_scores(seqs, q, softmax_scale=softmax_scale)
            n_keep = min(n_keep, scores.shape[-1])
            blocks = select_blocks(scores, n_keep, min(keep_first, n_keep))
            return self.decode_blocks(seqs, q, blocks, out, softmax_scale)
