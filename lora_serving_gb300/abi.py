"""Thin binding of ``liblora.so`` (the C ABI declared in include/lora.h): ctypes, and
csrc/pycalls.c for the calls between a decode step's projections.

Argument marshalling only: every function here has the name of the C entry
point it calls, takes torch tensors (device memory for kernel entry points,
host numpy arrays for the host helpers), reads their pointers and leading
dimensions, and raises ``LoraError`` on a non-OK status.  There is no
fallback: if the CUDA library is missing the import fails loudly.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import numpy as np

try:
    import torch
except ImportError:   # the host helpers (metadata, adapter preparation) do without it
    torch = None

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblora.so")
CALLS_PATH = os.path.join(_HERE, "_pycalls.so")

LORA_MAX_RANK = 128
LORA_BGMV_MAX_RANK = 32
LORA_MAX_PROJ = 4
LORA_DEV_SLOT_OUT_OF_RANGE = 0x1
LORA_DEV_BAD_SEGMENT = 0x2
LORA_APPLY_X_READY = 0x1
LORA_APPLY_NO_PDL = 0x2
LORA_APPLY_Y_READY = 0x4
LORA_DEV_TIMEOUT = 0x4
LORA_DEV_BAD_PAGE = 0x8
LORA_DEV_BAD_POSITION = 0x10
LORA_DEV_NO_PAGES = 0x20
LORA_MAX_ROPE_AXES = 3
LORA_KEEP_LAYERS = 64
LORA_BF16, LORA_F32 = 0, 1

STATUS = {
    0: "LORA_OK", 1: "LORA_ERR_INVALID_ARG", 2: "LORA_ERR_SHAPE",
    3: "LORA_ERR_RANK_EXCEEDS_SLOT", 4: "LORA_ERR_SLOT_RANGE", 5: "LORA_ERR_ALIGNMENT",
    6: "LORA_ERR_METADATA", 7: "LORA_ERR_WORKSPACE", 8: "LORA_ERR_CUDA",
}

# Every symbol include/lora.h declares.
EXPORTS = (
    "lora_bgmv_shrink", "lora_bgmv_expand", "lora_sgmv_shrink", "lora_sgmv_expand",
    "lora_apply", "lora_apply_workspace_bytes", "lora_build_metadata",
    "lora_prepare_adapter", "lora_slot_rank", "lora_read_device_status", "lora_status_string",
    "lora_kernel_launch_count", "lora_apply_noalloc", "lora_merge", "lora_merge_batch", "lora_linear",
    "lora_slots_create", "lora_slots_destroy", "lora_slots_register", "lora_slots_acquire",
    "lora_slots_slot_of", "lora_slots_stats",
    "lora_rms_norm", "lora_kv4_block_bytes", "lora_kv4_append", "lora_kv4_read", "lora_kv4_attend",
    "lora_kv4_attend_workspace_bytes", "lora_kv4_plan", "lora_kv4_attend_tree", "lora_kv4_keep", "lora_logits_adjust",
)
LORA_NOALLOC_SCRATCH_BYTES = 16 << 20


class LoraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{fn} returned {self.name}")


class lora_proj_t(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("out_off", ctypes.c_int), ("width", ctypes.c_int)]


class lora_meta_t(ctypes.Structure):
    _fields_ = [("lora_ids", ctypes.c_void_p), ("n_rows", ctypes.c_int), ("n_prefill", ctypes.c_int),
                ("seg_starts", ctypes.c_void_p), ("seg_slot", ctypes.c_void_p), ("n_segs", ctypes.c_int),
                ("max_seg_len", ctypes.c_int),
                ("perm", ctypes.c_void_p), ("gseg_starts", ctypes.c_void_p), ("gseg_slot", ctypes.c_void_p),
                ("n_gsegs", ctypes.c_int), ("max_gseg_len", ctypes.c_int)]


class lora_kv4_cache_t(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_kv", ctypes.c_int), ("head_dim", ctypes.c_int)]


class lora_kv4_batch_t(ctypes.Structure):
    _fields_ = [("q_starts", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("ld_table", ctypes.c_int), ("n_seqs", ctypes.c_int), ("n_rows", ctypes.c_int),
                ("max_q_len", ctypes.c_int), ("max_ctx_len", ctypes.c_int), ("held", ctypes.c_void_p)]


class lora_kv4_pool_t(ctypes.Structure):
    _fields_ = [("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("n_free_out", ctypes.c_void_p), ("held_out", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("ld_table", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int)]


class plan_args_t(ctypes.Structure):
    """plan_t of csrc/pycalls.c: what a store.KV4Plan keeps of lora_kv4_plan's arguments."""
    _fields_ = [("q_starts", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p), ("row_seq", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("n_seqs", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("max_q_len", ctypes.c_int32), ("max_ctx_len", ctypes.c_int32),
                ("pool", lora_kv4_pool_t)]


class lora_logits_rules_t(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("prompt_lens", ctypes.c_void_p), ("token_lens", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("n_bias", ctypes.c_void_p),
                ("ld_tokens", ctypes.c_int), ("ld_bias", ctypes.c_int), ("n_seqs", ctypes.c_int)]


_lib = None


def load(path: str | None = None):
    """Loads liblora.so once.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing: run lora_serving_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "lora_bgmv_shrink": [P, i32, P, i32, P, P, i32, i32, i32, i32, P, P],
        "lora_bgmv_expand": [P, i32, i32, i32, P, i32, P, P, i32, i32, i32, P, P],
        "lora_sgmv_shrink": [P, i32, P, i32, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, P, P],
        "lora_sgmv_expand": [P, i32, i32, i32, P, i32, P, P, P, i32, P, i32, i32, i32, i32, i32, P, P],
        "lora_apply": [P, i32, P, i32, i32, P, i32, i32, i32, P, P, sz, ctypes.c_uint32, P, P],
        "lora_apply_noalloc": [P, i32, P, i32, i32, P, i32, i32, i32, P, ctypes.c_uint32, P, P],
        "lora_apply_workspace_bytes": [i32, i32, i32],
        "lora_build_metadata": [P, i32, i32, i32, P, P, P, P, P, P, P, P, P],
        "lora_prepare_adapter": [P, P, i32, i32, i32, ctypes.c_double, i32, i32, P, P],
        "lora_slot_rank": [P, i32],
        "lora_read_device_status": [P, P, P],
        "lora_status_string": [i32],
        "lora_merge": [P, i32, i32, i32, P, P, i32, i32, P],
        "lora_merge_batch": [i32, P, P, P, P, P, P, i32, i32, P],
        "lora_linear": [P, i32, P, i32, i32, P, i32, P, i32, i32, i32, P, P, sz, P, P],
        "lora_slots_create": [i32, P, P, P, P, i32, i32, i32, P],
        "lora_slots_register": [P, ctypes.c_int64, P, P, i32, ctypes.c_double, i32],
        "lora_slots_acquire": [P, P, i32, P, P],
        "lora_slots_slot_of": [P, ctypes.c_int64],
        "lora_slots_stats": [P, P],
        "lora_rms_norm": [P, i32, P, i32, P, i32, i32, P, i32, P, i32, P, i32, P, i32, i32, ctypes.c_float, P],
        "lora_kv4_block_bytes": [i32, i32],
        "lora_kv4_append": [P, i32, P, i32, i32, i32, i32, i32, P, i32, i32, P, i32, P, i32, P, P, P, P],
        "lora_kv4_read": [P, i32, P, i32, P, P, P, P],
        "lora_kv4_attend": [P, i32, P, i32, i32, ctypes.c_float, i32, P, P, P, sz, P, P],
        "lora_kv4_attend_workspace_bytes": [i32, i32, i32, i32],
        "lora_kv4_plan": [P, P, P, P, P, P, P, P, i32, i32, i32, i32, P, P, P],
        "lora_kv4_attend_tree": [P, i32, P, i32, i32, ctypes.c_float, i32, P, i32, P, P, P, sz, P, P],
        "lora_kv4_keep": [P, i32, P, P, P, i32, P, P, P],
        "lora_logits_adjust": [P, i32, i32, P, i32, i32, i32, i32, P, P, P, P, i32, P, P, i32, i32, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("lora_apply_workspace_bytes", "lora_kv4_block_bytes", "lora_kv4_attend_workspace_bytes"):
        getattr(lib, name).restype = ctypes.c_size_t
    lib.lora_status_string.restype = ctypes.c_char_p
    lib.lora_kernel_launch_count.argtypes = []
    lib.lora_kernel_launch_count.restype = ctypes.c_uint64
    lib.lora_slots_destroy.argtypes = [P]
    lib.lora_slots_destroy.restype = None
    _lib = lib
    return lib


_calls = None


def _load_calls():
    """The module csrc/pycalls.c, bound to the library: the calls between a
    step's projections, whose kernels take less time than ctypes takes to
    convert their arguments."""
    global _calls
    lib = load()
    if torch is None:
        raise RuntimeError("lora_rms_norm, lora_kv4_* and lora_logits_adjust take torch tensors, and torch cannot be imported")
    if not os.path.exists(CALLS_PATH):
        raise RuntimeError(f"extension {CALLS_PATH} is missing: run lora_serving_gb300.build() with a C compiler and Python's headers")
    spec = importlib.util.spec_from_file_location("lora_serving_gb300._pycalls", CALLS_PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    fns = tuple(ctypes.cast(f, ctypes.c_void_p).value
                for f in (lib.lora_rms_norm, lib.lora_kv4_append, lib.lora_kv4_read, lib.lora_kv4_attend, lib.lora_kv4_plan,
                          lib.lora_kv4_attend_tree, lib.lora_kv4_keep, lib.lora_logits_adjust))
    mod.bind(fns, (torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn), _cur_device, _raw_stream)
    _calls = mod
    return mod


def _check(fn: str, st: int):
    if st != 0:
        raise LoraError(fn, st)


def _p(t) -> int:
    """Device/host pointer of a torch tensor, numpy array or raw int (0 = NULL)."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _ld(t) -> int:
    return int(t.stride(0))


_DTYPES = torch and {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "u8": torch.uint8,
                     "e4m3": torch.float8_e4m3fn}


def _dev(t, name: str, dtype: str | None = None, mat: bool = False) -> int:
    """Device pointer of a kernel argument, after the checks the C ABI cannot
    make: a torch tensor on a CUDA device (a host pointer handed to a kernel
    is an illegal address), of the element type the kernel reads, and for
    row-major operands (mat) 2-D with unit column stride, so that the row
    stride is the leading dimension.  None (NULL) and raw integer pointers
    pass unchecked."""
    if t is None or isinstance(t, int):
        return _p(t)
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not _DTYPES[dtype]:
        raise ValueError(f"{name} must be {_DTYPES[dtype]}, got {t.dtype}")
    if mat and (t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1)):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.data_ptr()


if torch and hasattr(torch._C, "_cuda_getCurrentRawStream"):   # the stream's handle without a Stream object around it (3 us)
    _cur_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
else:
    _cur_device = lambda: torch.cuda.current_device()  # noqa: E731
    _raw_stream = lambda dev: torch.cuda.current_stream(dev).cuda_stream  # noqa: E731


def _current_stream() -> int:
    return _raw_stream(_cur_device()) if torch.cuda.is_initialized() else torch.cuda.current_stream().cuda_stream


def _stream(stream) -> int:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------ kernels ----

def lora_bgmv_shrink(v, x, A, lora_ids, *, h_in, r_slot, n_slots, dev_status=None, stream=None):
    n_rows = int(lora_ids.numel())
    _check("lora_bgmv_shrink", load().lora_bgmv_shrink(
        _dev(v, "v", "f32", True), _ld(v), _dev(x, "x", "bf16", True), _ld(x), _dev(A, "A", "bf16"),
        _dev(lora_ids, "lora_ids", "i32"), n_rows, h_in, r_slot, n_slots, _dev(dev_status, "dev_status", "i32"),
        _stream(stream)))


def lora_bgmv_expand(y, y_off, width, v, B, lora_ids, *, r_slot, n_slots, dev_status=None,
                     stream=None, v_col=0):
    n_rows = int(lora_ids.numel())
    vp = _dev(v, "v", "f32", True) + 4 * v_col
    _check("lora_bgmv_expand", load().lora_bgmv_expand(
        _dev(y, "y", "bf16", True), _ld(y), y_off, width, vp, _ld(v), _dev(B, "B", "bf16"),
        _dev(lora_ids, "lora_ids", "i32"), n_rows, r_slot, n_slots, _dev(dev_status, "dev_status", "i32"),
        _stream(stream)))


def lora_sgmv_shrink(v, x, A, seg_starts, seg_slot, n_segs, row_perm, n_pos, *, h_in, r_slot,
                     n_slots, max_seg_len=0, dev_status=None, stream=None):
    _check("lora_sgmv_shrink", load().lora_sgmv_shrink(
        _dev(v, "v", "f32", True), _ld(v), _dev(x, "x", "bf16", True), _ld(x), _dev(A, "A", "bf16"),
        _dev(seg_starts, "seg_starts", "i32"), _dev(seg_slot, "seg_slot", "i32"), n_segs,
        _dev(row_perm, "row_perm", "i32"), n_pos, int(x.shape[0]), max_seg_len, h_in, r_slot, n_slots,
        _dev(dev_status, "dev_status", "i32"), _stream(stream)))


def lora_sgmv_expand(y, y_off, width, v, B, seg_starts, seg_slot, n_segs, row_perm, n_pos, *,
                     r_slot, n_slots, max_seg_len=0, dev_status=None, stream=None, v_col=0):
    vp = _dev(v, "v", "f32", True) + 4 * v_col
    _check("lora_sgmv_expand", load().lora_sgmv_expand(
        _dev(y, "y", "bf16", True), _ld(y), y_off, width, vp, _ld(v), _dev(B, "B", "bf16"),
        _dev(seg_starts, "seg_starts", "i32"), _dev(seg_slot, "seg_slot", "i32"), n_segs,
        _dev(row_perm, "row_perm", "i32"), n_pos, int(y.shape[0]), max_seg_len, r_slot, n_slots,
        _dev(dev_status, "dev_status", "i32"), _stream(stream)))


def make_projs(projs):
    """projs: sequence of (A_store, B_store, out_off, width) -> ctypes array."""
    arr = (lora_proj_t * len(projs))()
    for i, (A, B, off, w) in enumerate(projs):
        arr[i].A, arr[i].B, arr[i].out_off, arr[i].width = _p(A), _p(B), int(off), int(w)
    return arr


def lora_apply(y, x, h_in, projs, r_slot, n_slots, meta, workspace, *, flags=0, dev_status=None,
               stream=None):
    """projs: ctypes array from make_projs(); meta: lora_meta_t; workspace: device tensor;
    flags: LORA_APPLY_* bits."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("lora_apply", load().lora_apply(
        _dev(y, "y", "bf16", True), _ld(y), _dev(x, "x", "bf16", True), _ld(x), h_in, ctypes.addressof(projs),
        len(projs), r_slot, n_slots, ctypes.addressof(meta), _dev(workspace, "workspace"), ws_bytes, int(flags),
        _dev(dev_status, "dev_status", "i32"), _stream(stream)))


def lora_apply_noalloc(y, x, h_in, projs, r_slot, n_slots, meta, *, flags=0, dev_status=None, stream=None):
    """lora_apply with the library's built-in scratch instead of a workspace
    (for callers that cannot allocate device memory when they call in)."""
    _check("lora_apply_noalloc", load().lora_apply_noalloc(
        _dev(y, "y", "bf16", True), _ld(y), _dev(x, "x", "bf16", True), _ld(x), h_in, ctypes.addressof(projs),
        len(projs), r_slot, n_slots, ctypes.addressof(meta), int(flags), _dev(dev_status, "dev_status", "i32"),
        _stream(stream)))


def lora_linear(y, x, h_in, W, projs, r_slot, n_slots, meta, workspace, *, dev_status=None, stream=None):
    """y[:, off_p + c] = bf16(x W^T + B'_p (A_p x)) for every projection of
    projs (ctypes array from make_projs(), tiling W's rows in order); W is
    the stacked base weight [n_out][h_in] (row stride ld); y is written."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("lora_linear", load().lora_linear(
        _dev(y, "y", "bf16", True), _ld(y), _dev(x, "x", "bf16", True), _ld(x), h_in, _dev(W, "W", "bf16", True),
        _ld(W), ctypes.addressof(projs), len(projs), r_slot, n_slots, ctypes.addressof(meta),
        _dev(workspace, "workspace"), ws_bytes, _dev(dev_status, "dev_status", "i32"), _stream(stream)))


def lora_merge(W, A, B, sign, *, stream=None):
    """W [out][h_in] (row stride ld) += sign * B A, one bf16 rounding; A is one
    adapter slot [r_slot][h_in] of the A store, B the same slot [out][r_slot]
    of the scaled B store; sign +1 merges, -1 unmerges."""
    out, h_in = int(W.shape[0]), int(W.shape[1])
    r_slot = int(A.shape[0])
    _check("lora_merge", load().lora_merge(_dev(W, "W", "bf16", True), _ld(W), out, h_in, _dev(A, "A", "bf16", True),
                                           _dev(B, "B", "bf16", True), r_slot, int(sign), _stream(stream)))


def lora_merge_batch(Ws, As, Bs, sign, *, stream=None):
    """lora_merge over every (W, A, B) of the lists in one launch (per 32);
    all A share the slot rank (their row count)."""
    n = len(Ws)
    P = ctypes.c_void_p
    arr_w, arr_a, arr_b = (P * max(1, n))(), (P * max(1, n))(), (P * max(1, n))()
    ld = (ctypes.c_int * max(1, n))()
    out = (ctypes.c_int * max(1, n))()
    h_in = (ctypes.c_int * max(1, n))()
    for i, (W, A, B) in enumerate(zip(Ws, As, Bs)):
        arr_w[i] = _dev(W, f"Ws[{i}]", "bf16", True)
        arr_a[i], arr_b[i] = _dev(A, f"As[{i}]", "bf16", True), _dev(B, f"Bs[{i}]", "bf16", True)
        ld[i], out[i], h_in[i] = _ld(W), int(W.shape[0]), int(W.shape[1])
    r_slot = int(As[0].shape[0]) if n else 8
    _check("lora_merge_batch", load().lora_merge_batch(n, arr_w, ld, out, h_in, arr_a, arr_b, r_slot, int(sign),
                                                       _stream(stream)))


def lora_rms_norm(x, weight, eps, *, residual=None, residual_out=None, y=None, y8=None, scales=None, group=0,
                  stream=None):
    """h = bf16(x + residual) -> residual_out; n = h / sqrt(mean(h^2) + eps) * weight
    -> y (bf16) and/or y8 (float8_e4m3fn) with fp32 scales [n_rows][groups], one
    per `group` (128) columns or, with group 0, per row."""
    st = (_calls or _load_calls()).rms_norm(x, weight, eps, residual, residual_out, y, y8, scales, group, stream)
    if st:
        raise LoraError("lora_rms_norm", st)


def lora_kv4_block_bytes(page_size, head_dim) -> int:
    return int(load().lora_kv4_block_bytes(page_size, head_dim))


def lora_kv4_append(q_out, x, cache, batch, *, n_heads, q_off, k_off, v_off, rope=None, positions=None,
                    axis_pairs=None, dev_status=None, stream=None):
    """Rotates q (-> q_out) and k of the fused rows x and stores k and v in
    `cache` (store.KV4Cache) at the places `batch` (store.KV4Batch) gives.
    rope: fp32 [max_pos][pairs][2] (cos, sin) or None; positions: int32
    [n_rows][n_axes] or None; axis_pairs: pairs of each axis (default: all
    on one axis)."""
    st = (_calls or _load_calls()).kv4_append(q_out, x, cache.addr, batch.addr, n_heads, q_off, k_off, v_off, rope,
                                              positions, axis_pairs, dev_status, stream)
    if st:
        raise LoraError("lora_kv4_append", st)


def lora_kv4_read(k, v, cache, batch, *, dev_status=None, stream=None):
    """k, v [n_rows][n_kv * head_dim] <- the cached values of the rows' places."""
    st = (_calls or _load_calls()).kv4_read(k, v, cache.addr, batch.addr, dev_status, stream)
    if st:
        raise LoraError("lora_kv4_read", st)


def lora_kv4_attend(out, q, cache, batch, workspace, *, n_heads, scale, window=0, dev_status=None, stream=None):
    """out [n_rows][n_heads * head_dim] <- causal attention of q over the cache
    (the last `window` positions, 0: all)."""
    st = (_calls or _load_calls()).kv4_attend(out, q, cache.addr, batch.addr, workspace, n_heads, scale, window,
                                              dev_status, stream)
    if st:
        raise LoraError("lora_kv4_attend", st)


def lora_kv4_attend_workspace_bytes(n_heads, n_kv, head_dim, max_q_len) -> int:
    return int(load().lora_kv4_attend_workspace_bytes(n_heads, n_kv, head_dim, max_q_len))


def lora_kv4_plan(plan, q_lens, lens, *, depths=None, dev_status=None, stream=None):
    """A step's tables and pages: `plan` (store.KV4Plan) gets the row starts,
    lengths, pages, and each row's sequence, position and slot, from int32
    q_lens (rows that each sequence brings; -1: it has ended) and lens (cached
    positions); depths: int32 [max_rows], the rows' depths in drafted trees."""
    st = (_calls or _load_calls()).kv4_plan(plan.addr, q_lens, lens, depths, dev_status, stream)
    if st:
        raise LoraError("lora_kv4_plan", st)


def lora_kv4_attend_tree(out, q, cache, batch, tree, workspace, *, n_heads, scale, window=0, dev_status=None, stream=None):
    """out [n_rows][n_heads * head_dim] <- attention of drafted trees' rows over
    the cache: the positions before the sequence's first row (the last `window`
    of them by the row's depth, 0: all), and of its rows those whose bits are
    set in the row's int32 words of `tree` [n_rows][words]."""
    st = (_calls or _load_calls()).kv4_attend_tree(out, q, cache.addr, batch.addr, tree, workspace, n_heads, scale, window,
                                                   dev_status, stream)
    if st:
        raise LoraError("lora_kv4_attend_tree", st)


def lora_kv4_keep(layers, batch, n_keep, path, *, lens=None, dev_status=None, stream=None):
    """In every cache of `layers` (store.KV4Layers) the rows path[s][:n_keep[s]]
    of sequence s of `batch` move up to follow its context; lens <- the
    sequences' cached positions from now on.  int32 n_keep [n_seqs], path
    [n_seqs][columns], lens [n_seqs]."""
    st = (_calls or _load_calls()).kv4_keep(layers.addr, layers.n, batch.addr, n_keep, path, lens, dev_status, stream)
    if st:
        raise LoraError("lora_kv4_keep", st)


def lora_logits_adjust(out, logits, rules=None, *, row_seq=None, drafts=None, tree=None, q_starts=None, allowed=None,
                       allowed_rows=None, dev_status=None, stream=None):
    """out <- logits [n_rows][vocab] (bf16 or fp32 each) under the penalties and
    biases of `rules` (store.LogitsRules) for each row's request (row_seq: int32
    [n_rows], -1: not written; default: row t is request t's), with the drafted
    tokens on the row's path (drafts [n_rows], tree [n_rows][words], q_starts)
    counted in, and -infinity where the row's set of `allowed` (int32
    [sets][words], a bit per token; allowed_rows: set of each row, -1: none)
    lacks the token."""
    st = (_calls or _load_calls()).logits_adjust(out, logits, rules.addr if rules is not None else 0, row_seq, drafts, tree,
                                                 q_starts, allowed, allowed_rows, dev_status, stream)
    if st:
        raise LoraError("lora_logits_adjust", st)


class lora_slot_stats_t(ctypes.Structure):
    _fields_ = [("registered", ctypes.c_uint64), ("host_evictions", ctypes.c_uint64), ("hits", ctypes.c_uint64),
                ("loads", ctypes.c_uint64), ("slot_evictions", ctypes.c_uint64)]


class SlotManager:
    """The adapter slot manager (lora_slots_*): a host cache of prepared
    adapters feeding the GPU slots of the stores.  A_stores / B_stores: one
    device tensor per projection ([n_slots][r_slot][h_in], [n_slots][w][r_slot]),
    or None for the policy alone."""

    def __init__(self, h_in, width, n_slots, r_slot, max_cpu, A_stores=None, B_stores=None):
        self.n_proj = len(h_in)
        hi = (ctypes.c_int * self.n_proj)(*h_in)
        wd = (ctypes.c_int * self.n_proj)(*width)
        if A_stores is not None:
            self._a = (ctypes.c_void_p * self.n_proj)(*[_dev(t, "A_stores", "bf16") for t in A_stores])
            self._b = (ctypes.c_void_p * self.n_proj)(*[_dev(t, "B_stores", "bf16") for t in B_stores])
            a, b = ctypes.addressof(self._a), ctypes.addressof(self._b)
        else:
            a = b = 0
        self._h = ctypes.c_void_p()
        _check("lora_slots_create", load().lora_slots_create(self.n_proj, ctypes.addressof(hi), ctypes.addressof(wd),
                                                             a, b, n_slots, r_slot, max_cpu, ctypes.byref(self._h)))

    def close(self):
        if self._h:
            load().lora_slots_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def register(self, adapter_id, A_list, B_list, r, alpha, use_rslora=False):
        """A_list[p]: host uint16 bits [r][h_in_p]; B_list[p]: [w_p][r] (unscaled)."""
        A = [np.ascontiguousarray(a, dtype=np.uint16) for a in A_list]
        B = [np.ascontiguousarray(b, dtype=np.uint16) for b in B_list]
        ap = (ctypes.c_void_p * self.n_proj)(*[a.ctypes.data for a in A])
        bp = (ctypes.c_void_p * self.n_proj)(*[b.ctypes.data for b in B])
        _check("lora_slots_register", load().lora_slots_register(self._h, int(adapter_id), ctypes.addressof(ap),
                                                                 ctypes.addressof(bp), int(r), float(alpha),
                                                                 int(bool(use_rslora))))

    def acquire(self, adapter_ids, stream=0) -> np.ndarray:
        """Adapter ids of a batch (-1 = base) -> slot ids, loading what is missing."""
        ids = np.ascontiguousarray(adapter_ids, dtype=np.int64)
        out = np.empty(ids.size, np.int32)
        st = stream if isinstance(stream, int) else _stream(stream)
        _check("lora_slots_acquire", load().lora_slots_acquire(self._h, ids.ctypes.data, int(ids.size),
                                                               out.ctypes.data, st))
        return out

    def slot_of(self, adapter_id) -> int:
        return int(load().lora_slots_slot_of(self._h, int(adapter_id)))

    def stats(self) -> dict:
        s = lora_slot_stats_t()
        _check("lora_slots_stats", load().lora_slots_stats(self._h, ctypes.byref(s)))
        return {f: int(getattr(s, f)) for f, _ in s._fields_}


def lora_apply_workspace_bytes(n_rows, n_proj, r_slot) -> int:
    return int(load().lora_apply_workspace_bytes(n_rows, n_proj, r_slot))


def lora_read_device_status(dev_status, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check("lora_read_device_status", load().lora_read_device_status(
        _dev(dev_status, "dev_status", "i32"), ctypes.addressof(out), _stream(stream)))
    return out.value


# ------------------------------------------------------- host helpers ----

def lora_build_metadata(ids: np.ndarray, n_prefill: int, n_slots: int):
    """Returns dict of int32 arrays seg_starts, seg_slot, perm, gseg_starts,
    gseg_slot and ints n_segs, max_seg_len, n_gsegs, max_gseg_len."""
    ids = np.ascontiguousarray(ids, np.int32)
    T = ids.size
    D = T - n_prefill
    seg_starts = np.zeros(n_prefill + 1, np.int32)
    seg_slot = np.zeros(max(n_prefill, 1), np.int32)
    perm = np.zeros(max(D, 1), np.int32)
    gseg_starts = np.zeros(n_slots + 2, np.int32)
    gseg_slot = np.zeros(n_slots + 1, np.int32)
    S, MS, G, MG = (ctypes.c_int(0) for _ in range(4))
    _check("lora_build_metadata", load().lora_build_metadata(
        _p(ids), T, n_prefill, n_slots, _p(seg_starts), _p(seg_slot), ctypes.addressof(S),
        ctypes.addressof(MS), _p(perm), _p(gseg_starts), _p(gseg_slot), ctypes.addressof(G),
        ctypes.addressof(MG)))
    s, g = S.value, G.value
    return dict(seg_starts=seg_starts[: s + 1].copy(), seg_slot=seg_slot[:s].copy(), n_segs=s,
                max_seg_len=MS.value, perm=perm[:D].copy(), gseg_starts=gseg_starts[: g + 1].copy(),
                gseg_slot=gseg_slot[:g].copy(), n_gsegs=g, max_gseg_len=MG.value)


def lora_prepare_adapter(A: np.ndarray, B: np.ndarray, alpha: float, use_rslora: bool, r_slot: int,
                         A_slot_out: np.ndarray | None = None, B_slot_out: np.ndarray | None = None):
    """A [r][h_in], B [out][r] (uint16 bf16 bits) -> padded (A_slot, B'_slot)."""
    A = np.ascontiguousarray(A, np.uint16)
    B = np.ascontiguousarray(B, np.uint16)
    r, h_in = A.shape
    out = B.shape[0]
    if B.shape[1] != r:
        raise ValueError("lora_B must be [out][r] with the rank of lora_A")
    if A_slot_out is None:
        A_slot_out = np.empty((r_slot, h_in), np.uint16)
    if B_slot_out is None:
        B_slot_out = np.empty((out, r_slot), np.uint16)
    assert A_slot_out.flags.c_contiguous and B_slot_out.flags.c_contiguous
    _check("lora_prepare_adapter", load().lora_prepare_adapter(
        _p(A), _p(B), r, h_in, out, float(alpha), int(bool(use_rslora)), r_slot,
        _p(A_slot_out), _p(B_slot_out)))
    return A_slot_out, B_slot_out


def lora_slot_rank(ranks) -> int:
    arr = np.ascontiguousarray(ranks, np.int32)
    return int(load().lora_slot_rank(_p(arr), arr.size))


def lora_kernel_launch_count() -> int:
    return int(load().lora_kernel_launch_count())


def lora_status_string(status: int) -> str:
    return load().lora_status_string(status).decode()
