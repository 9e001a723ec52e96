"""Python binding of libverifyhead.so (restricted-vocabulary MTP draft head and
greedy speculative verification, GB300 / sm_103a).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  If the compiled
library is missing, every call raises: there is no fallback.

Entry points mirror the C ABI in include/verifyhead.h:
    mtp_draft_head_argmax, mtp_draft_head_argmax_nvfp4,
    spec_verify_greedy (spec_verify_greedy_path), vh_workspace_bytes,
    vh_add_rmsnorm (add_rmsnorm, add_rmsnorm_q8, add_rmsnorm_grad),
    vh_logits_logprobs (logits_logprobs, logits_logprobs_grad), vh_head_logprobs (head_logprobs),
    vh_nvfp4_quantize (nvfp4_quantize, nvfp4_quantize_tiles), vh_nvfp4_tile (nvfp4_tile),
    vh_nvfp4_dequantize (nvfp4_dequantize, nvfp4_dequantize_tiles), vh_nvfp4_matmul (nvfp4_matmul),
    vh_logits_process (logits_process, logits_process_grad).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libverifyhead.so")

VH_OK = 0
VH_ERR_NULL = -1
VH_ERR_SHAPE = -2
VH_ERR_ALIGN = -3
VH_ERR_WORKSPACE = -4
VH_ERR_LAUNCH = -5
VH_ERR_DEVICE = -6

VH_PATH_AUTO = 0
VH_PATH_CUDA_CORE = 1
VH_PATH_TENSOR = 2
VH_PATH_WARP_MMA = 3

VH_F32 = 0
VH_BF16 = 1
VH_F16 = 2

VH_NORM_SAME = 0
VH_NORM_INT8 = 1
VH_NORM_E4M3 = 2

# Every symbol the header declares (checked by the ABI tests).
EXPORTS = (
    "vh_version", "vh_status_string", "vh_workspace_bytes", "mtp_draft_head_argmax",
    "mtp_draft_head_argmax_nvfp4", "spec_verify_greedy", "spec_verify_greedy_path",
    "mtp_draft_head_argmax_static_ws", "mtp_draft_head_argmax_gather", "vh_workspace_error_offset",
    "vh_selftest_bounded_wait", "spec_verify_greedy_nvfp4", "vh_verify_nvfp4_workspace_bytes",
    "mtp_draft_head_argmax_nvfp4_path", "vh_nvfp4_packed_bytes", "vh_nvfp4_pack",
    "mtp_draft_head_argmax_nvfp4_packed", "spec_verify_greedy_nvfp4_packed",
    "vh_add_rmsnorm", "vh_add_rmsnorm_grad", "vh_add_rmsnorm_grad_workspace_bytes", "vh_logits_logprobs",
    "vh_logits_logprobs_workspace_bytes", "vh_logits_logprobs_grad", "vh_head_logprobs",
    "vh_head_logprobs_workspace_bytes", "vh_nvfp4_tiles_bytes", "vh_nvfp4_quantize", "vh_nvfp4_tile",
    "vh_nvfp4_dequantize", "vh_nvfp4_matmul", "vh_logits_process", "vh_logits_process_grad",
)


class VHError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None
_debug_lib = None
_use_debug = False


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    from . import buildlib as _b
    return _b.build(force=force, verbose=verbose, debug=debug)


def _load(path: str):
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run verify_head_gb300.build() (nvcc, sm_103a)")
    L = ctypes.CDLL(path)
    _declare(L)
    return L


def lib():
    """The loaded library (raises if it has not been built).  Inside
    `debug_library()` this is the VH_DEBUG build."""
    global _lib
    if _use_debug:
        return _debug_lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


@contextlib.contextmanager
def debug_library():
    """Route every call in the block through libverifyhead_debug.so (built on
    first use): the same kernels with device-side index guards that set bit 2
    of the workspace error word instead of touching memory out of range."""
    global _debug_lib, _use_debug
    if _debug_lib is None:
        from . import buildlib as _b
        _debug_lib = _load(_b.build(debug=True))
    prev, _use_debug = _use_debug, True
    try:
        yield _debug_lib
    finally:
        _use_debug = prev


class LogitsRules(ctypes.Structure):
    """vh_logits_rules."""
    _fields_ = [("history", ctypes.c_void_p), ("history_stride", ctypes.c_int64), ("history_width", ctypes.c_int),
                ("history_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p), ("draft_ids", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("temperature", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("n_bias", ctypes.c_int), ("allowed", ctypes.c_void_p), ("allowed_stride", ctypes.c_int64)]


def _declare(L):
    """ctypes signatures of every exported entry point."""
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.vh_version.restype = i32
    L.vh_version.argtypes = []
    L.vh_status_string.restype = ctypes.c_char_p
    L.vh_status_string.argtypes = [i32]
    L.vh_workspace_bytes.restype = sz
    L.vh_workspace_bytes.argtypes = [i32]
    L.mtp_draft_head_argmax.restype = i32
    L.mtp_draft_head_argmax.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]
    L.mtp_draft_head_argmax_nvfp4.restype = i32
    L.mtp_draft_head_argmax_nvfp4.argtypes = [vp, vp, vp, ctypes.c_float, vp, i32, i32, i32, vp, vp, vp, sz, vp]
    L.spec_verify_greedy.restype = i32
    L.spec_verify_greedy.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.spec_verify_greedy_nvfp4.restype = i32
    L.spec_verify_greedy_nvfp4.argtypes = [vp, vp, vp, ctypes.c_float, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz,
                                           vp]
    L.vh_workspace_error_offset.restype = sz
    L.vh_workspace_error_offset.argtypes = []
    L.vh_selftest_bounded_wait.restype = i32
    L.vh_selftest_bounded_wait.argtypes = [vp, ctypes.c_uint, vp]
    L.mtp_draft_head_argmax_gather.restype = i32
    L.mtp_draft_head_argmax_gather.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
    L.mtp_draft_head_argmax_static_ws.restype = i32
    L.mtp_draft_head_argmax_static_ws.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp]
    L.vh_verify_nvfp4_workspace_bytes.restype = sz
    L.vh_verify_nvfp4_workspace_bytes.argtypes = [i32, i32]
    L.mtp_draft_head_argmax_nvfp4_path.restype = i32
    L.mtp_draft_head_argmax_nvfp4_path.argtypes = [vp, vp, vp, ctypes.c_float, vp, i32, i32, i32, vp, vp, vp, sz, vp,
                                                   i32]
    L.vh_nvfp4_packed_bytes.restype = sz
    L.vh_nvfp4_packed_bytes.argtypes = [i32, i32]
    L.vh_nvfp4_pack.restype = i32
    L.vh_nvfp4_pack.argtypes = [vp, vp, i32, i32, vp, sz, vp]
    L.mtp_draft_head_argmax_nvfp4_packed.restype = i32
    L.mtp_draft_head_argmax_nvfp4_packed.argtypes = [vp, vp, ctypes.c_float, vp, i32, i32, i32, vp, vp, vp, sz, vp]
    L.spec_verify_greedy_nvfp4_packed.restype = i32
    L.spec_verify_greedy_nvfp4_packed.argtypes = [vp, vp, ctypes.c_float, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz,
                                                  vp]
    i64, f32 = ctypes.c_int64, ctypes.c_float
    L.vh_add_rmsnorm.restype = i32
    L.vh_add_rmsnorm.argtypes = [vp, vp, vp, i32, i32, i32, i32, i64, i64, f32, f32, vp, i64, i32, vp, i64, vp, vp]
    L.vh_add_rmsnorm_grad_workspace_bytes.restype = sz
    L.vh_add_rmsnorm_grad_workspace_bytes.argtypes = [i32, i32]
    L.vh_add_rmsnorm_grad.restype = i32
    L.vh_add_rmsnorm_grad.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, i64, f32, f32, vp, i64, vp, vp, sz,
                                      vp]
    L.vh_logits_logprobs_workspace_bytes.restype = sz
    L.vh_logits_logprobs_workspace_bytes.argtypes = [i32, i32, i32]
    L.vh_logits_logprobs.restype = i32
    L.vh_logits_logprobs.argtypes = [vp, i32, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.vh_logits_logprobs_grad.restype = i32
    L.vh_logits_logprobs_grad.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, i64, vp]
    L.vh_head_logprobs_workspace_bytes.restype = sz
    L.vh_head_logprobs_workspace_bytes.argtypes = [i32, i32, i32]
    L.vh_head_logprobs.restype = i32
    L.vh_head_logprobs.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.vh_nvfp4_tiles_bytes.restype = sz
    L.vh_nvfp4_tiles_bytes.argtypes = [i32, i32]
    L.vh_nvfp4_quantize.restype = i32
    L.vh_nvfp4_quantize.argtypes = [vp, i32, i32, i32, i64, f32, vp, vp, vp, vp]
    L.vh_nvfp4_tile.restype = i32
    L.vh_nvfp4_tile.argtypes = [vp, vp, i32, i32, vp, sz, vp]
    L.vh_nvfp4_dequantize.restype = i32
    L.vh_nvfp4_dequantize.argtypes = [vp, vp, i32, i32, f32, vp, i32, vp, i64, vp]
    L.vh_nvfp4_matmul.restype = i32
    L.vh_nvfp4_matmul.argtypes = [vp, f32, vp, vp, f32, vp, i32, i32, i32, i32, vp, i64, vp]
    rules = ctypes.POINTER(LogitsRules)
    L.vh_logits_process.restype = i32
    L.vh_logits_process.argtypes = [vp, i32, i32, i32, i64, i32, rules, vp, i32, i64, vp]
    L.vh_logits_process_grad.restype = i32
    L.vh_logits_process_grad.argtypes = [vp, vp, i32, i32, i32, i64, i64, i32, rules, vp, i64, vp]
    L.spec_verify_greedy_path.restype = i32
    L.spec_verify_greedy_path.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp, i32]


def status_string(status: int) -> str:
    return lib().vh_status_string(int(status)).decode()


def vh_workspace_bytes(rows: int) -> int:
    return int(lib().vh_workspace_bytes(int(rows)))


def vh_verify_nvfp4_workspace_bytes(rows: int, H: int) -> int:
    return int(lib().vh_verify_nvfp4_workspace_bytes(int(rows), int(H)))


def workspace_error(ws) -> int:
    """The error word of a workspace tensor: 0, or bit 1 (a bounded wait
    expired) and / or bit 2 (an index guard of the debug build fired) set by
    some call that used it.  Copies 4 bytes to the host (synchronising)."""
    off = int(lib().vh_workspace_error_offset())
    return int(ws[off:off + 4].cpu().view(__import__("torch").int32).item())


def _check(status: int, where: str):
    if status != VH_OK:
        raise VHError(status, where)


# ----------------------------------------------------------------------------
# torch-facing helpers (device memory and streams only).

def _torch():
    import torch
    return torch


def _ptr(t):
    # a plain int: the declared c_void_p argument types convert it
    return None if t is None else t.data_ptr()


_raw_stream = None  # torch's raw current-stream query, when this torch build has one


def _stream_ptr(stream):
    """cudaStream_t of `stream`, or of torch's current stream on the current device."""
    global _raw_stream
    torch = _torch()
    if stream is None:
        if _raw_stream is None:
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", False)
        if _raw_stream:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("verify_head_gb300 takes CUDA tensors only")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous (row-major)")


def workspace(rows: int, device=None):
    """A zeroed workspace for calls producing up to `rows` argmax rows."""
    torch = _torch()
    return torch.zeros(vh_workspace_bytes(rows), dtype=torch.uint8, device=device or "cuda")


def verify_nvfp4_workspace(rows: int, H: int, device=None):
    """A zeroed workspace for spec_verify_greedy_nvfp4 with `rows` hidden rows of width H."""
    torch = _torch()
    return torch.zeros(vh_verify_nvfp4_workspace_bytes(rows, H), dtype=torch.uint8, device=device or "cuda")


def mtp_draft_head_argmax(hidden, W_cand, cand_ids, ids=None, maxlogit=None, ws=None, stream=None):
    """hidden [B,H] bf16, W_cand [Vc,H] bf16, cand_ids [Vc] int32 -> (ids [B] int32, maxlogit [B] fp32)."""
    torch = _torch()
    _require_cuda(hidden, W_cand, cand_ids)
    B, H = hidden.shape
    Vc = W_cand.shape[0]
    if W_cand.shape[1] != H or cand_ids.numel() != Vc or hidden.element_size() != 2 or W_cand.element_size() != 2:
        raise ValueError("shape/dtype mismatch")
    if ids is None:
        ids = torch.empty(B, dtype=torch.int32, device=hidden.device)
    if maxlogit is None:
        maxlogit = torch.empty(B, dtype=torch.float32, device=hidden.device)
    if ws is None:
        ws = workspace(B, hidden.device)
    st = lib().mtp_draft_head_argmax(_ptr(hidden), _ptr(W_cand), _ptr(cand_ids), B, H, Vc, _ptr(ids), _ptr(maxlogit),
                                     _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(st, "mtp_draft_head_argmax")
    return ids, maxlogit


def mtp_draft_head_argmax_gather(hidden, W_full, row_ids, ids=None, maxlogit=None, ws=None, stream=None):
    """hidden [B,H] bf16, W_full [V,H] bf16, row_ids [n] int32 (rows of W_full to score, any order)
    -> (ids [B] int32 = winning row ids, maxlogit [B] fp32)."""
    torch = _torch()
    _require_cuda(hidden, W_full, row_ids)
    B, H = hidden.shape
    V = W_full.shape[0]
    if W_full.shape[1] != H or hidden.element_size() != 2 or W_full.element_size() != 2:
        raise ValueError("shape/dtype mismatch")
    if ids is None:
        ids = torch.empty(B, dtype=torch.int32, device=hidden.device)
    if maxlogit is None:
        maxlogit = torch.empty(B, dtype=torch.float32, device=hidden.device)
    if ws is None:
        ws = workspace(B, hidden.device)
    st = lib().mtp_draft_head_argmax_gather(_ptr(hidden), _ptr(W_full), _ptr(row_ids), B, H, row_ids.numel(), V,
                                            _ptr(ids), _ptr(maxlogit), _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(st, "mtp_draft_head_argmax_gather")
    return ids, maxlogit


def mtp_draft_head_argmax_nvfp4(hidden, Wq, scales, tensor_scale, cand_ids, ids=None, maxlogit=None, ws=None,
                                stream=None, path: int = VH_PATH_AUTO):
    """hidden [B,H] bf16, Wq [Vc,H/2] uint8, scales [Vc,H/16] uint8 (E4M3), tensor_scale float.
    `path` picks the kernel family (VH_PATH_AUTO / VH_PATH_CUDA_CORE / VH_PATH_TENSOR)."""
    torch = _torch()
    _require_cuda(hidden, Wq, scales, cand_ids)
    B, H = hidden.shape
    Vc = Wq.shape[0]
    if Wq.shape[1] * 2 != H or tuple(scales.shape) != (Vc, H // 16) or cand_ids.numel() != Vc:
        raise ValueError("shape mismatch")
    if ids is None:
        ids = torch.empty(B, dtype=torch.int32, device=hidden.device)
    if maxlogit is None:
        maxlogit = torch.empty(B, dtype=torch.float32, device=hidden.device)
    if ws is None:
        ws = workspace(B, hidden.device)
    st = lib().mtp_draft_head_argmax_nvfp4_path(_ptr(hidden), _ptr(Wq), _ptr(scales), float(tensor_scale),
                                                _ptr(cand_ids), B, H, Vc, _ptr(ids), _ptr(maxlogit), _ptr(ws),
                                                ws.numel(), _stream_ptr(stream), int(path))
    _check(st, "mtp_draft_head_argmax_nvfp4")
    return ids, maxlogit


def spec_verify_greedy(hidden, W_full, draft_ids, B: int, k: int, accept_len=None, next_ids=None, row_maxlogit=None,
                       ws=None, stream=None, path: int = VH_PATH_AUTO, want_maxlogit: bool = True):
    """hidden [B*(k+1),H] bf16, W_full [V,H] bf16, draft_ids [B,k] int32
    -> (accept_len [B], next_ids [B*(k+1)], row_maxlogit [B*(k+1)] or None).
    `path`: VH_PATH_AUTO / VH_PATH_CUDA_CORE / VH_PATH_TENSOR / VH_PATH_WARP_MMA."""
    torch = _torch()
    _require_cuda(hidden, W_full, draft_ids)
    R, H = hidden.shape
    V = W_full.shape[0]
    if R != B * (k + 1) or W_full.shape[1] != H or draft_ids.numel() != B * k:
        raise ValueError("shape mismatch")
    dev = hidden.device
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    if next_ids is None:
        next_ids = torch.empty(R, dtype=torch.int32, device=dev)
    if row_maxlogit is None and want_maxlogit:
        row_maxlogit = torch.empty(R, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(R, dev)
    st = lib().spec_verify_greedy_path(_ptr(hidden), _ptr(W_full), _ptr(draft_ids), B, k, H, V, _ptr(accept_len),
                                       _ptr(next_ids), _ptr(row_maxlogit), _ptr(ws), ws.numel(), _stream_ptr(stream),
                                       int(path))
    _check(st, "spec_verify_greedy")
    return accept_len, next_ids, row_maxlogit


def spec_verify_greedy_nvfp4(hidden, Wq, scales, tensor_scale, draft_ids, B: int, k: int, accept_len=None,
                             next_ids=None, row_maxlogit=None, ws=None, stream=None, want_maxlogit: bool = True):
    """hidden [B*(k+1),H] bf16, Wq [V,H/2] uint8, scales [V,H/16] uint8, draft_ids [B,k] int32
    -> (accept_len [B], next_ids [B*(k+1)], row_maxlogit or None)."""
    torch = _torch()
    _require_cuda(hidden, Wq, scales, draft_ids)
    R, H = hidden.shape
    V = Wq.shape[0]
    if R != B * (k + 1) or Wq.shape[1] * 2 != H or tuple(scales.shape) != (V, H // 16) or draft_ids.numel() != B * k:
        raise ValueError("shape mismatch")
    dev = hidden.device
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    if next_ids is None:
        next_ids = torch.empty(R, dtype=torch.int32, device=dev)
    if row_maxlogit is None and want_maxlogit:
        row_maxlogit = torch.empty(R, dtype=torch.float32, device=dev)
    if ws is None:
        ws = verify_nvfp4_workspace(R, H, dev)
    st = lib().spec_verify_greedy_nvfp4(_ptr(hidden), _ptr(Wq), _ptr(scales), float(tensor_scale), _ptr(draft_ids), B,
                                        k, H, V, _ptr(accept_len), _ptr(next_ids), _ptr(row_maxlogit), _ptr(ws),
                                        ws.numel(), _stream_ptr(stream))
    _check(st, "spec_verify_greedy_nvfp4")
    return accept_len, next_ids, row_maxlogit


def vh_nvfp4_packed_bytes(V: int, H: int) -> int:
    return int(lib().vh_nvfp4_packed_bytes(V, H))


def nvfp4_pack(Wq, scales, packed=None, stream=None):
    """Wq [V,H/2] uint8, scales [V,H/16] uint8 (row-major, CUDA) -> the tiled
    copy (uint8 CUDA tensor of vh_nvfp4_packed_bytes(V, H) bytes) that the
    *_nvfp4_packed calls read.  Done once per head (the weights are static)."""
    torch = _torch()
    _require_cuda(Wq, scales)
    V, H = Wq.shape[0], Wq.shape[1] * 2
    if tuple(scales.shape) != (V, H // 16):
        raise ValueError("shape mismatch")
    n = vh_nvfp4_packed_bytes(V, H)
    if n == 0:
        raise VHError(VH_ERR_SHAPE, "nvfp4_pack")
    if packed is None:
        packed = torch.empty(n, dtype=torch.uint8, device=Wq.device)
    st = lib().vh_nvfp4_pack(_ptr(Wq), _ptr(scales), V, H, _ptr(packed), packed.numel(), _stream_ptr(stream))
    _check(st, "vh_nvfp4_pack")
    return packed


def mtp_draft_head_argmax_nvfp4_packed(hidden, packed, tensor_scale, cand_ids, ids=None, maxlogit=None, ws=None,
                                       stream=None):
    """hidden [B,H] bf16, packed = nvfp4_pack(...) of the candidate table (Vc = cand_ids.numel() rows)."""
    torch = _torch()
    _require_cuda(hidden, packed, cand_ids)
    B, H = hidden.shape
    Vc = cand_ids.numel()
    if packed.numel() < vh_nvfp4_packed_bytes(Vc, H) or hidden.element_size() != 2:
        raise ValueError("shape mismatch")
    if ids is None:
        ids = torch.empty(B, dtype=torch.int32, device=hidden.device)
    if maxlogit is None:
        maxlogit = torch.empty(B, dtype=torch.float32, device=hidden.device)
    if ws is None:
        ws = workspace(B, hidden.device)
    st = lib().mtp_draft_head_argmax_nvfp4_packed(_ptr(hidden), _ptr(packed), float(tensor_scale), _ptr(cand_ids), B,
                                                  H, Vc, _ptr(ids), _ptr(maxlogit), _ptr(ws), ws.numel(),
                                                  _stream_ptr(stream))
    _check(st, "mtp_draft_head_argmax_nvfp4_packed")
    return ids, maxlogit


def spec_verify_greedy_nvfp4_packed(hidden, packed, tensor_scale, draft_ids, B: int, k: int, V: int, accept_len=None,
                                    next_ids=None, row_maxlogit=None, ws=None, stream=None,
                                    want_maxlogit: bool = True):
    """hidden [B*(k+1),H] bf16, packed = nvfp4_pack(...) of the full V-row head, draft_ids [B,k] int32
    -> (accept_len [B], next_ids [B*(k+1)], row_maxlogit or None)."""
    torch = _torch()
    _require_cuda(hidden, packed, draft_ids)
    R, H = hidden.shape
    if R != B * (k + 1) or draft_ids.numel() != B * k or packed.numel() < vh_nvfp4_packed_bytes(V, H):
        raise ValueError("shape mismatch")
    dev = hidden.device
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    if next_ids is None:
        next_ids = torch.empty(R, dtype=torch.int32, device=dev)
    if row_maxlogit is None and want_maxlogit:
        row_maxlogit = torch.empty(R, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(R, dev)
    st = lib().spec_verify_greedy_nvfp4_packed(_ptr(hidden), _ptr(packed), float(tensor_scale), _ptr(draft_ids), B, k,
                                               H, V, _ptr(accept_len), _ptr(next_ids), _ptr(row_maxlogit), _ptr(ws),
                                               ws.numel(), _stream_ptr(stream))
    _check(st, "spec_verify_greedy_nvfp4_packed")
    return accept_len, next_ids, row_maxlogit


# ----------------------------------------------------------------------------
# Norm and log probabilities.  None of these calls is recorded by autograd: results of inputs that require a gradient are
# cut off from them, and the gradients are the _grad calls' (to be called from a torch.autograd.Function, say).

_dtypes = {}  # torch dtype -> vh_dtype
_f32 = _i32 = None  # torch.float32, torch.int32
_current_device = None  # torch's query of the current device
_compiled = None  # the compiled marshalling (csrc/marshal.cpp); False where it has not been built


def _setup():
    """Fills the names above on the first call (torch is imported no earlier than it is needed)."""
    global _f32, _i32, _current_device, _raw_stream
    torch = _torch()
    if _raw_stream is None:
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", False)
    _dtypes.update({torch.float32: VH_F32, torch.bfloat16: VH_BF16, torch.float16: VH_F16})
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _f32, _i32 = torch.float32, torch.int32


def _load_marshal():
    """The compiled marshalling that was built for this interpreter and this torch, or None."""
    from importlib import machinery, util
    from . import buildlib as _b
    _torch()
    path = _b.marshal_path()
    if not os.path.exists(path):
        return None
    try:
        name = __name__ + "._marshal"
        spec = util.spec_from_file_location(name, path, loader=machinery.ExtensionFileLoader(name, path))
        m = util.module_from_spec(spec)
        spec.loader.exec_module(m)
        return m
    except ImportError:
        return None


def _compiled_calls():
    """The compiled marshalling, bound to the loaded library, or False.  It takes the usual calls (outputs and
    workspace given, torch's current stream) and leaves every other to the checks below."""
    global _compiled
    if _use_debug:
        return False
    if _compiled is None:
        L = lib()
        m = _load_marshal()
        if m is None:
            _compiled = False
        else:
            for name in ("vh_add_rmsnorm", "vh_add_rmsnorm_grad", "vh_logits_logprobs", "vh_logits_logprobs_grad",
                         "vh_head_logprobs", "vh_nvfp4_tiles_bytes", "vh_nvfp4_quantize", "vh_nvfp4_dequantize",
                         "vh_nvfp4_matmul", "vh_logits_process", "vh_logits_process_grad"):
                m.bind(name, ctypes.cast(getattr(L, name), ctypes.c_void_p).value)
            _compiled = m
    return _compiled


def _dtype(t, name):
    d = _dtypes.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: float32, bfloat16 or float16 wanted, not {t.dtype}")
    return d


def _device(t):
    """Device index of a call's first tensor, which must be the current device (the launch goes there)."""
    if _f32 is None:
        _setup()
    d = t.get_device()
    if d < 0:
        raise ValueError("verify_head_gb300 takes CUDA tensors only")
    if d != _current_device():
        raise ValueError(f"the tensors are on device {d}, not on the current device")
    return d


def _stream_on(stream, dev):
    """cudaStream_t of `stream`, or of torch's current stream on device `dev`."""
    return _raw_stream(dev) if stream is None and _raw_stream else _stream_ptr(stream)


def _int32(*sizes):
    """Refuses sizes that the C ABI's ints do not hold (ctypes would pass their low 32 bits on)."""
    for n in sizes:
        if not -0x80000000 <= n <= 0x7FFFFFFF:
            raise ValueError(f"a size of {n} is past 32 bits")


def _place(t, name, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name}: a CUDA tensor on device {dev} wanted")


def _rows(t, name, dev, shape, dtype):
    """Checks a 2-D CUDA tensor of that shape and type whose rows are contiguous; returns the elements between rows."""
    # the usual case in as few queries as possible: the checks are most of a small call's time on the host
    if t.is_contiguous() and t.dtype is dtype and t.shape == shape and t.get_device() == dev and len(shape) == 2:
        return shape[1] or 1
    _place(t, name, dev)
    if t.dim() != 2 or t.shape != shape:
        raise ValueError(f"{name}: shape mismatch")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {dtype} wanted, not {t.dtype}")
    rows, width = shape
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.stride(0) if rows > 1 else max(width, 1)


def _vector(t, name, dev, n, dtype):
    """Checks a contiguous CUDA tensor of n elements and returns its address (None passes)."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _place(t, name, dev)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous elements wanted")
    raise ValueError(f"{name}: {dtype} wanted, not {t.dtype}")


def _workspace(ws, dev):
    """Checks a workspace given by the caller; returns its size."""
    _place(ws, "ws", dev)
    if not ws.is_contiguous() or ws.element_size() != 1:
        raise ValueError("ws: a contiguous uint8 tensor wanted")
    return ws.numel()


def _allocating(stream):
    """Tensors made in this block belong to the stream the call runs on (they are cleared and reused in its order)."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _norm_weight(weight, H, dtype, dev):
    """(address, whether it is fp32) of a norm's weight."""
    if weight is None:
        return None, 0
    f32 = weight.dtype is _f32
    return _vector(weight, "weight", dev, H, _f32 if f32 else dtype), int(f32)


def _empty_rows(x):
    return _torch().empty(x.shape, dtype=x.dtype, device=x.device)


def _add_rmsnorm(where, x, residual, weight, eps, weight_offset, y, out_dtype, kind, h, scales, stream):
    dev = _device(x)
    dt = _dtype(x, "x")
    shape, dtype = x.shape, x.dtype
    xs = _rows(x, "x", dev, shape, dtype)
    T, H = shape
    _int32(T, H)
    rp, rs = (residual.data_ptr(), _rows(residual, "residual", dev, shape, dtype)) if residual is not None else (None, 0)
    hp, hs = (h.data_ptr(), _rows(h, "h", dev, shape, dtype)) if h is not None else (None, 0)
    ys = _rows(y, "q" if kind else "y", dev, shape, out_dtype)
    w, w32 = _norm_weight(weight, H, dtype, dev)
    st = lib().vh_add_rmsnorm(
        x.data_ptr(), rp, w, dt, w32, T, H, xs, rs, eps, weight_offset, y.data_ptr(), ys, kind, hp, hs,
        _vector(scales, "scales", dev, T, _f32), _stream_on(stream, dev))
    _check(st, where)


def add_rmsnorm(x, residual=None, weight=None, eps: float = 1e-6, weight_offset: float = 0.0, y=None, h=None,
                stream=None):
    """y = rmsnorm(x + residual) * (weight + weight_offset) and the sum h, both in x's type.
    x, residual [T,H] fp32 / bf16 / fp16 (rows may be strided), weight [H] of x's type or fp32.
    h may be `residual` itself (updated in place); without a residual h is x and nothing is written.
    -> (y, h)"""
    if stream is None and y is not None:
        m = _compiled_calls()
        if m:
            st = m.add_rmsnorm(x, residual, weight, eps, weight_offset, y, h, None)
            if st <= 0:
                _check(st, "add_rmsnorm")
                return y, (x if h is None else h)
    if y is None or (residual is not None and h is None):
        with _allocating(stream):
            y = _empty_rows(x) if y is None else y
            h = _empty_rows(x) if residual is not None and h is None else h
    _add_rmsnorm("add_rmsnorm", x, residual, weight, eps, weight_offset, y, x.dtype, VH_NORM_SAME, h, None, stream)
    return y, (x if h is None else h)


def add_rmsnorm_q8(x, residual=None, weight=None, eps: float = 1e-6, weight_offset: float = 0.0, q=None, scales=None,
                   h=None, dtype=None, stream=None):
    """add_rmsnorm with 8-bit rows: q [T,H] (torch.int8, or torch.float8_e4m3fn; `dtype` where q is not given) and
    scales [T] fp32 with q * scales[:, None] standing for the normed rows, for layers of the caller's that take 8-bit rows.
    -> (q, scales, h)"""
    if stream is None and q is not None and scales is not None and dtype is None:
        m = _compiled_calls()
        if m:
            st = m.add_rmsnorm(x, residual, weight, eps, weight_offset, q, h, scales)
            if st <= 0:
                _check(st, "add_rmsnorm_q8")
                return q, scales, (x if h is None else h)
    torch = _torch()
    if q is None or scales is None or (residual is not None and h is None):
        with _allocating(stream):
            q = torch.empty(x.shape, dtype=dtype or torch.int8, device=x.device) if q is None else q
            scales = torch.empty(x.shape[0], dtype=torch.float32, device=x.device) if scales is None else scales
            h = _empty_rows(x) if residual is not None and h is None else h
    if dtype is not None and q.dtype != dtype:
        raise ValueError(f"q: {dtype} wanted, not {q.dtype}")
    kind = {torch.int8: VH_NORM_INT8, torch.float8_e4m3fn: VH_NORM_E4M3}.get(q.dtype)
    if kind is None:
        raise ValueError(f"q: int8 or float8_e4m3fn wanted, not {q.dtype}")
    _add_rmsnorm("add_rmsnorm_q8", x, residual, weight, eps, weight_offset, q, q.dtype, kind, h, scales, stream)
    return q, scales, (x if h is None else h)


def add_rmsnorm_grad_workspace(T: int, H: int, device=None):
    torch = _torch()
    _int32(T, H)
    return torch.empty(int(lib().vh_add_rmsnorm_grad_workspace_bytes(T, H)), dtype=torch.uint8, device=device or "cuda")


def add_rmsnorm_grad(dy, h, weight=None, eps: float = 1e-6, weight_offset: float = 0.0, dh=None, dx=None, dweight=None,
                     ws=None, stream=None):
    """Gradient of add_rmsnorm from the sum h that it returned: dx [T,H] is the gradient of x and of the residual
    alike (dh, the gradient that reaches h, included), dweight [H] fp32 (None without a weight).  -> (dx, dweight)"""
    if stream is None and dx is not None:
        m = _compiled_calls()
        if m:
            st = m.add_rmsnorm_grad(dy, h, weight, eps, weight_offset, dh, dx, dweight, ws)
            if st <= 0:
                _check(st, "add_rmsnorm_grad")
                return dx, dweight
    torch = _torch()
    dev = _device(h)
    dt = _dtype(h, "h")
    shape, dtype = h.shape, h.dtype
    hs = _rows(h, "h", dev, shape, dtype)
    T, H = shape
    _int32(T, H)
    dys = _rows(dy, "dy", dev, shape, dtype)
    ep, es = (dh.data_ptr(), _rows(dh, "dh", dev, shape, dtype)) if dh is not None else (None, 0)
    w, w32 = _norm_weight(weight, H, dtype, dev)
    if weight is None and dweight is not None:
        raise ValueError("dweight without a weight")
    if dx is None or (weight is not None and (dweight is None or ws is None)):
        with _allocating(stream):
            dx = _empty_rows(h) if dx is None else dx
            if weight is not None:
                dweight = torch.empty(H, dtype=torch.float32, device=h.device) if dweight is None else dweight
                ws = add_rmsnorm_grad_workspace(T, H, h.device) if ws is None else ws
    dxs = _rows(dx, "dx", dev, shape, dtype)
    st = lib().vh_add_rmsnorm_grad(dy.data_ptr(), h.data_ptr(), w, ep, dt, w32, T, H, dys, hs, es, eps, weight_offset,
                                   dx.data_ptr(), dxs, _vector(dweight, "dweight", dev, H, _f32), _ptr(ws),
                                   0 if ws is None else _workspace(ws, dev), _stream_on(stream, dev))
    _check(st, "add_rmsnorm_grad")
    return dx, dweight


def _logprob_outputs(R, top_n, like, dev, stream, tokens, outs, make_ws):
    """The five outputs and the workspace, those not given newly made -> (outputs, their addresses and the
    workspace's, its size)."""
    logprob, entropy, lse, top_ids, top_logprobs, ws = outs
    if logprob is None or entropy is None or lse is None or top_ids is None or top_logprobs is None or ws is None:
        torch = _torch()
        with _allocating(stream):
            shapes = ((R,), (R,), (R,), (R, top_n), (R, top_n))
            outs = [torch.empty(s, dtype=_i32 if i == 3 else _f32, device=like.device) if g is None else g
                    for i, (s, g) in enumerate(zip(shapes, outs[:5]))] + [make_ws() if ws is None else ws]
        logprob, entropy, lse, top_ids, top_logprobs, ws = outs
    at = [_vector(logprob, "logprob", dev, R, _f32), _vector(entropy, "entropy", dev, R, _f32),
          _vector(lse, "lse", dev, R, _f32), None, None, ws.data_ptr(), _workspace(ws, dev)]
    if top_n > 0:
        at[3] = _vector(top_ids, "top_ids", dev, R * top_n, _i32)
        at[4] = _vector(top_logprobs, "top_logprobs", dev, R * top_n, _f32)
    if tokens is None:
        at[0] = None
    return outs, at


def _logprob_results(outs, tokens):
    return tuple(outs[:5]) if tokens is not None else (None, *outs[1:5])


def logits_logprobs_workspace(R: int, V: int, top_n: int = 0, device=None):
    """A zeroed workspace for logits_logprobs calls of this R, V and top_n."""
    torch = _torch()
    _int32(R, V, top_n)
    n = int(lib().vh_logits_logprobs_workspace_bytes(R, V, top_n))
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def logits_logprobs(logits, tokens, top_n: int = 0, logprob=None, entropy=None, lse=None, top_ids=None,
                    top_logprobs=None, ws=None, stream=None):
    """logits [R,V] fp32 / bf16 / fp16 (rows may be strided), tokens [R] int32 (outside [0,V): no token, logprob 0;
    None: logprob is None)  -> (logprob [R], entropy [R], lse [R], top_ids [R,top_n] int32, top_logprobs [R,top_n])."""
    if stream is None and ws is not None:
        m = _compiled_calls()
        if m:
            st = m.logits_logprobs(logits, tokens, top_n, logprob, entropy, lse, top_ids, top_logprobs, ws)
            if st <= 0:
                _check(st, "logits_logprobs")
                return logprob if tokens is not None else None, entropy, lse, top_ids, top_logprobs
    dev = _device(logits)
    dt = _dtype(logits, "logits")
    shape = logits.shape
    stride = _rows(logits, "logits", dev, shape, logits.dtype)
    R, V = shape
    _int32(R, V, top_n)
    tp = _vector(tokens, "tokens", dev, R, _i32)
    outs, at = _logprob_outputs(R, top_n, logits, dev, stream, tokens,
                                (logprob, entropy, lse, top_ids, top_logprobs, ws),
                                lambda: logits_logprobs_workspace(R, V, top_n, logits.device))
    st = lib().vh_logits_logprobs(logits.data_ptr(), dt, R, V, stride, tp, top_n, *at, _stream_on(stream, dev))
    _check(st, "logits_logprobs")
    return _logprob_results(outs, tokens)


def logits_logprobs_grad(logits, tokens, lse, entropy=None, g_logprob=None, g_entropy=None, dlogits=None, stream=None):
    """Gradient of logits_logprobs' logprob and entropy (their gradients [R] fp32, either may be None) with respect to
    the logits, from the lse and entropy it returned; dlogits may be `logits` itself.  Rows that hold nothing but a far mask
    value (-1e10, the type's lowest) want gradients of 0: their lse in fp32 says too little.  -> dlogits [R,V]"""
    if stream is None and dlogits is not None:
        m = _compiled_calls()
        if m:
            st = m.logits_logprobs_grad(logits, tokens, lse, entropy, g_logprob, g_entropy, dlogits)
            if st <= 0:
                _check(st, "logits_logprobs_grad")
                return dlogits
    dev = _device(logits)
    dt = _dtype(logits, "logits")
    shape, dtype = logits.shape, logits.dtype
    stride = _rows(logits, "logits", dev, shape, dtype)
    R, V = shape
    _int32(R, V)
    if dlogits is None:
        with _allocating(stream):
            dlogits = _empty_rows(logits)
    ds = _rows(dlogits, "dlogits", dev, shape, dtype)
    st = lib().vh_logits_logprobs_grad(
        logits.data_ptr(), dt, R, V, stride, _vector(tokens, "tokens", dev, R, _i32), _vector(lse, "lse", dev, R, _f32),
        _vector(entropy, "entropy", dev, R, _f32), _vector(g_logprob, "g_logprob", dev, R, _f32),
        _vector(g_entropy, "g_entropy", dev, R, _f32), dlogits.data_ptr(), ds, _stream_on(stream, dev))
    _check(st, "logits_logprobs_grad")
    return dlogits


def head_logprobs_workspace(R: int, V: int, top_n: int = 0, device=None):
    """A workspace for head_logprobs calls of this R, V and top_n (about 4 V bytes per row with alternatives)."""
    torch = _torch()
    _int32(R, V, top_n)
    ws = torch.empty(int(lib().vh_head_logprobs_workspace_bytes(R, V, top_n)), dtype=torch.uint8, device=device or "cuda")
    ws[:8192].zero_()
    return ws


def head_logprobs(hidden, W_full, tokens, top_n: int = 0, logprob=None, entropy=None, lse=None, top_ids=None,
                  top_logprobs=None, ws=None, stream=None):
    """logits_logprobs of the scores hidden @ W_full.T, which are not returned: hidden [R,H] bf16, W_full [V,H] bf16,
    tokens [R] int32 -> (logprob [R], entropy [R], lse [R], top_ids [R,top_n] int32, top_logprobs [R,top_n])."""
    if stream is None and ws is not None:
        m = _compiled_calls()
        if m:
            st = m.head_logprobs(hidden, W_full, tokens, top_n, logprob, entropy, lse, top_ids, top_logprobs, ws)
            if st <= 0:
                _check(st, "head_logprobs")
                return logprob if tokens is not None else None, entropy, lse, top_ids, top_logprobs
    dev = _device(hidden)
    _place(W_full, "W_full", dev)
    _require_cuda(hidden, W_full)
    bf16 = _torch().bfloat16
    R, H = hidden.shape
    V = W_full.shape[0]
    _int32(R, H, V, top_n)
    if W_full.shape[1] != H or hidden.dtype != bf16 or W_full.dtype != bf16:
        raise ValueError("shape/dtype mismatch")
    tp = _vector(tokens, "tokens", dev, R, _i32)
    outs, at = _logprob_outputs(R, top_n, hidden, dev, stream, tokens,
                                (logprob, entropy, lse, top_ids, top_logprobs, ws),
                                lambda: head_logprobs_workspace(R, V, top_n, hidden.device))
    st = lib().vh_head_logprobs(hidden.data_ptr(), W_full.data_ptr(), tp, R, H, V, top_n, *at, _stream_on(stream, dev))
    _check(st, "head_logprobs")
    return _logprob_results(outs, tokens)


# ----------------------------------------------------------------------------
# 4-bit rows.  As above, nothing here is recorded by autograd.


def vh_nvfp4_tiles_bytes(rows: int, H: int) -> int:
    """Bytes of a 4-bit matrix [rows, H] in the tiled layout."""
    _int32(rows, H)
    return int(lib().vh_nvfp4_tiles_bytes(rows, H))


def _scale(scale, name, dev, rows):
    """(number, address) of a tensor scale (a number) or row scales (fp32 [rows])."""
    if isinstance(scale, _torch().Tensor):
        return 0.0, _vector(scale, name, dev, rows, _f32)
    return float(scale), None


def _bytes(t, name, dev, shape):
    """Checks a contiguous uint8 CUDA tensor of that shape (or of at least that many bytes, where it is a number)."""
    _place(t, name, dev)
    fits = t.numel() >= shape if isinstance(shape, int) else t.shape == shape
    if t.dtype != _torch().uint8 or not t.is_contiguous() or not fits:
        raise ValueError(f"{name}: contiguous uint8 {shape if isinstance(shape, tuple) else f'of {shape} bytes'} wanted")
    return t.data_ptr()


def _quantize(where, x, tensor_scale, codes, scales, row_scales, stream):
    dev = _device(x)
    dt = _dtype(x, "x")
    stride = _rows(x, "x", dev, x.shape, x.dtype)
    T, H = x.shape
    _int32(T, H)
    cp = _bytes(codes, "codes", dev, (T, H // 2)) if scales is not None else _bytes(codes, "tiles", dev, vh_nvfp4_tiles_bytes(T, H))
    sp = _bytes(scales, "scales", dev, (T, H // 16)) if scales is not None else None
    rp = None
    if tensor_scale is None:
        rp = _vector(row_scales, "row_scales", dev, T, _f32)
    elif row_scales is not None:
        raise ValueError("row_scales are the output of a call without a tensor scale")
    st = lib().vh_nvfp4_quantize(x.data_ptr(), dt, T, H, stride, 0.0 if tensor_scale is None else float(tensor_scale), cp, sp,
                                 rp, _stream_on(stream, dev))
    _check(st, where)


def nvfp4_quantize(x, tensor_scale=None, codes=None, scales=None, row_scales=None, stream=None):
    """Rows x [T,H] (fp32 / bf16 / fp16, may be strided, H % 16 == 0) to block-scaled 4 bits with a tensor scale (a number),
    or with a scale of its own for each row: codes [T,H/2] uint8, scales [T,H/16] uint8 (E4M3), as the *_nvfp4 calls take
    them with a tensor scale.  -> (codes, scales, row_scales [T] fp32 or None)"""
    if stream is None and codes is not None and scales is not None:
        m = _compiled_calls()
        if m:
            st = m.nvfp4_quantize(x, tensor_scale, codes, scales, row_scales)
            if st <= 0:
                _check(st, "nvfp4_quantize")
                return codes, scales, row_scales
    torch = _torch()
    _device(x)
    if x.dim() != 2:
        raise ValueError("x: shape mismatch")
    T, H = x.shape
    with _allocating(stream):
        codes = torch.empty(T, H // 2, dtype=torch.uint8, device=x.device) if codes is None else codes
        scales = torch.empty(T, H // 16, dtype=torch.uint8, device=x.device) if scales is None else scales
        if row_scales is None and tensor_scale is None:
            row_scales = torch.empty(T, dtype=torch.float32, device=x.device)
    _quantize("nvfp4_quantize", x, tensor_scale, codes, scales, row_scales, stream)
    return codes, scales, row_scales


def nvfp4_quantize_tiles(x, tensor_scale=None, tiles=None, row_scales=None, stream=None):
    """nvfp4_quantize into the tiled layout that nvfp4_matmul takes.  -> (tiles, row_scales [T] fp32 or None)"""
    if stream is None and tiles is not None:
        m = _compiled_calls()
        if m:
            st = m.nvfp4_quantize(x, tensor_scale, tiles, None, row_scales)
            if st <= 0:
                _check(st, "nvfp4_quantize_tiles")
                return tiles, row_scales
    torch = _torch()
    _device(x)
    if x.dim() != 2:
        raise ValueError("x: shape mismatch")
    T, H = x.shape
    with _allocating(stream):
        tiles = torch.empty(vh_nvfp4_tiles_bytes(T, H), dtype=torch.uint8, device=x.device) if tiles is None else tiles
        if row_scales is None and tensor_scale is None:
            row_scales = torch.empty(T, dtype=torch.float32, device=x.device)
    _quantize("nvfp4_quantize_tiles", x, tensor_scale, tiles, None, row_scales, stream)
    return tiles, row_scales


def nvfp4_tile(codes, scales, tiles=None, stream=None):
    """codes [V,H/2] uint8, scales [V,H/16] uint8 (row-major) -> the tiled copy that nvfp4_matmul takes.  Done once for a
    weight (not the layout of nvfp4_pack, which serves the heads' argmax)."""
    torch = _torch()
    dev = _device(codes)
    if codes.dim() != 2:
        raise ValueError("codes: shape mismatch")
    V, H = codes.shape[0], codes.shape[1] * 2
    _int32(V, H)
    cp, sp = _bytes(codes, "codes", dev, (V, H // 2)), _bytes(scales, "scales", dev, (V, H // 16))
    n = vh_nvfp4_tiles_bytes(V, H)
    if tiles is None:
        with _allocating(stream):
            tiles = torch.empty(n, dtype=torch.uint8, device=codes.device)
    st = lib().vh_nvfp4_tile(cp, sp, V, H, _bytes(tiles, "tiles", dev, n), tiles.numel(), _stream_on(stream, dev))
    _check(st, "nvfp4_tile")
    return tiles


def _dequantize(where, codes, scales, T, H, scale, out, dtype, stream):
    dev = _device(codes)
    _int32(T, H)
    cp = _bytes(codes, "codes", dev, (T, H // 2)) if scales is not None else _bytes(codes, "tiles", dev, vh_nvfp4_tiles_bytes(T, H))
    sp = _bytes(scales, "scales", dev, (T, H // 16)) if scales is not None else None
    if out is None:
        with _allocating(stream):
            out = _torch().empty(T, H, dtype=dtype or _torch().bfloat16, device=codes.device)
    elif dtype is not None and out.dtype != dtype:
        raise ValueError(f"out: {dtype} wanted, not {out.dtype}")
    g, gp = _scale(scale, "scale", dev, T)
    st = lib().vh_nvfp4_dequantize(cp, sp, T, H, g, gp, _dtype(out, "out"), out.data_ptr(),
                                   _rows(out, "out", dev, (T, H), out.dtype), _stream_on(stream, dev))
    _check(st, where)
    return out


def nvfp4_dequantize(codes, scales, scale, out=None, dtype=None, stream=None):
    """Values of 4-bit rows, code * block scale * scale: codes [T,H/2], scales [T,H/16] uint8, scale a number or the row
    scales [T] fp32; out [T,H] fp32 / bf16 / fp16 (bf16 where neither out nor dtype is given).  -> out"""
    if stream is None and out is not None and dtype is None:
        m = _compiled_calls()
        if m:
            st = m.nvfp4_dequantize(codes, scales, scale, out)
            if st <= 0:
                _check(st, "nvfp4_dequantize")
                return out
    _device(codes)
    if codes.dim() != 2 or scales is None:
        raise ValueError("codes, scales: shape mismatch")
    return _dequantize("nvfp4_dequantize", codes, scales, codes.shape[0], codes.shape[1] * 2, scale, out, dtype, stream)


def nvfp4_dequantize_tiles(tiles, scale, T: int, H: int, out=None, dtype=None, stream=None):
    """nvfp4_dequantize from the tiled layout of a [T,H] matrix (its gradient's product takes the values).  -> out"""
    return _dequantize("nvfp4_dequantize_tiles", tiles, None, T, H, scale, out, dtype, stream)


def nvfp4_matmul(x_tiles, x_scale, w_tiles, w_scale, T: int, V: int, H: int, out=None, dtype=None, stream=None):
    """out[t,v] = sum over h of X[t,h] W[v,h] of two 4-bit matrices in the tiled layout, X [T,H] (nvfp4_quantize_tiles) and W
    [V,H] (nvfp4_tile, nvfp4_quantize_tiles); each scale is a number or the row scales (fp32 [T], [V]).  out [T,V] fp32 /
    bf16 / fp16, rows may be strided (bf16 where neither out nor dtype is given): logits of a 4-bit head, say.  -> out"""
    if stream is None and out is not None and dtype is None:
        m = _compiled_calls()
        if m:
            st = m.nvfp4_matmul(x_tiles, x_scale, w_tiles, w_scale, T, V, H, out)
            if st <= 0:
                _check(st, "nvfp4_matmul")
                return out
    dev = _device(x_tiles)
    _int32(T, V, H)
    xp = _bytes(x_tiles, "x_tiles", dev, vh_nvfp4_tiles_bytes(T, H))
    wp = _bytes(w_tiles, "w_tiles", dev, vh_nvfp4_tiles_bytes(V, H))
    if out is None:
        with _allocating(stream):
            out = _torch().empty(T, V, dtype=dtype or _torch().bfloat16, device=x_tiles.device)
    elif dtype is not None and out.dtype != dtype:
        raise ValueError(f"out: {dtype} wanted, not {out.dtype}")
    xg, xgp = _scale(x_scale, "x_scale", dev, T)
    wg, wgp = _scale(w_scale, "w_scale", dev, V)
    st = lib().vh_nvfp4_matmul(xp, xg, xgp, wp, wg, wgp, T, V, H, _dtype(out, "out"), out.data_ptr(),
                               _rows(out, "out", dev, (T, V), out.dtype), _stream_on(stream, dev))
    _check(st, "nvfp4_matmul")
    return out


# ----------------------------------------------------------------------------
# Processing of logits.

_RULES = ("history", "history_len", "prompt_len", "draft_ids", "repetition", "frequency", "presence", "bias_ids", "bias",
          "allowed", "temperature")


def _rows_or_none(t, name, dev, rows, dtype, least=0):
    """(address, elements between rows, width) of a 2-D tensor of that many rows, or of none."""
    if t is None:
        return None, 0, 0
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] < least:
        raise ValueError(f"{name}: shape mismatch")
    return t.data_ptr(), _rows(t, name, dev, t.shape, dtype), t.shape[1]


def _rules(dev, R, V, rules):
    """(vh_logits_rules, rows per sequence) of the rules given, all by the name of the call's argument."""
    S = next((len(rules[k]) for k in _RULES if k != "allowed" and rules[k] is not None), R)
    if S < 1 or R % S != 0:
        raise ValueError(f"{R} rows are not a whole number for each of {S} sequences")
    per = R // S
    r = LogitsRules()
    r.history, r.history_stride, r.history_width = _rows_or_none(rules["history"], "history", dev, S, _i32)
    for name, dtype in (("history_len", _i32), ("prompt_len", _i32), ("repetition", _f32), ("frequency", _f32),
                        ("presence", _f32), ("temperature", _f32)):
        setattr(r, name, _vector(rules[name], name, dev, S, dtype))
    d = rules["draft_ids"]
    if d is not None and d.shape != (S, per - 1):
        raise ValueError(f"draft_ids: ({S}, {per - 1}) wanted")
    r.draft_ids = _vector(d, "draft_ids", dev, S * (per - 1), _i32)
    ids, bias = rules["bias_ids"], rules["bias"]
    if (ids is None) != (bias is None) or (ids is not None and (ids.dim() != 2 or ids.shape != bias.shape or len(ids) != S)):
        raise ValueError("bias_ids, bias: shape mismatch")
    r.n_bias = ids.shape[1] if ids is not None else 0
    r.bias_ids, r.bias = _vector(ids, "bias_ids", dev, S * r.n_bias, _i32), _vector(bias, "bias", dev, S * r.n_bias, _f32)
    r.allowed, r.allowed_stride, _ = _rows_or_none(rules["allowed"], "allowed", dev, R, _i32, (V + 31) // 32)
    return r, per


def logits_process(logits, history=None, history_len=None, prompt_len=None, draft_ids=None, repetition=None, frequency=None,
                   presence=None, bias_ids=None, bias=None, allowed=None, temperature=None, out=None, stream=None):
    """Biases, penalties for repeated tokens, temperature and grammar masks on logits [R,V] (fp32 / bf16 / fp16, rows may be
    strided), whose rows are R / S after one another for each of S sequences (a verify round's k + 1 positions, or one):
        z = logits + bias;  z / repetition or (z <= 0) z * repetition for tokens in the history;
        z - frequency * n - presence * [n > 0], n the times a token has been output;  z / temperature;  -inf where not allowed
    history [S,L] int32 (the prompt's tokens first; ids outside [0,V) are passed over), history_len, prompt_len [S] int32;
    draft_ids [S,R/S-1] int32: row j also counts the first j; repetition, frequency, presence, temperature [S] fp32
    (temperature 0: greedy, as 1); bias_ids [S,n] int32 with bias [S,n] fp32 (the last entry of an id counts); allowed
    [R,>=ceil(V/32)] int32, bit v % 32 of word v / 32.  Every rule may be None.
    out: logits' type or fp32, may be `logits` itself (which takes longer).  -> out"""
    if stream is None and out is not None:
        m = _compiled_calls()
        if m:
            st = m.logits_process(logits, history, history_len, prompt_len, draft_ids, repetition, frequency, presence, bias_ids,
                                  bias, allowed, temperature, out)
            if st <= 0:
                _check(st, "logits_process")
                return out
    dev = _device(logits)
    dt = _dtype(logits, "logits")
    shape = logits.shape
    stride = _rows(logits, "logits", dev, shape, logits.dtype)
    R, V = shape
    _int32(R, V)
    rules = dict(zip(_RULES, (history, history_len, prompt_len, draft_ids, repetition, frequency, presence, bias_ids, bias,
                              allowed, temperature)))
    r, per = _rules(dev, R, V, rules)
    if out is None:
        with _allocating(stream):
            out = _empty_rows(logits)
    if out.dtype != logits.dtype and out.dtype != _f32:
        raise ValueError(f"out: {logits.dtype} or float32 wanted, not {out.dtype}")
    st = lib().vh_logits_process(logits.data_ptr(), dt, R, V, stride, per, ctypes.byref(r), out.data_ptr(), _dtypes[out.dtype],
                                 _rows(out, "out", dev, shape, out.dtype), _stream_on(stream, dev))
    _check(st, "logits_process")
    return out


def logits_process_grad(dout, logits, history=None, history_len=None, prompt_len=None, draft_ids=None, repetition=None,
                        frequency=None, presence=None, bias_ids=None, bias=None, allowed=None, temperature=None, dlogits=None,
                        stream=None):
    """Gradient of logits_process with respect to the logits, from dout [R,V] of their type (0 where not allowed); dlogits
    may be `dout` itself (which takes longer).  The other arguments as there.  -> dlogits"""
    if stream is None and dlogits is not None:
        m = _compiled_calls()
        if m:
            st = m.logits_process_grad(dout, logits, history, history_len, prompt_len, draft_ids, repetition, frequency, presence,
                                       bias_ids, bias, allowed, temperature, dlogits)
            if st <= 0:
                _check(st, "logits_process_grad")
                return dlogits
    dev = _device(logits)
    dt = _dtype(logits, "logits")
    shape, dtype = logits.shape, logits.dtype
    stride = _rows(logits, "logits", dev, shape, dtype)
    R, V = shape
    _int32(R, V)
    rules = dict(zip(_RULES, (history, history_len, prompt_len, draft_ids, repetition, frequency, presence, bias_ids, bias,
                              allowed, temperature)))
    r, per = _rules(dev, R, V, rules)
    if dlogits is None:
        with _allocating(stream):
            dlogits = _empty_rows(logits)
    st = lib().vh_logits_process_grad(dout.data_ptr(), logits.data_ptr(), dt, R, V, _rows(dout, "dout", dev, shape, dtype),
                                      stride, per, ctypes.byref(r), dlogits.data_ptr(),
                                      _rows(dlogits, "dlogits", dev, shape, dtype), _stream_on(stream, dev))
    _check(st, "logits_process_grad")
    return dlogits
