"""ctypes binding of libtopktopp (include/topktopp.h).

Argument marshalling only: tensors are turned into device pointers and the
current HIP stream, and every step of the filter runs in the library's HIP
kernels. If the library has not been built this module raises instead of
falling back to anything else.
"""

from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import operator
import os
import struct
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libtopktopp.so")

TOPKTOPP_F32, TOPKTOPP_F16, TOPKTOPP_BF16 = 0, 1, 2
STATUS_NAMES = {0: "OK", 1: "ERR_NULLPTR", 2: "ERR_INVALID", 3: "ERR_RUNTIME"}
EXPORTED_SYMBOLS = (
    "apply_top_k_top_p",
    "apply_top_k_top_p_ex",
    "apply_top_k_top_p_min_p",
    "apply_top_k_top_p_min_p_with_sorted",
    "apply_top_k_top_p_strided",
    "apply_top_k_top_p_with_sorted",
    "apply_top_k_top_p_with_sorted_ex",
    "beam_backtrace",
    "beam_reorder_states",
    "beam_search_select",
    "beam_search_select_workspace",
    "cache_pages_compact",
    "cache_pages_fork",
    "cache_pages_resize",
    "cache_pages_resize_workspace",
    "sample_top_k_top_p",
    "speculative_verify",
    "speculative_verify_workspace",
    "top_k_top_p_sorted_survivors",
    "topktopp_last_error",
    "topktopp_set_plan_policy",
)

_lib = None


TOPKTOPP_MAX_BEAMS, TOPKTOPP_MAX_CANDIDATES, TOPKTOPP_MAX_DRAFTS = 128, 256, 255


class BeamState(ctypes.Structure):
    """topktopp_beam_state: a state's memory, strides and run in bytes."""

    _fields_ = [
        ("data", ctypes.c_void_p),
        ("row_stride", ctypes.c_int64),
        ("size", ctypes.c_int64 * 3),
        ("stride", ctypes.c_int64 * 3),
        ("positions", ctypes.c_int64),
        ("position_stride", ctypes.c_int64),
        ("run", ctypes.c_int64),
    ]


class TopKTopPError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libtopktopp.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it first (python -m top_logits_filtering_amd.build); "
            "there is no fallback implementation"
        )
    lib = ctypes.CDLL(p)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.apply_top_k_top_p.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp]
    lib.apply_top_k_top_p.restype = i32
    lib.apply_top_k_top_p_with_sorted.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    lib.apply_top_k_top_p_with_sorted.restype = i32
    lib.apply_top_k_top_p_min_p.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, vp]
    lib.apply_top_k_top_p_min_p.restype = i32
    lib.apply_top_k_top_p_min_p_with_sorted.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp, vp, vp, vp]
    lib.apply_top_k_top_p_min_p_with_sorted.restype = i32
    lib.apply_top_k_top_p_ex.argtypes = [vp, i64, i32, i64, i64, vp, vp, vp, vp, i64, vp]
    lib.apply_top_k_top_p_ex.restype = i32
    lib.apply_top_k_top_p_with_sorted_ex.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, vp, vp, vp, i64, vp, i64, vp]
    lib.apply_top_k_top_p_with_sorted_ex.restype = i32
    lib.apply_top_k_top_p_strided.argtypes = [vp, i64, i64, i32, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp]
    lib.apply_top_k_top_p_strided.restype = i32
    lib.sample_top_k_top_p.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]
    lib.sample_top_k_top_p.restype = i32
    lib.top_k_top_p_sorted_survivors.argtypes = [vp, i32, i64, i64, vp, vp, vp, i64, vp, vp, vp, vp]
    lib.top_k_top_p_sorted_survivors.restype = i32
    lib.beam_search_select.argtypes = [vp, i64, i32, i64, i64, i64, vp, vp, ctypes.c_int32, vp, i64, vp, vp, vp, vp,
                                       i64, vp]
    lib.beam_search_select.restype = i32
    lib.beam_search_select_workspace.argtypes = [i32, i64, i64, i64, i64]
    lib.beam_search_select_workspace.restype = i64
    lib.beam_reorder_states.argtypes = [vp, i64, vp, i64, i64, vp, vp]
    lib.beam_reorder_states.restype = i32
    lib.beam_backtrace.argtypes = [vp, vp, i64, i64, i64, vp, vp, i64, ctypes.c_int32, vp, vp]
    lib.beam_backtrace.restype = i32
    lib.speculative_verify.argtypes = [vp, i64, i32, i64, i64, i64, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, i64, vp]
    lib.speculative_verify.restype = i32
    lib.speculative_verify_workspace.argtypes = [i32, i64, i64, i64, i32]
    lib.speculative_verify_workspace.restype = i64
    lib.cache_pages_fork.argtypes = [vp, i64, i64, vp, vp, i64, i64, vp, i64, i64, vp]
    lib.cache_pages_fork.restype = i32
    lib.cache_pages_resize.argtypes = [vp, i64, i64, i64, vp, vp, vp, i64, i64, vp, i64, vp, i64, vp]
    lib.cache_pages_resize.restype = i32
    lib.cache_pages_resize_workspace.argtypes = [i64, i64]
    lib.cache_pages_resize_workspace.restype = i64
    lib.cache_pages_compact.argtypes = [vp, i64, i64, i64, vp, i64, i64, i64, vp, vp, i64, vp, vp]
    lib.cache_pages_compact.restype = i32
    lib.topktopp_last_error.argtypes = []
    lib.topktopp_last_error.restype = ctypes.c_char_p
    lib.topktopp_set_plan_policy.argtypes = [i32]
    lib.topktopp_set_plan_policy.restype = i32
    if path is None:
        _lib = lib
    return lib


def last_error() -> str:
    return load_library().topktopp_last_error().decode()


def set_plan_policy(policy: int) -> int:
    """0 auto (candidate plan), 1 multi-pass plan, 2 candidate plan re-reading global memory."""
    prev = load_library().topktopp_set_plan_policy(int(policy))
    if prev < 0:
        raise ValueError(f"unknown plan policy {policy}")
    return prev


_DTYPE_CODES = None


def _dtype_code(t) -> int:
    global _DTYPE_CODES
    if _DTYPE_CODES is None:
        import torch

        _DTYPE_CODES = {torch.float32: TOPKTOPP_F32, torch.float16: TOPKTOPP_F16, torch.bfloat16: TOPKTOPP_BF16}
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _rows(t):
    """(pointer, row stride in elements) of a 2-D tensor whose rows are
    contiguous; None for None."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if t.dim() != 2:
        raise ValueError("expected a 2-D [B, V] tensor")
    B, V = t.shape
    if V > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride 1 along the last dimension)")
    ld = t.stride(0) if B > 1 else V
    return t.data_ptr(), ld


def _rows_contiguous(t) -> bool:
    """Rows contiguous and disjoint: a view the row-strided entry points take."""
    B, V = t.shape
    return (V <= 1 or t.stride(1) == 1) and (B <= 1 or t.stride(0) >= V)


def _entries(t, B):
    """(pointer, stride in elements) of a [B] parameter vector of any stride;
    (None, 0) for None."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if t.dim() != 1 or t.shape[0] != B:
        raise ValueError(f"expected a 1-D tensor of {B} entries, got shape {tuple(t.shape)}")
    return t.data_ptr(), t.stride(0)


def _check_vector(t, B, dtype, name):
    """A per-row parameter or output: None, or a 1-D tensor of B entries of `dtype`."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != B:
        raise ValueError(f"{name} must be a 1-D tensor of {B} entries, got shape {tuple(t.shape)}")


def _check_matrix(t, shape, dtype, name):
    """None, or a 2-D tensor of `shape` and `dtype`."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be [{shape[0]}, {shape[1]}], got shape {tuple(t.shape)}")


def _check_params(B, dtype, p, k, min_p):
    """p and min_p [B] in the logits dtype, k [B] int32 (each optional)."""
    import torch

    _check_vector(p, B, dtype, "p")
    _check_vector(k, B, torch.int32, "k")
    _check_vector(min_p, B, dtype, "min_p")


def _check_device(device, *tensors):
    """Every given tensor on the GPU, on `device`."""
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if t.device != device:
            raise ValueError(f"tensors must share one device: {t.device} and {device}")


def _stream(stream, device) -> int:
    """The HIP stream handle to launch on: the given one, else torch's current
    stream of the tensors' device."""
    if stream is None:
        import torch

        return torch._C._cuda_getCurrentRawStream(device.index)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int):
    if status != 0:
        raise TopKTopPError(status, last_error())


def apply_top_k_top_p(logits, p=None, k=None, out=None, stream=None, min_p=None):
    """Filter raw logits [B, V]; p [B] (logits dtype), k [B] (int32) and min_p
    [B] (logits dtype, the min-p stage) are optional. Every operand may be a
    strided view: row-strided ones (rows contiguous, e.g. a slice of a padded
    vocabulary) take the vector kernels, any other view (a transpose, a
    column step, parameters with a stride) the element-wise strided kernel."""
    import torch

    lib = load_library()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [B, V]")
    B, V = logits.shape
    if out is None:
        out = torch.empty((B, V), dtype=logits.dtype, device=logits.device)
    _check_matrix(out, (B, V), logits.dtype, "out")
    _check_params(B, logits.dtype, p, k, min_p)
    _check_device(logits.device, logits, out, p, k, min_p)
    st = _stream(stream, logits.device)
    params = [t for t in (p, k, min_p) if t is not None]
    if not (_rows_contiguous(logits) and _rows_contiguous(out) and all(t.is_contiguous() for t in params)):
        if not (logits.is_cuda and out.is_cuda):
            raise ValueError("tensors must live on the GPU")
        (pp, ps), (kp, ks), (mp, ms) = _entries(p, B), _entries(k, B), _entries(min_p, B)
        status = lib.apply_top_k_top_p_strided(logits.data_ptr(), logits.stride(0), logits.stride(1),
                                               _dtype_code(logits), B, V, pp, ps, kp, ks, mp, ms, out.data_ptr(),
                                               out.stride(0), out.stride(1), st)
        _check(status)
        return out
    (xp, ldx), (op, ldo) = _rows(logits), _rows(out)
    if ldx != V or ldo != V:
        status = lib.apply_top_k_top_p_ex(xp, ldx, _dtype_code(logits), B, V, _ptr(p), _ptr(k), _ptr(min_p), op, ldo,
                                          st)
    elif min_p is None:
        status = lib.apply_top_k_top_p(xp, _dtype_code(logits), B, V, _ptr(p), _ptr(k), op, st)
    else:
        status = lib.apply_top_k_top_p_min_p(xp, _dtype_code(logits), B, V, _ptr(p), _ptr(k), _ptr(min_p), op, st)
    _check(status)
    return out


def apply_top_k_top_p_with_sorted(sorted_value, sorted_indices, p=None, k=None, logits=None, out=None,
                                  stream=None, min_p=None):
    """Filter pre-sorted rows (ascending sorted_value, int32 sorted_indices);
    min_p [B] (logits dtype) adds the min-p stage."""
    import torch

    lib = load_library()
    if sorted_value.dim() != 2:
        raise ValueError("sorted_value must be 2-D [B, V]")
    B, V = sorted_value.shape
    if out is None:
        out = torch.empty((B, V), dtype=sorted_value.dtype, device=sorted_value.device)
    _check_matrix(sorted_indices, (B, V), torch.int32, "sorted_indices")
    _check_matrix(logits, (B, V), sorted_value.dtype, "logits")
    _check_matrix(out, (B, V), sorted_value.dtype, "out")
    _check_params(B, sorted_value.dtype, p, k, min_p)
    _check_device(sorted_value.device, sorted_value, sorted_indices, logits, out, p, k, min_p)
    st = _stream(stream, sorted_value.device)
    (sp, lds), (ip, ldi), (xp, ldx), (op, ldo) = _rows(sorted_value), _rows(sorted_indices), _rows(logits), _rows(out)
    if lds != V or ldi != V or ldo != V or (logits is not None and ldx != V):
        status = lib.apply_top_k_top_p_with_sorted_ex(
            sp, lds, ip, ldi, _dtype_code(sorted_value), B, V, _ptr(p), _ptr(k), _ptr(min_p), xp, ldx, op, ldo, st
        )
    elif min_p is None:
        status = lib.apply_top_k_top_p_with_sorted(
            _ptr(sorted_value), _ptr(sorted_indices), _dtype_code(sorted_value), B, V, _ptr(p), _ptr(k),
            _ptr(logits), _ptr(out), st
        )
    else:
        status = lib.apply_top_k_top_p_min_p_with_sorted(
            _ptr(sorted_value), _ptr(sorted_indices), _dtype_code(sorted_value), B, V, _ptr(p), _ptr(k),
            _ptr(min_p), _ptr(logits), _ptr(out), st
        )
    _check(status)
    return out


def sample_top_k_top_p(logits, p=None, k=None, min_p=None, q=None, eps=0.0, out=None, selected=None, stream=None):
    """Filter logits [B, V] and pick one index per row (int32 [B], returned).

    q [B, V] float32 by descending survivor rank (QSample), or None (the
    argmax). out, if given, receives the filtered logits; otherwise the rows
    are only read."""
    import torch

    lib = load_library()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [B, V]")
    B, V = logits.shape
    if q is not None and (q.dtype != torch.float32 or tuple(q.shape) != (B, V)):
        raise ValueError("q must be float32 [B, V]")
    if selected is None:
        selected = torch.empty((B,), dtype=torch.int32, device=logits.device)
    _check_matrix(out, (B, V), logits.dtype, "out")
    _check_vector(selected, B, torch.int32, "selected")
    _check_params(B, logits.dtype, p, k, min_p)
    _check_device(logits.device, logits, p, k, min_p, q, out, selected)
    status = lib.sample_top_k_top_p(
        _ptr(logits), _dtype_code(logits), B, V, _ptr(p), _ptr(k), _ptr(min_p), _ptr(q), float(eps), _ptr(out),
        _ptr(selected), _stream(stream, logits.device)
    )
    _check(status)
    return selected


def top_k_top_p_sorted_survivors(logits, p=None, k=None, min_p=None, cap=1024, with_probs=True, stream=None,
                                 out=None):
    """The filter's survivors in descending order: (probs [B, cap] float32 or
    None, indices [B, cap] int32, counts [B] int32). Ranks past a row's
    survivors hold probability 0 and index -1. ``out`` may give the three
    buffers (probs may be None); they are then filled and returned."""
    import torch

    lib = load_library()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [B, V]")
    B, V = logits.shape
    dev = logits.device
    if out is not None:
        probs, indices, counts = out
        if (tuple(indices.shape) != (B, cap) or tuple(counts.shape) != (B,)
                or (probs is not None and tuple(probs.shape) != (B, cap))):
            raise ValueError("out buffers must be probs [B, cap], indices [B, cap], counts [B]")
    else:
        probs = torch.empty((B, cap), dtype=torch.float32, device=dev) if with_probs else None
        indices = torch.empty((B, cap), dtype=torch.int32, device=dev)
        counts = torch.empty((B,), dtype=torch.int32, device=dev)
    _check_matrix(probs, (B, cap), torch.float32, "probs")
    _check_matrix(indices, (B, cap), torch.int32, "indices")
    _check_vector(counts, B, torch.int32, "counts")
    _check_params(B, logits.dtype, p, k, min_p)
    _check_device(dev, logits, p, k, min_p, probs, indices, counts)
    status = lib.top_k_top_p_sorted_survivors(
        _ptr(logits), _dtype_code(logits), B, V, _ptr(p), _ptr(k), _ptr(min_p), int(cap), _ptr(probs), _ptr(indices),
        _ptr(counts), _stream(stream, dev)
    )
    _check(status)
    return probs, indices, counts


_pack_pointer = struct.Struct("=Q").pack
_NO_POINTER = bytes(8)
_NULL_SCOPE = contextlib.nullcontext()


def _scope(stream, device):
    """(stream handle, context): the given stream, or torch's current one of
    the tensors' device, and the context in which buffers for it are allocated
    and kernels launched (that stream current, and its device)."""
    import torch

    if device.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
        if torch._C._cuda_getDevice() == device.index:
            return handle, _NULL_SCOPE
        return handle, torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):  # a handle; 0 is the default stream's
        stream = torch.cuda.ExternalStream(int(stream), device=device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream's device {stream.device} is not the tensors' device {device}")
    return int(stream.cuda_stream), torch.cuda.stream(stream)


def _check_dense(t, shape, dtype, name, device):
    """A contiguous tensor of `shape` and `dtype` on the GPU of index `device`
    (-1: the CPU, where nothing runs)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != device:
        raise ValueError(f"tensors must share one device: {name} is on {t.device}")


def beam_search_select_workspace(dtype, N, K, V, n=None):
    """Bytes of the workspace that beam_search_select takes for logits
    [N * K, V] of torch dtype `dtype` and n continuations (default K)."""
    import torch

    size = load_library().beam_search_select_workspace(
        _dtype_code(torch.empty(0, dtype=dtype)), int(N), int(K), int(V), int(K if n is None else n))
    if size < 0:
        raise TopKTopPError(2, last_error())
    return size


def beam_search_select(logits, scores, n=None, finished=None, end_token=None, weights=None, out=None, workspace=None,
                       stream=None):
    """The n best continuations (default K) of each prompt over its K beams and
    the vocabulary: (scores [N, n] float32, parents [N, n] int32, tokens [N, n]
    int32), best first.

    logits [N * K, V], rows contiguous, any row stride from V on; scores [N, K] float32,
    the beams' accumulated log-probabilities. A continuation of beam b with
    token v scores scores[b] + log_softmax(logits[b])[v]. finished [N, K]
    bool: such a beam goes on as itself only, with end_token and its score.
    weights [N, K] float32 > 0 multiply the scores for the ranking (length
    normalisation), not in what is returned. Beams whose score is -inf and
    tokens whose logit is -inf are left out; ranks without a continuation hold
    score -inf, parent -1, token -1. out: the three tensors to fill; workspace:
    a uint8 tensor of beam_search_select_workspace() bytes, not used by any
    other call that may run at the same time (each call allocates one else).
    No gradients: what is returned does not depend on logits or scores for
    autograd, whether or not these require grad."""
    import torch

    lib = _lib or load_library()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [N * K, V]")
    if scores.dim() != 2:
        raise ValueError("scores must be 2-D [N, K]")
    (R, V), (N, K) = logits.shape, scores.shape
    if N * K != R:
        raise ValueError(f"logits must have N * K = {N * K} rows, got {R}")
    ldx, step = logits.stride()
    if step != 1 and V > 1:
        raise ValueError("rows must be contiguous (stride 1 along the last dimension)")
    if R <= 1:
        ldx = V
    n = K if n is None else int(n)
    dtype = _dtype_code(logits)
    dev = logits.get_device()
    _check_dense(scores, (N, K), torch.float32, "scores", dev)
    p_finished = p_weights = None
    if finished is not None:
        _check_dense(finished, (N, K), torch.uint8 if finished.dtype == torch.uint8 else torch.bool, "finished", dev)
        if end_token is None:
            raise ValueError("finished needs end_token")
        if not 0 <= end_token < 2 ** 31:
            raise ValueError(f"end_token must be an int32 >= 0, got {end_token}")
        p_finished = finished.data_ptr()
    if weights is not None:
        _check_dense(weights, (N, K), torch.float32, "weights", dev)
        p_weights = weights.data_ptr()
    handle, scope = _scope(stream, logits.device)
    given = out is not None
    with scope:
        if not given:
            out = (torch.empty((N, n), dtype=torch.float32, device=logits.device),
                   torch.empty((N, n), dtype=torch.int32, device=logits.device),
                   torch.empty((N, n), dtype=torch.int32, device=logits.device))
        o_scores, o_parents, o_tokens = out
        _check_dense(o_scores, (N, n), torch.float32, "out scores", dev)
        _check_dense(o_parents, (N, n), torch.int32, "out parents", dev)
        _check_dense(o_tokens, (N, n), torch.int32, "out tokens", dev)
        if o_scores.requires_grad and torch.is_grad_enabled():
            raise ValueError("out scores that require grad can only be written under no_grad")
        if workspace is None:
            size = lib.beam_search_select_workspace(dtype, N, K, V, n)
            if size < 0:
                raise TopKTopPError(2, last_error())
            workspace = torch.empty(size, dtype=torch.uint8, device=logits.device)
        else:
            size = workspace.numel()
            _check_dense(workspace, workspace.shape, torch.uint8, "workspace", dev)
        status = lib.beam_search_select(
            logits.data_ptr(), ldx, dtype, N, K, V, scores.data_ptr(), p_finished,
            0 if finished is None else int(end_token), p_weights, n, o_scores.data_ptr(), o_parents.data_ptr(),
            o_tokens.data_ptr(), workspace.data_ptr(), size, handle)
    _check(status)
    if given:
        torch.autograd.graph.increment_version(out)
    return out


@functools.lru_cache(maxsize=256)
def _state_layout(shape, strides, itemsize, batch_dim, seq_dim):
    """A tensor's axes as a BeamState has them: (row_stride, sizes, strides,
    positions, position_stride, run), strides and run in bytes. Axes that lie
    side by side are joined. seq_dim None: no axis is the positions."""
    axes = sorted((strides[d] * itemsize, shape[d]) for d in range(len(shape))
                  if d not in (batch_dim, seq_dim) and shape[d] != 1)
    run = itemsize
    while axes and axes[0][0] == run:
        run *= axes.pop(0)[1]
    joined = []
    for stride, size in axes:
        if joined and stride == joined[-1][0] * joined[-1][1]:
            joined[-1] = (joined[-1][0], joined[-1][1] * size)
        else:
            joined.append((stride, size))
    positions, position_stride = (1, run) if seq_dim is None else (shape[seq_dim], strides[seq_dim] * itemsize)
    if seq_dim is None and len(joined) == 4:  # without lengths the positions are an axis like any other
        position_stride, positions = joined.pop()
    if len(joined) > 3:
        raise ValueError(f"a state of shape {shape} and strides {strides} has too many separate axes")
    # the last of the three has the smallest stride
    joined = [(run, 1)] * (3 - len(joined)) + joined[::-1]
    return (strides[batch_dim] * itemsize, tuple(n for _, n in joined), tuple(b for b, _ in joined), positions,
            position_stride, run)


@functools.lru_cache(maxsize=256)
def _state_bytes(shape, strides, itemsize, batch_dim, seq_dim, rows):
    """A BeamState as bytes, without the data pointer it begins with."""
    dims = len(shape)
    if not -dims <= batch_dim < dims:
        raise ValueError(f"a state of {dims} axes has no batch_dim {batch_dim}")
    if shape[batch_dim] != rows:
        raise ValueError(f"a state must have N * K = {rows} rows, got shape {tuple(shape)}")
    if seq_dim is not None:
        if not -dims <= seq_dim < dims or (seq_dim - batch_dim) % dims == 0:
            raise ValueError(f"a state of {dims} axes has no seq_dim {seq_dim} beside batch_dim {batch_dim}")
        seq_dim %= dims
    if 0 in shape:
        return bytes(ctypes.sizeof(BeamState) - 8)  # nothing to move
    row_stride, sizes, steps, positions, step, run = _state_layout(tuple(shape), strides, itemsize, batch_dim % dims,
                                                                   seq_dim)
    return struct.pack("=10q", row_stride, *sizes, *steps, positions, step, run)


def beam_reorder_states(states, parents, batch_dim=0, seq_dim=None, lengths=None, stream=None):
    """Every state's rows follow their beams, in place: along batch_dim (of
    size N * K) row i * K + b becomes what row i * K + parents[i, b] was.

    states: a tensor or a sequence of them (the caches of all layers, any
    dtype and strides), all with the rows along batch_dim. parents [N, K]
    int32; a row whose parent lies outside [0, K) stays as it is. lengths [N]
    int32 (needs seq_dim): only positions below lengths[i] along seq_dim are
    moved. Returns states. Gradients do not flow through the move: a state that
    requires grad is refused unless under no_grad, and one that was saved for a
    backward pass counts as modified, as with torch's in-place operations."""
    import torch

    lib = _lib or load_library()
    tensors = [states] if isinstance(states, torch.Tensor) else list(states)
    if parents.dim() != 2:
        raise ValueError("parents must be 2-D [N, K]")
    N, K = parents.shape
    dev = parents.get_device()
    _check_dense(parents, (N, K), torch.int32, "parents", dev)
    if lengths is not None:
        _check_dense(lengths, (N,), torch.int32, "lengths", dev)
        if seq_dim is None:
            raise ValueError("lengths needs seq_dim")
    seq = None if lengths is None else seq_dim
    descs = []
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"tensors must share one device: a state is on {t.device}")
        if t.is_neg() or (t.is_complex() and t.is_conj()):
            raise ValueError("a state must not be a lazily conjugated or negated view")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError("a state that requires grad can only be reordered under no_grad")
        descs.append(_pack_pointer(t.data_ptr()))
        descs.append(_state_bytes(t.shape, t.stride(), t.element_size(), batch_dim, seq, N * K))
    descs = b"".join(descs)
    handle, scope = _scope(stream, parents.device)
    with scope:
        status = lib.beam_reorder_states(descs, len(tensors), parents.data_ptr(), N, K,
                                         None if lengths is None else lengths.data_ptr(), handle)
    _check(status)
    torch.autograd.graph.increment_version(tensors)
    return states


def beam_backtrace(tokens, parents, beams=None, lengths=None, pad=-1, out=None, stream=None):
    """The sequences of a search's history: tokens and parents [T, N, K] int32
    are what was picked in each step. Hypothesis m of prompt i ends after
    lengths[i, m] steps at beam beams[i, m] (int32 [N, M]; default: every beam,
    after all T steps). Returns int32 [N, M, T]: each step's token, `pad`
    behind the end and before a parent outside [0, K)."""
    import torch

    lib = _lib or load_library()
    if tokens.dim() != 3:
        raise ValueError("tokens must be 3-D [T, N, K]")
    T, N, K = tokens.shape
    ends = beams if beams is not None else lengths
    if ends is not None and ends.dim() != 2:
        raise ValueError("beams and lengths must be 2-D [N, M]")
    M = K if ends is None else ends.shape[1]
    if not -2 ** 31 <= pad < 2 ** 31:
        raise ValueError(f"pad must be an int32, got {pad}")
    dev = tokens.get_device()
    _check_dense(tokens, (T, N, K), torch.int32, "tokens", dev)
    _check_dense(parents, (T, N, K), torch.int32, "parents", dev)
    if beams is not None:
        _check_dense(beams, (N, M), torch.int32, "beams", dev)
    if lengths is not None:
        _check_dense(lengths, (N, M), torch.int32, "lengths", dev)
    handle, scope = _scope(stream, tokens.device)
    given = out is not None
    with scope:
        if not given:
            out = torch.empty((N, M, T), dtype=torch.int32, device=tokens.device)
        _check_dense(out, (N, M, T), torch.int32, "out", dev)
        status = lib.beam_backtrace(tokens.data_ptr(), parents.data_ptr(), T, N, K,
                                    None if beams is None else beams.data_ptr(),
                                    None if lengths is None else lengths.data_ptr(), M, int(pad), out.data_ptr(),
                                    handle)
    _check(status)
    if given:
        torch.autograd.graph.increment_version(out)
    return out


def _row_strided(t, name, shape, dtype, device):
    """The row stride of a 2-D tensor with contiguous rows; checks it like _check_dense."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got shape {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"tensors must share one device: {name} is on {t.device}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name}: rows must be contiguous (stride 1 along the last dimension)")
    return shape[1] if shape[0] <= 1 else ld


@functools.lru_cache(maxsize=256)
def _verify_bytes(dtype, N, D, V, draft_logits):
    size = load_library().speculative_verify_workspace(dtype, N, D, V, draft_logits)
    if size < 0:
        raise TopKTopPError(2, last_error())
    return size


@functools.lru_cache(maxsize=256)
def _resize_bytes(R, P):
    size = load_library().cache_pages_resize_workspace(R, P)
    if size < 0:
        raise TopKTopPError(2, last_error())
    return size


def speculative_verify_workspace(dtype, N, D, V, draft_logits=False):
    """Bytes of the workspace that speculative_verify takes for N sequences of
    D drafts, V tokens and torch dtype `dtype`, with draft logits or without."""
    import torch

    return _verify_bytes(_dtype_code(torch.empty(0, dtype=dtype)), int(N), int(D), int(V), int(bool(draft_logits)))


def speculative_verify(logits, drafts, uniforms=None, draft_logits=None, parents=None, lengths=None, out=None,
                       workspace=None, stream=None):
    """How many drafted tokens stand, and the token behind them: (tokens
    [N, D + 1] int32, accepted [N] int32, path [N, D] int32 or None).

    logits [N * (D + 1), V], rows contiguous, any row stride from V on: of each
    sequence, what follows its last token and each of its drafts, ready to be
    sampled from (divided by the temperature, filtered tokens at -inf). drafts
    [N, D] int32; uniforms [N, D + 1] float32 in [0, 1): one for each row's
    acceptance, and the last one for the token behind. draft_logits [N * D, V]
    (as logits): what each draft was drawn from; without, drafts count as
    proposals that were not drawn. parents [N, D] int32: the drafts form a tree,
    draft j behind draft parents[i, j] < j or, for -1, behind the last token;
    default: a chain. lengths [N] int32: drafts that count (default D). Without
    uniforms the verification is greedy.

    tokens holds the accepted drafts, the token behind them and -1; path (with
    parents) the accepted drafts' numbers and -1. Draft w behind an accepted one
    stands if u[w] q(d) < p(d); where it does not, the token is drawn from
    max(p - q, 0). A chain is faster without parents. A row with a NaN or +inf or nothing above -inf accepts
    nothing and gives -1. out: the three tensors to fill (path None without
    parents, or wherever it is not needed); workspace: a uint8 tensor of
    speculative_verify_workspace() bytes, not used by any other call that may
    run at the same time (each call allocates one else). No gradients."""
    import torch

    lib = _lib or load_library()
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [N * (D + 1), V]")
    if drafts.dim() != 2:
        raise ValueError("drafts must be 2-D [N, D]")
    (R, V), (N, D) = logits.shape, drafts.shape
    if N * (D + 1) != R:
        raise ValueError(f"logits must have N * (D + 1) = {N * (D + 1)} rows, got {R}")
    dtype, dev = _dtype_code(logits), logits.get_device()
    ldx = _row_strided(logits, "logits", (R, V), logits.dtype, dev)
    _check_dense(drafts, (N, D), torch.int32, "drafts", dev)
    ldq, p_draft, p_uniforms, p_parents, p_lengths = V, None, None, None, None
    if uniforms is not None:
        _check_dense(uniforms, (N, D + 1), torch.float32, "uniforms", dev)
        p_uniforms = uniforms.data_ptr()
    if draft_logits is not None:
        if uniforms is None:
            raise ValueError("draft_logits needs uniforms")
        if parents is not None:
            raise ValueError("draft_logits cannot go with parents")
        ldq = _row_strided(draft_logits, "draft_logits", (N * D, V), logits.dtype, dev)
        p_draft = draft_logits.data_ptr() or None
    if parents is not None:
        _check_dense(parents, (N, D), torch.int32, "parents", dev)
        p_parents = parents.data_ptr() or None
    if lengths is not None:
        _check_dense(lengths, (N,), torch.int32, "lengths", dev)
        p_lengths = lengths.data_ptr()
    handle, scope = _scope(stream, logits.device)
    given = out is not None
    with scope:
        if not given:
            out = (torch.empty((N, D + 1), dtype=torch.int32, device=logits.device),
                   torch.empty((N,), dtype=torch.int32, device=logits.device),
                   None if parents is None else torch.empty((N, D), dtype=torch.int32, device=logits.device))
        tokens, accepted, path = out
        _check_dense(tokens, (N, D + 1), torch.int32, "out tokens", dev)
        _check_dense(accepted, (N,), torch.int32, "out accepted", dev)
        if path is not None:
            _check_dense(path, (N, D), torch.int32, "out path", dev)
        if workspace is None:
            size = _verify_bytes(dtype, N, D, V, int(p_draft is not None))
            workspace = torch.empty(size, dtype=torch.uint8, device=logits.device)
        else:
            size = workspace.numel()
            _check_dense(workspace, workspace.shape, torch.uint8, "workspace", dev)
        status = lib.speculative_verify(
            logits.data_ptr(), ldx, dtype, N, D, V, drafts.data_ptr(), p_uniforms, p_draft, ldq, p_parents, p_lengths,
            tokens.data_ptr(), accepted.data_ptr(), None if path is None else path.data_ptr(), workspace.data_ptr(),
            size, handle)
    _check(status)
    if given:
        torch.autograd.graph.increment_version([t for t in out if t is not None])
    return out


def _page_table(tables, lengths, uses, R):
    """(row stride, C, P) of a page table of R rows, checked."""
    import torch

    if tables.dim() != 2:
        raise ValueError("tables must be 2-D [rows, pages of a row]")
    dev, C = tables.get_device(), tables.shape[1]
    ld = _row_strided(tables, "tables", (R, C), torch.int32, dev)
    if lengths is not None:
        _check_dense(lengths, (R,), torch.int32, "lengths", dev)
    if uses is None:
        return ld, C, 0
    if uses.dim() != 1:
        raise ValueError("uses must be 1-D [pages]")
    _check_dense(uses, uses.shape, torch.int32, "uses", dev)
    return ld, C, uses.shape[0]


_shape_of, _dtype_of, _requires_grad_of = map(operator.attrgetter, ("shape", "dtype", "requires_grad"))


def _page_caches(caches, P, page_size, page_dim, slot_dim, dev):
    """(tensors, their descriptions) of caches of P pages."""
    import torch

    Tensor = torch.Tensor
    tensors = [caches] if isinstance(caches, Tensor) else list(caches)
    # maps and sets, as a step of the interpreter for each property of each tensor takes longer than the call
    if set(map(Tensor.get_device, tensors)) - {dev}:
        raise ValueError("tensors must share one device: a cache is on another")
    if torch.is_grad_enabled() and any(map(_requires_grad_of, tensors)):
        raise ValueError("a cache that requires grad can only be changed under no_grad")
    if any(map(Tensor.is_neg, tensors)):
        raise ValueError("a cache must not be a lazily negated view")
    shapes, strides, dtypes = set(map(_shape_of, tensors)), set(map(Tensor.stride, tensors)), set(map(_dtype_of, tensors))
    for dtype in dtypes:
        if dtype.is_complex and any(map(Tensor.is_conj, tensors)):
            raise ValueError("a cache must not be a lazily conjugated view")
    for shape in shapes:
        dims = len(shape)
        if not (-dims <= page_dim < dims and -dims <= slot_dim < dims) or (page_dim - slot_dim) % dims == 0:
            raise ValueError(f"a cache of {dims} axes has no page_dim {page_dim} and slot_dim {slot_dim}")
        if shape[page_dim] != P or shape[slot_dim] != page_size:
            raise ValueError(f"a cache must have {P} pages of {page_size} slots, got shape {tuple(shape)}")
    if len(shapes) == len(strides) == len(dtypes) == 1:  # the caches of a model's layers: one description for all
        t = tensors[0]
        descs = _NO_POINTER + _state_bytes(t.shape, t.stride(), t.element_size(), page_dim, slot_dim, P)
        words = memoryview(bytearray(descs * len(tensors))).cast("q")
        words[::len(descs) // 8] = array.array("q", map(Tensor.data_ptr, tensors))
        return tensors, bytes(words)
    return tensors, b"".join(_pack_pointer(t.data_ptr()) +
                             _state_bytes(t.shape, t.stride(), t.element_size(), page_dim, slot_dim, P) for t in tensors)


def cache_pages_fork(tables, lengths, parents, uses, page_size, stream=None):
    """The rows of a page table follow their beams, in place: row i * K + b
    becomes what row i * K + parents[i, b] was. The pages are not touched; rows
    that come from one share them until one grows (cache_pages_resize).

    tables [N * K, C] int32, rows contiguous: position t of a row lies in page
    tables[row, t // page_size]; lengths [N * K] int32, the positions that a row
    holds; uses [P] int32, how many held entries name each page (0: free). All
    three are changed; begin with lengths and uses of 0. parents [N, K] int32, a
    row whose parent lies outside [0, K) stays as it is. Returns tables."""
    import torch

    lib = _lib or load_library()
    if parents.dim() != 2:
        raise ValueError("parents must be 2-D [N, K]")
    N, K = parents.shape
    ld, C, P = _page_table(tables, lengths, uses, N * K)
    _check_dense(parents, (N, K), torch.int32, "parents", tables.get_device())
    handle, scope = _scope(stream, tables.device)
    with scope:
        status = lib.cache_pages_fork(tables.data_ptr(), ld, C, lengths.data_ptr(), parents.data_ptr(), N, K,
                                      uses.data_ptr(), P, int(page_size), handle)
    _check(status)
    torch.autograd.graph.increment_version((tables, lengths, uses))
    return tables


def cache_pages_resize_workspace(R, P):
    """Bytes of the workspace that cache_pages_resize takes for R rows and P pages."""
    return _resize_bytes(int(R), int(P))


def cache_pages_resize(tables, lengths, new_lengths, uses, page_size, caches=None, page_dim=0, slot_dim=1,
                       workspace=None, stream=None):
    """Row r of a page table is to hold new_lengths[r] positions, in place.

    Rows that become shorter give back the pages behind their new end (entries
    become -1); then those that grow get theirs, in order of the rows, the free
    pages of the lowest numbers first. A row that is going to write into its last
    page, which is not full and used by other rows as well, gets a page of its own
    in its place, with the slots that it holds copied in all caches; the last of
    several such rows keeps the page if no other uses it. From the first row that
    cannot be served on, rows that would grow stay as they are: `lengths` becomes
    new_lengths for all others, so comparing the two tells. Lengths outside
    [0, C * page_size] leave their row as it is.

    tables, lengths, uses: as for cache_pages_fork; new_lengths [R] int32. caches:
    a tensor or a sequence of them, any dtype and strides, with the pages along
    page_dim and their slots along slot_dim, none beginning within another (views
    that interleave, as keys and values of one tensor may, go as that tensor);
    without, nothing can be copied, and the first row that would have to be counts
    as not served. workspace: a uint8
    tensor of cache_pages_resize_workspace() bytes, not used by any other call that
    may run at the same time. Returns lengths."""
    import torch

    lib = _lib or load_library()
    if lengths.dim() != 1:
        raise ValueError("lengths must be 1-D [rows]")
    R = lengths.shape[0]
    ld, C, P = _page_table(tables, lengths, uses, R)
    dev = tables.get_device()
    _check_dense(new_lengths, (R,), torch.int32, "new_lengths", dev)
    tensors, descs = [], None
    if caches is not None:
        tensors, descs = _page_caches(caches, P, int(page_size), page_dim, slot_dim, dev)
    handle, scope = _scope(stream, tables.device)
    with scope:
        if workspace is None:
            size = _resize_bytes(R, P)
            workspace = torch.empty(size, dtype=torch.uint8, device=tables.device)
        else:
            size = workspace.numel()
            _check_dense(workspace, workspace.shape, torch.uint8, "workspace", dev)
        status = lib.cache_pages_resize(tables.data_ptr(), ld, R, C, lengths.data_ptr(), new_lengths.data_ptr(),
                                        uses.data_ptr(), P, int(page_size), descs, len(tensors),
                                        workspace.data_ptr(), size, handle)
    _check(status)
    torch.autograd.graph.increment_version([tables, lengths, uses, *tensors])
    return lengths


def cache_pages_compact(caches, tables, starts, path, counts, page_dim=0, slot_dim=1, stream=None):
    """The entries of accepted paths move behind one another, in place: in every
    cache, position starts[i] + j of sequence i becomes what position
    starts[i] + path[i, j] was, for j < counts[i].

    caches: as for cache_pages_resize; tables [N, C] int32, rows contiguous:
    position t lies in page tables[i, t // slots]; starts and counts [N] int32;
    path [N, D] int32, ascending, as speculative_verify gives it (a path ends
    before a number that is not larger than the one before). The pages written to
    must be those of one sequence only. Returns caches."""
    import torch

    lib = _lib or load_library()
    if path.dim() != 2:
        raise ValueError("path must be 2-D [N, D]")
    N, D = path.shape
    ld, C, _ = _page_table(tables, None, None, N)
    dev = tables.get_device()
    _check_dense(path, (N, D), torch.int32, "path", dev)
    _check_dense(starts, (N,), torch.int32, "starts", dev)
    _check_dense(counts, (N,), torch.int32, "counts", dev)
    if not isinstance(caches, torch.Tensor):
        caches = list(caches)
        if not caches:
            return caches
    first = caches if isinstance(caches, torch.Tensor) else caches[0]
    dims = first.dim()
    if not (-dims <= page_dim < dims and -dims <= slot_dim < dims):
        raise ValueError(f"a cache of {dims} axes has no page_dim {page_dim} and slot_dim {slot_dim}")
    P, page_size = first.shape[page_dim], first.shape[slot_dim]
    tensors, descs = _page_caches(caches, P, page_size, page_dim, slot_dim, dev)
    handle, scope = _scope(stream, tables.device)
    with scope:
        status = lib.cache_pages_compact(descs, len(tensors), P, page_size, tables.data_ptr(), ld, N, C,
                                         starts.data_ptr(), path.data_ptr(), D, counts.data_ptr(), handle)
    _check(status)
    torch.autograd.graph.increment_version(tensors)
    return caches
