"""ctypes binding of libtopktopp (include/topktopp.h).

Argument marshalling only: tensors are turned into device pointers and the
current HIP stream, and every step of the filter runs in the library's HIP
kernels. If the library has not been built this module raises instead of
falling back to anything else.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
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
    "sample_top_k_top_p",
    "top_k_top_p_sorted_survivors",
    "topktopp_last_error",
    "topktopp_set_plan_policy",
)

_lib = None


TOPKTOPP_MAX_BEAMS, TOPKTOPP_MAX_CANDIDATES = 128, 256


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
