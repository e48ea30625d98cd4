"""Binding of libdet.so (the HIP library), with the C interface's names: ctypes, and for the
language-model operators, whose calls are small, an extension (csrc/lm_binding.cpp).

Argument marshalling only: tensors become device pointers and sizes, the workspace is a
torch uint8 tensor from the caching allocator, and the current torch stream is passed
through.  Every step of every operation runs in the library's kernels; there is no CPU or
PyTorch fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdet.so")

DET_F32 = 0
DET_F64 = 1
DET_I32 = 2      # det_scan only
DET_F16 = 3      # the language-model operators only, like DET_BF16
DET_BF16 = 4
DET_E4M3 = 5     # det_rms_norm's 8-bit output only
DET_I64 = 6      # token ids, like DET_I32
DET_SCAN_EXCLUSIVE = 1
DET_SCAN_REVERSE = 2
DET_BIAS_BIDIRECTIONAL = 1
DET_BIAS_CAUSAL = 2
DET_GATE_SIGMOID = 1

_STATUS = {
    0: "DET_SUCCESS",
    1: "DET_ERROR_INVALID_VALUE",
    2: "DET_ERROR_UNSUPPORTED",
    3: "DET_ERROR_TOO_LARGE",
    4: "DET_ERROR_WORKSPACE",
    5: "DET_ERROR_LAUNCH",
}


class DetError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)}")
        self.status = status


class ScanWaitError(RuntimeError):
    """A look-back wait of det_scan gave up (its health word is set): the output is unspecified."""


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdet.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python __graft_entry__.py` "
                           "(hipcc --offload-arch=gfx950); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, sz, u, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint, ctypes.c_int
    L.det_sum_workspace_size.argtypes, L.det_sum_workspace_size.restype = [i64, i], sz
    L.det_sum.argtypes, L.det_sum.restype = [p, i64, i, p, p, sz, p], i
    L.det_sum_noalloc.argtypes, L.det_sum_noalloc.restype = [p, i64, i, p, p], i
    L.det_scan_workspace_size.argtypes, L.det_scan_workspace_size.restype = [i64, i, u, i64], sz
    L.det_scan.argtypes, L.det_scan.restype = [p, p, i64, i, u, p, i64, p, sz, p], i
    L.det_scatter_add_workspace_size.argtypes = [i64, i64, i64, i]
    L.det_scatter_add_workspace_size.restype = sz
    L.det_scatter_add.argtypes = [p, p, i64, i64, i, p, i64, p, p, p, sz, p]
    L.det_scatter_add.restype = i
    L.det_scatter_sub.argtypes = [p, p, i64, i64, i, p, i64, p, p, p, sz, p]
    L.det_scatter_sub.restype = i
    L.det_scatter_add_running_workspace_size.argtypes = [i64, i64, i64, i]
    L.det_scatter_add_running_workspace_size.restype = sz
    L.det_scatter_add_running.argtypes = [p, p, i64, i64, i, p, i64, p, p, p, sz, p]
    L.det_scatter_add_running.restype = i
    d = ctypes.c_double
    L.det_rms_norm.argtypes = [p, i64, p, i64, p, i64, i64, i, d, p, p, i, i64, p, p, p]
    L.det_rms_norm.restype = i
    L.det_rms_norm_backward_workspace_size.argtypes = [i64, i64, i]
    L.det_rms_norm_backward_workspace_size.restype = sz
    L.det_rms_norm_backward.argtypes = [p, i64, p, i64, p, p, p, i64, i64, i64, i, p, p, p, sz, p]
    L.det_rms_norm_backward.restype = i
    L.det_relative_bias.argtypes = [p, i64, i64, i64, u, i64, i64, i64, i64, p, p, p, i64, i64,
                                    i64, i, p, p]
    L.det_relative_bias.restype = i
    L.det_relative_bias_backward_workspace_size.argtypes = [i64, i64, i64, i64, i64, i]
    L.det_relative_bias_backward_workspace_size.restype = sz
    L.det_relative_bias_backward.argtypes = [p, i64, i64, i64, i64, i64, i64, u, i64, i64, i64,
                                             i64, p, p, i, p, p, p, sz, p]
    L.det_relative_bias_backward.restype = i
    L.det_token_logprobs.argtypes = [p, i64, p, i64, i64, i, d, p, p, p, i64, p, p, p]
    L.det_token_logprobs.restype = i
    L.det_token_logprobs_backward.argtypes = [p, i64, p, p, p, p, p, i64, i64, i, d, p, i64, p]
    L.det_token_logprobs_backward.restype = i
    L.det_layer_norm.argtypes = [p, i64, p, i64, p, p, i64, i64, i, d, p, p, p, p, p]
    L.det_layer_norm.restype = i
    L.det_layer_norm_backward_workspace_size.argtypes = [i64, i64, i]
    L.det_layer_norm_backward_workspace_size.restype = sz
    L.det_layer_norm_backward.argtypes = [p, i64, p, i64, p, p, p, p, i64, i64, i64, i, p, p, p, p,
                                          sz, p]
    L.det_layer_norm_backward.restype = i
    L.det_embedding.argtypes = [p, i64, p, i, i64, i64, i64, i, d, p, p]
    L.det_embedding.restype = i
    L.det_embedding_backward_workspace_size.argtypes = [i64, i64, i64, i]
    L.det_embedding_backward_workspace_size.restype = sz
    L.det_embedding_backward.argtypes = [p, i64, p, i, i64, i64, i64, i, d, p, p, sz, p]
    L.det_embedding_backward.restype = i
    for size in (L.det_gated_scan_workspace_size, L.det_gated_scan_backward_workspace_size,
                 L.det_linear_cross_entropy_workspace_size,
                 L.det_linear_cross_entropy_backward_workspace_size):
        size.argtypes, size.restype = [i64, i64, i64, i], sz
    L.det_gated_scan.argtypes = [p, p, p, p, u, i64, i64, i64, i, p, p, p, sz, p]
    L.det_gated_scan.restype = i
    L.det_gated_scan_backward.argtypes = [p, p, p, p, p, p, p, u, i64, i64, i64, i, p, p, p, p, sz, p]
    L.det_gated_scan_backward.restype = i
    L.det_linear_cross_entropy.argtypes = [p, i64, p, i64, p, i64, i64, i64, i, d, p, p, p, sz, p]
    L.det_linear_cross_entropy.restype = i
    L.det_linear_cross_entropy_backward.argtypes = [p, i64, p, i64, p, p, p, i64, i64, i64, i, d, p,
                                                    p, p, sz, p]
    L.det_linear_cross_entropy_backward.restype = i
    L.det_spec_version.argtypes, L.det_spec_version.restype = [], i
    L.det_spec_constants.argtypes = [ctypes.POINTER(i64)] * 4
    L.det_spec_constants.restype = None
    L.det_status_string.argtypes, L.det_status_string.restype = [i], ctypes.c_char_p
    L.det_scan_error.argtypes, L.det_scan_error.restype = [p, p, p], i
    L.det_debug_set_launch.argtypes, L.det_debug_set_launch.restype = [i, i], i
    L.det_debug_set_sum_chunk.argtypes, L.det_debug_set_sum_chunk.restype = [i], i
    L.det_debug_last_launch.argtypes = [ctypes.POINTER(i64)] * 3
    L.det_debug_last_launch.restype = None
    L.det_debug_set_scan_delay.argtypes, L.det_debug_set_scan_delay.restype = [u, i], i
    L.det_debug_set_scan_anchors.argtypes, L.det_debug_set_scan_anchors.restype = [i, i], i
    L.det_debug_kernel_timing.argtypes, L.det_debug_kernel_timing.restype = [i], i
    L.det_debug_kernel_report.argtypes = [ctypes.c_char_p, sz]
    L.det_debug_kernel_report.restype = sz
    _lib = L
    return L


def _dtype_code(t: torch.Tensor, allow_int: bool = False) -> int:
    if t.dtype == torch.float32:
        return DET_F32
    if t.dtype == torch.float64:
        return DET_F64
    if allow_int and t.dtype == torch.int32:
        return DET_I32
    raise TypeError(f"det supports float32 and float64{' and int32' if allow_int else ''}, "
                    f"got {t.dtype}")


def _dev_ptr(t: Optional[torch.Tensor]):
    # plain integers: ctypes passes them as void* (the argument types are declared)
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("det operates on device tensors")
    return t.data_ptr()


# the current stream's raw handle without building a torch Stream object per call (what
# torch.cuda.current_stream(device).cuda_stream returns), when this torch has the accessor
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index if device.index is not None
                           else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace of {nbytes} bytes needed")
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _check(st: int, what: str):
    if st != 0:
        raise DetError(st, what)


def _flat(t: torch.Tensor) -> torch.Tensor:
    if not t.is_contiguous():
        raise ValueError("det needs contiguous tensors (views with an offset are fine)")
    return t


# ------------------------------------------------------------------ sum

@functools.lru_cache(maxsize=256)
def det_sum_workspace_size(n: int, dtype_code: int) -> int:
    return lib().det_sum_workspace_size(n, dtype_code)


def det_sum(x: torch.Tensor, out: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Reproducible sum of all elements of ``x``; returns a 0-d tensor (or fills ``out``)."""
    x = _flat(x)
    dt = _dtype_code(x)
    n = x.numel()
    if out is None:
        out = torch.empty((), dtype=x.dtype, device=x.device)
    dev = x.device
    w = _workspace(det_sum_workspace_size(n, dt), dev, ws)
    _check(lib().det_sum(_dev_ptr(x), n, dt, _dev_ptr(out), _dev_ptr(w), w.numel(),
                         _stream(dev)), "det_sum")
    return out


def det_sum_noalloc(x: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """det_sum through the entry point that allocates nothing (its partials live in the
    library's per-GPU array); ``out`` (one element, dtype of x) is filled and returned.  Calls
    that overlap in time on one GPU race."""
    x = _flat(x)
    dt = _dtype_code(x)
    if out.dtype != x.dtype or out.numel() != 1:
        raise ValueError("out must be one element of x's dtype")
    _check(lib().det_sum_noalloc(_dev_ptr(x), x.numel(), dt, _dev_ptr(out), _stream(x.device)),
           "det_sum_noalloc")
    return out


# ------------------------------------------------------------------ scan

@functools.lru_cache(maxsize=256)
def det_scan_workspace_size(n: int, dtype_code: int, flags: int = 0, num_segments: int = 0) -> int:
    return lib().det_scan_workspace_size(n, dtype_code, flags, num_segments)


def det_scan(x: torch.Tensor, y: Optional[torch.Tensor] = None, exclusive: bool = False,
             reverse: bool = False, offsets: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None, check: bool = False,
             health: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Reproducible prefix sum of ``x`` (1-D).  ``offsets``: int64 device tensor [S+1]
    (0 = o_0 <= ... <= o_S = n) for a segmented scan.  int32 ``x`` gives wrapping integer
    sums (the slot-allocation scan of count-scan-write).

    The library's look-back waits are bounded; one that gives up leaves ``y`` unspecified and
    sets the workspace's health word.  ``health`` (device int32, one element) receives that
    word without synchronising; ``check=True`` waits for the scan and raises ScanWaitError
    when the word is set."""
    x = _flat(x)
    dt = _dtype_code(x, allow_int=True)
    n = x.numel()
    if y is None:
        y = torch.empty_like(x)
    flags = (DET_SCAN_EXCLUSIVE if exclusive else 0) | (DET_SCAN_REVERSE if reverse else 0)
    nseg = 0
    if offsets is not None:
        if offsets.dtype != torch.int64:
            raise TypeError("offsets must be int64")
        offsets = _flat(offsets)
        nseg = offsets.numel() - 1
    dev = x.device
    w = _workspace(det_scan_workspace_size(n, dt, flags, max(nseg, 0)), dev, ws)
    _check(lib().det_scan(_dev_ptr(x), _dev_ptr(y), n, dt, flags, _dev_ptr(offsets), nseg,
                          _dev_ptr(w), w.numel(), _stream(dev)), "det_scan")
    if check or health is not None:
        h = health if health is not None else torch.empty((), dtype=torch.int32, device=x.device)
        if h.dtype != torch.int32 or h.numel() != 1:
            raise ValueError("health must be an int32 tensor with one element")
        _check(lib().det_scan_error(_dev_ptr(w), _dev_ptr(h), _stream(x.device)),
               "det_scan_error")
        if check and int(h.item()) != 0:
            raise ScanWaitError("det_scan: a look-back wait gave up; the output is unspecified")
    return y


def det_scan_error(ws: torch.Tensor) -> torch.Tensor:
    """Health word of the last scan run in workspace ``ws`` (device int32: 0 = normal)."""
    out = torch.empty((), dtype=torch.int32, device=ws.device)
    _check(lib().det_scan_error(_dev_ptr(ws), _dev_ptr(out), _stream(ws.device)), "det_scan_error")
    return out


# ------------------------------------------------------------------ scatter-add

@functools.lru_cache(maxsize=256)
def det_scatter_add_workspace_size(n: int, num_out: int, row_len: int, dtype_code: int) -> int:
    return lib().det_scatter_add_workspace_size(n, num_out, row_len, dtype_code)


@functools.lru_cache(maxsize=256)
def det_scatter_add_running_workspace_size(n: int, num_out: int, row_len: int,
                                           dtype_code: int) -> int:
    return lib().det_scatter_add_running_workspace_size(n, num_out, row_len, dtype_code)


def _scatter(entry: str, values: torch.Tensor, index: torch.Tensor, out: torch.Tensor,
             prev: Optional[torch.Tensor], n_skipped: Optional[torch.Tensor],
             ws: Optional[torch.Tensor]) -> torch.Tensor:
    values = _flat(values)
    index = _flat(index)
    out = _flat(out)
    dt = _dtype_code(values)
    if out.dtype != values.dtype:
        raise TypeError("values and out must share a dtype")
    if index.dtype != torch.int32:
        raise TypeError("index must be int32")
    n = index.numel()
    row_len = values.numel() // n if n else (out[0].numel() if out.dim() > 1 and len(out) else 1)
    if n and values.numel() != n * row_len:
        raise ValueError("values and index disagree on n")
    if row_len < 1:
        row_len = 1
    num_out = out.numel() // row_len
    if out.numel() != num_out * row_len:
        raise ValueError("out is not a whole number of rows")
    if prev is not None:
        prev = _flat(prev)
        if prev.numel() != n * row_len or prev.dtype != values.dtype:
            raise ValueError("prev must match values")
    if n_skipped is not None and (n_skipped.dtype != torch.int64 or n_skipped.numel() < 1):
        raise ValueError("n_skipped must be an int64 tensor with one element")
    size_fn = (det_scatter_add_running_workspace_size if entry == "det_scatter_add_running"
               else det_scatter_add_workspace_size)
    dev = values.device
    w = _workspace(size_fn(n, num_out, row_len, dt), dev, ws)
    _check(getattr(lib(), entry)(_dev_ptr(values), _dev_ptr(index), n, row_len, dt, _dev_ptr(out),
                                 num_out, _dev_ptr(prev), _dev_ptr(n_skipped), _dev_ptr(w),
                                 w.numel(), _stream(dev)), entry)
    return out


def det_scatter_add(values: torch.Tensor, index: torch.Tensor, out: torch.Tensor,
                    prev: Optional[torch.Tensor] = None, n_skipped: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``out[index[i]] += values[i]`` along axis 0 in the fixed order; returns ``out``.

    ``values``: [n] or [n, *row]; ``index``: int32 [n]; ``out``: [num_out] or [num_out, *row].
    ``prev`` (same shape as values) receives the destination rows before the call;
    ``n_skipped`` (int64, one element) receives the number of out-of-range indices."""
    return _scatter("det_scatter_add", values, index, out, prev, n_skipped, ws)


def det_scatter_sub(values: torch.Tensor, index: torch.Tensor, out: torch.Tensor,
                    prev: Optional[torch.Tensor] = None, n_skipped: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``out[index[i]] -= values[i]``: the values negated, then added in the fixed order of
    det_scatter_add (arguments as there); returns ``out``."""
    return _scatter("det_scatter_sub", values, index, out, prev, n_skipped, ws)


def det_scatter_add_running(values: torch.Tensor, index: torch.Tensor, out: torch.Tensor,
                            prev: torch.Tensor, n_skipped: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """det_scatter_add whose ``prev`` (required, shape of values) receives the running value:
    the destination's initial value plus the earlier contributions (ascending source index),
    summed by the exclusive segmented det_scan of the destination-grouped members; the first
    member of a destination gets the initial value itself.  Returns ``out``."""
    if prev is None:
        raise ValueError("det_scatter_add_running needs prev")
    return _scatter("det_scatter_add_running", values, index, out, prev, n_skipped, ws)


class _Gather(torch.autograd.Function):
    """``values[index]`` along axis 0; the gradient scatters back through det_scatter_add."""

    @staticmethod
    def forward(ctx, values, index):
        ctx.save_for_backward(index)
        ctx.shape = values.shape
        return values.index_select(0, index.long())

    @staticmethod
    def backward(ctx, grad_out):
        (index,) = ctx.saved_tensors
        grad = torch.zeros(ctx.shape, dtype=grad_out.dtype, device=grad_out.device)
        det_scatter_add(grad_out.contiguous(), index, grad)
        return grad, None


def gather(values: torch.Tensor, index: torch.Tensor) -> torch.Tensor:
    """Rows ``values[index[i]]`` (``index`` int32, in range).  The forward pass only moves data;
    in the backward pass the gradient rows that share a source row are accumulated by
    det_scatter_add, so the gradient's bits do not depend on scheduling (the gather case of the
    Warp guide's "Tape and Backward Passes")."""
    if index.dtype != torch.int32:
        raise TypeError("index must be int32")
    if index.numel() and (int(index.min()) < 0 or int(index.max()) >= values.shape[0]):
        raise IndexError("gather index out of range")
    return _Gather.apply(values, index)


# ------------------------------------------------------------------ language-model operators

_lm = None


def _lm_binding():
    """The extension that marshals these operators' arguments (raises if it has not been built)."""
    global _lm
    if _lm is None:
        lib()
        try:
            from . import _lm_binding as _lm
        except ImportError as e:
            raise RuntimeError(f"{os.path.join(_HERE, '_lm_binding.so')} cannot be loaded ({e}): "
                               "build it with `python __graft_entry__.py`; there is no fallback "
                               "path") from e
    return _lm


def _row_stride(t: torch.Tensor, what: str) -> int:
    """Elements between neighbouring rows of ``t`` (its last dimension is a row)."""
    return _lm_binding().row_stride(t, what)


class RmsNorm(NamedTuple):
    """y; h = x + residual as stored (x itself without a residual) and rstd, which the backward
    pass takes; scales of an 8-bit y, else None."""
    y: torch.Tensor
    h: torch.Tensor
    rstd: torch.Tensor
    scales: Optional[torch.Tensor]


def det_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, quant: Optional[torch.dtype] = None,
                 group: int = 0) -> RmsNorm:
    """Root-mean-square norm of the rows (last dimension) of ``x + residual``, times ``weight``.

    x, residual: [..., d] of one type (float32, float16, bfloat16), rows contiguous and evenly
    spaced; weight: [d].  Computed in f32; a row's bits depend on that row alone.
    ``quant=torch.float8_e4m3fn``: y holds 8-bit codes and scales [..., ceil(d / group)] their
    scales, one for every ``group`` (32, 64, 128) neighbouring channels, or with ``group=0``
    one a row; y * scale stands for the normed value."""
    if quant is not None and quant != torch.float8_e4m3fn:
        raise TypeError(f"quant must be torch.float8_e4m3fn, got {quant}")
    return RmsNorm(*_lm_binding().rms_norm(x, weight, eps, residual, quant is not None, group))


@functools.lru_cache(maxsize=256)
def det_rms_norm_backward_workspace_size(rows: int, d: int, dtype_code: int) -> int:
    return lib().det_rms_norm_backward_workspace_size(rows, d, dtype_code)


def det_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                          rstd: torch.Tensor, dh: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of det_rms_norm's ``y``; ``h`` and ``rstd`` as det_rms_norm returned them.
    ``dh``: the gradient that reaches h from elsewhere (the residual stream), added to dx.  dx is
    also the residual's gradient.  dweight's sum over the rows has an order fixed by their
    number."""
    return _lm_binding().rms_norm_backward(dy, h, weight, rstd, dh, ws)


def _bias_flags(bidirectional: bool, causal: bool) -> int:
    return (DET_BIAS_BIDIRECTIONAL if bidirectional else 0) | (DET_BIAS_CAUSAL if causal else 0)


def det_relative_bias(table: torch.Tensor, q: int, k: int, scores: Optional[torch.Tensor] = None,
                      max_distance: int = 128, bidirectional: bool = True, causal: bool = False,
                      q_offset: Union[int, torch.Tensor] = 0,
                      lengths: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A learned relative position bias [batch, heads, q, k], added to ``scores`` where given.

    table: [buckets, heads]; the bias of query i and key j is the row of the bucket that
    j - (i + q_offset) falls into: near distances have a bucket each, farther ones share them by
    the logarithm up to ``max_distance``; ``bidirectional`` gives keys after the query the
    second half of the buckets.  Masked places are -inf: keys after the query when ``causal``,
    and keys and queries at or past ``lengths`` (int32 [batch]).  ``q_offset``: query 0's
    position among the keys, a whole number or int32 [batch].  Without scores, lengths or a
    tensor of offsets batch is 1: one bias serves every sequence.  ``scores``: [batch, heads,
    q, k] of the table's type, rows contiguous, other strides free; ``out`` may be scores."""
    several = torch.is_tensor(q_offset)
    return _lm_binding().relative_bias(table, q, k, scores, max_distance,
                                       _bias_flags(bidirectional, causal),
                                       0 if several else q_offset, q_offset if several else None,
                                       lengths, out)


@functools.lru_cache(maxsize=256)
def det_relative_bias_backward_workspace_size(batch: int, heads: int, q: int, k: int,
                                              num_buckets: int, dtype_code: int) -> int:
    return lib().det_relative_bias_backward_workspace_size(batch, heads, q, k, num_buckets,
                                                           dtype_code)


def det_relative_bias_backward(dout: torch.Tensor, num_buckets: int, max_distance: int = 128,
                               bidirectional: bool = True, causal: bool = False,
                               q_offset: Union[int, torch.Tensor] = 0,
                               lengths: Optional[torch.Tensor] = None,
                               dscores: Optional[torch.Tensor] = None,
                               ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient [num_buckets, heads]: ``dout`` [batch, heads, q, k] summed by buckets
    over the unmasked places, in an order fixed by the sizes (arguments as for
    det_relative_bias).  ``dscores`` (contiguous, dout's shape and type; may be dout itself)
    receives the scores' gradient: dout with zeros at the masked places."""
    several = torch.is_tensor(q_offset)
    return _lm_binding().relative_bias_backward(dout, num_buckets, max_distance,
                                                _bias_flags(bidirectional, causal),
                                                0 if several else q_offset,
                                                q_offset if several else None, lengths, dscores, ws)


class TokenLogprobs(NamedTuple):
    """Float32 logp, entropy and lse of every row; top_logp and top_ids (int64) [..., top], None
    without alternatives."""
    logp: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logp: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]


def det_token_logprobs(logits: torch.Tensor, targets: torch.Tensor, scale: float = 1.0,
                       top: int = 0) -> TokenLogprobs:
    """Log probabilities of ``targets`` under softmax(scale * logits), with each row's entropy and
    its ``top`` likeliest tokens (ties to the lower id).

    logits: [..., vocab], rows contiguous and evenly spaced (a slice of a padded vocabulary is
    fine); targets: int64 [...]; one outside the vocabulary (such as -100) is not scored and its
    logp is 0, but its entropy is returned like any other's: a loss that adds entropies leaves
    those out itself.  A row's bits depend on its logits and the scale alone."""
    return TokenLogprobs(*_lm_binding().token_logprobs(logits, targets, scale, top))


def det_token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                                dlogp: torch.Tensor, entropy: Optional[torch.Tensor] = None,
                                dentropy: Optional[torch.Tensor] = None, scale: float = 1.0,
                                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The logits' gradient for ``dlogp`` and, where given, ``dentropy`` (float32 [...]); ``lse``
    and ``entropy`` as det_token_logprobs returned them for these logits and this scale.  ``out``
    (logits' shape and type, rows contiguous and evenly spaced) may be logits itself."""
    return _lm_binding().token_logprobs_backward(logits, targets, lse, dlogp, entropy, dentropy,
                                                 scale, out)


class _RmsNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        r = det_rms_norm(x, weight, eps, residual)
        ctx.save_for_backward(r.h, weight, r.rstd)
        ctx.set_materialize_grads(False)
        ctx.residual = residual is not None
        return (r.y, r.h) if ctx.residual else r.y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        if dy is None and dh is None:
            return None, None, None, None
        dy = torch.zeros_like(h) if dy is None else dy.contiguous()
        dx, dweight = det_rms_norm_backward(dy, h, weight, rstd,
                                            None if dh is None else dh.contiguous())
        return dx, dweight, dx if ctx.residual else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6):
    """Differentiable det_rms_norm: y, or (y, h = x + residual) with a residual."""
    return _RmsNormFn.apply(x, weight, residual, eps)


class _RelativeBias(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, scores, q, k, how, q_offset, lengths):
        out = det_relative_bias(table, q, k, scores, q_offset=q_offset, lengths=lengths, **how)
        ctx.how, ctx.buckets, ctx.scored = how, table.shape[0], scores is not None
        tensor = torch.is_tensor(q_offset)
        ctx.save_for_backward(q_offset if tensor else None, lengths)
        ctx.q_offset = None if tensor else q_offset
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        offsets, lengths = ctx.saved_tensors
        dout = dout.contiguous()
        masked = ctx.how["causal"] or lengths is not None
        want = ctx.scored and ctx.needs_input_grad[1]
        dscores = torch.empty_like(dout) if want and masked else dout if want else None
        dtable = det_relative_bias_backward(
            dout, ctx.buckets, q_offset=offsets if offsets is not None else ctx.q_offset,
            lengths=lengths, dscores=dscores if masked else None, **ctx.how)
        return dtable, dscores, None, None, None, None, None


def relative_bias(table: torch.Tensor, q: int, k: int, scores: Optional[torch.Tensor] = None,
                  max_distance: int = 128, bidirectional: bool = True, causal: bool = False,
                  q_offset: Union[int, torch.Tensor] = 0,
                  lengths: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable det_relative_bias (gradients of the table and the scores)."""
    how = {"max_distance": max_distance, "bidirectional": bidirectional, "causal": causal}
    return _RelativeBias.apply(table, scores, q, k, how, q_offset, lengths)


class _TokenLogprobsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, scale):
        r = det_token_logprobs(logits, targets, scale)
        ctx.save_for_backward(logits, targets, r.lse, r.entropy)
        ctx.set_materialize_grads(False)
        ctx.scale = scale
        return r.logp, r.entropy

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dlogp, dentropy):
        logits, targets, lse, entropy = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None
        dlogp = torch.zeros_like(lse) if dlogp is None else dlogp.contiguous()
        dlogits = det_token_logprobs_backward(
            logits, targets, lse, dlogp, entropy,
            None if dentropy is None else dentropy.contiguous(), ctx.scale)
        return dlogits, None, None


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, scale: float = 1.0):
    """Differentiable det_token_logprobs: (logp, entropy), the entropy of unscored rows too."""
    return _TokenLogprobsFn.apply(logits, targets, scale)


class LayerNorm(NamedTuple):
    """y; h = x + residual as stored (x itself without a residual), mean and rstd, which the backward
    pass takes."""
    y: torch.Tensor
    h: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor


def det_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, residual: Optional[torch.Tensor] = None) -> LayerNorm:
    """Layer norm of the rows (last dimension) of ``x + residual``, times ``weight``, plus ``bias``.

    x, residual: [..., d] of one type (float32, float16, bfloat16), rows contiguous and evenly
    spaced; weight, bias: [d].  Computed in f32, the variance about the mean; a row's bits depend on
    that row alone."""
    return LayerNorm(*_lm_binding().layer_norm(x, weight, bias, eps, residual))


@functools.lru_cache(maxsize=256)
def det_layer_norm_backward_workspace_size(rows: int, d: int, dtype_code: int) -> int:
    return lib().det_layer_norm_backward_workspace_size(rows, d, dtype_code)


def det_layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                            mean: torch.Tensor, rstd: torch.Tensor,
                            dh: Optional[torch.Tensor] = None, bias: bool = True,
                            ws: Optional[torch.Tensor] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(dx, dweight, dbias) of det_layer_norm's ``y``; ``h``, ``mean`` and ``rstd`` as det_layer_norm
    returned them.  ``dh``: the gradient that reaches h from elsewhere (the residual stream), added
    to dx.  dx is also the residual's gradient.  ``bias=False``: no dbias (None).  The sums over the
    rows have an order fixed by their number."""
    return _lm_binding().layer_norm_backward(dy, h, weight, mean, rstd, dh, bias, ws)


def det_embedding(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """``scale * table[tokens]``: [..., d] for tokens [...] (int32 or int64), zeros for a token outside
    the vocabulary (such as -1 for padding).

    table: [vocab, d] (float32, float16, bfloat16), rows contiguous and evenly spaced."""
    return _lm_binding().embedding(table, tokens, scale)


@functools.lru_cache(maxsize=256)
def det_embedding_backward_workspace_size(n: int, vocab: int, d: int, dtype_code: int) -> int:
    return lib().det_embedding_backward_workspace_size(n, vocab, d, dtype_code)


def det_embedding_backward(dout: torch.Tensor, tokens: torch.Tensor, vocab: int,
                           scale: float = 1.0, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient [vocab, d]: ``scale`` times the sum of ``dout`` [..., d] over each token's
    places, in their order, in f32 (a token with more than 64 places: blocks of 64, joined in
    double); zeros for tokens that do not occur."""
    return _lm_binding().embedding_backward(dout, tokens, vocab, scale, ws)


class GatedScan(NamedTuple):
    """h of every step, and float32 state behind the last one."""
    h: torch.Tensor
    state: torch.Tensor


def det_gated_scan(gate: torch.Tensor, x: torch.Tensor, state: Optional[torch.Tensor] = None,
                   sigmoid: bool = False, lengths: Optional[torch.Tensor] = None,
                   state_out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None) -> GatedScan:
    """The gated linear recurrence h[t] = a[t] h[t-1] + b[t] of every channel.

    gate, x: [batch, steps, d], contiguous, of one type (float32, float16, bfloat16).  a = gate (at
    most 1 in magnitude) and b = x, or with ``sigmoid`` a = sigmoid(gate) and b = (1 - a) x.
    ``state``: float32 [batch, d], h before the first step (zeros).  ``lengths``: int32 [batch]; steps
    at or past a sequence's length keep its state and have h = 0.  ``state_out`` receives the state;
    up to 8 steps it may be ``state`` itself, which a decoding loop then updates in place.  Computed
    in f32; the bits of a step depend on its own channel and the steps before it alone."""
    return GatedScan(*_lm_binding().gated_scan(gate, x, state, sigmoid, lengths, state_out, ws))


@functools.lru_cache(maxsize=256)
def det_gated_scan_workspace_size(batch: int, steps: int, d: int, dtype_code: int) -> int:
    return lib().det_gated_scan_workspace_size(batch, steps, d, dtype_code)


@functools.lru_cache(maxsize=256)
def det_gated_scan_backward_workspace_size(batch: int, steps: int, d: int, dtype_code: int) -> int:
    return lib().det_gated_scan_backward_workspace_size(batch, steps, d, dtype_code)


def det_gated_scan_backward(dh: torch.Tensor, gate: torch.Tensor, x: torch.Tensor, h: torch.Tensor,
                            state: Optional[torch.Tensor] = None,
                            dstate: Optional[torch.Tensor] = None, sigmoid: bool = False,
                            lengths: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(dgate, dx, the first state's gradient or None without ``state``) for ``dh`` and, where given,
    ``dstate`` (float32 [batch, d], the last state's).  ``h`` as det_gated_scan returned it, the other
    arguments as they were handed to it; all contiguous."""
    return _lm_binding().gated_scan_backward(dh, gate, x, h, state, dstate, sigmoid, lengths, ws)


class LinearCrossEntropy(NamedTuple):
    """Float32 loss and lse of every row."""
    loss: torch.Tensor
    lse: torch.Tensor


@functools.lru_cache(maxsize=256)
def det_linear_cross_entropy_workspace_size(rows: int, vocab: int, d: int, dtype_code: int) -> int:
    return lib().det_linear_cross_entropy_workspace_size(rows, vocab, d, dtype_code)


@functools.lru_cache(maxsize=256)
def det_linear_cross_entropy_backward_workspace_size(rows: int, vocab: int, d: int,
                                                     dtype_code: int) -> int:
    return lib().det_linear_cross_entropy_backward_workspace_size(rows, vocab, d, dtype_code)


def det_linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                             scale: float = 1.0,
                             ws: Optional[torch.Tensor] = None) -> LinearCrossEntropy:
    """Cross entropy of softmax(scale * x weight^T) at ``targets``, the logits never in memory.

    x: [..., d]; weight: [vocab, d] of the same type (float32, float16, bfloat16), rows of both
    contiguous and evenly spaced; targets: int64 [...]; one outside the vocabulary (such as -100) has
    loss 0.  Matrix instructions with f32 sums, whose order depends on the sizes alone."""
    return LinearCrossEntropy(*_lm_binding().linear_cross_entropy(x, weight, targets, scale, ws))


def det_linear_cross_entropy_backward(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                                      lse: torch.Tensor, dloss: torch.Tensor, scale: float = 1.0,
                                      ws: Optional[torch.Tensor] = None
                                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) for ``dloss`` (float32 [...]); ``lse`` as det_linear_cross_entropy returned it for
    these x, weight and scale.  The logits are made again in pieces of the vocabulary."""
    return _lm_binding().linear_cross_entropy_backward(x, weight, targets, lse, dloss, scale, ws)


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps):
        r = det_layer_norm(x, weight, bias, eps, residual)
        ctx.save_for_backward(r.h, weight, r.mean, r.rstd)
        ctx.set_materialize_grads(False)
        ctx.residual, ctx.bias = residual is not None, bias is not None
        return (r.y, r.h) if ctx.residual else r.y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, mean, rstd = ctx.saved_tensors
        if dy is None and dh is None:
            return None, None, None, None, None
        dy = torch.zeros_like(h) if dy is None else dy.contiguous()
        dx, dweight, dbias = det_layer_norm_backward(
            dy, h, weight, mean, rstd, None if dh is None else dh.contiguous(), ctx.bias)
        return dx, dweight, dbias, dx if ctx.residual else None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, eps: float = 1e-5):
    """Differentiable det_layer_norm: y, or (y, h = x + residual) with a residual."""
    return _LayerNormFn.apply(x, weight, bias, residual, eps)


class _EmbeddingFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return det_embedding(table, tokens, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        (tokens,) = ctx.saved_tensors
        return det_embedding_backward(dout.contiguous(), tokens, ctx.vocab, ctx.scale), None, None


def embedding(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """Differentiable det_embedding (gradient of the table)."""
    return _EmbeddingFn.apply(table, tokens, scale)


class _GatedScanFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, state, sigmoid, lengths):
        r = det_gated_scan(gate, x, state, sigmoid, lengths)
        ctx.save_for_backward(gate, x, state, lengths, r.h)
        ctx.set_materialize_grads(False)
        ctx.sigmoid = sigmoid
        return r.h, r.state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dstate):
        gate, x, state, lengths, h = ctx.saved_tensors
        if dh is None and dstate is None:
            return None, None, None, None, None
        dh = torch.zeros_like(h) if dh is None else dh.contiguous()
        dgate, dx, first = det_gated_scan_backward(
            dh, gate, x, h, state, None if dstate is None else dstate.contiguous(), ctx.sigmoid,
            lengths)
        return dgate, dx, first, None, None


def gated_scan(gate: torch.Tensor, x: torch.Tensor, state: Optional[torch.Tensor] = None,
               sigmoid: bool = False, lengths: Optional[torch.Tensor] = None):
    """Differentiable det_gated_scan: (h, state), with gradients of gate, x and the first state."""
    return _GatedScanFn.apply(gate, x, state, sigmoid, lengths)


class _LinearCrossEntropyFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, scale):
        r = det_linear_cross_entropy(x, weight, targets, scale)
        ctx.save_for_backward(x, weight, targets, r.lse)
        ctx.scale = scale
        return r.loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        x, weight, targets, lse = ctx.saved_tensors
        dx, dweight = det_linear_cross_entropy_backward(x, weight, targets, lse, dloss.contiguous(),
                                                        ctx.scale)
        return dx, dweight, None, None


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         scale: float = 1.0) -> torch.Tensor:
    """Differentiable det_linear_cross_entropy: the loss of every row (gradients of x and weight)."""
    return _LinearCrossEntropyFn.apply(x, weight, targets, scale)


# ------------------------------------------------------------------ introspection

def det_spec_version() -> int:
    return lib().det_spec_version()


def det_spec_constants():
    v, l_, a, a2 = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    lib().det_spec_constants(ctypes.byref(v), ctypes.byref(l_), ctypes.byref(a), ctypes.byref(a2))
    return v.value, l_.value, a.value, a2.value


def det_status_string(status: int) -> str:
    return lib().det_status_string(status).decode()


def det_debug_set_launch(grid_wgs: int = 0, extra_lds_bytes: int = 0) -> None:
    """Test hook: workgroups of the sum and look-back scan kernels (0 = default; may exceed the
    resident count) and extra dynamic LDS per workgroup (lowers occupancy)."""
    _check(lib().det_debug_set_launch(grid_wgs, extra_lds_bytes), "det_debug_set_launch")


def det_debug_set_sum_chunk(chunk_log2: int = 0) -> None:
    """Test hook: elements per partial of the sum's first level, as a power of two (0 = 14)."""
    _check(lib().det_debug_set_sum_chunk(chunk_log2), "det_debug_set_sum_chunk")


def det_debug_last_launch() -> dict:
    """Test hook: {sum_grid, scan_grid, scan_per_cu} of the library's most recent launches."""
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    lib().det_debug_last_launch(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    return {"sum_grid": a.value, "scan_grid": b.value, "scan_per_cu": c.value}


def det_debug_set_scan_delay(seed: int = 0, max_us: int = 0) -> None:
    """Test hook: seeded pauses of up to ``max_us`` microseconds before the look-back scan's
    status publications (0 = off)."""
    _check(lib().det_debug_set_scan_delay(seed & 0xFFFFFFFF, max_us), "det_debug_set_scan_delay")


def det_debug_set_scan_anchors(A: int = 0, A2: int = 0) -> None:
    """Test hook: scan anchor constants (0 = the spec's 256)."""
    _check(lib().det_debug_set_scan_anchors(A, A2), "det_debug_set_scan_anchors")


def det_debug_kernel_timing(enable: bool) -> None:
    """Test hook: bracket every library kernel launch with HIP events (drops earlier records)."""
    _check(lib().det_debug_kernel_timing(1 if enable else 0), "det_debug_kernel_timing")


def det_debug_kernel_report() -> dict:
    """Wait for the recorded launches; {kernel: (launches, total_ms, average_ms)}."""
    L = lib()
    need = L.det_debug_kernel_report(None, 0)
    buf = ctypes.create_string_buffer(need)
    L.det_debug_kernel_report(buf, need)
    rep = {}
    for line in buf.value.decode().splitlines():
        if line.startswith("#"):
            raise RuntimeError("kernel timing: " + line[1:].strip())
        name, cnt, tot, avg = line.rsplit(" ", 3)
        rep[name] = (int(cnt), float(tot), float(avg))
    return rep
