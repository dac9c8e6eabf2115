"""The operators around the top-k of a sparse-attention indexer.

A thin binding over the C ABI in ``include/indexer_ops.h``, in the manner of the
package's top-k calls: tensors are checked and marshalled, the work runs in the
library's sm_103a kernels on the tensors' device and the current torch stream (or
``stream``), and nothing falls back to torch. A decode step, with a paged cache
``codes`` [pages, page_size, 128] (float8_e4m3fn) and ``scales`` [pages, page_size, 1]:

    freqs, scale = indexer_rotary_freqs(64, device="cuda")
    q = indexer_rotary(q, positions, freqs, start=64, scale=scale)       # [B, H, 128]
    k = indexer_rotary(k, positions, freqs, start=64, scale=scale)       # [B, 1, 128]
    indexer_cache_write(k[:, 0], slots, codes, scales)
    q8, w = indexer_quantise(q, weights=weights)
    s = indexer_scores(q8[:, None], w[:, None], codes, scales, page_table, seq_lens[:, None], n)
    picked = topk_transform_paged(s, seq_lens, page_table, page_size, k=1024)
    rows = indexer_cache_read(codes, scales, picked)                     # [B, 1024, 128] bf16
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _check, load_library

__all__ = [
    "indexer_rotary", "indexer_rotary_freqs", "indexer_quantise", "indexer_cache_write",
    "indexer_cache_read", "indexer_scores", "indexer_guard_hits", "indexer_reset_guard_hits",
    "INDEXER_BLOCK", "INDEXER_MAX_HEADS",
]

INDEXER_BLOCK = 128
INDEXER_MAX_HEADS = 128

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_LAYOUTS = {"half": 0, "interleaved": 1}
_FORMATS = {"fp32": 0, "pow2": 1}


class IndexerCache(ctypes.Structure):
    """ctypes copy of indexer_cache_t (include/indexer_ops.h)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("code_page_stride", ctypes.c_int64),
                ("code_token_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("dim", ctypes.c_int32)]


def declare(lib: ctypes.CDLL) -> None:
    """Sets the C signatures on a freshly loaded library."""
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sig = {
        "indexer_rotary": [vp, i64, i64, vp, vp, i32, i64, i32, i32, i32, i32, i32, f32, i32, vp, i64,
                           i64, vp],
        "indexer_quantise": [vp, i64, i64, i32, i64, i32, i32, i32, vp, vp, vp, vp],
        "indexer_cache_write": [vp, i64, i32, i64, vp, i32, vp, vp],
        "indexer_cache_read": [vp, vp, i64, i32, vp, vp],
        "indexer_scores": [vp, vp, vp, vp, i64, vp, i32, i32, i32, i64, vp, vp],
        "indexer_guard_hits": [ctypes.POINTER(ctypes.c_uint64)],
        "indexer_reset_guard_hits": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    lib.indexer_cache_bytes.restype = ctypes.c_size_t
    lib.indexer_cache_bytes.argtypes = []
    if lib.indexer_cache_bytes() != ctypes.sizeof(IndexerCache):
        raise RuntimeError("indexer_cache_t layout differs between the library and this binding")


# ---------------------------------------------------------------- checks and the call

def _tensor(t, name: str, dtypes, device=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (the library has no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


_INT32, _FP32, _FP64, _E4M3 = (torch.int32,), (torch.float32,), (torch.float64,), (torch.float8_e4m3fn,)


def _contiguous(t, name: str, dtypes, shape, device) -> None:
    _tensor(t, name, dtypes, device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor of shape {tuple(shape)}, "
                         f"got {tuple(t.shape)}")


def _rows(x, name: str):
    """(tokens, heads, dim, token stride, head stride) of a [tokens, dim] or
    [tokens, heads, dim] tensor with unit column stride."""
    _tensor(x, name, _DTYPES)
    if x.dim() not in (2, 3) or (x.shape[-1] > 1 and x.stride(-1) != 1):
        raise ValueError(f"{name} must be [tokens, dim] or [tokens, heads, dim] with unit inner stride")
    if x.dim() == 2:
        return x.shape[0], 1, x.shape[1], x.stride(0), 0
    return x.shape[0], x.shape[1], x.shape[2], x.stride(0), x.stride(1)


def _choice(value, table, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}")
    return table[value]


def _call(what: str, device, stream, *args) -> None:
    fn = getattr(load_library(), what)
    s = torch.cuda.current_stream(device) if stream is None else stream
    if torch.cuda.current_device() == device.index:
        st = fn(*args, s.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, s.cuda_stream)
    if st != 0:
        _check(st, what)


def _fresh(shape, dtype, device, stream):
    """An output of this call: in use on `stream`, where one is given, until the call's
    kernel has ended."""
    out = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        out.record_stream(stream)
    return out


def _cache(codes, scales, device=None) -> IndexerCache:
    _tensor(codes, "codes", _E4M3, device)
    device = codes.device
    _tensor(scales, "scales", _FP32, device)
    if codes.dim() != 3 or codes.shape[2] < 1 or (codes.shape[2] > 1 and codes.stride(2) != 1):
        raise ValueError("codes must be [pages, page_size, dim] with unit inner stride")
    pages, size, dim = codes.shape
    nb = -(-dim // INDEXER_BLOCK)
    if tuple(scales.shape) != (pages, size, nb) or (nb > 1 and scales.stride(2) != 1):
        raise ValueError(f"scales must be [{pages}, {size}, {nb}] (one for each {INDEXER_BLOCK} columns) "
                         "with unit inner stride")
    if size < 1:
        raise ValueError("a page must hold at least one row")
    if pages * size > 2**31 - 1:
        raise ValueError("a cache holds at most 2**31 - 1 rows")
    c = IndexerCache(codes.data_ptr(), scales.data_ptr(), pages, codes.stride(0), codes.stride(1),
                     scales.stride(0), scales.stride(1), size, dim)
    for t, name, width in ((codes, "codes", dim), (scales, "scales", nb)):
        # rows apart from each other: pages outside rows, or rows outside pages
        axes = sorted((t.stride(i), t.shape[i]) for i in (0, 1) if t.shape[i] > 1)
        for stride, count in axes:
            if stride < width:
                raise ValueError(f"{name}: rows must not overlap")
            width += (count - 1) * stride
    return c


# ---------------------------------------------------------------- rotary positions

def indexer_rotary_freqs(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None,
                         factor: float = 1.0, original_len: int = 4096, beta_fast: float = 32.0,
                         beta_slow: float = 1.0, device="cuda") -> tuple[torch.Tensor, float]:
    """(freqs, scale) for indexer_rotary: fp64 radians per position of the rot_dim / 2
    pairs, base ** (-2 i / rot_dim), and the factor of sine and cosine.

    scaling, for contexts `factor` times the trained `original_len`: None; "linear" (all
    frequencies divided by factor); "ntk" (a larger base: the slowest pair divided by
    factor, the fastest kept); "yarn" (pairs that turn more than beta_fast times within
    original_len kept, those that turn less than beta_slow times divided by factor, those
    between blended; scale = 0.1 ln(factor) + 1)."""
    if rot_dim < 2 or rot_dim % 2 != 0:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    freqs, scale = base ** (-2.0 * i / rot_dim), 1.0
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "yarn":
        if not beta_fast > beta_slow:
            raise ValueError("beta_fast must be above beta_slow")
        turns = original_len * freqs / (2.0 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        freqs = freqs * keep + freqs / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    return freqs.to(device), scale


def _rotary(x, positions, freqs, layout, start, scale, transpose, out, stream):
    tokens, heads, dim, ts, hs = _rows(x, "x")
    if out is None:
        out = _fresh(x.shape, x.dtype, x.device, stream)
    ots, ohs = out.stride(0), out.stride(1) if x.dim() == 3 else 0
    _call("indexer_rotary", x.device, stream, x.data_ptr(), ts, hs, positions.data_ptr(),
          freqs.data_ptr(), _DTYPES[x.dtype], tokens, heads, dim, 2 * freqs.shape[0], start, layout,
          scale, transpose, out.data_ptr(), ots, ohs)
    return out


class _Rotary(torch.autograd.Function):
    """The rotation is linear in x: its gradient is the transposed rotation, by this same function."""

    @staticmethod
    def forward(ctx, x, positions, freqs, layout, start, scale, transpose):
        ctx.save_for_backward(positions, freqs)
        ctx.how = layout, start, scale, transpose
        return _rotary(x, positions, freqs, layout, start, scale, transpose, None, None)

    @staticmethod
    def backward(ctx, grad):
        positions, freqs = ctx.saved_tensors
        layout, start, scale, transpose = ctx.how
        if grad.shape[-1] > 1 and grad.stride(-1) != 1:
            grad = grad.contiguous()
        grad = _Rotary.apply(grad, positions, freqs, layout, start, scale, not transpose)
        return grad, None, None, None, None, None, None


def indexer_rotary(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, *,
                   layout: str = "half", start: int = 0, scale: float = 1.0,
                   transpose: bool = False, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Rotary positions on columns [start, start + 2 * len(freqs)) of x ([tokens, dim] or
    [tokens, heads, dim], bf16, fp16 or fp32, unit inner stride); the other columns are copied.

    Pair i turns by positions[t] * freqs[i] radians (positions int32 [tokens], freqs fp64,
    see indexer_rotary_freqs) and is multiplied by `scale`. layout: "half" pairs column
    start + i with start + len(freqs) + i, "interleaved" pairs 2i with 2i + 1. Angles keep
    their precision at any position. transpose: the rotation of a gradient (by the opposite
    angle, with the same scale). out: a tensor like x, or x itself for a call in place.
    Differentiable in x (twice too); a call with `out` or `stream` is not."""
    how = _choice(layout, _LAYOUTS, "layout")
    tokens, _, dim, _, _ = _rows(x, "x")
    _tensor(positions, "positions", _INT32, x.device)
    if positions.dim() != 1 or positions.shape[0] != tokens or (tokens > 1 and positions.stride(0) != 1):
        raise ValueError(f"positions must be a contiguous int32 vector of length {tokens}")
    _tensor(freqs, "freqs", _FP64, x.device)
    if freqs.dim() != 1 or freqs.shape[0] < 1 or (freqs.shape[0] > 1 and freqs.stride(0) != 1):
        raise ValueError("freqs must be a contiguous fp64 vector of at least one frequency")
    start = int(start)
    if start < 0 or start + 2 * freqs.shape[0] > dim:
        raise ValueError(f"columns [{start}, {start + 2 * freqs.shape[0]}) do not lie within the row of {dim}")
    if torch.is_grad_enabled() and x.requires_grad:
        if out is not None or stream is not None:
            raise ValueError("a differentiable call takes neither out nor stream")
        return _Rotary.apply(x, positions, freqs, how, start, float(scale), bool(transpose))
    if out is not None:
        _tensor(out, "out", (x.dtype,), x.device)
        if out.shape != x.shape or (dim > 1 and out.stride(-1) != 1):
            raise ValueError(f"out must have x's shape {tuple(x.shape)} and unit inner stride")
        if torch.is_grad_enabled() and out.requires_grad:
            raise ValueError("out must not require a gradient")
        if _overlap(x, out) and not (out.data_ptr() == x.data_ptr() and out.stride() == x.stride()):
            raise ValueError("out must be x itself or not overlap it")
    return _rotary(x, positions, freqs, how, start, float(scale), bool(transpose), out, stream)


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the spans of memory of two tensors meet."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    if a.numel() == 0 or b.numel() == 0:
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


# ---------------------------------------------------------------- 8-bit rows and cache

def indexer_quantise(x: torch.Tensor, *, scale_format: str = "fp32",
                     weights: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales): rows of x ([tokens, dim] or [tokens, heads, dim]) as e4m3, with one
    fp32 scale for each block of 128 columns; the values they stand for are codes * scales.

    scale_format: "fp32" (amax / 448) or "pow2" (the next power of two). weights: fp32
    [tokens, heads] (or [tokens]), for rows of one block: scales then holds
    weights * scale, of the same shape, as indexer_scores takes it. A block that holds an
    infinity or a NaN becomes NaN throughout. codes, scales: contiguous outputs."""
    fmt = _choice(scale_format, _FORMATS, "scale_format")
    tokens, heads, dim, ts, hs = _rows(x, "x")
    if dim < 1:
        raise ValueError("rows must have at least one column")
    nb = -(-dim // INDEXER_BLOCK)
    dev = x.device
    if weights is not None:
        if nb != 1:
            raise ValueError(f"weights need rows of one block (at most {INDEXER_BLOCK} columns), got {dim}")
        _contiguous(weights, "weights", _FP32, x.shape[:-1], dev)
    scale_shape = x.shape[:-1] if weights is not None else (*x.shape[:-1], nb)
    if codes is None:
        codes = _fresh(x.shape, torch.float8_e4m3fn, dev, stream)
    else:
        _contiguous(codes, "codes", _E4M3, x.shape, dev)
    if scales is None:
        scales = _fresh(scale_shape, torch.float32, dev, stream)
    else:
        _contiguous(scales, "scales", _FP32, scale_shape, dev)
    _call("indexer_quantise", dev, stream, x.data_ptr(), ts, hs, _DTYPES[x.dtype], tokens, heads, dim,
          fmt, None if weights is None else weights.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def indexer_cache_write(x: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor,
                        scales: torch.Tensor, *, scale_format: str = "fp32", stream=None) -> None:
    """Quantises the rows of x ([tokens, dim]) as indexer_quantise does and writes row t at
    slots[t] = page * page_size + offset of a cache: codes [pages, page_size, dim]
    float8_e4m3fn, scales [pages, page_size, ceil(dim / 128)] fp32 (views of one buffer are
    fine). Slot -1: the row is not written. Another slot outside the cache is not written
    either, and counted (indexer_guard_hits). Slots should differ from each other."""
    fmt = _choice(scale_format, _FORMATS, "scale_format")
    tokens, _, dim, ts, _ = _rows(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [tokens, dim]")
    cache = _cache(codes, scales, x.device)
    if dim != cache.dim:
        raise ValueError(f"x has rows of {dim} columns, the cache {cache.dim}")
    _tensor(slots, "slots", _INT32, x.device)
    if slots.dim() != 1 or slots.shape[0] != tokens or (tokens > 1 and slots.stride(0) != 1):
        raise ValueError(f"slots must be a contiguous int32 vector of length {tokens}")
    _call("indexer_cache_write", x.device, stream, x.data_ptr(), ts, _DTYPES[x.dtype], tokens,
          slots.data_ptr(), fmt, ctypes.addressof(cache))


def indexer_cache_read(codes: torch.Tensor, scales: torch.Tensor, slots: torch.Tensor, *,
                       dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """The cache rows at `slots` (int32, contiguous, any shape; the positions that
    topk_transform_paged writes are such slots) as `dtype`: [*slots.shape, dim]. Slot -1
    gives zeros; another slot outside the cache too, and is counted (indexer_guard_hits)."""
    kind = _choice(dtype, _DTYPES, "dtype")
    cache = _cache(codes, scales)
    dev = codes.device
    _tensor(slots, "slots", _INT32, dev)
    if not slots.is_contiguous():
        raise ValueError("slots must be contiguous")
    shape = (*slots.shape, cache.dim)
    if out is None:
        out = _fresh(shape, dtype, dev, stream)
    else:
        _contiguous(out, "out", (dtype,), shape, dev)
    _call("indexer_cache_read", dev, stream, ctypes.addressof(cache), slots.data_ptr(), slots.numel(),
          kind, out.data_ptr())
    return out


# ---------------------------------------------------------------- scores

def indexer_scores(q: torch.Tensor, weights: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, row_len: int, *,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The indexer's scores, fp32 [batch * queries, row_len], as topk_transform_* takes them:

        scale_j * sum_h weights[b, n, h] * relu(q[b, n, h] . k_j)

    for j < seq_lens[b, n] (clamped to [0, row_len]) and -inf after that. q: float8_e4m3fn
    [batch, queries, heads, 128] (one query a sequence for decode, several drafted tokens,
    or a prompt's chunk), weights fp32 [batch, queries, heads] with the scale of q folded in
    (indexer_quantise with weights), both contiguous; the cache's codes
    [pages, page_size, 128] and scales [pages, page_size, 1]; page_table int32 [batch, P]
    with P * page_size >= row_len; seq_lens int32 [batch, queries]. Positions on a page
    outside the cache get -inf and are counted (indexer_guard_hits)."""
    _tensor(q, "q", _E4M3)
    dev = q.device
    if q.dim() != 4 or q.shape[3] != INDEXER_BLOCK or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [batch, queries, heads, {INDEXER_BLOCK}] tensor")
    batch, queries, heads, _ = q.shape
    if not 1 <= heads <= INDEXER_MAX_HEADS:
        raise ValueError(f"heads must be in [1, {INDEXER_MAX_HEADS}], got {heads}")
    _contiguous(weights, "weights", _FP32, (batch, queries, heads), dev)
    cache = _cache(codes, scales, dev)
    if cache.dim != INDEXER_BLOCK:
        raise ValueError(f"the cache's rows must have {INDEXER_BLOCK} columns, got {cache.dim}")
    if (q.data_ptr() | codes.data_ptr() | (codes.stride(0) if codes.shape[0] > 1 else 0)
            | (codes.stride(1) if codes.shape[1] > 1 else 0)) % 16:
        raise ValueError("q and every row of codes must start on 16 bytes")
    row_len = int(row_len)
    if not 1 <= row_len <= 2**31 - 1:
        raise ValueError(f"row_len must be in [1, 2**31 - 1], got {row_len}")
    _tensor(page_table, "page_table", _INT32, dev)
    if page_table.dim() != 2 or page_table.shape[0] != batch or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be [batch, pages] int32 with unit inner stride")
    if page_table.shape[1] * cache.page_size < row_len:
        raise ValueError("page_table has too few pages for the rows")
    pt_stride = page_table.stride(0) if batch > 1 else page_table.shape[1]
    if pt_stride < page_table.shape[1]:
        raise ValueError("page_table rows must not overlap (use .contiguous() on expanded tables)")
    _contiguous(seq_lens, "seq_lens", _INT32, (batch, queries), dev)
    shape = (batch * queries, row_len)
    if out is None:
        out = _fresh(shape, torch.float32, dev, stream)
    else:
        _contiguous(out, "out", _FP32, shape, dev)
    _call("indexer_scores", dev, stream, q.data_ptr(), weights.data_ptr(), ctypes.addressof(cache),
          page_table.data_ptr(), pt_stride, seq_lens.data_ptr(), batch, queries, heads, row_len,
          out.data_ptr())
    return out


def indexer_guard_hits() -> int:
    """Slots and page ids outside the cache that calls on the current device have met (each
    at least once); waits for the device's pending work."""
    n = ctypes.c_uint64(0)
    _check(load_library().indexer_guard_hits(ctypes.byref(n)), "indexer_guard_hits")
    return int(n.value)


def indexer_reset_guard_hits() -> None:
    _check(load_library().indexer_reset_guard_hits(), "indexer_reset_guard_hits")
