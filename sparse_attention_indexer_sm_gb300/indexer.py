"""The operators around the top-k of a sparse-attention indexer.

A thin binding over the C ABI in ``include/indexer_ops.h``, in the manner of the
package's top-k calls: tensors are checked and marshalled (in ``csrc/indexer_binding.cpp``),
the work runs in the library's sm_103a kernels on the tensors' device and the current torch
stream (or ``stream``, which the caller orders behind the work that makes the inputs), and
nothing falls back to torch. A decode step, with a paged cache
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
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import TopkError, _build, _check, load_library

__all__ = [
    "indexer_rotary", "indexer_rotary_freqs", "indexer_quantise", "indexer_cache_write",
    "indexer_cache_read", "indexer_scores", "indexer_guard_hits", "indexer_reset_guard_hits",
    "INDEXER_BLOCK", "INDEXER_MAX_HEADS",
]

INDEXER_BLOCK = 128
INDEXER_MAX_HEADS = 128

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_LAYOUTS = {"half": 0, "interleaved": 1}
_RAMPS = {"turns": 0, "pairs": 1}
_FORMATS = {"fp32": 0, "pow2": 1}

_binding = None


def _load_binding():
    """The compiled binding (raises if it has not been built)."""
    global _binding
    if _binding is None:
        load_library()
        path = _build.binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (python -m "
                               "sparse_attention_indexer_sm_gb300.build, or __graft_entry__.build())")
        loader = importlib.machinery.ExtensionFileLoader("indexer_binding", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("indexer_binding", loader))
        loader.exec_module(module)
        module.set_error(TopkError)
        _binding = module
    return _binding


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
        "indexer_set_scores_failure": [i32],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    lib.indexer_cache_bytes.restype = ctypes.c_size_t
    lib.indexer_cache_bytes.argtypes = []
    if lib.indexer_cache_bytes() != ctypes.sizeof(IndexerCache):
        raise RuntimeError("indexer_cache_t layout differs between the library and this binding")


def _choice(value, table, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}")
    return table[value]


def _on(stream, call, *args):
    """A call on a stream of the caller's. Its tensors are in use there until its kernel has ended: none of their memory
    is handed out again before that. (Outputs that it makes come from that stream's memory.)"""
    out = call(*args, stream.cuda_stream)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


# ---------------------------------------------------------------- rotary positions

def indexer_rotary_freqs(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None,
                         factor: float = 1.0, original_len: int = 4096, beta_fast: float = 32.0,
                         beta_slow: float = 1.0, ramp: str = "turns",
                         device="cuda") -> tuple[torch.Tensor, float]:
    """(freqs, scale) for indexer_rotary: fp64 radians per position of the rot_dim / 2
    pairs, base ** (-2 i / rot_dim), and the factor of sine and cosine.

    scaling, for contexts `factor` times the trained `original_len`: None; "linear" (all
    frequencies divided by factor); "ntk" (a larger base: the slowest pair divided by
    factor, the fastest kept); "yarn" (pairs that turn more than beta_fast times within
    original_len kept, those that turn less than beta_slow times divided by factor, those
    between blended; scale = 0.1 ln(factor) + 1).

    ramp, how yarn blends: "turns", linearly in the number of turns; or "pairs", linearly in
    the pair's index between the pairs that turn beta_fast times (rounded down) and beta_slow
    times (rounded up), as the method's published code does and the checkpoints trained with
    it expect: take the one that the model was trained with. A model that puts the factor
    into its softmax ignores `scale`."""
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
        if _choice(ramp, _RAMPS, "ramp") == 0:
            turns = original_len * freqs / (2.0 * math.pi)
            keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        else:
            low, high = (rot_dim * math.log(original_len / (2.0 * math.pi * b)) / (2.0 * math.log(base))
                         for b in (beta_fast, beta_slow))
            low, high = max(math.floor(low), 0), min(math.ceil(high), rot_dim - 1)
            keep = 1.0 - ((i - low) / max(high - low, 1)).clamp(0.0, 1.0)
        freqs = freqs * keep + freqs / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    return freqs.to(device), scale


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
    Differentiable in x by backward (twice too); a call with `out` or `stream` is not, and
    forward-mode tangents are refused."""
    f = (_binding or _load_binding()).rotary
    how = _choice(layout, _LAYOUTS, "layout")
    if stream is not None:
        return _on(stream, f, x, positions, freqs, how, start, scale, transpose, out)
    return f(x, positions, freqs, how, start, scale, transpose, out, None)


# ---------------------------------------------------------------- 8-bit rows and cache

def indexer_quantise(x: torch.Tensor, *, scale_format: str = "fp32",
                     weights: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales): rows of x ([tokens, dim] or [tokens, heads, dim]) as e4m3, with one
    fp32 scale for each block of 128 columns; the values they stand for are codes * scales.

    scale_format: "fp32" (amax / 448) or "pow2" (the next power of two). weights: fp32
    [tokens, heads] (or [tokens]), for rows of one block: scales then holds
    weights * scale, of the same shape, as indexer_scores takes it. A block that holds an
    infinity or a NaN becomes NaN throughout. codes, scales: contiguous outputs. There is no
    gradient: tensors that require one are refused while gradients are recorded."""
    f = (_binding or _load_binding()).quantise
    fmt = _choice(scale_format, _FORMATS, "scale_format")
    if stream is not None:
        return _on(stream, f, x, fmt, weights, codes, scales)
    return f(x, fmt, weights, codes, scales, None)


def indexer_cache_write(x: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor,
                        scales: torch.Tensor, *, scale_format: str = "fp32", stream=None) -> None:
    """Quantises the rows of x ([tokens, dim]) as indexer_quantise does and writes row t at
    slots[t] = page * page_size + offset of a cache: codes [pages, page_size, dim]
    float8_e4m3fn, scales [pages, page_size, ceil(dim / 128)] fp32 (views of one buffer are
    fine). Slot -1: the row is not written. Another slot outside the cache is not written
    either, and counted (indexer_guard_hits). Slots should differ from each other. There is
    no gradient, as in indexer_quantise."""
    f = (_binding or _load_binding()).cache_write
    fmt = _choice(scale_format, _FORMATS, "scale_format")
    if stream is not None:
        _on(stream, f, x, slots, codes, scales, fmt)
    else:
        f(x, slots, codes, scales, fmt, None)


def indexer_cache_read(codes: torch.Tensor, scales: torch.Tensor, slots: torch.Tensor, *,
                       dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """The cache rows at `slots` (int32, contiguous, any shape; the positions that
    topk_transform_paged writes are such slots) as `dtype`: [*slots.shape, dim]. Slot -1
    gives zeros; another slot outside the cache too, and is counted (indexer_guard_hits).
    There is no gradient, as in indexer_quantise."""
    f = (_binding or _load_binding()).cache_read
    kind = _choice(dtype, _DTYPES, "dtype")
    if stream is not None:
        return _on(stream, f, codes, scales, slots, kind, out)
    return f(codes, scales, slots, kind, out, None)


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
    outside the cache get -inf and are counted (indexer_guard_hits). There is no gradient, as
    in indexer_quantise."""
    f = (_binding or _load_binding()).scores
    if stream is not None:
        return _on(stream, f, q, weights, codes, scales, page_table, seq_lens, row_len, out)
    return f(q, weights, codes, scales, page_table, seq_lens, row_len, out, None)


def indexer_guard_hits() -> int:
    """Slots and page ids outside the cache that calls on the current device have met (each
    at least once); waits for the device's pending work."""
    n = ctypes.c_uint64(0)
    _check(load_library().indexer_guard_hits(ctypes.byref(n)), "indexer_guard_hits")
    return int(n.value)


def indexer_reset_guard_hits() -> None:
    _check(load_library().indexer_reset_guard_hits(), "indexer_reset_guard_hits")
