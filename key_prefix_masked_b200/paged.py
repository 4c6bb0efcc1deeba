"""Serving around the prefix-masked attention: q and k as a projection leaves them, a paged
key/value cache, and attention of each sequence's new tokens over its pages.

    q, k = attn_qk_norm_rope(q, k, positions, inv_freq, q_weight=wq, k_weight=wk)
    attn_cache_write(k, v, slots, k_cache, v_cache)
    out, lse = attn_paged_fwd(q, k_cache, v_cache, block_table, kv_len, q_start, max_q)

``attn_cache_read`` copies sequences back from their pages into the [B, H, T, D] prefix
layout of ``attn_prefix_fwd``.  ``PagedCache`` holds a pool of pages and runs the three
calls in order.  As in the rest of the package, every step runs in the C library; this
module checks and marshals arguments.
"""
from __future__ import annotations

import math
import struct

import torch

from . import _binding
from ._binding import _check, lib

CACHE_BF16 = 0
CACHE_E4M3 = 1

_CACHE = struct.Struct("4P6q5i4x")      # attn_cache
_OPERAND = struct.Struct("3P2i6q")      # attn_rope_operand
_STRIDES = struct.Struct("3q")          # attn_strides


_functions = {}
# The current stream's handle by device index.  The public accessor builds a Stream object
# on every call (2 us); this one is what generated torch code uses.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name, device, *args):
    """The library's function `name` on the device's current stream, with that device current."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib(), name)
    index = device.index
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(st, name)


def _new(shape, strides, dtype, device):
    """An uninitialised tensor (empty_strided skips a microsecond of torch.empty's argument handling)."""
    return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _new_like(t):
    """An uninitialised contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


_CONTIGUOUS = (0, 0, 0)                 # what the library takes for contiguous


def _strides4(t, name):
    """(page or batch, head, row) strides of a [*, H, T, D] view; a dim of size 1 gets a stride that
    is never used but passes the checks."""
    if t.is_contiguous():
        return _CONTIGUOUS
    B, H, T, D = t.shape
    b, h, s, d = t.stride()
    if d != 1 and D != 1:
        raise ValueError(f"{name}: the head dim must be contiguous (stride 1)")
    if T == 1:
        s = D
    if H == 1:
        h = T * D
    if B == 1:
        b = H * T * D
    if s == 0:
        raise ValueError(f"{name}: rows may not be broadcast")
    return b, h, s


def _strides3(t, name):
    """(0, head, token) strides of a [T, H, D] view (not zeros for a contiguous one: the rotation,
    which takes [B, H, T, D], would read those otherwise)."""
    T, H, D = t.shape
    if t.is_contiguous():
        return 0, D, H * D
    s, h, d = t.stride()
    if d != 1 and D != 1:
        raise ValueError(f"{name}: the head dim must be contiguous (stride 1)")
    if T == 1:
        s = H * D
    if H == 1:
        h = D
    if s == 0:
        raise ValueError(f"{name}: rows may not be broadcast")
    return 0, h, s


def _bf16(t, dim, name):
    if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() not in dim:
        raise ValueError(f"{name} must be a bf16 CUDA tensor of {' or '.join(map(str, dim))} dimensions")


def _int32(t, shape, name, device):
    if t.dtype != torch.int32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on {device}")


def _not_overlapping(t, name):
    """Rows that are written must not share memory (a broadcast head or batch)."""
    if not t.is_contiguous() and any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError(f"{name} may not be a broadcast view")


# ---------------------------------------------------------------------------------- norm and rotation
def rope_inv_freq(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_context=None, beta_fast=32.0,
                  beta_slow=1.0, device="cuda"):
    """(inv_freq, attn_factor) for attn_qk_norm_rope: fp64 [rotary_dim / 2] angles per position.

    scaling, for contexts `factor` times as long as the trained one:
      None      base^(-2i / rotary_dim)
      "linear"  the same divided by factor (positions interpolated)
      "ntk"     base * factor^(rotary_dim / (rotary_dim - 2)): the slowest pair interpolated, the fastest kept
      "yarn"    by parts: pairs that turn more than beta_fast times over original_context are kept, those
                that turn less than beta_slow times are divided by factor; attn_factor
                0.1 ln(factor) + 1 on the rotated values.  Between, a linear ramp in the pair's index,
                from the last pair that is kept to the first that is divided in full: what the
                published models use (the code released with arXiv 2309.00071)
      "yarn_turns"  the same with the ramp linear in the number of turns (that paper's equations)
    """
    R = int(rotary_dim)
    if R < 2 or R % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not factor >= 1.0 or not base > 0.0:
        raise ValueError("factor must be at least 1 and base positive")
    i = torch.arange(0, R, 2, dtype=torch.float64)
    attn_factor = 1.0
    if scaling == "ntk":
        if R < 4:
            raise ValueError("scaling 'ntk' needs rotary_dim >= 4")
        base = base * factor ** (R / (R - 2))
    f = float(base) ** (-i / R)
    if scaling == "linear":
        f = f / factor
    elif scaling in ("yarn", "yarn_turns"):
        if not original_context or not original_context > 0:
            raise ValueError(f"scaling {scaling!r} needs original_context")
        if not beta_fast > beta_slow > 0.0 or not base > 1.0:
            raise ValueError(f"scaling {scaling!r} needs beta_fast > beta_slow > 0 and base > 1")
        if scaling == "yarn":
            # a pair i of base^(-2i/R) turns n times where i = R ln(context / (2 pi n)) / (2 ln base)
            first, last = (R * math.log(original_context / (2 * math.pi * n)) / (2 * math.log(base)) for n in (beta_fast, beta_slow))
            first, last = max(math.floor(first), 0), min(math.ceil(last), R - 1)
            keep = 1.0 - ((i / 2 - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
        else:
            turns = original_context * f / (2 * math.pi)
            keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        attn_factor = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), attn_factor


def _operand(x, out, weight, name):
    """(output, packed attn_rope_operand) of one operand; makes the output where none is given."""
    shape = x.shape
    st = _strides4 if len(shape) == 4 else _strides3
    x_st = st(x, name)
    if out is None:
        out = _new_like(x)
        out_st = x_st if x.is_contiguous() else st(out, name)
    else:
        if out.shape != shape or out.dtype != torch.bfloat16 or out.device != x.device:
            raise ValueError(f"{name}_out must be a bf16 tensor of {name}'s shape on {x.device}")
        _not_overlapping(out, name + "_out")
        out_st = st(out, name + "_out")
    w = 0
    fp32 = False
    if weight is not None:
        dtype = weight.dtype
        fp32 = dtype == torch.float32
        if (not (fp32 or dtype == torch.bfloat16) or weight.device != x.device or weight.shape != shape[-1:]
                or not weight.is_contiguous()):
            raise ValueError(f"{name}_weight must be a contiguous bf16 or fp32 tensor [D] on {x.device}")
        w = weight.data_ptr()
    return out, _OPERAND.pack(x.data_ptr(), out.data_ptr(), w, shape[1], fp32, *x_st, *out_st)


def attn_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                      attn_factor=1.0, q_out=None, k_out=None):
    """Per-head RMS norm and rotation by position (attn_qk_norm_rope): returns (q_out, k_out).

    q: bf16 [T, Hq, D] (tokens first) or [B, H, T, D], views included (e.g. slices of a packed
    projection); k: the same with its own head count, or None.  positions: int32 [T], or [B, T].
    inv_freq: fp64 [R/2] (rope_inv_freq), R <= D elements of each head are rotated; None: norm only.
    A weight that is None leaves its operand unnormalised.  q_out may be q (in place)."""
    _bf16(q, (3, 4), "q")
    shape, dev = q.shape, q.device
    four = len(shape) == 4
    B, T = (shape[0], shape[2]) if four else (1, shape[0])
    D = shape[-1]
    R = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or inv_freq.device != dev or not inv_freq.is_contiguous():
            raise ValueError(f"inv_freq must be a contiguous fp64 tensor [R / 2] on {dev}")
        R = 2 * inv_freq.numel()
        _int32(positions, (B, T) if four else (T,), "positions", dev)
    if k is not None:
        _bf16(k, (len(shape),), "k")
        ks = k.shape
        if k.device != dev or ks[-1] != D or ks[0] != shape[0] or (four and ks[2] != T):
            raise ValueError("k must have q's tokens, head dim and device")
    if q.numel() == 0 or (k is not None and k.numel() == 0):
        raise ValueError("q and k may not be empty")
    q_out, op_q = _operand(q, q_out, q_weight, "q")
    op_k = None
    if k is not None:
        k_out, op_k = _operand(k, k_out, k_weight, "k")
    _call("attn_qk_norm_rope", dev, op_q, op_k, positions.data_ptr() if R else None,
          inv_freq.data_ptr() if R else None, B, T, D, R, bool(interleaved), eps, attn_factor)
    return q_out, k_out if k is not None else None


# ---------------------------------------------------------------------------------- cache
def _cache(k_cache, v_cache, k_scale, v_scale):
    """The packed attn_cache of a pool's tensors."""
    dtype, shape = k_cache.dtype, k_cache.shape
    e4m3 = dtype == torch.float8_e4m3fn
    if not k_cache.is_cuda or len(shape) != 4 or not (e4m3 or dtype == torch.bfloat16):
        raise ValueError("k_cache must be a bf16 or float8_e4m3fn CUDA tensor [num_pages, Hkv, page_size, D]")
    if v_cache.shape != shape or v_cache.dtype != dtype or v_cache.device != k_cache.device:
        raise ValueError("v_cache must match k_cache")
    P, H, page, D = shape
    if e4m3:
        for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if (s is None or s.dtype != torch.uint8 or s.device != k_cache.device or s.shape != shape[:3]
                    or not s.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous uint8 tensor [num_pages, Hkv, page_size]")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("bf16 pages have no scales")
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr() if e4m3 else 0,
                       v_scale.data_ptr() if e4m3 else 0, *_strides4(k_cache, "k_cache"),
                       *_strides4(v_cache, "v_cache"), P, page, H, D, CACHE_E4M3 if e4m3 else CACHE_BF16)


def attn_cache_write(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None):
    """Stores rows k, v (bf16 [T, Hkv, D], views included) at slots (int32 [T], page * page_size + row;
    negative: skipped) of the pages (attn_cache_write).

    k_cache, v_cache: [num_pages, Hkv, page_size, D], views of other layouts included, bf16, or
    float8_e4m3fn with k_scale, v_scale uint8 [num_pages, Hkv, page_size].  The slots of one call must
    be distinct."""
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    _not_overlapping(k_cache, "k_cache")
    _not_overlapping(v_cache, "v_cache")
    _bf16(k, (3,), "k")
    _bf16(v, (3,), "v")
    shape, pool, dev = k.shape, k_cache.shape, k.device
    T = shape[0]
    if v.shape != shape or shape[1] != pool[1] or shape[2] != pool[3]:
        raise ValueError("k and v must be [T, Hkv, D] with the cache's Hkv and D")
    if dev != k_cache.device or v.device != dev:
        raise ValueError("all tensors must be on one device")
    _int32(slots, (T,), "slots", dev)
    if T == 0:
        return
    _call("attn_cache_write", dev, c, k.data_ptr(), v.data_ptr(), _STRIDES.pack(*_strides3(k, "k")),
          _STRIDES.pack(*_strides3(v, "v")), slots.data_ptr(), T)


def _table(block_table, kv_len, device):
    shape = block_table.shape
    if block_table.dtype != torch.int32 or block_table.device != device or len(shape) != 2 or (
            block_table.stride(1) != 1 and shape[1] != 1):
        raise ValueError(f"block_table must be an int32 tensor [B, max_pages] on {device} with contiguous rows")
    B, n = shape
    if B == 0 or n == 0:
        raise ValueError("block_table may not be empty")
    _int32(kv_len, (B,), "kv_len", device)
    return B, n


def attn_cache_read(k_cache, v_cache, block_table, kv_len, Tk=None, k_scale=None, v_scale=None, k_out=None, v_out=None):
    """Sequences read back from their pages as contiguous prefixes (attn_cache_read): (k, v) bf16
    [B, Hkv, Tk, D], as attn_prefix_fwd takes them.

    block_table: int32 [B, max_pages]; kv_len: int32 [B].  Rows at or beyond kv_len[b] are left as
    they were (uninitialised where k_out, v_out are made here).  Tk: by default max_pages * page_size."""
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    B, n = _table(block_table, kv_len, dev)
    _, H, page, D = k_cache.shape
    k_st = v_st = None                  # contiguous
    if k_out is None or v_out is None:
        if k_out is not None or v_out is not None:
            raise ValueError("k_out and v_out are given together")
        Tk = n * page if Tk is None else int(Tk)
        k_out = _new((B, H, Tk, D), (H * Tk * D, Tk * D, D, 1), torch.bfloat16, dev)
        v_out = torch.empty_like(k_out)
    else:
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if (t.dim() != 4 or t.shape[:2] != (B, H) or t.shape[3] != D or t.dtype != torch.bfloat16
                    or t.device != dev or t.shape != k_out.shape or Tk not in (None, t.shape[2])):
                raise ValueError(f"{name} must be a bf16 tensor [B, Hkv, Tk, D] on {dev}")
            _not_overlapping(t, name)
        Tk = k_out.shape[2]
        k_st, v_st = _STRIDES.pack(*_strides4(k_out, "k_out")), _STRIDES.pack(*_strides4(v_out, "v_out"))
    if Tk == 0:
        return k_out, v_out
    _call("attn_cache_read", dev, c, block_table.data_ptr(), block_table.stride(0), n, kv_len.data_ptr(),
          k_out.data_ptr(), v_out.data_ptr(), k_st, v_st, B, Tk)
    return k_out, v_out


# ---------------------------------------------------------------------------------- attention
def attn_paged_fwd(q, k_cache, v_cache, block_table, kv_len, q_start=None, max_q=None, causal=True, scale=None,
                   k_scale=None, v_scale=None, workspace=None, out=None, lse=None, need_lse=True):
    """Attention of each sequence's new tokens over its pages (attn_paged_fwd): (out bf16 [T, Hq, D],
    lse fp32 [T, Hq]).

    q: bf16 [T, Hq, D], sequence b's rows at [q_start[b], q_start[b+1]) (int32 [B + 1]); without
    q_start one row per sequence.  max_q: an upper bound on a sequence's rows.  By default it is T, which is
    right but makes a batch of few rows each run as if one sequence had them all, several times slower: give
    it with q_start.  The
    pages hold the new tokens' keys too; with `causal`, the rows are the last positions of their
    sequence.  Rows outside every sequence are left as they were (uninitialised where out is made
    here).  workspace: a buffer of attn_paged_workspace_bytes, allocated here when not given."""
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    B, n = _table(block_table, kv_len, k_cache.device)
    _bf16(q, (3,), "q")
    shape, dev = q.shape, q.device
    T, Hq, D = shape
    _, Hkv, page, Dc = k_cache.shape
    if D != Dc or dev != k_cache.device:
        raise ValueError("q must have the cache's head dim and device")
    if Hq == 0 or Hkv == 0 or Hq % Hkv:
        raise ValueError("q's head count must be a multiple of the cache's")
    if q_start is not None:
        _int32(q_start, (B + 1,), "q_start", dev)
    elif T != B:
        raise ValueError("without q_start, q must have one row per sequence")
    out_st = None                       # contiguous
    if out is None:
        out = _new_like(q)
    elif out.shape != shape or out.dtype != torch.bfloat16 or out.device != dev:
        raise ValueError("out must be a bf16 tensor of q's shape on q's device")
    else:
        _not_overlapping(out, "out")
        out_st = _STRIDES.pack(*_strides3(out, "out"))
    if lse is not None:
        if lse.shape != (T, Hq) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous fp32 tensor [T, Hq] on q's device")
    elif need_lse:
        lse = _new((T, Hq), (Hq, 1), torch.float32, dev)
    if T == 0:
        return out, lse
    scale = D ** -0.5 if scale is None else scale
    max_q = 1 if q_start is None else T if max_q is None else int(max_q)
    bytes_of = _functions.get("attn_paged_workspace_bytes")
    if bytes_of is None:
        bytes_of = _functions["attn_paged_workspace_bytes"] = lib().attn_paged_workspace_bytes
    need = bytes_of(B, T, Hq, Hkv, D, page, n, max_q)
    if need and workspace is None:
        workspace = _new((need,), (1,), torch.uint8, dev)
    elif need and (workspace.device != dev or not workspace.is_contiguous()
                   or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must be a contiguous CUDA buffer of at least {need} bytes")
    _call("attn_paged_fwd", dev, c, q.data_ptr(), _STRIDES.pack(*_strides3(q, "q")), block_table.data_ptr(),
          block_table.stride(0), n, kv_len.data_ptr(), None if q_start is None else q_start.data_ptr(), out.data_ptr(),
          out_st, None if lse is None else lse.data_ptr(),
          workspace.data_ptr() if need else None, B, T, Hq, max_q, bool(causal), scale)
    return out, lse


class PagedCache:
    """A pool of key/value pages and the serving step over it.

    quantised: e4m3 rows with a power-of-two scale each, otherwise bf16.  Which page belongs to
    which sequence is the caller's (block_table, slots)."""

    def __init__(self, num_pages, page_size, Hkv, D, quantised=False, device=None):
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        shape = (int(num_pages), int(Hkv), int(page_size), int(D))
        dtype = torch.float8_e4m3fn if quantised else torch.bfloat16
        self.page_size = int(page_size)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8 if quantised else dtype, device=dev).view(dtype)
                          for _ in range(2))
        self.scales = {}
        if quantised:
            self.scales = {n: torch.full(shape[:3], 127, dtype=torch.uint8, device=dev) for n in ("k_scale", "v_scale")}

    def write(self, k, v, slots):
        attn_cache_write(k, v, slots, self.k, self.v, **self.scales)

    def read(self, block_table, kv_len, Tk=None):
        return attn_cache_read(self.k, self.v, block_table, kv_len, Tk, **self.scales)

    def attend(self, q, block_table, kv_len, q_start=None, max_q=None, **kw):
        return attn_paged_fwd(q, self.k, self.v, block_table, kv_len, q_start, max_q, **self.scales, **kw)

    def step(self, q, k, v, positions, slots, block_table, kv_len, q_start=None, max_q=None, inv_freq=None, rope=None,
             **kw):
        """One serving step of new tokens: q [T, Hq, D], k, v [T, Hkv, D] as the projection leaves
        them.  Norm and rotation (`rope`: further arguments of attn_qk_norm_rope), the new rows into
        their slots, attention over the pages.  kv_len counts the new tokens.  Returns (out, lse)."""
        q, k = attn_qk_norm_rope(q, k, positions, inv_freq, **(rope or {}))
        self.write(k, v, slots)
        return self.attend(q, block_table, kv_len, q_start, max_q, **kw)
