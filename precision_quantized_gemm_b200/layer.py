"""The operators between a decoder layer's quantised products: the norm that
makes a product's operand, the rotary cache write, the cache read and the
attention over the quantised cache.  Argument marshalling over the C ABI, as
in the package's own module; the formulas stand in include/qgemm.h.

    r = norm(residual, w, x, fmt=QG_FP8_DYNAMIC)          # r.h, r.operand
    qkv = run(QG_FP8_DYNAMIC, r.operand, Wqkv).view(T, Hq + 2 * Hkv, D)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    q = cache_write(cache, k, v, slots, q=q, rope=rope, positions=positions)
    o = attend(cache, q, q_offsets, kv_len, page_table, tree_mask=mask, max_q=most)

Shapes, types and strides are checked here (ValueError); sizes, alignment and
options by the library (QGemmError).  ``stream``: the torch stream to launch
on (default: the current stream of the tensors' device).  Buffers these
functions allocate come from that stream's pool; tensors of other streams are
the caller's to order, as with any torch operation.
"""
from __future__ import annotations

import ctypes
import functools
import math
from collections import namedtuple

from . import (NORM_KINDS, QG_NORM_NONE, QG_NVFP4, QGEMM_ATTEND_MAX_Q, Operand, Workspace, _torch, check, lib, qg_attend,
               qg_cache, qg_cache_write, qg_norm, qg_operand, qgemm_operand_bytes)

__all__ = ["Cache", "NormResult", "Rope", "attend", "cache_read", "cache_write", "norm", "rope_frequencies"]

NormResult = namedtuple("NormResult", "h y operand")


# ------------------------------------------------------- C-named entry points --
def qgemm_norm(n, M, N, fmt, out, static_amax_ptr, stream):
    return lib().qgemm_norm(ctypes.byref(n), M, N, fmt, ctypes.byref(out) if out is not None else None,
                            static_amax_ptr, stream)


def qgemm_cache_bytes(fmt, pages, page_size, kv_heads, head_dim):
    """(bytes of k or v, bytes of k_scale or v_scale) of a cache."""
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    check(lib().qgemm_cache_bytes(fmt, pages, page_size, kv_heads, head_dim, ctypes.byref(c), ctypes.byref(s)),
          "qgemm_cache_bytes")
    return c.value, s.value


def qgemm_cache_write(cache, w, tokens, stream):
    return lib().qgemm_cache_write(ctypes.byref(cache), ctypes.byref(w), tokens, stream)


def qgemm_cache_read(cache, slots_ptr, tokens, k_ptr, ldk, v_ptr, ldv, stream):
    return lib().qgemm_cache_read(ctypes.byref(cache), slots_ptr, tokens, k_ptr, ldk, v_ptr, ldv, stream)


def qgemm_attend_workspace_size(cache, a):
    return lib().qgemm_attend_workspace_size(ctypes.byref(cache), ctypes.byref(a))


def qgemm_attend(cache, a, ws_ptr, ws_bytes, stream):
    return lib().qgemm_attend(ctypes.byref(cache), ctypes.byref(a), ws_ptr, ws_bytes, stream)


# ------------------------------------------------------------------- checking --
torch = None  # imported at the first call, as in the package's own module


def _ready(device, stream) -> bool:
    """Whether the launch goes where the caller stands: the current stream of
    the current device, which is the tensors'.  (The raw accessors cost a
    tenth of torch.cuda.current_stream(), half of a small call.)"""
    global torch
    if torch is None:
        torch = _torch()
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    return stream is None and device.index == torch._C._cuda_getDevice()


def _there(device, stream):
    """Makes the tensors' device and the stream to launch on current."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("the stream is not one of the tensors' device")
    return torch.cuda.stream(stream)


def _here(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _stride(name, stride):
    # the structures' strides are 32-bit, and ctypes would cut a larger one
    if stride > 0x7fffffff:
        raise ValueError(f"{name}: a row stride below 2^31 elements wanted")
    return stride


def _rows(name, t, rows, width, device):
    """A bf16 matrix [rows, width] with contiguous rows; its row stride."""
    if t.dtype != torch.bfloat16 or t.shape != (rows, width) or t.device != device:
        raise ValueError(f"{name}: bf16 [{rows}, {width}] on {device} wanted")
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return _stride(name, t.stride(0)) if rows > 1 else width


def _heads(name, t, tokens, heads, dim, device):
    """A bf16 tensor [tokens, heads, dim] whose heads lie side by side; its token stride."""
    if t.dtype != torch.bfloat16 or t.shape != (tokens, heads, dim) or t.device != device:
        raise ValueError(f"{name}: bf16 [{tokens}, {heads}, {dim}] on {device} wanted")
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != dim):
        raise ValueError(f"{name}: a token's heads must lie side by side")
    return _stride(name, st[0]) if tokens > 1 else heads * dim


def _ints(name, t, shape, device, dtype=None):
    dtype = dtype or torch.int32
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} on {device} wanted")
    return t.data_ptr()


def _vector(name, t, width, device):
    if t is None:
        return None
    if t.dtype != torch.bfloat16 or t.shape != (width,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous bf16 [{width}] on {device} wanted")
    return t.data_ptr()


# ----------------------------------------------------------------------- norm --
def norm(residual, weight, x=None, *, bias=None, kind="rms", post_weight=None, post_bias=None, gate=None,
         block_scale=1.0, residual_scale=1.0, eps=1e-6, weight_offset=0.0, fmt=None, out=None, h=None, y=None,
         static_amax=None, stream=None) -> NormResult:
    """h = residual_scale * residual + block_scale * gate * P(x); y = norm(h).

    ``residual`` (or None) and the block's output ``x`` (or None): bf16 [M, N].
    ``kind``: "rms" or "layer", for the norm of h (``weight``, ``bias``; weight
    None: only h) and for P (with ``post_weight``; else P is the identity).
    ``gate``: bf16 [N] or [M, N].  ``fmt`` (a format): y becomes the operand
    ``out`` (allocated if None) of the next ``run``; without it y is bf16.
    ``h`` / ``y``: bf16 [M, N] buffers for them; h is also returned when x is
    given or nothing else is asked for, and may be ``residual`` (in place).
    NVFP4 needs ``static_amax``.  Returns NormResult(h, y, operand)."""
    first = residual if residual is not None else x
    if first is None or first.dim() != 2:
        raise ValueError("residual or x: bf16 [M, N] wanted")
    code = NORM_KINDS.get(kind, QG_NORM_NONE)
    if code == QG_NORM_NONE:
        raise ValueError("kind is 'rms' or 'layer'")
    if weight is None and (fmt is not None or out is not None or y is not None):
        raise ValueError("y needs a weight")
    if out is not None and fmt is None:
        fmt = out.fmt
    if out is not None and (out.fmt != fmt or out.is_weight):
        raise ValueError("out is not an activation operand of this format")
    M, N = first.shape
    dev = first.device
    if not _ready(dev, stream):
        with _there(dev, stream):
            return norm(residual, weight, x, bias=bias, kind=kind, post_weight=post_weight, post_bias=post_bias,
                        gate=gate, block_scale=block_scale, residual_scale=residual_scale, eps=eps,
                        weight_offset=weight_offset, fmt=fmt, out=out, h=h, y=y, static_amax=static_amax)
    # (new_empty takes half the time of torch.empty; the inputs' types are checked below)
    if h is None and (x is not None or weight is None):
        h = first.new_empty((M, N))
    if weight is not None and fmt is None and y is None:
        y = first.new_empty((M, N))
    if fmt is not None and out is None:
        out = _operand(fmt, M, N, dev)
    elif out is not None and out.q.device != dev:
        raise ValueError(f"out: an operand on {dev} wanted")
    a = qg_norm(residual_scale=residual_scale, block_scale=block_scale, eps=eps, weight_offset=weight_offset)
    if residual is not None:
        a.ldr, a.residual = _rows("residual", residual, M, N, dev), residual.data_ptr()
    if x is not None:
        a.ldx, a.x = _rows("x", x, M, N, dev), x.data_ptr()
    if h is not None:
        a.ldh, a.h = _rows("h", h, M, N, dev), h.data_ptr()
    if y is not None:
        a.ldy, a.y = _rows("y", y, M, N, dev), y.data_ptr()
    if gate is not None:
        if gate.dim() == 1:
            a.gate = _vector("gate", gate, N, dev)
        else:
            a.ldg, a.gate = _rows("gate", gate, M, N, dev), gate.data_ptr()
    if weight is not None:
        a.pre_norm, a.pre_weight = code, _vector("weight", weight, N, dev)
    if bias is not None:
        a.pre_bias = _vector("bias", bias, N, dev)
    if post_weight is not None:
        a.post_norm, a.post_weight = code, _vector("post_weight", post_weight, N, dev)
    if post_bias is not None:
        a.post_bias = _vector("post_bias", post_bias, N, dev)
    amax = None
    if static_amax is not None:
        if static_amax.dtype != torch.float32 or static_amax.numel() != 1 or static_amax.device != dev:
            raise ValueError(f"static_amax: one fp32 value on {dev} wanted")
        amax = static_amax.data_ptr()
    check(lib().qgemm_norm(a, M, N, fmt if fmt is not None else 0, out.c if out is not None else None, amax, _here(dev)),
          "qgemm_norm")
    return NormResult(h, y, out)


@functools.lru_cache(maxsize=1024)
def _operand_bytes(fmt, M, N):
    return qgemm_operand_bytes(fmt, False, M, N)


def _operand(fmt, M, N, dev):
    """An activation operand that the norm fills: nothing to clear beforehand,
    and a tensor scale for NVFP4 only."""
    qb, sb = _operand_bytes(fmt, M, N)
    o = Operand.__new__(Operand)
    o.fmt, o.is_weight, o.rows, o.K = fmt, False, M, N
    o.q = torch.empty(qb, dtype=torch.uint8, device=dev)
    o.scale = torch.empty(sb, dtype=torch.uint8, device=dev)
    o.global_scale = torch.empty(4, dtype=torch.float32, device=dev) if fmt == QG_NVFP4 else None
    o.c = qg_operand(o.q.data_ptr(), o.scale.data_ptr(),
                     o.global_scale.data_ptr() if fmt == QG_NVFP4 else None, M, N)
    return o


# ----------------------------------------------------------------------- rope --
def rope_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int = 8192, low: float = 1.0, high: float = 4.0, fast: float = 32.0, slow: float = 1.0,
                     device="cuda"):
    """(frequency, magnitude) of a rotary embedding of ``dim`` channels:
    frequency[j] = base^(-2j / dim) radians per position, float64 [dim / 2],
    rescaled for contexts ``factor`` times the ``original`` one:
      None      unscaled
      "linear"  all frequencies / factor
      "base"    base * factor^(dim / (dim - 2)): the slowest pair / factor, the fastest kept
      "bands"   pairs that turn more than ``high`` times in the original context kept, fewer than ``low`` / factor,
                a linear blend in the number of turns between
      "ramp"    pairs that turn more than ``fast`` times kept, fewer than ``slow`` / factor, a linear blend in the
                pair's index between; magnitude 0.1 ln(factor) + 1"""
    torch = _torch()
    if dim <= 0 or dim % 2 or factor < 1.0:
        raise ValueError("dim: an even number; factor: at least 1")
    j = torch.arange(dim // 2, dtype=torch.float64)
    if scaling == "base":
        base = base * factor ** (dim / (dim - 2)) if dim > 2 else base
    f = float(base) ** (-2.0 * j / dim)
    magnitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    elif scaling == "ramp":
        def index(turns):  # the pair that turns so many times in the original context
            return dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        # (the upper end may lie past the last pair, which is then blended, too)
        first, last = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), dim - 1)
        keep = 1 - ((j - first) / max(last - first, 1e-3)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling: None, 'linear', 'base', 'bands' or 'ramp'")
    return f.to(device), magnitude


class Rope:
    """Rotary positions of a head's first ``2 * len(frequency)`` channels:
    ``frequency`` float64 [R / 2] radians per position (rope_frequencies),
    channel pairs (j, j + R / 2), or (2j, 2j + 1) when ``interleaved``."""

    def __init__(self, frequency, interleaved: bool = False, magnitude: float = 1.0):
        torch = _torch()
        if frequency.dtype != torch.float64 or frequency.dim() != 1 or not frequency.is_contiguous():
            raise ValueError("frequency: contiguous float64 [R / 2] wanted")
        self.frequency, self.interleaved, self.magnitude = frequency, bool(interleaved), float(magnitude)
        self.dim = 2 * frequency.numel()


# ---------------------------------------------------------------------- cache --
class Cache:
    """A paged key / value cache quantised per (token, head): ``fmt``
    QG_FP8_DYNAMIC (e4m3) or QG_W8A8_INT8.  Allocates zeroed buffers, or wraps
    given ones: k, v uint8 [pages, kv_heads, page_size, head_dim], k_scale,
    v_scale fp32 [pages, kv_heads, page_size].  Slot s is place s % page_size
    of page s // page_size."""

    def __init__(self, fmt: int, pages: int | None = None, page_size: int | None = None, kv_heads: int | None = None,
                 head_dim: int | None = None, device="cuda", k=None, v=None, k_scale=None, v_scale=None):
        torch = _torch()
        if k is None:
            if None in (pages, page_size, kv_heads, head_dim) or any(t is not None for t in (v, k_scale, v_scale)):
                raise ValueError("pages, page_size, kv_heads and head_dim, or all four buffers, wanted")
            qgemm_cache_bytes(fmt, pages, page_size, kv_heads, head_dim)
            shape = (pages, kv_heads, page_size)
            k, v = (torch.zeros(*shape, head_dim, dtype=torch.uint8, device=device) for _ in range(2))
            k_scale, v_scale = (torch.zeros(*shape, dtype=torch.float32, device=device) for _ in range(2))
        if k.dim() != 4:
            raise ValueError("k: uint8 [pages, kv_heads, page_size, head_dim] wanted")
        for name, t, shape, dtype in (("k", k, k.shape, torch.uint8), ("v", v, k.shape, torch.uint8),
                                      ("k_scale", k_scale, k.shape[:3], torch.float32),
                                      ("v_scale", v_scale, k.shape[:3], torch.float32)):
            if t is None or t.dtype != dtype or t.shape != shape or t.device != k.device or not t.is_contiguous():
                raise ValueError(f"{name}: contiguous {dtype} {list(shape)} on {k.device} wanted")
        self.fmt = fmt
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        qgemm_cache_bytes(fmt, self.pages, self.page_size, self.kv_heads, self.head_dim)
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.device
        self.c = qg_cache(fmt, self.pages, self.page_size, self.kv_heads, self.head_dim, k.data_ptr(), v.data_ptr(),
                          k_scale.data_ptr(), v_scale.data_ptr())


def cache_write(cache: Cache, k, v, slots, q=None, rope: Rope | None = None, positions=None, q_out=None, stream=None):
    """Quantises keys and values (bf16 [T, kv_heads, head_dim], any token
    stride) into the cache's ``slots`` (int32 [T]; below 0: a padded token,
    not written; the others must differ), rotating keys by ``rope`` at
    ``positions`` (int32 [T]).  ``q`` (bf16 [T, q_heads, head_dim]) is rotated
    alongside into ``q_out`` (allocated if None, may be q), which is returned."""
    if k.dim() != 3:
        raise ValueError("k: bf16 [tokens, kv_heads, head_dim] wanted")
    T, dev, D = k.shape[0], cache.device, cache.head_dim
    if not _ready(dev, stream):
        with _there(dev, stream):
            return cache_write(cache, k, v, slots, q=q, rope=rope, positions=positions, q_out=q_out)
    a = qg_cache_write(ldk=_heads("k", k, T, cache.kv_heads, D, dev), ldv=_heads("v", v, T, cache.kv_heads, D, dev),
                       k=k.data_ptr(), v=v.data_ptr(), slots=_ints("slots", slots, (T,), dev))
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q: bf16 [tokens, q_heads, head_dim] wanted")
        Hq = q.shape[1]
        if q_out is None:
            q_out = q.new_empty((T, Hq, D))
        a.q_heads, a.ldq, a.ldqo = Hq, _heads("q", q, T, Hq, D, dev), _heads("q_out", q_out, T, Hq, D, dev)
        a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rope is not None:
        if positions is None or rope.frequency.device != dev:
            raise ValueError(f"a rope needs positions, and its frequency on {dev}")
        a.positions, a.frequency = _ints("positions", positions, (T,), dev), rope.frequency.data_ptr()
        a.rope_dim, a.interleaved, a.magnitude = rope.dim, rope.interleaved, rope.magnitude
    check(lib().qgemm_cache_write(cache.c, a, T, _here(dev)), "qgemm_cache_write")
    return q_out


def cache_read(cache: Cache, slots, k=None, v=None, stream=None):
    """Keys and values of ``slots`` (int32 [T]; below 0: a zero row) as bf16
    [T, kv_heads, head_dim]; returns (k, v)."""
    T, dev = slots.shape[0], cache.device
    if not _ready(dev, stream):
        with _there(dev, stream):
            return cache_read(cache, slots, k=k, v=v)
    shape = (T, cache.kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=torch.bfloat16, device=dev) if k is None else k
    v = k.new_empty(shape) if v is None else v
    check(lib().qgemm_cache_read(cache.c, _ints("slots", slots, (T,), dev), T, k.data_ptr(),
                                 _heads("k", k, *shape, dev), v.data_ptr(), _heads("v", v, *shape, dev), _here(dev)),
          "qgemm_cache_read")
    return k, v


# ------------------------------------------------------------------ attention --
def attend(cache: Cache, q, q_offsets, kv_len, page_table, *, tree_mask=None, scale: float | None = None,
           max_q: int | None = None, out=None, lse=None, workspace: Workspace | None = None, stream=None):
    """Attention of each sequence's newest tokens over the cache (qgemm_attend).

    q: bf16 [T, q_heads, head_dim]; q_offsets int32 [B + 1]: sequence b's
    tokens are rows q_offsets[b] .. q_offsets[b + 1]; kv_len int32 [B]: its
    positions, those tokens' own (already written) included; page_table int32
    [B, max_pages].  tree_mask int64 [T, words]: bit j of a token's words says
    whether it sees its sequence's drafted token j (None: causal).  max_q: the
    most tokens of one sequence, at most 256; a sequence's tokens past it get
    no output (default: T, refused above 256).  scale:
    default head_dim ** -0.5.  lse: fp32 [T, q_heads] buffer for the log sums.
    Returns out (bf16
    [T, q_heads, head_dim]); rows that belong to no sequence are not written."""
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError("q: bf16 [tokens, q_heads, head_dim], page_table: int32 [batch, max_pages] wanted")
    if tree_mask is not None and (tree_mask.dim() != 2 or tree_mask.shape[1] == 0):
        raise ValueError("tree_mask: int64 [tokens, words], at least one word, wanted")
    T, Hq, D = q.shape
    B, pages = page_table.shape
    dev = cache.device
    if max_q is None:
        # the lengths are on the device: one sequence may have all tokens
        if T > QGEMM_ATTEND_MAX_Q:
            raise ValueError(f"more than {QGEMM_ATTEND_MAX_Q} tokens: max_q, the most of one sequence, wanted")
        max_q = T
    if not _ready(dev, stream):
        with _there(dev, stream):
            return attend(cache, q, q_offsets, kv_len, page_table, tree_mask=tree_mask, scale=scale, max_q=max_q,
                          out=out, lse=lse, workspace=workspace)
    out = q.new_empty((T, Hq, D)) if out is None else out
    a = qg_attend(ldq=_heads("q", q, T, Hq, cache.head_dim, dev), ldo=_heads("out", out, T, Hq, D, dev),
                  q=q.data_ptr(), out=out.data_ptr(), q_offsets=_ints("q_offsets", q_offsets, (B + 1,), dev),
                  kv_len=_ints("kv_len", kv_len, (B,), dev), page_table=_ints("page_table", page_table, (B, pages), dev),
                  q_heads=Hq, batch=B, tokens=T, max_pages=pages,
                  max_q=max_q,
                  scale=D ** -0.5 if scale is None else scale)
    if lse is not None:
        a.lse = _ints("lse", lse, (T, Hq), dev, torch.float32)
    if tree_mask is not None:
        a.mask_words = tree_mask.shape[1]
        a.tree_mask = _ints("tree_mask", tree_mask, (T, a.mask_words), dev, torch.int64)
    L = lib()
    workspace = workspace or Workspace(dev)
    wsp, wsb = workspace.scratch(L.qgemm_attend_workspace_size(cache.c, a))
    if workspace.buf.device != dev:
        raise ValueError(f"workspace: one on {dev} wanted")
    check(L.qgemm_attend(cache.c, a, wsp, wsb, _here(dev)), "qgemm_attend")
    return out
