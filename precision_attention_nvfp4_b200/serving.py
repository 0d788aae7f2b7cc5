"""Serving: rotary positions, a paged KV cache in FP8, attention over it.

  rotary_table(dim, ...)                -> RotaryTable (frequencies on the device)
  rotary(x, positions, table)           -> x rotated; transpose=True: its gradient
  kv_cache(pages, heads, page, d)       -> KvCache (zeroed)
  cache_write(cache, k, v, slots, ...)  quantises K (rotated) and V rows into the cache, rotates Q
  cache_read(cache, slots)              -> (k, v) rows in bf16
  tree_mask(parents)                    -> (words, depth) of a tree of drafted tokens
  cache_attention(q, cache, ...)        -> (out, lse): one query a sequence, a chunk of a prompt, a drafted tree

As in the rest of the package every call marshals torch tensors into the C ABI
and enqueues kernels on the current stream of the tensors' device. The results
carry no autograd graph: tensors that require a gradient are refused while
gradients are recorded, and dual tensors of forward mode. Caller's outputs
(out, lse, q_out) count as written in place.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Optional, Sequence, Tuple

import torch

from torch.autograd import forward_ad as _forward_ad
from torch.autograd.graph import increment_version as _written  # a caller's tensor was written in place

from . import _lib

__all__ = ["RotaryTable", "rotary_table", "rotary", "KvCache", "kv_cache", "cache_write", "cache_read", "tree_mask",
           "cache_attention"]

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}
_LAYOUTS = {"half": 0, "interleaved": 1}
_BF16 = torch.bfloat16
_rows, _table, _cache, _queries = _lib.ROWS.pack, _lib.ROTARY_TABLE.pack, _lib.KV_CACHE.pack, _lib.CACHE_QUERIES.pack


# the current stream's handle without a Stream object around it (4 of a small call's 12 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev: torch.device, where: str, *args) -> None:
    """Calls the library's ``where`` on ``dev`` and its current stream."""
    fn, index = getattr(_lib.load(), where), dev.index
    if torch.cuda.current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st:
        _lib.check(st, where)


def _rows3(x: torch.Tensor, name: str, dev: Optional[torch.device] = None) -> bytes:
    """[T, H, d] bf16 rows on a CUDA device, their channels contiguous."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{name}: expected a tensor [T, H, d]")
    st, sh, sd = x.stride()
    _check_rows(x, name, sd, dev)
    T, H, d = x.shape
    return _rows(x.data_ptr(), 1, T, H, d, 0, st, sh)


def _check_rows(x: torch.Tensor, name: str, sd: int, dev: Optional[torch.device]) -> None:
    if x.dtype != _BF16 or (sd != 1 and x.numel() > 0):
        raise ValueError(f"{name}: expected CUDA bf16 rows with contiguous channels")
    if x.device != dev if dev is not None else not x.is_cuda:
        raise ValueError(f"{name}: expected a tensor on {dev or 'a CUDA device'}")
    _no_graph(x, name)


def _no_graph(x: torch.Tensor, name: str) -> None:
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, but this call records no graph (detach it; the gradient of "
                         "rotary is rotary with transpose=True)")
    # (outside of a dual level, -1, there are no tangents: 1 us of a small call for its tensors)
    if getattr(_forward_ad, "_current_level", 0) >= 0 and _forward_ad.unpack_dual(x).tangent is not None:
        raise ValueError(f"{name}: carries a forward-mode tangent, which this call would drop (unpack it; rotary is "
                         "linear: the tangent of its result is rotary of the tangent)")


def _vector(x: torch.Tensor, name: str, n: int, dtype: torch.dtype, dev: torch.device) -> int:
    if (not isinstance(x, torch.Tensor) or x.dtype != dtype or x.device != dev or x.numel() != n
            or not x.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {n} elements on {dev}")
    return x.data_ptr()


def _writable(x: torch.Tensor, name: str) -> None:
    """Refuses a tensor whose elements share memory (an expanded one)."""
    extent = 1
    for stride, size in sorted((st, n) for st, n in zip(x.stride(), x.shape) if n > 1):
        if stride < extent:
            raise ValueError(f"{name}: its elements overlap in memory")
        extent = stride * (size - 1) + extent


def _span(x: torch.Tensor) -> Tuple[int, int]:
    a = x.data_ptr()
    return a, a + (sum((n - 1) * st for n, st in zip(x.shape, x.stride())) + 1) * x.element_size()


def _meet(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two tensors of one type and number of dimensions share an element: exactly where their strides agree
    (heads of one projection lie between one another's), by their spans where they do not."""
    if x.numel() == 0 or y.numel() == 0:
        return False
    (a, b), (c, d) = _span(x), _span(y)
    if a >= d or c >= b:
        return False
    return _layouts_meet(c - a, x.element_size(), tuple(x.shape), x.stride(), tuple(y.shape), y.stride())


@functools.lru_cache(maxsize=256)
def _layouts_meet(distance, size, shape_x, strides_x, shape_y, strides_y) -> bool:
    apart, odd = divmod(distance, size)
    if odd:
        return True
    dims = []  # stride, and the least and the most of the difference of the two indices
    for sx, sy, nx, ny in zip(strides_x, strides_y, shape_x, shape_y):
        if nx > 1 and ny > 1 and sx != sy:
            return True
        if nx > 1 or ny > 1:
            dims.append((sx if nx > 1 else sy, 1 - ny, nx - 1))
    dims.sort(reverse=True)

    def reach(left, i):  # is some index difference in dims[i:] worth `left` elements?
        if i == len(dims):
            return left == 0
        stride, low, high = dims[i]
        if stride == 0:
            return reach(left, i + 1)
        # what the dims after this one can make up for
        down, up = (sum(dim[0] * dim[k] for dim in dims[i + 1:]) for k in (1, 2))
        first, last = max(low, -((up - left) // stride)), min(high, (left - down) // stride)
        return any(reach(left - z * stride, i + 1) for z in range(first, last + 1))

    return reach(apart, 0)


def _apart(x: torch.Tensor, y: torch.Tensor, name: str) -> None:
    """x may be y itself, but not reach into it otherwise."""
    if not (x.data_ptr() == y.data_ptr() and x.stride() == y.stride() and x.shape == y.shape):
        if _meet(x, y):
            raise ValueError(f"{name}: overlaps an input")


def _disjoint(x: torch.Tensor, y: torch.Tensor, name: str) -> None:
    if x.numel() == 0 or y.numel() == 0:
        return
    (a, b), (c, d) = _span(x), _span(y)
    if a < d and c < b:
        raise ValueError(f"{name}: overlaps an input")


# ------------------------------------------------------------------------------------------------ rotary
@dataclasses.dataclass(frozen=True)
class RotaryTable:
    turns: torch.Tensor  # int64 [dim / 2]: turns a position, as 64-bit fractions
    dim: int             # rotated channels
    layout: str          # "half" or "interleaved"
    magnitude: float     # factor on the rotated channels

    def to(self, device) -> "RotaryTable":
        return dataclasses.replace(self, turns=self.turns.to(device))

    def _c(self, dev: torch.device) -> bytes:
        t = self.turns
        if t.device != dev:
            raise ValueError(f"table: expected on {dev}")
        return _table(t.data_ptr(), self.dim, _LAYOUTS[self.layout], self.magnitude)

    def __post_init__(self):
        if self.layout not in _LAYOUTS:
            raise ValueError("layout must be 'half' or 'interleaved'")
        if self.turns.dtype != torch.int64 or self.turns.numel() != self.dim // 2 or not self.turns.is_contiguous():
            raise ValueError("turns must be a contiguous int64 tensor of dim / 2 elements")


def rotary_table(dim: int, *, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
                 original_length: float = 8192.0, fast: Optional[float] = None, slow: Optional[float] = None,
                 magnitude: Optional[float] = None, device="cuda") -> RotaryTable:
    """The frequencies of a rotary embedding of the first ``dim`` channels (a
    multiple of 16). ``scaling``: "none", "linear", "ntk", "yarn" or
    "wavelength" (fpattn_rotary_turns in include/fpattn.h has the formulas),
    by ``factor`` from a model trained for ``original_length`` tokens;
    ``fast`` and ``slow`` bound the ramp of the last two (32 and 1 turns for
    yarn, 4 and 1 for wavelength); ``magnitude`` multiplies the rotated
    channels (default 1, for yarn 0.1 ln(factor) + 1)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if magnitude is not None and not magnitude > 0:
        raise ValueError("magnitude must be positive")
    spec = _lib.RotarySpec(int(dim), _SCALINGS[scaling], float(base), float(factor), float(original_length),
                           float(fast if fast is not None else (32.0 if scaling == "yarn" else 4.0)),
                           float(slow if slow is not None else 1.0), float(magnitude or 0.0))
    turns = torch.empty(max(int(dim) // 2, 1), dtype=torch.int64)
    mag = ctypes.c_float(0.0)
    _lib.check(_lib.load().fpattn_rotary_turns(ctypes.byref(spec), turns.data_ptr(), ctypes.byref(mag)),
               "fpattn_rotary_turns")
    return RotaryTable(turns.to(device), int(dim), layout, mag.value)


def rotary(x: torch.Tensor, positions: torch.Tensor, table: RotaryTable, *, transpose: bool = False,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotates the first ``table.dim`` channels of bf16 rows by their positions.

    x: [T, H, d] (tokens first, as a projection leaves them) with positions
    [T], or [B, H, N, d] (the layout of ``attention``) with positions [N] or
    [B, N], int64. Any strides that keep a row contiguous and 16-byte aligned.
    ``out`` may be ``x``. ``transpose`` applies the transposed rotation: given
    the gradient of the result it returns the gradient of x."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("x: expected [T, H, d] or [B, H, N, d]")
    _check_rows(x, "x", x.stride(-1), None)
    dev, caller_out = x.device, out is not None
    if not caller_out:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        if not isinstance(out, torch.Tensor) or out.shape != x.shape:
            raise ValueError("out: expected a tensor of x's shape")
        _check_rows(out, "out", out.stride(-1), dev)
        _writable(out, "out")
        _apart(out, x, "out")
    if x.dim() == 3:
        (T, H, d), B = x.shape, 1
        st, sh, _ = x.stride()
        xr = _rows(x.data_ptr(), 1, T, H, d, 0, st, sh)
        st, sh, _ = out.stride()
        orow = _rows(out.data_ptr(), 1, T, H, d, 0, st, sh)
    else:
        B, H, T, d = x.shape
        sb, sh, st, _ = x.stride()
        xr = _rows(x.data_ptr(), B, T, H, d, sb, st, sh)
        sb, sh, st, _ = out.stride()
        orow = _rows(out.data_ptr(), B, T, H, d, sb, st, sh)
    per_b = isinstance(positions, torch.Tensor) and positions.dim() == 2
    if per_b and (x.dim() != 4 or tuple(positions.shape) != (B, T)):
        raise ValueError("positions: expected [B, N]")
    pos = _vector(positions, "positions", B * T if per_b else T, torch.int64, dev)
    if out.numel() > 0:
        _launch(dev, "fpattn_rotary", xr, table._c(dev), pos, 1 if per_b else 0, 1 if transpose else 0, orow)
        if caller_out:
            _written(out)
    return out


# ------------------------------------------------------------------------------------------------ cache
@dataclasses.dataclass(frozen=True)
class KvCache:
    """A paged KV cache in FP8: a row (K or V of one token and KV head) is d
    E4M3 codes and a power-of-two exponent; value = E4M3(code) * 2^(exp - 127),
    exponent byte 255 marks a row of NaN."""
    k_codes: torch.Tensor  # uint8 [pages, H, page_size, d]
    v_codes: torch.Tensor  # uint8 [pages, H, page_size, d]
    exps: torch.Tensor     # uint8 [pages, H, 2, page_size]: K, V

    def __post_init__(self):
        k, v, e = self.k_codes, self.v_codes, self.exps
        for name, t in (("k_codes", k), ("v_codes", v), ("exps", e)):
            if (not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda or t.dim() != 4
                    or not t.is_contiguous() or t.device != k.device):
                raise ValueError(f"{name}: expected a contiguous 4-D uint8 tensor on one CUDA device")
        pages, heads, page, d = k.shape
        if v.shape != k.shape or tuple(e.shape) != (pages, heads, 2, page):
            raise ValueError("k_codes and v_codes must be [pages, H, page_size, d], exps [pages, H, 2, page_size]")

    @property
    def num_pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def num_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k_codes.shape[3]

    @property
    def device(self) -> torch.device:
        return self.k_codes.device

    def _c(self) -> bytes:
        k = self.k_codes
        return _cache(k.data_ptr(), self.v_codes.data_ptr(), self.exps.data_ptr(), *k.shape)


def kv_cache(num_pages: int, num_heads: int, page_size: int, head_dim: int, device="cuda") -> KvCache:
    """An empty cache (codes 0): page_size 16, 32, 64 or 128 tokens, head_dim
    64 or 128, 2 * head_dim + 2 bytes a token and head."""
    if page_size not in (16, 32, 64, 128) or head_dim not in (64, 128) or num_pages < 1 or num_heads < 1:
        raise ValueError("kv_cache: page_size must be 16, 32, 64 or 128, head_dim 64 or 128, counts positive")
    k, v = (torch.zeros((num_pages, num_heads, page_size, head_dim), dtype=torch.uint8, device=device)
            for _ in range(2))
    return KvCache(k, v, torch.zeros((num_pages, num_heads, 2, page_size), dtype=torch.uint8, device=device))


def cache_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
                rotary: Optional[RotaryTable] = None, positions: Optional[torch.Tensor] = None,
                q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                nonfinite_flag: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Quantises the K and V rows of T tokens into the cache, in one launch.

    k, v: bf16 [T, H, d] (slices of a fused projection will do). slots: int64
    [T], page * page_size + offset; a slot outside the cache (-1) writes
    nothing; the slots of a call are distinct. With ``rotary`` and
    ``positions`` (int64 [T]) K is rotated in fp32 before it is quantised, and
    ``q`` [T, any heads, d], when given, is rotated too and returned (in
    ``q_out``, which may be ``q``). ``nonfinite_flag``: device int32, set to 1
    when a row holds a non-finite value (that row is stored as NaN)."""
    dev = cache.device
    kr, vr = _rows3(k, "k", dev), _rows3(v, "v", dev)
    T, H, d = k.shape
    if v.shape != k.shape or H != cache.num_heads or d != cache.head_dim:
        raise ValueError("k, v: expected [T, H, d] with the cache's H and d")
    slot_p = _vector(slots, "slots", T, torch.int64, dev)
    tab = pos_p = None
    if rotary is not None:
        tab = rotary._c(dev)
        pos_p = _vector(positions, "positions", T, torch.int64, dev)
    elif positions is not None or q is not None:
        raise ValueError("positions and q go with a rotary table")
    qr = orow = None
    caller_q_out = False
    if q is not None:
        qr = _rows3(q, "q", dev)
        if q.shape[0] != T or q.shape[2] != d:
            raise ValueError("q: expected [T, heads, d] of k's T and d")
        caller_q_out = q_out is not None
        if not caller_q_out:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif not isinstance(q_out, torch.Tensor) or q_out.shape != q.shape:
            raise ValueError("q_out: expected a tensor of q's shape")
        orow = _rows3(q_out, "q_out", dev)
        if caller_q_out:
            _writable(q_out, "q_out")
            _apart(q_out, q, "q_out")
            # (q's heads may lie between those of k and v in one projection)
            if _meet(q_out, k) or _meet(q_out, v):
                raise ValueError("q_out: overlaps k or v")
        if q.shape[1] == 0:
            qr = orow = None
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    flag_p = None
    if nonfinite_flag is not None:
        flag_p = _vector(nonfinite_flag, "nonfinite_flag", 1, torch.int32, dev)
    if T > 0:
        _launch(dev, "fpattn_cache_write", cache._c(), kr, vr, slot_p, tab, pos_p, qr, orow, flag_p)
        if caller_q_out:
            _written(q_out)
    return q_out


def cache_read(cache: KvCache, slots: torch.Tensor, *,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The K and V rows at ``slots`` (int64 [T]) in bf16, exactly: (k, v), each
    [T, H, d]; zeros for a slot outside the cache. ``out``: a pair of tensors
    to fill, of any strides that keep a row contiguous (a transposed view of
    the [H, N, d] layout of ``attention``, say). Rows that are read and
    written again (the accepted ones of a drafted tree, moved) keep their
    values."""
    dev = cache.device
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots: expected a 1-D tensor")
    T, H, d = slots.shape[0], cache.num_heads, cache.head_dim
    slot_p = _vector(slots, "slots", T, torch.int64, dev)
    if out is None:
        k = slots.new_empty((T, H, d), dtype=_BF16)
        v = torch.empty_like(k)
    else:
        k, v = out
        for name, t in (("out[0]", k), ("out[1]", v)):
            if not isinstance(t, torch.Tensor) or tuple(t.shape) != (T, H, d):
                raise ValueError(f"{name}: expected [T, H, d] = {(T, H, d)}")
            _writable(t, name)
    kr, vr = _rows3(k, "out[0]", dev), _rows3(v, "out[1]", dev)
    if out is not None and _meet(k, v):
        raise ValueError("out: the two tensors are the same memory, or share some")
    if T > 0:
        _launch(dev, "fpattn_cache_read", cache._c(), slot_p, kr, vr)
        if out is not None:
            _written(k)
            _written(v)
    return k, v


# ------------------------------------------------------------------------------------------------ attention
def tree_mask(parents: Sequence[int], device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """What the tokens of a drafted tree see of one another (host planner):
    parents[i] < i is the token before token i, -1 for a first one. Returns
    (words int64 [n, ceil(n / 64)] for cache_attention, depth int64 [n]: a
    token's position is the number of cached tokens before the tree plus its
    depth)."""
    p = torch.tensor([int(x) for x in parents], dtype=torch.int32)
    n = p.numel()
    if n < 1:
        raise ValueError("parents: expected at least one token")
    words = torch.zeros((n, (n + 63) // 64), dtype=torch.int64)
    depth = torch.zeros(n, dtype=torch.int32)
    _lib.check(_lib.load().fpattn_tree_mask(p.data_ptr(), n, words.shape[1], words.data_ptr(), depth.data_ptr()),
               "fpattn_tree_mask")
    return words.to(device), depth.to(device=device, dtype=torch.int64)


def cache_attention(q: torch.Tensor, cache: KvCache, page_table: torch.Tensor, lengths: torch.Tensor, *,
                    q_start: Optional[torch.Tensor] = None, max_queries: Optional[int] = None,
                    tree_mask: Optional[torch.Tensor] = None, causal: bool = True, softmax_scale: float = 0.0,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True):
    """softmax(q K^T * scale) V over the cached tokens of every sequence.

    q: bf16 [B, T, Hq, d] (T queries for every sequence), or [rows, Hq, d] with
    ``q_start`` (int32 [B + 1]): the queries of sequence b are rows q_start[b]
    .. q_start[b + 1] - 1, at most ``max_queries`` of them (default: all rows;
    a close bound saves planning; of a sequence with more, the rows behind are
    left as they were or filled). Hq is a multiple of the cache's heads.
    page_table: int32 [B, max_pages]; lengths: int32 [B], cached tokens of each
    sequence, those of these queries included (write them first).

    Query i of n of a sequence of L tokens is its token L - n + i and sees the
    tokens up to itself; with ``tree_mask`` (int64 words [B, T, W], [T, W] for
    one tree shared by all, or [rows, W] with q_start; see the function
    tree_mask) the tokens before L - n and those whose bit is set; with
    causal=False every one.

    Returns (out bf16 of q's shape, lse float32 of q's shape without d, or
    None). Rows behind the last sequence are left as they are; a query that
    sees no token gets out = 0, lse = -inf."""
    dev = cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != (4 if q_start is None else 3):
        raise ValueError("q: expected [B, T, Hq, d], or [rows, Hq, d] with q_start")
    _check_rows(q, "q", q.stride(-1), dev)
    if (not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.dtype != torch.int32
            or page_table.device != dev or page_table.shape[1] < 1
            or (page_table.stride(1) != 1 and page_table.shape[1] > 1)):
        raise ValueError(f"page_table: expected int32 [B, max_pages] on {dev}, its rows contiguous")
    B = page_table.shape[0]
    hq, d = q.shape[-2:]
    if d != cache.head_dim or hq % cache.num_heads != 0:
        raise ValueError("q: expected the cache's d and a multiple of its heads")
    len_p = _vector(lengths, "lengths", B, torch.int32, dev)
    if q_start is None:
        if q.shape[0] != B:
            raise ValueError("q and page_table must have one B")
        T = q.shape[1]
        if max_queries not in (None, T):
            raise ValueError("max_queries goes with q_start")
        sb, st, sh, _ = q.stride()
        rows = (q.data_ptr(), B, T, hq, d, sb, st, sh)
        start_p = None
    else:
        T = q.shape[0] if max_queries is None else int(max_queries)
        if T < 1 and q.shape[0] > 0:
            raise ValueError("max_queries must be at least 1")
        T = min(T, q.shape[0])
        rows = (q.data_ptr(), 1, q.shape[0], hq, d, 0, q.stride(0), q.stride(1))
        start_p = _vector(q_start, "q_start", B + 1, torch.int32, dev)
    tree_p, words, tree_b = None, 0, 0
    if tree_mask is not None:
        if (not isinstance(tree_mask, torch.Tensor) or tree_mask.dtype != torch.int64 or tree_mask.device != dev
                or tree_mask.dim() < 2 or not tree_mask.is_contiguous() or tree_mask.shape[-1] * 64 < T):
            raise ValueError(f"tree_mask: expected contiguous int64 words [..., W] on {dev} with 64 W >= the queries")
        words = tree_mask.shape[-1]
        lead = tuple(tree_mask.shape[:-1])
        if q_start is not None:
            if lead != (q.shape[0],):
                raise ValueError("tree_mask: expected [rows, W]")
        elif lead == (B, T):
            tree_b = T * words
        elif lead != (T,):
            raise ValueError("tree_mask: expected [B, T, W] or [T, W]")
        tree_p = tree_mask.data_ptr()
    written = []
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif (not isinstance(out, torch.Tensor) or out.dtype != torch.bfloat16 or out.device != dev
          or out.shape != q.shape or not out.is_contiguous()):
        raise ValueError(f"out: expected a contiguous bf16 tensor of q's shape on {dev}")
    else:
        _no_graph(out, "out")
        _disjoint(out, q, "out")
        written.append(out)
    if lse is None:
        if return_lse:
            lse = q.new_empty(q.shape[:-1], dtype=torch.float32)
    elif (not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or lse.device != dev
          or lse.shape != q.shape[:-1] or not lse.is_contiguous()):
        raise ValueError(f"lse: expected a contiguous float32 tensor of q's shape without d on {dev}")
    else:
        _no_graph(lse, "lse")
        written.append(lse)
        _disjoint(lse, q, "lse")
        if out.numel() > 0 and lse.numel() > 0 and _span(out)[0] < _span(lse)[1] and _span(lse)[0] < _span(out)[1]:
            raise ValueError("out and lse overlap")
    if out.numel() == 0 or B == 0:
        return out, lse
    desc = _queries(*rows, start_p or 0, B, T, page_table.data_ptr(), page_table.shape[1], page_table.stride(0), len_p,
                    1 if causal else 0, tree_p or 0, words, tree_b, softmax_scale)
    need = _workspace_bytes(dev.index, B, T, hq, page_table.shape[1], q_start is None, *cache.k_codes.shape)
    # allocated for this call: two calls, or two captured graphs, never share one
    ws = cache.exps.new_empty(need)
    _launch(dev, "fpattn_cache_attention", cache._c(), desc, out.data_ptr(), None if lse is None else lse.data_ptr(),
            ws.data_ptr(), need)
    for x in written:
        _written(x)
    return out, lse


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(device, B, T, hq, max_pages, uniform, pages, heads, page, d) -> int:
    """fpattn_cache_attention_workspace of calls of these sizes (it follows no pointer)."""
    p = 256
    rows = (p, B if uniform else 1, T, hq, d, 0, 8 * hq, 8)
    with torch.cuda.device(device):
        return _lib.load().fpattn_cache_attention_workspace(
            _cache(p, p, p, pages, heads, page, d),
            _queries(*rows, 0 if uniform else p, B, T, p, max_pages, max_pages, p, 1, 0, 0, 0, 0.0))
