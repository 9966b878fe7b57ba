"""Python side of the decode calls of include/st.h: one step of a beam decode
over an int8 paged cache. Argument marshalling and checks only, as in the
package; every step runs in the library's CUDA kernels.

A step, for R rows (beams) with `have` tokens each:

    slots, sources, start, lens, report = st_kv_plan(table, have, add, num_blocks, block_size, T)
    assert report[2:].tolist() == [0, 0]                           # else some rows got no slots: see st_kv_plan
    st_kv_append(cache, k, v, slots, sources)                      # per layer
    out = st_kv_attend(cache, q, table, start, lens, max_q)        # per layer
    scores, parents, tokens, finished = st_beam_select(logits, scores, keep)
    table, have = (x.flatten(0, 1) for x in st_beam_reorder([table.view(B, K, -1), lens.view(B, K)], parents))

Tensors are on the current CUDA device; work goes to the current stream, or to
`stream`. Nothing waits. There are no backward passes: tensors that require a
gradient are refused outside torch.no_grad(). Call each function once before
capturing it in a graph.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Sequence

import torch

from . import _BeamExtras, _KvCache, _check, _stream, lib

ST_BF16, ST_F16, ST_F32 = 0, 1, 2
_DTYPES = {torch.bfloat16: ST_BF16, torch.float16: ST_F16, torch.float32: ST_F32}
_HALVES = (torch.bfloat16, torch.float16)
_I8, _I32, _I64, _F32, _BOOL = torch.int8, torch.int32, torch.int64, torch.float32, torch.bool


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _wrong(x, dtype, shape, name: str):
    _need(isinstance(x, torch.Tensor) and x.dtype == dtype, f"{name} must be a tensor of {dtype}")
    _need(x.shape == shape, f"{name} must have shape {tuple(shape)}, not {tuple(x.shape)}")
    _need(False, f"{name} must be contiguous")


def _array(x: torch.Tensor, dtype, shape, name: str) -> int:
    """The address of a dense tensor of this type and shape."""
    if not isinstance(x, torch.Tensor) or x.dtype is not dtype or x.shape != shape or not x.is_contiguous():
        _wrong(x, dtype, shape, name)
    if dtype is _F32 and (x.requires_grad or x.is_neg()):
        _not_plain(x, name)
    return x.data_ptr()


try:  # torch.empty on the current device with its cost halved (what torch's own generated code calls)
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    def _empty_strided_cuda(shape, strides, dtype):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")


def _empty(shape, dtype, stream):
    """A new tensor on the current device, in the allocator's books of the stream that will use it."""
    shape, strides, n = tuple(shape), [], 1
    for size in shape[::-1]:
        strides.append(n)
        n *= size or 1
    strides = tuple(strides[::-1])
    if stream is None:
        return _empty_strided_cuda(shape, strides, dtype)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        return _empty_strided_cuda(shape, strides, dtype)


_TOP, _FAR = (1 << 31) - 1, (1 << 63) - 1  # the marshalling would cut larger numbers to their low bits


def _too_far(*numbers):
    _need(False, f"sizes and numbers must be within {64 if max(map(abs, numbers)) > _FAR else 32} bits, not {max(numbers, key=abs)}")


def _not_plain(x: torch.Tensor, name: str):
    """For a tensor that requires a gradient (what the calls write is not recorded, so that it would be lost) or whose
    memory does not hold its values."""
    _need(not (x.requires_grad and torch.is_grad_enabled()),
          f"{name} requires a gradient and the decode calls have none: make them under torch.no_grad()")
    _need(not (x.is_neg() or x.is_conj()), f"{name} is a view that negates or conjugates: resolve it first (resolve_neg, resolve_conj)")


def _on_gpu(x: torch.Tensor, name: str):
    if not x.is_cuda:
        raise ValueError(f"{name} must be on the current CUDA device")


def _empty1(n, dtype, stream):
    return _empty_strided_cuda((n,), (1,), dtype) if stream is None else _empty((n,), dtype, stream)


def _empty2(n, m, dtype, stream):
    return _empty_strided_cuda((n, m), (m, 1), dtype) if stream is None else _empty((n, m), dtype, stream)


@functools.lru_cache(maxsize=256)
def _select_workspace(B: int, K: int, V: int, keep: int) -> int:
    need = ctypes.c_int64(0)
    _check(lib().st_beam_select_workspace(B, K, V, keep, ctypes.byref(need)), "st_beam_select_workspace")
    return need.value


@functools.lru_cache(maxsize=256)
def _attend_workspace(kv_heads: int, size: int, dim: int, T: int, heads: int, R: int, max_q: int, max_len: int) -> int:
    need = ctypes.c_int64(0)
    c = _KvCache(None, None, None, None, 1, kv_heads, size, dim)  # (the number of blocks does not matter)
    _check(lib().st_kv_attend_workspace(ctypes.byref(c), T, heads, R, max_q, max_len, ctypes.byref(need)),
           "st_kv_attend_workspace")
    return need.value


def _room(workspace) -> int:
    """Bytes of a workspace given: all of them behind its address."""
    _need(isinstance(workspace, torch.Tensor) and workspace.is_contiguous(), "workspace must be a contiguous tensor")
    return workspace.numel() * workspace.element_size()


class KvCache:
    """An int8 paged cache over caller-owned tensors: k, v int8 [num_blocks,
    kv_heads, block_size, head_dim] and their scales float32 [num_blocks,
    kv_heads]. KvCache.empty allocates one. The calls read the tensors' addresses here, so its fields do not change:
    other tensors need another KvCache."""

    __slots__ = ("_tensors", "_shape", "_c", "_ref")

    def __init__(self, k, v, k_scale, v_scale):
        shape = k.shape
        if len(shape) != 4:
            raise ValueError("k must be [num_blocks, kv_heads, block_size, head_dim]")
        scales = shape[:2]
        c = _KvCache(_array(k, _I8, shape, "k"), _array(v, _I8, shape, "v"), _array(k_scale, _F32, scales, "k_scale"),
                     _array(v_scale, _F32, scales, "v_scale"), *shape)
        self._tensors = k, v, k_scale, v_scale
        self._shape = shape
        self._c = c
        self._ref = ctypes.byref(c)

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    num_blocks = property(lambda self: self._shape[0])
    kv_heads = property(lambda self: self._shape[1])
    block_size = property(lambda self: self._shape[2])
    head_dim = property(lambda self: self._shape[3])

    @classmethod
    def empty(cls, num_blocks: int, kv_heads: int, block_size: int, head_dim: int, device="cuda"):
        shape = (num_blocks, kv_heads, block_size, head_dim)
        return cls(torch.zeros(shape, dtype=torch.int8, device=device), torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:2], device=device), torch.zeros(shape[:2], device=device))


def _vectors(x: torch.Tensor, heads: Optional[int], dim: int, name: str):
    """[T, heads, dim] of 16-bit floats with dense vectors; its address and strides."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _HALVES:
        raise ValueError(f"{name} must be a tensor of bfloat16 or float16")
    shape = x.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [T, {'heads' if heads is None else heads}, {dim}], not {tuple(shape)}")
    if x.requires_grad or x.is_neg():
        _not_plain(x, name)
    token, head, one = x.stride()
    if one != 1:
        raise ValueError(f"{name} must have dense vectors")
    # strides of extents of one say nothing
    return x.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def st_kv_plan(table: torch.Tensor, have: torch.Tensor, add: torch.Tensor, num_blocks: int, block_size: int, T: int,
               slots: Optional[torch.Tensor] = None, sources: Optional[torch.Tensor] = None,
               row_start: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
               report: Optional[torch.Tensor] = None, stream=None):
    """Blocks for the rows' next tokens: table int32 [R, max_blocks] (written in
    place), have and add int32 [R], room for T new tokens. Returns (slots int64
    [T], sources int32 [T], row_start int32 [R + 1], lens int32 [R], report
    int32 [4]); see st_kv_plan in include/st.h for what they hold. Rows that
    could not be served (report[2] of them) have lens -1 and no slots: append
    the others' tokens, free blocks, and plan again with have = torch.where(lens
    < 0, have, lens) and no tokens for the rows served."""
    if table.dim() != 2 or T < 0:
        raise ValueError("table must be [R, max_blocks], and T not negative")
    R, width = table.shape
    if not (R <= _TOP and width <= _TOP and -_TOP <= num_blocks <= _TOP and -_TOP <= block_size <= _TOP):
        _too_far(R, width, num_blocks, block_size)
    pt, ph, pa = _array(table, _I32, (R, width), "table"), _array(have, _I32, (R,), "have"), _array(add, _I32, (R,), "add")
    _on_gpu(table, "table")

    def made(x, n, dtype, name):
        if x is None:
            x = _empty1(n, dtype, stream)
            return x, x.data_ptr()
        return x, _array(x, dtype, (n,), name)

    slots, p0 = made(slots, T, _I64, "slots")
    sources, p1 = made(sources, T, _I32, "sources")
    row_start, p2 = made(row_start, R + 1, _I32, "row_start")
    lens, p3 = made(lens, R, _I32, "lens")
    report, p4 = made(report, 4, _I32, "report")
    status = lib().st_kv_plan(pt, ph, pa, R, width, num_blocks, block_size, T, p0, p1, p2, p3, p4, _stream(stream))
    if status:
        _check(status, "st_kv_plan")
    return slots, sources, row_start, lens, report


def st_kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                 sources: Optional[torch.Tensor] = None, stream=None):
    """Quantise keys and values [T, kv_heads, head_dim] (bfloat16 or float16,
    any multiple-of-8 strides) into the cache's slots int64 [T]."""
    _, heads, _, dim = cache._shape
    pk, kt, kh = _vectors(k, heads, dim, "k")
    pv, vt, vh = _vectors(v, heads, dim, "v")
    T = k.shape[0]
    if v.shape[0] != T or v.dtype is not k.dtype:
        raise ValueError("k and v must have the same tokens and type")
    _check(lib().st_kv_append(cache._ref, pk, pv, _DTYPES[k.dtype], T, kt, kh, vt, vh,
                              _array(slots, _I64, (T,), "slots"),
                              None if sources is None else _array(sources, _I32, (T,), "sources"),
                              _stream(stream)), "st_kv_append")


def st_kv_attend(cache: KvCache, q: torch.Tensor, table: torch.Tensor, row_start: torch.Tensor, lens: torch.Tensor,
                 max_q: int, max_len: Optional[int] = None, scale: Optional[float] = None, causal: bool = True,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of query tokens q [T, q_heads, head_dim] over the rows' cached
    tokens (table int32 [R, max_blocks], row_start int32 [R + 1], lens int32 [R]).
    max_q and max_len bound a row's query and cached tokens; scale defaults to
    head_dim ** -0.5. `out` rows behind row_start[R] are left as they were (a new `out` holds anything there)."""
    _, kv_heads, size, dim = cache._shape
    pq, qt, qh = _vectors(q, None, dim, "q")
    T, heads, _ = q.shape
    if table.dim() != 2:
        raise ValueError("table must be [R, max_blocks]")
    R, width = table.shape
    if max_len is None:
        max_len = width * size
    if not (R <= _TOP and width <= _TOP and heads <= _TOP and -_TOP <= max_q <= _TOP and -_FAR <= max_len <= _FAR):
        _too_far(R, width, heads, max_q, max_len)
    pt = _array(table, _I32, (R, width), "table")
    ps, pl = _array(row_start, _I32, (R + 1,), "row_start"), _array(lens, _I32, (R,), "lens")
    if out is None:
        _on_gpu(q, "q")
        if stream is None:
            out = _empty_strided_cuda((T, heads, dim), (heads * dim, dim, 1), q.dtype)
        else:
            out = _empty((T, heads, dim), q.dtype, stream)
        po, ot, oh = out.data_ptr(), heads * dim, dim
    else:
        _need(out.shape == q.shape and out.dtype == q.dtype, "out must be like q")
        po, ot, oh = _vectors(out, heads, dim, "out")
        # tokens apart from each other, and heads: one inside the other either way
        _need((T <= 1 or ot >= dim) and (heads <= 1 or oh >= dim) and
              (T <= 1 or heads <= 1 or ot >= (heads - 1) * oh + dim or oh >= (T - 1) * ot + dim), "out's vectors must not overlap")
    room = 0 if workspace is None else _room(workspace)
    need = _attend_workspace(kv_heads, size, dim, T, heads, R, max_q, max_len)
    if workspace is None and need:
        workspace, room = _empty1(need, torch.uint8, stream), need
    status = lib().st_kv_attend(cache._ref, pq, _DTYPES[q.dtype], T, heads, qt, qh, pt, width, ps, pl, R, max_q, max_len,
                                dim ** -0.5 if scale is None else scale, int(causal), po, ot, oh,
                                None if workspace is None else workspace.data_ptr(), room, _stream(stream))
    if status:
        _check(status, "st_kv_attend")
    return out


def st_beam_select(logits: torch.Tensor, scores: torch.Tensor, keep: int, allow: Optional[torch.Tensor] = None,
                   finished: Optional[torch.Tensor] = None, end_token: int = 0,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """The `keep` best (beam, token) pairs of each request from logits [B, K, V]
    (bfloat16, float16 or float32; vocabulary dense, beams evenly spaced) and
    scores float32 [B, K]. `allow` int32 [B, K, ceil(V / 32)] holds a bit per
    token (expanded dimensions are read as they are); `finished` bool [B, K]
    marks beams that only repeat end_token. Returns (scores [B, keep], parents int32, tokens
    int32, finished bool or None); missing pairs are -inf, -1, -1."""
    kind = _DTYPES.get(logits.dtype)
    if kind is None or logits.dim() != 3:
        raise ValueError("logits must be [B, K, V] bfloat16, float16 or float32")
    if logits.requires_grad or logits.is_neg():
        _not_plain(logits, "logits")
    B, K, V = logits.shape
    if not (B <= _TOP and K <= _TOP and V <= _TOP and -_TOP <= keep <= _TOP and -_TOP <= end_token <= _TOP):
        _too_far(B, K, V, keep, end_token)
    request, beam, one = logits.stride()
    if V > 1 and one != 1:
        raise ValueError("logits must have a dense vocabulary")
    stride = beam if K > 1 else request if B > 1 else V
    if B > 1 and K > 1 and request != K * stride:
        raise ValueError("logits' beams must be evenly spaced")
    pscores = _array(scores, _F32, (B, K), "scores")
    ex = out_finished = None
    if allow is not None or finished is not None:
        ex = _BeamExtras()
        if allow is not None:
            _need(allow.dtype in (torch.int32, torch.uint32) and tuple(allow.shape) == (B, K, (V + 31) // 32),
                  "allow must be int32 [B, K, ceil(V / 32)]")
            _need(allow.shape[2] <= 1 or allow.stride(2) == 1, "allow must have dense words")
            ex.allow, ex.allow_request_stride, ex.allow_beam_stride = allow.data_ptr(), allow.stride(0), allow.stride(1)
        if finished is not None:
            pf = _array(finished, _BOOL, (B, K), "finished")
            _on_gpu(finished, "finished")
            out_finished = _empty2(B, keep, torch.bool, stream)
            ex.finished, ex.out_finished = pf, out_finished.data_ptr()
            ex.end_token = end_token
    room = 0 if workspace is None else _room(workspace)
    _on_gpu(logits, "logits")
    need = _select_workspace(B, K, V, keep)
    out_scores = _empty2(B, keep, torch.float32, stream)
    out_parents, out_tokens = _empty2(B, keep, _I32, stream), _empty2(B, keep, _I32, stream)
    if workspace is None and need:
        workspace, room = _empty1(need, torch.uint8, stream), need
    _check(lib().st_beam_select(logits.data_ptr(), kind, stride, pscores, B, K, V, keep, out_scores.data_ptr(), out_parents.data_ptr(), out_tokens.data_ptr(),
                                None if ex is None else ctypes.byref(ex),
                                None if workspace is None else workspace.data_ptr(), room, _stream(stream)),
           "st_beam_select")
    return out_scores, out_parents, out_tokens, out_finished


def _rows(x: torch.Tensor, dim: int, what: str):
    """The stride between the beams of a tensor whose requests and beams are
    dimensions dim - 1 and dim, evenly spaced, with dense rows behind them."""
    shape, stride = x.shape, x.stride()
    if not x.is_contiguous():
        want = 1
        for n, s in zip(reversed(shape[dim + 1:]), reversed(stride[dim + 1:])):
            if n != 1 and s != want:
                raise ValueError(f"{what} must have dense rows")
            want *= n
        if shape[dim - 1] > 1 and shape[dim] > 1 and stride[dim - 1] != shape[dim] * stride[dim]:
            raise ValueError(f"{what} must have evenly spaced beams")
    return stride[dim] if shape[dim] > 1 else stride[dim - 1] if shape[dim - 1] > 1 else 0


def st_beam_reorder(states: Sequence[torch.Tensor], parents: torch.Tensor, out: Optional[Sequence[torch.Tensor]] = None,
                    beam_dim: int = 1, stream=None):
    """The states of the chosen beams: for each tensor, out[b, j] = states[b,
    parents[b, j]] (zeros where the parent is -1) with parents int32 [B, keep].
    The request and beam dimensions are beam_dim - 1 and beam_dim; beam_dim = 2
    takes tensors of several layers [layers, B, K, ...]. Up to 16 tensors go in
    one launch; `out` must not overlap them."""
    if parents.dim() != 2 or beam_dim not in (1, 2) or not len(states):
        raise ValueError("parents must be [B, keep], beam_dim 1 or 2, and states not empty")
    B, keep = parents.shape
    K = states[0].shape[beam_dim] if states[0].dim() > beam_dim else -1
    if not (B <= _TOP and K <= _TOP and keep <= _TOP):
        _too_far(B, K, keep)
    pp = _array(parents, _I32, (B, keep), "parents")
    rows = B * K
    made, words = [], []  # words: the eight of each st_beam_state
    for i, x in enumerate(states):
        shape = x.shape
        if len(shape) <= beam_dim or shape[beam_dim - 1] != B or shape[beam_dim] != K:
            raise ValueError(f"state {i} must have {B} requests of {K} beams at dimension {beam_dim}")
        if x.requires_grad or x.is_neg() or x.is_conj():
            _not_plain(x, f"state {i}")
        size = x.element_size()
        if out is None and beam_dim == 1 and stream is None and rows and x.is_contiguous():  # the usual case
            _on_gpu(x, f"state {i}")
            n = x.numel() // rows
            y = _empty_strided_cuda((B, keep, *shape[2:]), (keep * n, n, *x.stride()[2:]), x.dtype)
            made.append(y)
            n *= size
            words += (x.data_ptr(), y.data_ptr(), n, n, n, 1, 0, 0)
            continue
        new = shape[:beam_dim] + (keep,) + shape[beam_dim + 1:]
        step = _rows(x, beam_dim, f"state {i}")
        if out is None:
            _on_gpu(x, f"state {i}")
            y = _empty(new, x.dtype, stream)
        else:
            y = out[i]
            if y.shape != new or y.dtype != x.dtype:
                raise ValueError(f"out {i} must be {tuple(new)} {x.dtype}")
            _not_plain(y, f"out {i}")
        layers = (shape[0], size * x.stride(0), size * y.stride(0)) if beam_dim == 2 else (1, 0, 0)
        words += (x.data_ptr(), y.data_ptr(), size * math.prod(shape[beam_dim + 1:]), size * step,
                  size * _rows(y, beam_dim, f"out {i}"), *layers)
        made.append(y)
    status = lib().st_beam_reorder((ctypes.c_int64 * len(words))(*words), len(states), pp, B, K, keep, _stream(stream))
    if status:
        _check(status, "st_beam_reorder")
    return made


def st_decode_check(stream=None) -> int:
    """Synchronize and return the decode calls' device-side status (ST_OK or ST_ERR_DEVICE)."""
    return lib().st_decode_check(_stream(stream))
