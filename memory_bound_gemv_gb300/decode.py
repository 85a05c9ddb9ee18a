"""Binding of the decode-step operators: what stands between the GEMVs of a step.

``PagedKV`` describes a paged key-value cache once; the calls then take it with
the step's tensors: ``gemv_rope_append`` (rotary positions with several axes,
and the append), ``gemv_attn_paged`` (attention of one new token per
sequence), ``gemv_kv_evict_plan`` / ``gemv_kv_evict_apply`` (eviction by
accumulated attention weight; ``gemv_kv_evict`` does both) and
``gemv_norm_residual`` (the norms around a block with its gate and the
residual).  As in the rest of the package: argument checks and marshalling
only, no CPU fallback, C errors raised as ``GemvError``.  Lengths, slots and
page numbers stay on the device; one out of range is skipped and reported by
``gemv_get_device_error``.
"""

from __future__ import annotations

import ctypes
import math
import struct
import threading
import warnings
import weakref
from typing import Optional, Sequence

import memory_bound_gemv_gb300 as _mbg

ELEM_F32, ELEM_F16, ELEM_BF16 = 0, 1, 5
_ATTN_COUNTER_BYTES = 8192  # GEMV_ATTN_COUNTER_BYTES
NORM_LAYER, NORM_POST, NORM_UNIT_OFFSET = 1, 2, 4

torch = _Tensor = None  # looked up by _need_torch: importing the package does not import torch
_elems = {}
_quick = None  # csrc/binding.cpp


def _need_torch():
    global torch, _Tensor, _quick
    if torch is None:
        import torch as module

        _elems.update({module.float32: ELEM_F32, module.float16: ELEM_F16, module.bfloat16: ELEM_BF16})
        _quick = _load_binding(module)
        torch, _Tensor = module, module.Tensor


class _NoBinding:
    """Stands in for the compiled form: every call is left to the Python form."""

    def __getattr__(self, name):
        return lambda *args: -1


def _load_binding(module):
    """The compiled form of the calls below for the installed torch; it answers -1 where a call is not of the
    common kind, and the Python form then checks it and says why.  One that is missing or was made for another
    torch is built anew; where that cannot be, the Python form takes all calls, with a warning."""
    import importlib.machinery
    import importlib.util

    from . import build

    lib = _mbg.lib()
    try:
        if not build.binding_up_to_date():
            build.build()
        loader = importlib.machinery.ExtensionFileLoader("_mbgbinding", build.BINDING)
        binding = importlib.util.module_from_spec(importlib.util.spec_from_loader("_mbgbinding", loader))
        loader.exec_module(binding)
        if binding.torch_version != module.__version__:
            raise ImportError(f"made for torch {binding.torch_version}, this is {module.__version__}")
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"decode-step calls check their arguments in Python, a few microseconds slower each: {e}")
        return _NoBinding()
    binding.use(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
        "gemv_attn_paged", "gemv_rope_append", "gemv_kv_evict_plan", "gemv_kv_evict_apply", "gemv_norm_residual")))
    return binding


class _KvStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int64), ("scores", ctypes.c_void_p), ("stamps", ctypes.c_void_p),
                ("elem", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _declare(L):
    vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int
    sig = {
        "gemv_attn_paged": [vp, vp, vp],
        "gemv_kv_evict_plan": [vp, vp, i32, i32, i32, vp, i64, vp, vp],
        "gemv_kv_evict_apply": [vp, vp, i64, vp, vp, i32, vp],
        "gemv_rope_append": [vp, vp, vp],
        "gemv_norm_residual": [vp, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = st
    L.gemv_attn_paged_workspace.argtypes = [vp, i32, i32]
    L.gemv_attn_paged_workspace.restype = ctypes.c_size_t
    L.gemv_capture_id.argtypes = [vp]
    L.gemv_capture_id.restype = ctypes.c_uint64
    return L


# The argument structures of include/gemv.h, packed in one go.
_ATTN = struct.Struct("PqqPqqPPPPNiif0q")
_ROPE = struct.Struct("PqqPqqPqqPqqPqPPPPPiiiiii0q")
_NORM = struct.Struct("PqiPqiPqiPqiPqiPqiPqiPqiqqffI0q")


def _operand(t, name, dtype, shape, index):
    """Strides of a tensor of this type and shape, on CUDA device `index`, whose last dimension is contiguous."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape:
        strides = t.stride()
        if not strides or strides[-1] == 1 or shape[-1] <= 1:
            return strides
    _refuse(t, name, dtype, shape, index)


def _refuse(t, name, dtype, shape, index):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"the last dimension of {name} must be contiguous")


def _dense(t, name, dtype, shape, index):
    """Address of a contiguous tensor."""
    _operand(t, name, dtype, shape, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _count(value, name, least):
    """Refuses counts that the library's 32-bit arguments cannot hold (ctypes would cut them off)."""
    if not least <= value < 2 ** 31:
        raise ValueError(f"{name} must be at least {least} and below 2^31")


def _on(stream):
    """Context in which tensors belong to the stream that a call runs on."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)  # None: no change


class _Workspace:
    """Scratch memory of ``gemv_attn_paged`` calls that follow each other: (address, bytes, tensor).

    A call with weights is two launches: ``lock`` keeps those of another thread from coming between them."""

    def __init__(self, tensor):
        self._values = tensor.data_ptr(), tensor.numel(), tensor
        self.lock = threading.Lock()

    def __getitem__(self, i):
        return self._values[i]


# Workspaces that some handle holds, by device, stream, capture and size.
_shared = weakref.WeakValueDictionary()
_shared_lock = threading.Lock()


class PagedKV:
    """A paged key-value cache, described once.

    k, v: [pages, page_size, kv_heads, head_dim], float16 or bfloat16, any
    strides with a contiguous last dimension (a pool laid out [pages, kv_heads,
    page_size, head_dim] is passed transposed).  page_table: int32 [batch,
    max_pages], the pages of each sequence in order; entries behind a
    sequence's last page are never read.  scores (float32) and stamps (int32),
    [batch, kv_heads, max_pages * page_size]: the attention weight each slot
    has gathered and the number of its token, for eviction.

    The tensors are kept; their contents may change, their storage not.  For
    ``gemv_attn_paged`` there is a workspace per stream, and one per stream of
    each CUDA graph that calls are captured into.  Handles that need as much
    (a model's layers) share them, as calls on one stream follow each other.  A
    handle keeps what it has used until it is gone or ``release_workspaces`` is called.
    """

    def __init__(self, k, v, page_table, scores=None, stamps=None):
        _need_torch()
        if not isinstance(k, _Tensor) or k.dim() != 4:
            raise ValueError("k must be a tensor [pages, page_size, kv_heads, head_dim]")
        if k.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"k has dtype {k.dtype}, expected float16 or bfloat16")
        if min(k.shape[1:]) < 1:
            raise ValueError(f"k has shape {tuple(k.shape)}: pages need slots, heads and elements")
        index = k.get_device()
        _operand(k, "k", k.dtype, k.shape, max(index, 0))
        _operand(v, "v", k.dtype, k.shape, index)
        if not isinstance(page_table, _Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a tensor [batch, max_pages]")
        _operand(page_table, "page_table", torch.int32, page_table.shape, index)
        pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.batch, self.max_pages = page_table.shape
        self.capacity = self.max_pages * self.page_size
        self.device, self.index, self.dtype = k.device, index, k.dtype
        per_slot = (self.batch, self.kv_heads, self.capacity)
        if scores is not None:
            _dense(scores, "scores", torch.float32, per_slot, index)
        if stamps is not None:
            _dense(stamps, "stamps", torch.int32, per_slot, index)
        self.k, self.v, self.page_table, self.scores, self.stamps = k, v, page_table, scores, stamps
        self._s = _KvStruct(
            k.data_ptr(), v.data_ptr(), k.stride()[:3], v.stride()[:3], page_table.data_ptr(), page_table.stride(0),
            pages, None if scores is None else scores.data_ptr(), None if stamps is None else stamps.data_ptr(),
            _elems[k.dtype], self.page_size, self.max_pages, self.batch, self.kv_heads, self.head_dim)
        self._at = ctypes.addressof(self._s)
        self._workspaces = {}
        self._lib = _mbg.lib()

    def _workspace(self, q_heads, weights, ptr, stream):
        capture = 0
        if stream is not None or torch.cuda.is_current_stream_capturing():
            capture = self._lib.gemv_capture_id(ptr)
        key = (ptr, capture, q_heads, weights)
        got = self._workspaces.get(key)
        if got is None:
            n = max(self._lib.gemv_attn_paged_workspace(self._at, q_heads, 1 if weights else 0), _ATTN_COUNTER_BYTES)
            shared = (self.index, ptr, capture, n)
            with _shared_lock:
                got = _shared.get(shared)
                if got is None:
                    with _on(stream):
                        t = torch.empty(n, dtype=torch.uint8, device=self.device)
                        t[:_ATTN_COUNTER_BYTES].zero_()
                    got = _shared[shared] = _Workspace(t)
            self._workspaces[key] = got
        return got

    def release_workspaces(self):
        """Lets go of the workspaces that ``gemv_attn_paged`` has made: for handles that outlive CUDA graphs.

        A graph that calls with this handle were captured into must not be
        replayed afterwards.  Later calls make new ones."""
        self._workspaces.clear()


class RopeTable:
    """Frequencies of rotary positions with one or more axes, kept on the device.

    ``rot_dim`` leading elements of a head are turned, as rot_dim / 2 pairs:
    elements i and i + rot_dim / 2, or with ``pairs`` elements 2 i and 2 i + 1.
    ``sections``: how many consecutive pairs go by each axis (default: all by
    one).  Pair i turns with frequency theta^(-2 i / rot_dim); with ``per_axis``
    each axis has the whole ladder over its own pairs, theta^(-j / pairs of the
    axis).  ``frequencies`` (radians per position, below 2 pi) replaces them,
    for ladders stretched or scaled otherwise.
    """

    def __init__(self, rot_dim: int, sections: Optional[Sequence[int]] = None, theta: float = 10000.0,
                 pairs: bool = False, per_axis: bool = False, frequencies: Optional[Sequence[float]] = None,
                 device="cuda"):
        _need_torch()
        half = rot_dim // 2
        if rot_dim < 0 or rot_dim % 2:
            raise ValueError("rot_dim must be even and not negative")
        sections = [half] if sections is None else [int(n) for n in sections]
        if not 1 <= len(sections) <= 255 or min(sections) < 0 or sum(sections) != half:
            raise ValueError(f"sections must be 1 to 255 counts that add up to rot_dim / 2 = {half}")
        if frequencies is None:
            if not theta > 0:
                raise ValueError("theta must be positive")
            if per_axis:
                frequencies = [theta ** (-j / n) for n in sections for j in range(n)]
            else:
                frequencies = [theta ** (-2.0 * i / rot_dim) for i in range(half)]
        if len(frequencies) != half:
            raise ValueError(f"frequencies must have rot_dim / 2 = {half} values")
        turns = []
        for f in frequencies:
            if not 0 <= f < 2 * math.pi:
                raise ValueError("frequencies must lie in [0, 2 pi)")
            t = round(math.ldexp(f / (2 * math.pi), 64)) % (1 << 64)
            turns.append(t - (1 << 64) if t >= 1 << 63 else t)
        self.rot_dim, self.axes, self.pairs = rot_dim, len(sections), bool(pairs)
        self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self.axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], dtype=torch.uint8).to(device)
        self.index = self.turns.get_device()
        self._turns_at, self._axis_at = self.turns.data_ptr(), self.axis.data_ptr()
        self._packed = struct.pack("QQiiii", self._turns_at, self._axis_at, self.index, self.axes, rot_dim, self.pairs)


def gemv_attn_paged(cache: PagedKV, q, lengths, out=None, scale: Optional[float] = None, window: int = 0, lse=None,
                    accumulate: bool = False, scores_out=None, stream=None):
    """Attention of one new token per sequence over the cache; returns out.

    q: [batch, q_heads, head_dim] of the cache's type, any strides with a
    contiguous last dimension; lengths: int32 [batch], the slots in use (the
    new token's among them).  ``window``: only the last so many slots (0: all).
    ``lse``: float32 [batch, q_heads] that receives log(sum exp(score)).
    ``accumulate``: adds the weights, summed over the query heads of a cached
    head, to cache.scores, or with ``scores_out`` writes the sums there.  A
    sequence of length 0 gives zeros (and lse -inf)."""
    index = cache.index
    if scale is None:
        scale = cache.head_dim ** -0.5
    if not isinstance(q, _Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [batch, q_heads, head_dim]")
    heads = q.shape[1]
    s_ptr = 0
    if accumulate and cache.scores is not None:
        if scores_out is None:
            s_ptr = cache.scores.data_ptr()
        else:
            s_ptr = _dense(scores_out, "scores_out", torch.float32, cache.scores.shape, index)
    if heads and (s_ptr if accumulate else scores_out is None):
        ptr = _mbg._stream_ptr(stream)
        ws = cache._workspace(heads, accumulate, ptr, stream)
        result = out
        if result is None:
            with _on(stream):
                result = torch.empty(q.shape, dtype=cache.dtype, device=cache.device)
        with ws.lock:
            st = _quick.attn(cache._at, index, q, lengths, result, lse, s_ptr, ws[0], ws[1], scale, window, ptr)
        if st == 0:
            return result
    shape = (cache.batch, heads, cache.head_dim)
    qs = _operand(q, "q", cache.dtype, shape, index)
    if heads < 1 or heads % cache.kv_heads:
        raise ValueError(f"q has {heads} heads, expected a multiple of {cache.kv_heads}")
    n_ptr = _dense(lengths, "lengths", torch.int32, (cache.batch,), index)
    _count(window, "window", 0)
    if out is None:
        with _on(stream):
            out = torch.empty(shape, dtype=cache.dtype, device=cache.device)
        os = out.stride()
    else:
        os = _operand(out, "out", cache.dtype, shape, index)
    l_ptr = 0 if lse is None else _dense(lse, "lse", torch.float32, (cache.batch, heads), index)
    if accumulate and cache.scores is None:
        raise ValueError("accumulate needs a cache with scores")
    if scores_out is not None and not accumulate:
        raise ValueError("scores_out goes with accumulate=True")
    ptr = _mbg._stream_ptr(stream)
    ws = cache._workspace(heads, accumulate, ptr, stream)
    args = _ATTN.pack(q.data_ptr(), qs[0], qs[1], out.data_ptr(), os[0], os[1], n_ptr, l_ptr, s_ptr, ws[0], ws[1],
                      heads, window, scale)
    with ws.lock:
        st = cache._lib.gemv_attn_paged(cache._at, args, ptr)
    if st:
        _mbg._raise(st, "gemv_attn_paged")
    return out


def gemv_rope_append(cache: PagedKV, q, k, v, positions, slots, rope: RopeTable, q_out=None, seq=None, stamps=None,
                     stream=None):
    """Turns q and k by their positions, writes k and v to the cache; returns q_out.

    q: [tokens, q_heads, head_dim], k and v: [tokens, kv_heads, head_dim], all
    float32 (a GEMV's output), float16 or bfloat16; any strides with a
    contiguous last dimension, so parts of one QKV product will do.
    positions: int32 [axes, tokens].  slots: int32 [tokens], each token's slot
    in its sequence (negative: padding, not written).  seq: int32 [tokens], the
    tokens' sequences (default: token t belongs to sequence t).  stamps: int32
    [tokens], the tokens' numbers (default: the slots) for a cache with stamps.
    q_out: [tokens, q_heads, head_dim] of the cache's type."""
    index = cache.index
    if q_out is not None and _quick.rope(cache._at, index, rope._packed, q, k, v, positions, slots, seq, stamps, q_out,
                                         stream if stream is None else _mbg._stream_ptr(stream)) == 0:
        return q_out
    if not isinstance(q, _Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [tokens, q_heads, head_dim]")
    dtype = q.dtype
    elem = _elems.get(dtype)
    if elem is None:
        raise TypeError(f"q has dtype {dtype}, expected float32, float16 or bfloat16")
    tokens, heads, dim = q.shape
    q_shape, kv_shape = (tokens, heads, cache.head_dim), (tokens, cache.kv_heads, dim)
    qs = _operand(q, "q", dtype, q_shape, index)
    ks = _operand(k, "k", dtype, kv_shape, index)
    vs = _operand(v, "v", dtype, kv_shape, index)
    if rope.rot_dim > dim:
        raise ValueError(f"the rope turns {rope.rot_dim} elements, a head has {dim}")
    if rope.index != index:
        raise ValueError(f"the rope table is on {rope.turns.device}, expected {cache.device}")
    ps = _operand(positions, "positions", torch.int32, (rope.axes, tokens), index)
    per_token = (tokens,)
    s_ptr = _dense(slots, "slots", torch.int32, per_token, index)
    b_ptr = t_ptr = 0
    if seq is not None:
        b_ptr = _dense(seq, "seq", torch.int32, per_token, index)
    elif tokens > cache.batch:
        raise ValueError(f"{tokens} tokens for {cache.batch} sequences: seq is needed")
    if stamps is not None:
        t_ptr = _dense(stamps, "stamps", torch.int32, per_token, index)
    if q_out is None:
        with _on(stream):
            q_out = torch.empty(q_shape, dtype=cache.dtype, device=cache.device)
        os = q_out.stride()
    else:
        os = _operand(q_out, "q_out", cache.dtype, q_shape, index)
    st = cache._lib.gemv_rope_append(
        cache._at, _ROPE.pack(q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                              q_out.data_ptr(), os[0], os[1], positions.data_ptr(), ps[0], s_ptr, b_ptr, t_ptr,
                              rope._turns_at, rope._axis_at, elem, tokens, heads, rope.axes, rope.rot_dim, rope.pairs),
        _mbg._stream_ptr(stream))
    if st:
        _mbg._raise(st, "gemv_rope_append")
    return q_out


def _moves(cache, moves, counts):
    if not isinstance(moves, _Tensor) or moves.dim() != 4:
        raise ValueError("moves must be a tensor [batch, kv_heads, max_moves, 2]")
    room = moves.shape[2]
    return (_dense(moves, "moves", torch.int32, (cache.batch, cache.kv_heads, room, 2), cache.index), room,
            _dense(counts, "counts", torch.int32, (cache.batch, cache.kv_heads), cache.index))


def gemv_kv_evict_plan(cache: PagedKV, lengths, keep: int, sinks: int = 0, recent: int = 0, moves=None, counts=None,
                       stream=None):
    """Which slots move so that ``keep`` of each sequence and cached head stay; returns (moves, counts).

    Those that stay: slots whose stamp is below ``sinks`` or among the
    ``recent`` newest numbers, then the larger score, then the lower slot.
    moves: int32 [batch, kv_heads, max_moves, 2], the first counts[b, h] pairs
    (from, to) are written; max_moves at least min(keep, capacity - keep).
    Nothing in the cache changes."""
    if moves is not None and _quick.plan(cache._at, cache.index, lengths, keep, sinks, recent, moves, counts,
                                         stream if stream is None else _mbg._stream_ptr(stream)) == 0:
        return moves, counts
    if cache.scores is None or cache.stamps is None:
        raise ValueError("eviction needs a cache with scores and stamps")
    _count(keep, "keep", 1)
    _count(sinks, "sinks", 0)
    _count(recent, "recent", 0)
    n_ptr = _dense(lengths, "lengths", torch.int32, (cache.batch,), cache.index)
    most = max(1, min(keep, cache.capacity - keep))
    if moves is None or counts is None:
        with _on(stream):
            if moves is None:
                moves = torch.empty((cache.batch, cache.kv_heads, most, 2), dtype=torch.int32, device=cache.device)
            if counts is None:
                counts = torch.empty((cache.batch, cache.kv_heads), dtype=torch.int32, device=cache.device)
    m_ptr, room, c_ptr = _moves(cache, moves, counts)
    if room < most:
        raise ValueError(f"moves has room for {room}, at least {most} are needed")
    st = cache._lib.gemv_kv_evict_plan(cache._at, n_ptr, keep, sinks, recent, m_ptr, room, c_ptr,
                                       _mbg._stream_ptr(stream))
    if st:
        _mbg._raise(st, "gemv_kv_evict_plan")
    return moves, counts


def gemv_kv_evict_apply(cache: PagedKV, moves, counts, lengths, keep: int, stream=None):
    """Carries a plan out: keys, values, scores and stamps move, lengths is lowered to keep.

    ``lengths`` may be None (left to the caller).  A plan may be carried out on
    several caches that are filled alike."""
    if _quick.apply(cache._at, cache.index, moves, counts, lengths, keep,
                    stream if stream is None else _mbg._stream_ptr(stream)) == 0:
        return
    _count(keep, "keep", 1)
    m_ptr, room, c_ptr = _moves(cache, moves, counts)
    n_ptr = None if lengths is None else _dense(lengths, "lengths", torch.int32, (cache.batch,), cache.index)
    st = cache._lib.gemv_kv_evict_apply(cache._at, m_ptr, room, c_ptr, n_ptr, keep, _mbg._stream_ptr(stream))
    if st:
        _mbg._raise(st, "gemv_kv_evict_apply")


def gemv_kv_evict(cache: PagedKV, lengths, keep: int, sinks: int = 0, recent: int = 0, moves=None, counts=None,
                  stream=None):
    """``gemv_kv_evict_plan`` and ``gemv_kv_evict_apply`` in turn; returns (moves, counts)."""
    moves, counts = gemv_kv_evict_plan(cache, lengths, keep, sinks, recent, moves, counts, stream)
    gemv_kv_evict_apply(cache, moves, counts, lengths, keep, stream)
    return moves, counts


_NONE = (0, 0, 0)


def _rows(t, name, rows, width, index):
    """(address, row stride, type) of an operand [rows, width] or [width]."""
    if t is None:
        return _NONE
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = t.dtype
    elem = _elems.get(dtype)
    if elem is None:
        raise TypeError(f"{name} has dtype {dtype}, expected float32, float16 or bfloat16")
    if t.dim() == 1:
        _operand(t, name, dtype, (width,), index)
        return t.data_ptr(), 0, elem
    return t.data_ptr(), _operand(t, name, dtype, (rows, width), index)[0], elem


def gemv_norm_residual(y, x, post: bool = False, post_weight=None, gate=None, alpha: float = 1.0, pre_weight=None,
                       pre_bias=None, kind: str = "rms", unit_offset: bool = False, eps: float = 1e-6, out=None,
                       h=None, h_dtype=None, pre: bool = True, stream=None):
    """The norms around a block with its gate and the residual; returns (out, h).

        u = y;  u = norm(u) * post_weight (with post);  u = u * gate
        out = x + alpha * u;  h = norm(out) * pre_weight + pre_bias

    y (the block's output) and x (the residual): [rows, width], float32,
    float16 or bfloat16 each.  post_weight, gate, pre_weight, pre_bias: [width],
    or [rows, width] for values of each row; None leaves one out.
    ``kind``: 'rms' or 'layer' for both norms.  ``unit_offset``: pre_weight
    stands for 1 + pre_weight.  out: like x (may be x).  h: the next block's
    input, [rows, width], ``h_dtype`` float16 by default; ``pre=False``: none
    (h is None).  h is computed from the unrounded sum."""
    if torch is None:
        _need_torch()
    if kind != "rms" and kind != "layer":
        raise ValueError("kind must be 'rms' or 'layer'")
    if post_weight is not None and not post:
        raise ValueError("post_weight goes with post=True")
    if not pre and (pre_weight is not None or pre_bias is not None or h is not None):
        raise ValueError("pre_weight, pre_bias and h go with pre=True")
    flags = (NORM_LAYER if kind == "layer" else 0) | (NORM_POST if post else 0) | (NORM_UNIT_OFFSET if unit_offset else 0)
    if out is not None and (h is not None or not pre) and h_dtype is None and _quick.norm(
            y, x, gate, post_weight, pre_weight, pre_bias, out, h, alpha, eps, flags,
            stream if stream is None else _mbg._stream_ptr(stream)) == 0:
        return out, h
    if not isinstance(y, _Tensor) or y.dim() != 2:
        raise ValueError("y must be a tensor [rows, width]")
    if not isinstance(x, _Tensor) or x.dim() != 2:
        raise ValueError("x must be a tensor [rows, width]")
    rows, width = y.shape
    index = max(y.get_device(), 0)
    y_, x_ = _rows(y, "y", rows, width, index), _rows(x, "x", rows, width, index)
    if out is None or (pre and h is None):
        with _on(stream):
            if out is None:
                out = torch.empty((rows, width), dtype=x.dtype, device=y.device)
            if pre and h is None:
                h = torch.empty((rows, width), dtype=h_dtype or torch.float16, device=y.device)
    o_ = (out.data_ptr(), _operand(out, "out", x.dtype, (rows, width), index)[0], x_[2])
    h_ = _NONE
    if pre:
        h_ = _rows(h, "h", rows, width, index)
        if h.dim() != 2 or (h_dtype is not None and h.dtype is not h_dtype):
            _refuse(h, "h", h_dtype or h.dtype, (rows, width), index)
    st = _mbg.lib().gemv_norm_residual(
        _NORM.pack(*y_, *x_, *_rows(gate, "gate", rows, width, index),
                   *_rows(post_weight, "post_weight", rows, width, index),
                   *_rows(pre_weight, "pre_weight", rows, width, index),
                   *_rows(pre_bias, "pre_bias", rows, width, index), *o_, *h_, rows, width, alpha, eps, flags),
        _mbg._stream_ptr(stream))
    if st:
        _mbg._raise(st, "gemv_norm_residual")
    return out, h
