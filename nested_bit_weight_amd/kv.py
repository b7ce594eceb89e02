"""The key-value cache of a decode step: append, attend, evict.

What runs between a layer's qkv product and its o product, over one paged cache
(pools [pages][heads][page][dim] of bf16, or of 8 bits with a factor for each head, and
a table of page numbers for each sequence; see ``include/nbw.h`` for every detail):

    cache = KVCache(k_pool, v_pool, table)
    q_out, lens1 = kv_append(cache, k, v, lens, positions, q=q, rope=rope, pos=pos, acc=acc)
    out = kv_attend(cache, q_out, lens1, acc=acc)       # acc: running totals of the weights
    lens2 = kv_evict(cache, acc, pos, lens1, budget, recent=64, acc_out=acc2, pos_out=pos2)

As everywhere in this package the calls only marshal arguments, queue the work on the
current stream of the tensors' GPU, whichever GPU is the current one, and raise if the library is not built.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _lib, _raw_stream, _workspace

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class KVView(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("pages", _i64), ("heads", _i32), ("page", _i32), ("dim", _i32),
                ("dtype", _i32), ("k_scale", _vp), ("v_scale", _vp), ("table", _vp), ("rows", _i64),
                ("width", _i64), ("table_ld", _i64)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("q", _vp), ("q_out", _vp), ("k_ld", _i64), ("v_ld", _i64),
                ("q_ld", _i64), ("q_out_ld", _i64), ("tokens", _i64), ("q_heads", _i32), ("eps", _f32),
                ("cu", _vp), ("lens", _vp), ("positions", _vp), ("rope", _vp), ("rope_rows", _i64),
                ("q_norm", _vp), ("k_norm", _vp), ("pos", _vp), ("acc", _vp), ("lens_out", _vp)]


class AttendArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("out", _vp), ("q_ld", _i64), ("out_ld", _i64), ("q_heads", _i32), ("scale", _f32),
                ("lens", _vp), ("max_len", _i64), ("acc", _vp), ("acc_out", _vp), ("decay", _f32),
                ("workspace", _vp), ("workspace_bytes", _i64)]


class EvictArgs(ctypes.Structure):
    _fields_ = [("acc", _vp), ("pos", _vp), ("lens", _vp), ("budget", _i64), ("sink", _i64), ("recent", _i64),
                ("acc_out", _vp), ("pos_out", _vp), ("lens_out", _vp), ("max_len", _i64), ("workspace", _vp),
                ("workspace_bytes", _i64)]


SIZES_KEPT = 64
KV_DTYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


def declare(lib) -> None:
    """The C signatures of the cache's entry points."""
    pc = ctypes.POINTER(KVView)
    for name, args in (("nbw_kv_append", AppendArgs), ("nbw_kv_attend", AttendArgs), ("nbw_kv_evict", EvictArgs)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [pc, ctypes.POINTER(args), _vp], ctypes.c_int
    lib.nbw_kv_attend_workspace_bytes.argtypes = [pc, _i32, _i64, _i32]
    lib.nbw_kv_attend_workspace_bytes.restype = _i64
    lib.nbw_kv_evict_workspace_bytes.argtypes = [pc, _i64, _i64]
    lib.nbw_kv_evict_workspace_bytes.restype = _i64


# The GPU that kernels go to (the bare getter: the tensors are there, so the runtime is up).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_BF16, _F32, _INT32 = torch.bfloat16, torch.float32, torch.int32


def _is(t, name: str, dtype, shape, index: int) -> int:
    """Address of a contiguous tensor of this type and shape on GPU number ``index``."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on GPU {index}, got {t.device}")
    raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


class KVCache:
    """One layer's cache: pools ``k`` and ``v`` [pages][heads][page][dim] (bf16, or
    float8_e4m3fn with fp32 factors ``k_scale`` and ``v_scale`` [heads]) and the int32
    ``table`` [rows][width] of page numbers (its rows may lie further apart than width).

    The tensors stay the caller's; the object refers to them and may be kept as long as
    they live.  The numbers in the table may change between calls."""

    __slots__ = ("k", "v", "table", "k_scale", "v_scale", "view", "_ref", "rows", "heads", "page", "dim", "width",
                 "capacity", "pages", "device", "_dev", "_row", "_track", "_sizes")

    def __init__(self, k, v, table, k_scale=None, v_scale=None):
        for t, name in ((k, "k"), (v, "v"), (table, "table")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.device.type != "cuda":
                raise ValueError(f"{name} must be on a GPU")
        if k.dtype not in KV_DTYPES:
            raise TypeError(f"k must be torch.bfloat16 or torch.float8_e4m3fn, got {k.dtype}")
        if k.dim() != 4:
            raise ValueError("k must be [pages][heads][page][dim]")
        device = k.device
        index = k.get_device()
        _is(k, "k", k.dtype, k.shape, index)
        _is(v, "v", k.dtype, k.shape, index)
        if table.dtype != torch.int32 or table.dim() != 2 or table.device != device:
            raise ValueError("table must be an int32 [rows][width] tensor on the pools' GPU")
        rows, width = table.shape
        if (width > 1 and table.stride(1) != 1) or (rows > 1 and table.stride(0) < width):
            raise ValueError("table must have unit column stride and rows that do not overlap")
        pages, heads, page, dim = k.shape
        fp8 = k.dtype == torch.float8_e4m3fn
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if fp8 != (t is not None):
                raise ValueError(f"{name} goes with an 8-bit cache, and with no other")
            if fp8:
                _is(t, name, _F32, (heads,), index)
        self.k, self.v, self.table, self.k_scale, self.v_scale = k, v, table, k_scale, v_scale
        self.rows, self.width, self.pages, self.heads, self.page, self.dim = rows, width, pages, heads, page, dim
        self.capacity, self.device = width * page, device
        self._dev, self._row = index, (rows,)
        self._sizes = {}  # workspace bytes by the sizes that they depend on
        self._track = (rows, heads, self.capacity)
        self.view = KVView(k.data_ptr(), v.data_ptr(), pages, heads, page, dim, KV_DTYPES[k.dtype],
                           k_scale.data_ptr() if fp8 else None, v_scale.data_ptr() if fp8 else None,
                           table.data_ptr(), rows, width, table.stride(0) if rows > 1 else width)
        self._ref = ctypes.byref(self.view)
        if _lib().nbw_kv_evict_workspace_bytes(self._ref, 1, 1) < 0:
            raise ValueError(f"a cache of {pages} pages of {page} slots, {heads} heads of {dim} and a table of "
                             f"{rows} x {width} is outside what the library takes (dim 64, 128 or 256; pages of a "
                             f"power of two up to 4096 slots, 16-byte aligned; a row of at most 2^30 slots; "
                             f"rows x heads below 2^24)")

    def _heads(self, t, name: str, shape):
        """Address of a bf16 tensor of shape [n][heads][dim] and its stride from one token
        to the next (0: dense); tokens may lie apart, as in a slice of a wider product."""
        try:
            if t.dtype is _BF16 and t.get_device() == self._dev and t.shape == shape:
                if t.is_contiguous():
                    return t.data_ptr(), 0
                n, heads, dim = shape
                s0, s1, s2 = t.stride()
                if s2 == 1 and (s1 == dim or heads == 1) and (s0 >= heads * dim or n == 1):
                    return t.data_ptr(), s0 if n > 1 else 0
        except AttributeError:
            pass
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if t.get_device() != self._dev:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        raise ValueError(f"{name} must have contiguous heads, one after the other")

    def _queries(self, q, tokens: int):
        """Shape of q: [tokens][q_heads][dim], q_heads a multiple of the cache's heads."""
        if not isinstance(q, torch.Tensor):
            raise TypeError("q must be a torch.Tensor")
        shape = q.shape
        if len(shape) != 3 or shape[0] != tokens or shape[2] != self.dim or not shape[1] or shape[1] % self.heads:
            raise ValueError(f"q must be [{tokens}][q_heads][{self.dim}] with q_heads a multiple of {self.heads}, "
                             f"got {tuple(shape)}")
        return shape

    def attend_workspace_bytes(self, q_heads: int, max_len: int = 0, weights: bool = False) -> int:
        """Bytes of scratch kv_attend needs."""
        with torch.cuda.device(self._dev):  # they depend on its number of compute units
            return _bytes(_lib().nbw_kv_attend_workspace_bytes(self._ref, q_heads, max_len, int(weights)))

    def evict_workspace_bytes(self, budget: int, max_len: int = 0) -> int:
        """Bytes of scratch kv_evict needs."""
        return _bytes(_lib().nbw_kv_evict_workspace_bytes(self._ref, budget, max_len))

    def _scratch(self, workspace, query, sizes, stream: int):
        """Address and size of a call's workspace; "auto": the binding's buffer, of the
        bytes that ``query`` gives for ``sizes``."""
        if workspace is None:
            return None, 0
        if isinstance(workspace, str):
            if workspace != "auto":
                raise ValueError("workspace must be 'auto', a tensor or None")
            nbytes = self._sizes.get(sizes)
            if nbytes is None:
                nbytes = _bytes(query(self._ref, *sizes))
                if len(self._sizes) >= SIZES_KEPT:  # a bound that grows with every token passes by here once
                    self._sizes.clear()
                self._sizes[sizes] = nbytes
            if nbytes == 0:
                return None, 0
            workspace = _workspace(self._dev, stream, nbytes)
            return workspace.data_ptr(), workspace.numel()
        if workspace.get_device() != self._dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the cache's GPU")
        return workspace.data_ptr(), workspace.numel()


def _bytes(n: int) -> int:
    if n < 0:
        raise ValueError("bad arguments: query heads must be a multiple of the cache's heads, a budget within the "
                         "capacity, a bound of the lengths not negative, the work no more than one launch takes")
    return n


def kv_append(cache: KVCache, k, v, lens, positions, *, q=None, cu=None, rope=None, q_norm=None, k_norm=None,
              eps: float = 1e-6, q_out=None, pos=None, acc=None, lens_out=None):
    """New keys ``k`` and values ``v`` (bf16 [tokens][heads][dim]) go into the cache: one
    token for each row, or with ``cu`` (int32 [rows + 1], ascending from 0 to tokens) tokens
    cu[r]..cu[r+1]-1 for row r, from slot ``lens[r]`` on (int32 [rows]).

    ``positions``: int32 [tokens].  ``rope``: fp32 [max position + 1][dim], cosines then sines.
    ``k_norm``, ``q_norm``: bf16 [dim], weights of the heads' norms.  ``q``: bf16
    [tokens][q_heads][dim], normalised and rotated alongside into ``q_out`` (which may be q).
    ``pos`` and ``acc`` ([rows][heads][capacity], int32 and fp32) get the tokens' positions
    and zeros.  Returns (q_out or None, lens + new tokens)."""
    if _current_device() != cache._dev:
        with torch.cuda.device(cache._dev):
            return kv_append(cache, k, v, lens, positions, q=q, cu=cu, rope=rope, q_norm=q_norm, k_norm=k_norm, eps=eps,
                             q_out=q_out, pos=pos, acc=acc, lens_out=lens_out)
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    tokens, rows, heads, index = k.size(0) if k.dim() else 0, cache.rows, cache.heads, cache._dev
    shape = (tokens, heads, cache.dim)
    kp, k_ld = cache._heads(k, "k", shape)
    vp, v_ld = cache._heads(v, "v", shape)
    qp = qo = cu_p = None
    q_ld = qo_ld = q_heads = rope_rows = 0
    if cu is not None:
        cu_p = _is(cu, "cu", _INT32, (rows + 1,), index)
    elif tokens != rows:
        raise ValueError(f"without cu there is one token for each of the {rows} rows, got {tokens}")
    if q is not None:
        shape = cache._queries(q, tokens)
        q_heads = shape[1]
        qp, q_ld = cache._heads(q, "q", shape)
        if q_out is None:
            q_out = torch.empty(shape, dtype=q.dtype, device=q.device)
        qo, qo_ld = cache._heads(q_out, "q_out", shape)
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm go with q")
    if rope is not None:
        rope_rows = rope.size(0) if isinstance(rope, torch.Tensor) and rope.dim() == 2 else 0
        if rope_rows < 1:
            raise ValueError("rope must be an fp32 [positions][dim] tensor")
    if lens_out is None:
        lens_out = torch.empty(rows, dtype=_INT32, device=k.device)
    args = AppendArgs(
        kp, vp, qp, qo, k_ld, v_ld, q_ld, qo_ld, tokens, q_heads, eps, cu_p, _is(lens, "lens", _INT32, cache._row, index),
        _is(positions, "positions", _INT32, (tokens,), index),
        None if rope is None else _is(rope, "rope", _F32, (rope_rows, cache.dim), index), rope_rows,
        None if q_norm is None else _is(q_norm, "q_norm", _BF16, (cache.dim,), index),
        None if k_norm is None else _is(k_norm, "k_norm", _BF16, (cache.dim,), index),
        None if pos is None else _is(pos, "pos", _INT32, cache._track, index),
        None if acc is None else _is(acc, "acc", _F32, cache._track, index),
        _is(lens_out, "lens_out", _INT32, cache._row, index))
    st = _lib().nbw_kv_append(cache._ref, ctypes.byref(args), _raw_stream(index))
    if st:
        _check(st, "nbw_kv_append")
    return q_out, lens_out


def kv_attend(cache: KVCache, q, lens, *, scale: float | None = None, out=None, acc=None, acc_out=None,
              decay: float = 1.0, max_len: int | None = None, workspace="auto") -> torch.Tensor:
    """Attention of one new token for each row, ``q`` bf16 [rows][q_heads][dim], over the
    row's first ``lens`` slots (int32 [rows], the new token's among them): bf16
    [rows][q_heads][dim].  ``scale``: of the scores, 1/sqrt(dim) if None.

    With ``acc`` (fp32 [rows][heads][capacity]) ``acc_out`` (acc itself if None) becomes
    decay * acc + the softmax weights, added over the query heads of a head.  ``max_len``:
    a bound of the lengths, if one below the capacity is known.  ``workspace``: "auto" (the
    binding's buffer of this device and stream), or a uint8 tensor of at least
    ``cache.attend_workspace_bytes(...)`` bytes, as a captured graph should have."""
    index = cache._dev
    if _current_device() != index:
        with torch.cuda.device(index):
            return kv_attend(cache, q, lens, scale=scale, out=out, acc=acc, acc_out=acc_out, decay=decay, max_len=max_len,
                             workspace=workspace)
    shape = cache._queries(q, cache.rows)
    q_heads = shape[1]
    qp, q_ld = cache._heads(q, "q", shape)
    if scale is None:
        scale = 0.0
    else:
        scale = _f32(scale).value  # a number too small for fp32 would be 0, which stands for the default
        if not 0.0 < abs(scale) < 3e38:
            raise ValueError("scale must be finite and not 0 in fp32")
    if max_len is None:
        max_len = 0
    elif max_len < 1:
        raise ValueError("max_len must be at least 1")
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
    op, out_ld = cache._heads(out, "out", shape)
    acc_p = acc_o = None
    if acc is not None:
        acc_p = _is(acc, "acc", _F32, cache._track, index)
        acc_o = acc_p if acc_out is None else _is(acc_out, "acc_out", _F32, cache._track, index)
    elif acc_out is not None:
        raise ValueError("acc_out goes with acc")
    lib, stream = _lib(), _raw_stream(index)
    ws, ws_bytes = cache._scratch(workspace, lib.nbw_kv_attend_workspace_bytes, (q_heads, max_len, acc is not None), stream)
    args = AttendArgs(qp, op, q_ld, out_ld, q_heads, scale, _is(lens, "lens", _INT32, cache._row, index), max_len, acc_p,
                      acc_o, decay, ws, ws_bytes)
    st = lib.nbw_kv_attend(cache._ref, ctypes.byref(args), stream)
    if st:
        _check(st, "nbw_kv_attend")
    return out


def kv_evict(cache: KVCache, acc, pos, lens, budget: int, *, sink: int = 0, recent: int = 0, acc_out, pos_out,
             lens_out=None, max_len: int | None = None, workspace="auto") -> torch.Tensor:
    """Rows longer than ``budget`` keep, for each head, the budget slots with the largest
    totals ``acc`` (fp32 [rows][heads][capacity]; the lowest slot first among equals); the
    ones whose position ``pos`` (int32, same shape) is below ``sink`` or among the ``recent``
    last are kept in any case, whatever their totals (sink + recent <= budget).  Slots that stay past the budget move
    into the ones below it that go, in the pools, in ``acc_out`` and in ``pos_out`` (buffers
    of their own, of the same shapes).  Returns min(lens, budget) in ``lens_out``.
    ``max_len`` and ``workspace`` as for :func:`kv_attend`."""
    index, track = cache._dev, cache._track
    if _current_device() != index:
        with torch.cuda.device(index):
            return kv_evict(cache, acc, pos, lens, budget, sink=sink, recent=recent, acc_out=acc_out, pos_out=pos_out,
                            lens_out=lens_out, max_len=max_len, workspace=workspace)
    if max_len is None:
        max_len = 0
    elif max_len < 1:
        raise ValueError("max_len must be at least 1")
    if not 1 <= budget <= cache.capacity:
        raise ValueError(f"budget must be within 1..{cache.capacity}, got {budget}")
    if sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError("sink and recent must not be negative, nor more than the budget together")
    if lens_out is None:
        lens_out = torch.empty(cache.rows, dtype=_INT32, device=cache.device)
    lib, stream = _lib(), _raw_stream(index)
    ws, ws_bytes = cache._scratch(workspace, lib.nbw_kv_evict_workspace_bytes, (budget, max_len), stream)
    args = EvictArgs(_is(acc, "acc", _F32, track, index), _is(pos, "pos", _INT32, track, index),
                     _is(lens, "lens", _INT32, cache._row, index), budget, sink, recent,
                     _is(acc_out, "acc_out", _F32, track, index), _is(pos_out, "pos_out", _INT32, track, index),
                     _is(lens_out, "lens_out", _INT32, cache._row, index), max_len, ws, ws_bytes)
    st = lib.nbw_kv_evict(cache._ref, ctypes.byref(args), stream)
    if st:
        _check(st, "nbw_kv_evict")
    return lens_out
