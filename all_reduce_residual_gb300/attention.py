"""Attention of a tensor-parallel decode step on one shard's heads: rotary
positions, the append to a paged key-value cache, attention of each sequence's
new token over it, and the pages themselves.

A decode step of a layer, between two epilogues (``run``)::

    q = rotary_append(ws, q, k, v, positions, slots, table, cache)
    out, lse = paged_decode(ws, q, cache, block_table, lens)
    partial = out.flatten(1) @ w_o          # this shard's partial of run()

Like ``run``, these functions check shapes, dtypes and devices, allocate
outputs and scratch through torch, and pass torch's current stream (or
``stream``); everything else happens in libarf.so's kernels. With ``stream``,
outputs and scratch come from that stream's memory, so that nothing queued
elsewhere still uses them; the caller orders what the call reads, and what
later reads its outputs, as between any two streams. Nothing is read
back, so they can be captured into CUDA graphs. The checks and the call itself
are in the module _torch_ops (csrc/torch_ops.cpp), for the host's time. No
gradients are recorded: a tensor that requires one is refused unless gradients
are off (torch.no_grad, torch.inference_mode), and tensors that a call writes
count as modified in place.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os

import torch

from . import _binding as B

_CACHE_DTYPE = {torch.bfloat16: B.ARF_BF16, torch.float16: B.ARF_FP16, torch.float8_e4m3fn: B.ARF_E4M3}
_SCALING = {None: B.ARF_ROPE_NONE, "none": B.ARF_ROPE_NONE, "linear": B.ARF_ROPE_LINEAR, "ntk": B.ARF_ROPE_NTK,
            "yarn": B.ARF_ROPE_YARN}

if not os.path.exists(os.path.join(B.PKG, "_torch_ops.so")):
    raise RuntimeError(f"{B.PKG}/_torch_ops.so is not built: run `python -m all_reduce_residual_gb300.build` "
                       "(or __graft_entry__.build()) where torch is installed; there is no other implementation")
B.load()  # the library itself, before the module that links against it
from . import _torch_ops  # noqa: E402


def _raise(ws, st, what):
    raise B.ArfError(st, what, B.arf_last_cuda_error(ws.handle) if st == B.ARF_ERR_CUDA else 0)


def _int(x, bits, name):
    """x as a signed C integer of so many bits (ctypes would cut it off)."""
    x = operator.index(x)
    if not -(1 << (bits - 1)) <= x < 1 << (bits - 1):
        raise ValueError(f"{name}: {x} does not fit in {bits} bits")
    return x


def _share(delta, dims, row):
    """Whether two tensors of rows of `row` bytes, at offsets sum(i * stride)
    of 0 <= i < n for every (stride, n) of `dims`, have a byte in common when
    the second begins `delta` bytes after the first. The rows of one do not
    overlap (each stride is beyond all that is inside it); of other tensors
    no library call writes."""
    if any(n == 0 for _, n in dims):
        return False
    dims = sorted((d for d in dims if d[1] > 1), reverse=True)
    reach = row - 1 + sum(stride * (n - 1) for stride, n in dims)  # the largest distance of two bytes

    def meets(rest, reach, dims):
        if abs(rest) > reach:
            return False
        if not dims:
            return True
        (stride, n), *inner = dims
        if stride == 0:
            return meets(rest, reach, inner)
        return any(-n < i < n and meets(rest - i * stride, reach - stride * (n - 1), inner)
                   for i in (rest // stride, rest // stride + 1))

    return meets(delta, reach, dims)


def _base(t):
    """The tensor that t is a view of, which shares its version counter (one
    for all layers where they are views of one tensor), or t."""
    try:
        return t._base if t._is_view() else t
    except RuntimeError:  # a view that autograd does not follow
        return t


def _fixed(name):
    return property(lambda self: getattr(self, "_" + name))


class RotaryTable:
    """The angles per position of a model's rotary positions, on the device
    (arf_rotary_turns); made once and kept.

    rot_dim: leading elements of each head that rotate. layout: "half" pairs
    (i, i + rot_dim/2) or "interleaved" pairs (2i, 2i + 1). scaling: None,
    "linear", "ntk" or "yarn" with `factor`; original_length (the trained
    context), beta_fast and beta_slow are used by "yarn".

    "yarn" is the formula of its paper: the ramp between the pairs that slow
    down and those that do not is linear in the turns that a pair makes over
    original_length, and cos and sin are multiplied by 0.1 ln(factor) + 1.
    Models trained with another ramp (released code takes it linear in the
    pair's index), another factor or none have other angles: from_frequencies
    takes theirs.
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, scaling=None, factor: float = 1.0,
                 original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, layout: str = "half",
                 device=None):
        if scaling not in _SCALING:
            raise ValueError(f"unknown scaling {scaling!r}: None, linear, ntk or yarn")
        rot_dim = _int(rot_dim, 32, "rot_dim")
        if rot_dim > 1 << 20:
            raise ValueError(f"rot_dim: {rot_dim} is beyond every head size")
        turns = (ctypes.c_uint64 * max(1, rot_dim // 2))()
        mag = ctypes.c_float()
        st = B.arf_rotary_turns(rot_dim, base, _SCALING[scaling], factor, original_length, beta_fast, beta_slow,
                                turns, mag)
        if st != B.ARF_OK:
            raise B.ArfError(st, "arf_rotary_turns")
        self._set(turns, mag.value, layout, device)

    @classmethod
    def from_frequencies(cls, frequencies, magnitude: float = 1.0, layout: str = "half", device=None):
        """The table of a model's own frequencies: radians per position of
        each pair (a sequence or tensor, taken in binary64; 2 len(frequencies)
        leading elements of a head rotate), and a factor for cos and sin."""
        w, magnitude = [float(x) for x in frequencies], float(magnitude)
        if not 1 <= len(w) <= 1 << 19 or not all(map(math.isfinite, (*w, magnitude))):
            raise ValueError("frequencies: a finite number for each of 1 to 2^19 pairs; magnitude: finite")
        table = cls.__new__(cls)
        # as a fraction of a turn times 2^64, whole turns dropped
        turns = (ctypes.c_uint64 * len(w))(*(round(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for x in w))
        table._set(turns, magnitude, layout, device)
        return table

    def _set(self, turns, magnitude, layout, device):
        if layout not in ("half", "interleaved"):
            raise ValueError(f"unknown layout {layout!r}: half or interleaved")
        rot_dim = 2 * len(turns)
        self._rot_dim, self._layout, self._magnitude = rot_dim, layout, magnitude
        # torch has no 64-bit unsigned type that kernels need here: the same bits as int64
        host = torch.frombuffer(turns, dtype=torch.int64)
        self._turns = host.clone() if device is not None and torch.device(device).type == "cpu" else \
            host.to(device if device is not None else torch.device("cuda", torch.cuda.current_device()))
        self._struct = B.Rotary(self._turns.data_ptr(), rot_dim, int(layout == "interleaved"), magnitude)
        # what _torch_ops reads: the struct's address, and the device
        self._table_key = (ctypes.addressof(self._struct), self._turns.get_device())

    # the struct holds the table's address: a table is made anew, not changed
    rot_dim, layout, magnitude, turns, struct = map(_fixed, ("rot_dim", "layout", "magnitude", "turns", "struct"))


class KVCache:
    """A paged cache over the caller's page tensors (arf_kv_cache_t).

    k, v: [pages, page_size, kv_heads, D] (layout "nhd") or [pages, kv_heads,
    page_size, D] ("hnd"), of equal shape and strides, D contiguous; bf16,
    fp16 or float8_e4m3fn (which holds value / scale). They may be views of one
    tensor; a cache whose keys and values share elements can only be read.
    """

    def __init__(self, k, v, layout: str = "nhd", k_scale: float = 1.0, v_scale: float = 1.0):
        if layout not in ("nhd", "hnd"):
            raise ValueError(f"unknown layout {layout!r}: nhd or hnd")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or v.dtype != k.dtype:
            raise ValueError("k and v: two page tensors of equal shape, strides and dtype")
        if k.dtype not in _CACHE_DTYPE:
            raise ValueError(f"unsupported cache dtype {k.dtype}: bf16, fp16 or float8_e4m3fn")
        if k.requires_grad or v.requires_grad:
            raise ValueError("k and v: pages that require a gradient, which no call records: detach them")
        if k.device != v.device or not k.is_cuda:
            raise ValueError(f"k is on {k.device}, v on {v.device}: one CUDA device is needed")
        if k.stride(3) != 1 and k.shape[3] > 1:
            raise ValueError("the elements of a head must be contiguous")
        for n, name in zip(k.shape, ("pages", "page tensor", "page tensor", "head_dim")):
            _int(n, 32, name)
        pages, a, b, d = k.shape
        sp, sa, sb, _ = k.stride()
        (page_size, heads), (st, sh) = ((a, b), (sa, sb)) if layout == "nhd" else ((b, a), (sb, sa))
        self._k, self._v, self._layout = k, v, layout
        self._num_pages, self._page_size, self._kv_heads, self._head_dim = pages, page_size, heads, d
        self._struct = B.Cache(k.data_ptr(), v.data_ptr(), pages, page_size, heads, d, sp, st, sh,
                              _CACHE_DTYPE[k.dtype], k_scale, v_scale)
        # keys and values that share memory can be read; a call that writes
        # them would leave which of the two is there to chance
        es = k.element_size()
        shared = _share(v.data_ptr() - k.data_ptr(), [(sp * es, pages), (sa * es, a), (sb * es, b)], d * es)
        # what _torch_ops reads: the struct's address, the device, whether the
        # pages may be written, and the tensors whose versions count that
        self._cache_key = (ctypes.addressof(self._struct), k.get_device(), not shared, _base(k), _base(v))

    # the struct holds the pages' addresses: a cache of other pages is made anew
    k, v, layout, num_pages, page_size, kv_heads, head_dim, struct = map(
        _fixed, ("k", "v", "layout", "num_pages", "page_size", "kv_heads", "head_dim", "struct"))
    dtype, device = property(lambda self: self._k.dtype), property(lambda self: self._k.device)


def rotary(ws, q, k, positions, table: RotaryTable, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (k may be None) at
    positions [T] (int32). q_out / k_out are allocated when None; q_out=q and
    k_out=k work in place. Returns (q_out, k_out)."""
    r = _torch_ops.rotary(ws.handle.value, ws.device, q, k, positions, table, q_out, k_out, stream)
    if type(r) is int:
        _raise(ws, r, "arf_rotary")
    return r


def rotary_append(ws, q, k, v, positions, slots, table, cache: KVCache, q_out=None, stream=None):
    """Rotates q and k [T, heads, D] at positions [T] (int32) and writes the
    rotated k and v of token t to the cache at slots[t] (int64: page *
    page_size + row; negative: padding, nothing is written). Returns q_out.

    table=None appends k and v as they are; then q and positions must be None
    too. q=None rotates and appends k alone."""
    r = _torch_ops.rotary_append(ws.handle.value, ws.device, q, k, v, positions, slots, table, cache, q_out, stream)
    if type(r) is int:
        _raise(ws, r, "arf_rotary_append")
    return r


def paged_decode(ws, q, cache: KVCache, block_table, lens, scale=None, softcap: float = 0.0, window: int = 0,
                 out=None, lse=None, stream=None):
    """Attention of one new token per sequence: q [B, Hq, D] over the first
    lens[b] (int32) tokens of sequence b, whose pages block_table[b] (int32)
    names, or the last `window` of them (0: all). scale: D ** -0.5 when None;
    softcap > 0 caps scores at softcap * tanh(s / softcap). Returns (out [B,
    Hq, D], lse [B, Hq] float32); rows without tokens give 0 and -inf."""
    r = _torch_ops.paged_decode(ws.handle.value, ws.device, q, cache, block_table, lens, scale, softcap, window, out,
                                lse, stream)
    if type(r) is int:
        _raise(ws, r, "arf_paged_decode")
    return r


def copy_pages(ws, caches, src, dst, stream=None):
    """Copies page src[i] to page dst[i] in every cache of `caches` (one
    KVCache or a sequence of equal geometry). src, dst: host page numbers (a
    list or a CPU int32 tensor); no page may be a destination twice, or a
    source as well as a destination."""
    if isinstance(caches, KVCache):
        caches = (caches,)
    elif not isinstance(caches, (list, tuple)):
        caches = list(caches)
    st = _torch_ops.copy_pages(ws.handle.value, ws.device, caches, src, dst, stream)
    if st != B.ARF_OK:
        _raise(ws, st, "arf_copy_pages")


def bad_indices(ws) -> int:
    """Slots, table entries and lengths out of range that kernels have skipped
    since the last call (arf_workspace_bad_indices; waits for the device)."""
    n = ctypes.c_uint()
    st = B.arf_workspace_bad_indices(ws.handle, n)
    if st != B.ARF_OK:
        _raise(ws, st, "arf_workspace_bad_indices")
    return n.value


class PagePool:
    """Which sequence holds which pages of a cache (arf_pages_*): opening,
    growing, forking, closing and compacting, on the host."""

    def __init__(self, num_pages: int, page_size: int):
        self.handle = ctypes.c_void_p()
        self.page_size = page_size
        self._check(B.arf_pages_create(_int(num_pages, 32, "num_pages"), _int(page_size, 32, "page_size"), self.handle),
                    "arf_pages_create")

    @staticmethod
    def _check(st, what):
        if st != B.ARF_OK:
            raise B.ArfError(st, what)

    def open(self, tokens: int = 0) -> int:
        seq = ctypes.c_int32()
        self._check(B.arf_pages_open(self.handle, _int(tokens, 64, "tokens"), seq), "arf_pages_open")
        return seq.value

    def extend(self, seq: int, tokens: int = 1):
        """Returns the (src, dst) page copy to make first, or None."""
        src, dst = ctypes.c_int32(), ctypes.c_int32()
        self._check(B.arf_pages_extend(self.handle, _int(seq, 32, "sequence"), _int(tokens, 64, "tokens"), src, dst),
                    "arf_pages_extend")
        return (src.value, dst.value) if src.value >= 0 else None

    def fork(self, seq: int) -> int:
        child = ctypes.c_int32()
        self._check(B.arf_pages_fork(self.handle, _int(seq, 32, "sequence"), child), "arf_pages_fork")
        return child.value

    def free(self, seq: int) -> None:
        """Ends a sequence."""
        self._check(B.arf_pages_close(self.handle, _int(seq, 32, "sequence")), "arf_pages_close")

    def compact(self):
        """Moves pages down so that those in use come first; returns (src,
        dst), the copies to make with copy_pages, as CPU int32 tensors."""
        n = ctypes.c_int32()
        st = B.arf_pages_compact(self.handle, None, None, 0, n)
        while st == B.ARF_ERR_INVALID_ARG and n.value > 0:
            cap = n.value
            src, dst = torch.empty(cap, dtype=torch.int32), torch.empty(cap, dtype=torch.int32)
            st = B.arf_pages_compact(self.handle, src.data_ptr(), dst.data_ptr(), cap, n)
            if st == B.ARF_OK:
                return src[: n.value], dst[: n.value]
        self._check(st, "arf_pages_compact")
        return torch.empty(0, dtype=torch.int32), torch.empty(0, dtype=torch.int32)

    def pages(self, seq: int):
        """The sequence's page numbers, in order."""
        return self.block_table([seq])[0][0].tolist()[: self._size(seq)[0]]

    def length(self, seq: int) -> int:
        return self._size(seq)[1]

    def _size(self, seq):
        n, tokens = ctypes.c_int32(), ctypes.c_int64()
        self._check(B.arf_pages_table(self.handle, _int(seq, 32, "sequence"), None, 0, n, tokens), "arf_pages_table")
        return n.value, tokens.value

    def block_table(self, seqs, width: int | None = None):
        """(block_table [len(seqs), width], lens) as CPU int32 tensors for
        paged_decode; unused entries are -1."""
        seqs = [_int(s, 32, "sequence") for s in seqs]
        sizes = [self._size(s) for s in seqs]
        widest = max((n for n, _ in sizes), default=0)
        if width is not None and width < widest:
            raise ValueError(f"a sequence has {widest} pages, more than width {width}")
        width = widest if width is None else width
        table = torch.full((len(seqs), width), -1, dtype=torch.int32)
        n, tokens = ctypes.c_int32(), ctypes.c_int64()
        for i, s in enumerate(seqs):
            self._check(B.arf_pages_table(self.handle, s, table[i].data_ptr() if width else None, width, n, tokens),
                        "arf_pages_table")
        return table, torch.tensor([t for _, t in sizes], dtype=torch.int32)

    @property
    def free_pages(self) -> int:
        n = ctypes.c_int32()
        self._check(B.arf_pages_free(self.handle, n), "arf_pages_free")
        return n.value

    def close(self) -> None:
        if self.handle:
            B.arf_pages_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
