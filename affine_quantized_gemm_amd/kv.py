"""Paged K/V cache held in 4 bits: appending, attention, page bookkeeping.

Argument checks and marshalling only; every step runs in the HIP kernels of
``libqmm.so`` (``qmm_kv_*`` in ``include/qmm.h``, where the formats and
contracts are).  Tables, lengths and reference counts are int32 device
tensors that the kernels read when they run, so that a step that uses them
can be captured in a graph.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import (_DT, _lib, QMM_ERR_UNSUPPORTED, QmmError, _check, _dev, _dt, _expect, _same_device)

_I32 = torch.int32
ATTEND_ZEROED_BYTES = 65536  # QMM_KV_ATTEND_ZEROED_BYTES


class _Geometry(ctypes.Structure):  # qmm_kv_cache
    _fields_ = [("dt", ctypes.c_int32), ("group_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("layers", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("pool", ctypes.c_void_p)]


def record_words(head_dim: int, group_size: int, page_size: int, dtype=torch.float16) -> int:
    """int32 words of one record (one page of one layer and kv head)."""
    g = _Geometry(_dt(dtype), group_size, head_dim, 1, page_size, 1, 0, None)
    n = int(_lib.qmm_kv_record_bytes(ctypes.byref(g)))
    if n < 0:
        raise QmmError(n, f"head_dim={head_dim}, group_size={group_size}, page_size={page_size}")
    return n // 4


class KVCache:
    """A pool [layers, pages, kv_heads, words] (int32, GPU, contiguous) and its geometry.

    The pool is the caller's tensor (:meth:`empty` makes one).  Besides it the
    object keeps, for each stream that :meth:`attend` was called on without a
    workspace, one workspace; so calls on several streams may overlap, ordered
    by the caller as for any tensor.

    A call works on ``seqs`` sequences: ``tables`` [seqs, width] names their
    pages, ``lens`` [seqs] their lengths with the new tokens counted in.  The
    new tokens' rows are dense: without ``starts`` every sequence has the same
    number of them, else ``starts`` [seqs + 1] are the sequences' first rows
    and ``max_new`` bounds how many one has.
    """

    def __init__(self, pool: torch.Tensor, head_dim: int, group_size: int, page_size: int, dtype=torch.float16):
        words = record_words(head_dim, group_size, page_size, dtype)
        if pool.dim() != 4:
            raise ValueError(f"pool must be 4-D [layers, pages, kv_heads, words], got shape {tuple(pool.shape)}")
        layers, pages, kv_heads, _ = pool.shape
        _expect(pool, "pool", (layers, pages, kv_heads, words), (_I32,))
        _dev(pool, "pool")
        self.pool, self.dtype = pool, dtype
        self.layers, self.pages, self.kv_heads = layers, pages, kv_heads
        self.head_dim, self.group_size, self.page_size = head_dim, group_size, page_size
        self.device = pool.device
        self._scale = 1.0 / math.sqrt(head_dim)
        self._geometry = _Geometry(_DT[dtype], group_size, head_dim, kv_heads, page_size, layers, pages,
                                   pool.data_ptr())
        self._c = ctypes.byref(self._geometry)
        self._spaces: dict[int, torch.Tensor] = {}
        self._most_space = ATTEND_ZEROED_BYTES + 32768 * (head_dim + 4)  # the bound qmm.h gives
        if layers < 1 or kv_heads < 1:
            raise QmmError(QMM_ERR_UNSUPPORTED, f"pool {tuple(pool.shape)}")

    @classmethod
    def empty(cls, layers: int, pages: int, kv_heads: int, head_dim: int, group_size: int = 64, page_size: int = 64,
              dtype=torch.float16, device="cuda") -> "KVCache":
        """A cache with a pool of its own (contents unset: nothing reads a slot that was not appended to)."""
        words = record_words(head_dim, group_size, page_size, dtype)
        pool = torch.empty((layers, pages, kv_heads, words), dtype=_I32, device=device)
        return cls(pool, head_dim, group_size, page_size, dtype)

    # ---- checks (a call's host time is a good part of a small step: few attribute reads) ----

    def _ints(self, t, name, shape=None):
        if isinstance(t, torch.Tensor) and t.dtype is _I32 and t.is_contiguous() and t.device == self.device \
                and (shape is None or t.shape == shape):
            return t.data_ptr()
        raise ValueError(f"{name} must be a contiguous int32 tensor"
                         f"{'' if shape is None else ' of shape ' + str(tuple(shape))} on {self.device}")

    def _seqs(self, layer, rows, tables, lens, starts, max_new):
        """The arguments from cache to starts that append, read and attend share."""
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of {self.layers}")
        if tables.dim() != 2:
            raise ValueError(f"tables must be 2-D [seqs, width], got shape {tuple(tables.shape)}")
        seqs, width = tables.shape
        if starts is None:
            if max_new is None:
                max_new = rows // seqs if seqs else 0
            if rows != seqs * max_new:
                raise ValueError(f"{rows} rows are not the same number for each of {seqs} sequences: give starts")
            first = None
        else:
            if max_new is None:
                raise ValueError("starts needs max_new, a bound of one sequence's new tokens")
            first = self._ints(starts, "starts", (seqs + 1,))
            if rows > seqs * max_new:
                raise ValueError(f"{rows} rows are more than {seqs} sequences of at most {max_new}")
        return (self._c, layer, seqs, max_new, rows, self._ints(tables, "tables"), width,
                self._ints(lens, "lens", (seqs,)), first)

    def _rows(self, t, name, heads=None):
        """Address and strides of a [rows, heads, head_dim] operand (heads and rows may be strided)."""
        if t.dim() != 3 or t.shape[2] != self.head_dim or (heads is not None and t.shape[1] != heads):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                             f"[rows, {'heads' if heads is None else heads}, {self.head_dim}]")
        if t.dtype is not self.dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {self.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, expected {self.device}")
        r, h, d = t.stride()
        if d != 1:
            raise ValueError(f"{name}'s last axis must be contiguous")
        return t.data_ptr(), r, h

    def _new(self, shape, strides, dtype, stream):
        """A tensor of this call; where the call runs on another stream than the current one, that stream's."""
        if stream is None:
            return torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        with torch.cuda.stream(self._as_stream(stream)):
            return torch.empty_strided(shape, strides, dtype=dtype, device=self.device)

    def _as_stream(self, stream):
        return stream if isinstance(stream, torch.cuda.Stream) else \
            torch.cuda.ExternalStream(int(stream), device=self.device)

    def _space(self, workspace, need, stream):
        if workspace is None:
            if need == 0:
                return None, 0
            workspace = self._new((need,), (1,), torch.uint8, stream)
        else:
            _dev(workspace, "workspace")
            _same_device(self.pool, (workspace, "workspace"))
        # (a temporary's block goes back to the caching allocator, which hands it out again in stream order)
        return workspace, workspace.numel() * workspace.element_size()

    def _raw(self, stream) -> int:
        """Address of the stream of a call (torch's own lookup behind current_stream(), without the object)."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        return int(getattr(stream, "cuda_stream", stream))

    def attend_workspace(self, *sizes: int) -> torch.Tensor:
        """A workspace for :meth:`attend` calls (one per stream, or per captured graph): of the sizes given, as in
        :meth:`attend_workspace_bytes`, or without them of any sizes.  (Fewer sequences can need more.)"""
        need = self.attend_workspace_bytes(*sizes) if sizes else self._most_space
        return torch.zeros((max(need, 16),), dtype=torch.uint8, device=self.device)

    def _own_space(self, stream, raw: int, *sizes: int):
        """Workspace of an :meth:`attend` call that was not given one, and its bytes: the one kept for the stream,
        zeroed when made and large enough for every call.  A call that is being captured gets one of its own, of the
        sizes it needs, whose counters are zeroed in the graph; or none where it needs none."""
        if stream is None:
            if not torch.cuda.is_current_stream_capturing():
                kept = self._spaces.get(raw)
                if kept is None:
                    kept = self._spaces[raw] = torch.zeros((self._most_space,), dtype=torch.uint8, device=self.device)
                return kept, self._most_space
            need = self.attend_workspace_bytes(*sizes)
            if need == 0:
                return None, 0
            own = torch.empty((need,), dtype=torch.uint8, device=self.device)
            own[:ATTEND_ZEROED_BYTES].zero_()
            return own, need
        with torch.cuda.stream(self._as_stream(stream)):  # its state of capture, its memory
            return self._own_space(None, raw, *sizes)

    # ---- tokens ----

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor,
               starts: torch.Tensor | None = None, max_new: int | None = None, stream=None) -> None:
        """Quantize the new tokens' k and v [rows, kv_heads, head_dim] into their places in ``layer``."""
        rows = k.shape[0]
        if v.shape != k.shape:
            raise ValueError(f"v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
        _check(_lib.qmm_kv_append(*self._seqs(layer, rows, tables, lens, starts, max_new),
                                  *self._rows(k, "k", self.kv_heads), *self._rows(v, "v", self.kv_heads),
                                  self._raw(stream)), "qmm_kv_append")

    def read(self, layer: int, rows: int, tables: torch.Tensor, lens: torch.Tensor,
             starts: torch.Tensor | None = None, max_new: int | None = None, stream=None):
        """(k, v) [rows, kv_heads, head_dim]: what ``layer`` holds of the sequences' last tokens, dequantized."""
        args = self._seqs(layer, rows, tables, lens, starts, max_new)
        shape, strides = (rows, self.kv_heads, self.head_dim), (self.kv_heads * self.head_dim, self.head_dim, 1)
        k, v = self._new(shape, strides, self.dtype, stream), self._new(shape, strides, self.dtype, stream)
        _check(_lib.qmm_kv_read(*args, k.data_ptr(), v.data_ptr(), self._raw(stream)), "qmm_kv_read")
        return k, v

    def attend_workspace_bytes(self, seqs: int, max_new: int, rows: int, heads: int, max_len: int) -> int:
        """Bytes of workspace :meth:`attend` needs (0: none)."""
        n = int(_lib.qmm_kv_attend_workspace_bytes(self._c, seqs, max_new, rows, heads, max_len))
        if n < 0:
            raise QmmError(n, "qmm_kv_attend_workspace_bytes")
        return n

    def attend(self, layer: int, q: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor,
               starts: torch.Tensor | None = None, max_new: int | None = None, mask: torch.Tensor | None = None,
               scale: float | None = None, max_len: int | None = None, out: torch.Tensor | None = None,
               lse: bool | torch.Tensor = False, workspace: torch.Tensor | None = None, stream=None):
        """Attention of the new tokens' q [rows, heads, head_dim] over ``layer``: out [rows, heads, head_dim].

        A row sees all tokens before its sequence's new ones and of these the
        ones up to itself, or with ``mask`` (int64 [rows]) the new tokens j
        whose bit j its word has set.  A row that sees nothing gives zeros.
        ``scale`` defaults to 1/sqrt(head_dim).  ``max_len`` bounds the
        lengths for the split of the work (default: what the tables hold).
        ``workspace``: from :meth:`attend_workspace` (default: one that the
        cache keeps for the stream).
        ``lse``: True, or an fp32 tensor [rows, heads], for (out, lse).
        """
        ptr, qr, qh = self._rows(q, "q")
        rows, heads, _ = q.shape
        args = self._seqs(layer, rows, tables, lens, starts, max_new)
        if out is None:
            out = self._new((rows, heads, self.head_dim), (heads * self.head_dim, self.head_dim, 1), self.dtype, stream)
        else:
            _expect(out, "out", (rows, heads, self.head_dim), (self.dtype,))
            _dev(out, "out")
            _same_device(q, (out, "out"))
        if lse is True:
            lse = self._new((rows, heads), (heads, 1), torch.float32, stream)
        elif lse is not False:
            _expect(lse, "lse", (rows, heads), (torch.float32,))
            _dev(lse, "lse")
            _same_device(q, (lse, "lse"))
        if mask is not None:
            _expect(mask, "mask", (rows,), (torch.int64,))
            _dev(mask, "mask")
            _same_device(q, (mask, "mask"))
        if max_len is None:
            max_len = max(1, args[6] * self.page_size)
        raw = self._raw(stream)
        if workspace is None:
            workspace, nbytes = self._own_space(stream, raw, args[2], args[3], rows, heads, max_len)
        else:
            _dev(workspace, "workspace")
            _same_device(q, (workspace, "workspace"))
            nbytes = workspace.numel() * workspace.element_size()
        _check(_lib.qmm_kv_attend(*args, ptr, qr, qh, heads, self._scale if scale is None else scale,
                                  None if mask is None else mask.data_ptr(), out.data_ptr(),
                                  None if lse is False else lse.data_ptr(), max_len,
                                  None if workspace is None else workspace.data_ptr(), nbytes, raw), "qmm_kv_attend")
        return out if lse is False else (out, lse)

    # ---- pages ----

    def _book(self, tables, lens, refs):
        """seqs, tables, width, lens, refs of the page calls."""
        if tables.dim() != 2:
            raise ValueError(f"tables must be 2-D [seqs, width], got shape {tuple(tables.shape)}")
        seqs, width = tables.shape
        return (seqs, self._ints(tables, "tables"), width, self._ints(lens, "lens", (seqs,)),
                self._ints(refs, "refs", (self.pages,)))

    def pages_workspace_bytes(self, n: int) -> int:
        """Bytes of workspace of :meth:`reserve` (n sequences), :meth:`fork` (n pairs), :meth:`compact` (0)."""
        r = int(_lib.qmm_kv_pages_workspace_bytes(self._c, n))
        if r < 0:
            raise QmmError(r, "qmm_kv_pages_workspace_bytes")
        return r

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Page dst[i] <- page src[i] in every layer (int32 device tensors)."""
        n = src.numel()
        _check(_lib.qmm_kv_copy_pages(self._c, self._ints(src, "src", (n,)), self._ints(dst, "dst", (n,)), n,
                                      self._raw(stream)), "qmm_kv_copy_pages")

    def reserve(self, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, add: torch.Tensor,
                ok: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Room for add[s] more tokens of every sequence: pages taken, lens grown; returns ok [seqs] (1 or 0)."""
        book = self._book(tables, lens, refs)
        seqs = book[0]
        ap = self._ints(add, "add", (seqs,))
        if ok is None:
            ok = self._new((seqs,), (1,), _I32, stream)
        workspace, nbytes = self._space(workspace, self.pages_workspace_bytes(seqs), stream)
        _check(_lib.qmm_kv_reserve(self._c, *book, ap, self._ints(ok, "ok", (seqs,)),
                                   None if workspace is None else workspace.data_ptr(), nbytes, self._raw(stream)),
               "qmm_kv_reserve")
        return ok

    def fork(self, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, src: torch.Tensor,
             dst: torch.Tensor, ok: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
        """Sequence dst[i] becomes a copy of src[i]: whole pages shared, a partly filled last one copied.

        dst rows hold nothing before.  Returns ok [n]: 0 where no page was left."""
        book = self._book(tables, lens, refs)
        n = src.numel()
        if ok is None:
            ok = self._new((n,), (1,), _I32, stream)
        workspace, nbytes = self._space(workspace, self.pages_workspace_bytes(n), stream)
        _check(_lib.qmm_kv_fork(self._c, *book, self._ints(src, "src", (n,)), self._ints(dst, "dst", (n,)), n,
                                self._ints(ok, "ok", (n,)), None if workspace is None else workspace.data_ptr(),
                                nbytes, self._raw(stream)), "qmm_kv_fork")
        return ok

    def free(self, tables: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, which: torch.Tensor,
             stream=None) -> None:
        """Give up every page of the sequences ``which``; their rows become -1 and their lengths 0."""
        n = which.numel()
        _check(_lib.qmm_kv_free(self._c, *self._book(tables, lens, refs), self._ints(which, "which", (n,)), n,
                                self._raw(stream)), "qmm_kv_free")

    def compact(self, tables: torch.Tensor, refs: torch.Tensor, tables_out: torch.Tensor | None = None,
                refs_out: torch.Tensor | None = None, live: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
        """Move the live pages into the lowest ids; returns (tables, refs) rewritten for that.

        ``tables_out`` and ``refs_out`` may be ``tables`` and ``refs``; ``live``
        (int32 [1]) gets the number of live pages."""
        if tables.dim() != 2:
            raise ValueError(f"tables must be 2-D [seqs, width], got shape {tuple(tables.shape)}")
        seqs, width = tables.shape
        tp, rp = self._ints(tables, "tables"), self._ints(refs, "refs", (self.pages,))
        if tables_out is None:
            tables_out = self._new((seqs, width), (width, 1), _I32, stream)
        if refs_out is None:
            refs_out = self._new((self.pages,), (1,), _I32, stream)
        if live is None:
            live = self._new((1,), (1,), _I32, stream)
        workspace, nbytes = self._space(workspace, self.pages_workspace_bytes(0), stream)
        _check(_lib.qmm_kv_compact(self._c, seqs, tp, width, rp, self._ints(tables_out, "tables_out", (seqs, width)),
                                   self._ints(refs_out, "refs_out", (self.pages,)), self._ints(live, "live", (1,)),
                                   workspace.data_ptr(), nbytes, self._raw(stream)), "qmm_kv_compact")
        return tables_out, refs_out
