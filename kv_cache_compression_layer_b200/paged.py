"""Device buffers and calls of one paged 4-bit KV cache.

``PagedCache`` owns (or adopts) the arrays that include/kvcomp_paged.h
describes and checks what its methods are given (device, type, layout,
sizes); the work is done by the ``kv_paged_*`` entry points. Sequences are
named by their number in the cache; a method that takes ``layers=(first,
number)`` works on those layers of each sequence, one that does not on all.
Per-row tensors hold one entry per call row: (sequence in the order given,
layer, KV head).
"""
from __future__ import annotations

from contextlib import nullcontext
from typing import Optional, Sequence, Tuple

import torch

from . import (KV_BF16, KV_MAX_SEQ, kv_paged_append, kv_paged_attn, kv_paged_compact, kv_paged_copy, kv_paged_fork,
               kv_paged_free, kv_paged_load, kv_paged_page_bytes, kv_paged_rebuild, kv_paged_shape, kv_paged_ws_bytes,
               kv_read_device_status, make_paged_cache)


def on_stream(stream, device):
    """A context in which torch works on ``stream``: a torch stream, or a raw one's address (0: the default stream)."""
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


class PagedCache:
    """One cache: a pool of pages, the rows' page lists and lengths, and a workspace.

    ``pages`` [n_pages, page_bytes] uint8 (a pinned CPU tensor makes a cache that only copies
    reach: see ``copy_to``), ``table`` [rows, max_pages] and ``lens`` [rows] int32 adopt existing
    arrays, for instance a cache loaded from elsewhere; the holders' counts and the bitmap of free
    pages are made from them. Without them the cache starts empty.
    """

    def __init__(self, shape: kv_paged_shape, device=None, pages: Optional[torch.Tensor] = None,
                 table: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None):
        self.shape = shape
        if device is None:
            device = table.device if table is not None else "cuda"
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("the page lists are on a CUDA device (pages alone may be pinned host memory)")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        page_bytes = kv_paged_page_bytes(shape)
        if page_bytes == 0:
            raise ValueError("invalid shape")
        self.rows = shape.n_seqs * shape.n_layers * shape.n_kv_heads
        self.dtype = torch.bfloat16 if shape.dtype == KV_BF16 else torch.float32
        if (table is None) != (lens is None):
            raise ValueError("table and lens come together")
        self.on_host = pages is not None and pages.device.type == "cpu"
        if self.on_host and not pages.is_pinned():
            raise ValueError("pages on the host have to be pinned")
        if pages is None:
            pages = torch.zeros(shape.n_pages, page_bytes, dtype=torch.uint8, device=device)
        elif (pages.dtype != torch.uint8 or tuple(pages.shape) != (shape.n_pages, page_bytes)
              or not pages.is_contiguous()):
            raise ValueError(f"pages: a contiguous uint8 tensor of {(shape.n_pages, page_bytes)}")
        elif not self.on_host and pages.device != device:
            raise ValueError(f"pages: on {device}")
        if table is None:
            table = torch.zeros(self.rows, shape.max_pages, dtype=torch.int32, device=device)
            lens = torch.zeros(self.rows, dtype=torch.int32, device=device)
        self._is("table", table, torch.int32, self.rows * shape.max_pages)
        self._is("lens", lens, torch.int32, self.rows)
        self.pages, self.table, self.lens = pages, table, lens
        self.ref = torch.zeros(shape.n_pages, dtype=torch.int32, device=device)
        self.free_bits = torch.zeros((shape.n_pages + 31) // 32, dtype=torch.int32, device=device)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        with self._here():
            self.ws = torch.empty(kv_paged_ws_bytes(shape), dtype=torch.uint8, device=device)
            self.cache = make_paged_cache(self.pages, self.table, self.lens, self.ref, self.free_bits, self.status,
                                          self.ws)
            kv_paged_rebuild(shape, self.cache)

    # -- checks ----------------------------------------------------------------
    def _here(self):
        if self.device.index == torch.cuda.current_device():
            return nullcontext()
        return torch.cuda.device(self.device)

    def _on(self, stream):
        return self._here() if stream is None else on_stream(stream, self.device)

    def _is(self, name: str, x: torch.Tensor, dtype, numel: int, at_least: bool = False):
        if x.dtype != dtype or x.device != self.device or not x.is_contiguous():
            raise ValueError(f"{name}: a contiguous {dtype} tensor on {self.device}")
        if x.numel() < numel if at_least else x.numel() != numel:
            raise ValueError(f"{name}: {numel} elements, got {x.numel()}")

    def _call_rows(self, seqs: Sequence[int], layers: Optional[Tuple[int, int]]) -> Tuple[int, int, int]:
        l0, nl = (0, self.shape.n_layers) if layers is None else layers
        if l0 < 0 or nl < 1 or l0 + nl > self.shape.n_layers:
            raise ValueError(f"layers: (first, number) within {self.shape.n_layers}")
        if self.on_host:
            raise ValueError("the pages are on the host: copy the sequences to a cache on a device")
        if not 0 < len(seqs) <= KV_MAX_SEQ:
            raise ValueError(f"1 to {KV_MAX_SEQ} sequences a call")
        return l0, nl, len(seqs) * nl * self.shape.n_kv_heads

    # -- calls -----------------------------------------------------------------
    def append(self, seqs: Sequence[int], K: torch.Tensor, V: torch.Tensor, count: Optional[torch.Tensor] = None,
               src_off: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
               idx_off: Optional[torch.Tensor] = None, layers: Optional[Tuple[int, int]] = None, stream=None):
        """Quantises and stores tokens behind the rows' last.

        Without ``count``: K and V [call rows, n, head_dim] (or [call rows, head_dim] for one token
        each). With ``count`` (int32 [call rows]) and ``src_off`` (int64 [call rows]): K and V
        [n_src, head_dim], call row i taking its first count[i] rows from src_off[i] on, or with
        ``idx`` (int32) and ``idx_off`` (int64) rows src_off[i] + idx[idx_off[i] + t].
        """
        l0, nl, n = self._call_rows(seqs, layers)
        d = self.shape.head_dim
        if K.numel() % d or (K.dim() and K.shape[-1] != d):
            raise ValueError(f"K: rows of {d}")
        self._is("K", K, self.dtype, K.numel())
        self._is("V", V, self.dtype, K.numel())
        n_src = K.numel() // d
        n_each = 0
        if count is None:
            if src_off is not None or idx is not None:
                raise ValueError("src_off and idx go with count")
            if n_src % n:
                raise ValueError(f"K: a multiple of {n} rows")
            n_each = n_src // n
        else:
            self._is("count", count, torch.int32, n)
            if src_off is None:
                raise ValueError("count goes with src_off")
            self._is("src_off", src_off, torch.int64, n, at_least=True)
            if idx is not None:
                if idx_off is None:
                    raise ValueError("idx goes with idx_off")
                self._is("idx", idx, torch.int32, idx.numel())
                self._is("idx_off", idx_off, torch.int64, n, at_least=True)
                if idx.numel() == 0:  # an empty tensor has no address, which would mean "without idx":
                    idx = idx_off = None  # no token has a source
                    n_src = 0
        if count is None and n_src == 0:
            return
        with self._here():
            kv_paged_append(self.shape, self.cache, seqs, K, V, n_src, n_each, count, src_off, idx, idx_off, l0, nl,
                            stream)

    def load(self, seqs: Sequence[int], K_out: torch.Tensor, V_out: torch.Tensor, out_off: torch.Tensor,
             layers: Optional[Tuple[int, int]] = None, stream=None):
        """The rows' values: token t of call row i to row out_off[i] + t of K_out and V_out, while it is below
        out_off[i + 1] (int64 [call rows + 1], ascending)."""
        l0, nl, n = self._call_rows(seqs, layers)
        d = self.shape.head_dim
        if K_out.numel() % d or (K_out.dim() and K_out.shape[-1] != d):
            raise ValueError(f"K_out: rows of {d}")
        self._is("K_out", K_out, self.dtype, K_out.numel())
        self._is("V_out", V_out, self.dtype, K_out.numel())
        self._is("out_off", out_off, torch.int64, n + 1)
        if K_out.numel() == 0:
            return
        with self._here():
            kv_paged_load(self.shape, self.cache, seqs, out_off, K_out.numel() // d, K_out, V_out, l0, nl, stream)

    def attend(self, seqs: Sequence[int], q: torch.Tensor, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, n_q: int = 1, layers: Optional[Tuple[int, int]] = None,
               stream=None) -> torch.Tensor:
        """Attention of ``n_q`` query tokens a row, their own tokens appended before: q and out
        [call rows, n_q, group, head_dim] (any shape of as many elements), lse float32 [call rows,
        n_q, group] or None. Returns out (made on ``stream`` if it is not given)."""
        l0, nl, n = self._call_rows(seqs, layers)
        R = n_q * self.shape.group
        self._is("q", q, self.dtype, n * R * self.shape.head_dim)
        if lse is not None:
            self._is("lse", lse, torch.float32, n * R)
        if out is None:
            with self._on(stream):  # memory that `stream` may write to, whatever else is under way
                out = torch.empty_like(q)
        else:
            self._is("out", out, self.dtype, q.numel())
            if abs(out.data_ptr() - q.data_ptr()) < q.numel() * q.element_size():
                raise ValueError("out overlaps q")
        with self._here():
            kv_paged_attn(self.shape, self.cache, seqs, q, out, lse, n_q, l0, nl, stream)
        return out

    def fork(self, src: Sequence[int], dst: Sequence[int], stream=None):
        """dst[i] (empty) becomes a second holder of src[i]'s tokens; a src may be named more than once."""
        self._call_rows(src, None)
        with self._here():
            kv_paged_fork(self.shape, self.cache, src, dst, stream)

    def copy_to(self, other: "PagedCache", src: Sequence[int], dst: Sequence[int], stream=None):
        """Copies the pages of src[i] into pages of other's dst[i] (empty). Either cache's pages may be
        pinned host memory."""
        if other.device != self.device:
            raise ValueError("both caches keep their lists on one device")
        with self._here():
            kv_paged_copy(self.shape, self.cache, src, other.shape, other.cache, dst, stream)

    def compact(self, src: Sequence[int], dst: Sequence[int], idx: torch.Tensor, idx_off: torch.Tensor,
                count: torch.Tensor, stream=None):
        """dst[i] holds tokens idx[idx_off[r] + t], t < count[r], of src[i]'s rows r; dst[i] is src[i] (in place)
        or empty."""
        _, _, n = self._call_rows(src, None)
        self._is("idx", idx, torch.int32, idx.numel())
        self._is("idx_off", idx_off, torch.int64, n, at_least=True)
        self._is("count", count, torch.int32, n)
        if idx.numel() == 0:  # no list: a token that is asked for all the same has a position that no row has
            with self._on(stream):
                idx = torch.full((self.shape.max_pages * self.shape.page_tokens,), -1, dtype=torch.int32,
                                 device=self.device)
                idx_off = torch.zeros(n, dtype=torch.int64, device=self.device)
        with self._here():
            kv_paged_compact(self.shape, self.cache, src, dst, idx, idx_off, count, stream)

    def free(self, seqs: Sequence[int], stream=None):
        """The sequences become empty; pages that nothing else holds are free again."""
        with self._here():
            kv_paged_free(self.shape, self.cache, seqs, stream)

    # -- host views ------------------------------------------------------------
    def read_status(self) -> int:
        """The status word (KV_DEV_* bits) after all earlier work on the current stream (waits for it)."""
        with self._here():
            return kv_read_device_status(self.status)

    def free_pages(self) -> int:
        """Pages that no row holds (waits for earlier work)."""
        return int((self.ref == 0).sum())
