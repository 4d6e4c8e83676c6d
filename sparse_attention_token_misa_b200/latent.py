"""The latent key/value cache in 16, 8 or 4 bits and the attention that reads it.

Bindings of include/misa_latent.h (argument marshalling only), and LatentCache,
which keeps a cache, its lengths and the workspaces of one batch together.

A cache is a tensor [nseq, L, row]: bf16 rows of 576 ("bf16"), or uint8 rows of
656 ("mx8") or 400 bytes ("mx4").  The form is read off the tensor.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import _native as nat
from ._native import MLA_DQK, MLA_DV, _call, _p, _req, _shape

KV_FORMS = {"bf16": 0, "mx8": 1, "mx4": 2}       # MISA_KV_BF16, MISA_KV_MX8, MISA_KV_MX4
_ROW_BYTES = {"bf16": 1152, "mx8": 656, "mx4": 400}
_FORM_OF = {(torch.bfloat16, MLA_DQK): "bf16", (torch.uint8, 656): "mx8", (torch.uint8, 400): "mx4"}


def kv_row_bytes(form: str) -> int:
    """Bytes of one cache row in this form."""
    if form not in KV_FORMS:
        raise ValueError(f"form must be one of {tuple(KV_FORMS)}")
    return int(nat.lib().misa_kv_row_bytes(KV_FORMS[form]))


def alloc_kv_cache(nseq: int, L: int, form: str, device=None) -> torch.Tensor:
    """A cache of nseq sequences of L rows, zeroed (every row reads back as zeros)."""
    kv_row_bytes(form)
    if form == "bf16":
        return torch.zeros((nseq, L, MLA_DQK), dtype=torch.bfloat16, device=device or "cuda")
    return torch.zeros((nseq, L, _ROW_BYTES[form]), dtype=torch.uint8, device=device or "cuda")


def _cache_form(cache: torch.Tensor) -> str:
    shape = cache.shape
    form = _FORM_OF.get((cache.dtype, shape[2])) if len(shape) == 3 else None
    if form is not None:
        if cache.stride()[1:] != (shape[2], 1):
            raise ValueError("cache rows must be contiguous and follow one another")
        return form
    raise ValueError("cache: expected shape [nseq, L, 576] bf16 or [nseq, L, 656 or 400] uint8, got "
                     f"{tuple(cache.shape)} {cache.dtype}")


def _dims(t: torch.Tensor, name: str, *dims: int) -> None:
    """_shape for sizes that are all known: one comparison where they fit."""
    if t.shape != dims:
        _shape(t, name, *dims)


def _ptr(t):
    """The address of a tensor that _on has looked at."""
    return None if t is None else t.data_ptr()


def _seq_stride(cache: torch.Tensor) -> int:
    return int(cache.stride(0)) * cache.element_size() if cache.shape[0] > 1 else 0


def _idx_stride(idx: torch.Tensor) -> int:
    """Elements between the rows of idx (torch leaves any stride on a single row)."""
    return int(idx.stride(0)) if idx.shape[0] > 1 else idx.shape[1]


def _on(first: torch.Tensor, stream, *others):
    """A context with the device of `first` made current (the library launches
    there; every tensor has to be on it), and `stream`, so that what a call
    allocates for itself belongs to the stream that uses it."""
    device = first.get_device()
    if device < 0:
        _p(first)
    for t in others:
        if t is not None and t.get_device() != device:
            _p(t)
            raise ValueError(f"tensors on {first.device} and {t.device}")
    if stream is None and device == torch.cuda.current_device():
        return contextlib.nullcontext(torch.cuda.current_stream(device).cuda_stream)
    return _switched(first.device, stream)


@contextlib.contextmanager
def _switched(device: torch.device, stream):
    with torch.cuda.device(device):
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream is not None and stream.device != device:
            raise ValueError(f"tensors on {device}, stream on {stream.device}")
        with torch.cuda.stream(stream):
            yield torch.cuda.current_stream().cuda_stream


def append_kv(cache: torch.Tensor, lens: torch.Tensor, rows: torch.Tensor, counts: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> None:
    """misa_append_kv: rows [nseq, n_new, 576] bf16, the first counts[b] (None:
    all) of each sequence, go to rows [lens[b], lens[b] + counts[b]) of cache,
    quantised to its form.  lens is not advanced."""
    form = _cache_form(cache)
    _req(rows, torch.bfloat16, "rows")
    _req(lens, torch.int32, "lens")
    nseq, L_cap, _ = cache.shape
    _shape(rows, "rows", nseq, None, MLA_DQK)
    _dims(lens, "lens", nseq)
    if counts is not None:
        _dims(counts, "counts", nseq)
        _req(counts, torch.int32, "counts")
    if rows.shape[1] == 0:
        return
    with _on(cache, stream, lens, rows, counts, workspace) as s:
        ws = workspace if workspace is not None else nat.alloc_workspace(256, cache.device)
        _call("misa_append_kv", _ptr(rows), nseq, rows.shape[1], _ptr(counts), _ptr(lens), KV_FORMS[form], _ptr(cache),
              _seq_stride(cache), L_cap, _ptr(ws), ws.numel(), s)


def read_kv(cache: torch.Tensor, seq_of: torch.Tensor, idx: torch.Tensor | None = None,
            first: torch.Tensor | None = None, n: int | None = None, prefix_len: torch.Tensor | None = None,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """misa_read_kv -> [T, n, 576] bf16: the rows idx [T, n] (-1: zeros) of cache
    seq_of[t], or n rows from first[t] (None: 0) on, zeros at and past prefix_len[t]
    (None: the cache's length)."""
    form = _cache_form(cache)
    nseq, L, _ = cache.shape
    _req(seq_of, torch.int32, "seq_of"); _shape(seq_of, "seq_of", None)
    T = seq_of.shape[0]
    if idx is not None:
        if first is not None or prefix_len is not None or n is not None:
            raise ValueError("idx goes without first, n and prefix_len")
        _req(idx, torch.int32, "idx", contiguous=False); _shape(idx, "idx", T, None)
        if idx.stride(1) != 1:
            raise ValueError("idx rows must be contiguous")
        n = idx.shape[1]
    elif n is None:
        raise ValueError("read_kv takes idx or n")
    for name, t in (("first", first), ("prefix_len", prefix_len)):
        if t is not None:
            _req(t, torch.int32, name); _dims(t, name, T)
    if out is not None:
        _req(out, torch.bfloat16, "out"); _dims(out, "out", T, n, MLA_DQK)
    with _on(cache, stream, seq_of, idx, first, prefix_len, out, workspace) as s:
        if out is None:
            out = cache.new_empty((T, n, MLA_DQK), dtype=torch.bfloat16)
        ws = workspace if workspace is not None else nat.alloc_workspace(256, cache.device)
        _call("misa_read_kv", _ptr(cache), KV_FORMS[form], nseq, _seq_stride(cache), L, _ptr(seq_of), T, _ptr(idx),
              _idx_stride(idx) if idx is not None else 0, _ptr(first), _ptr(prefix_len), n, _ptr(out), _ptr(ws),
              ws.numel(), s)
    return out


def _attend(op: int, q, cache, seq_of, per_query, scale, out, lse, want_lse, workspace, stream):
    """Shared marshalling of the two attention calls; per_query is idx or prefix_len."""
    form = _cache_form(cache)
    sparse = op == nat.OP_SPARSE_MLA_Q
    if sparse and form == "bf16":
        raise ValueError("sparse_mla_q reads a quantised cache; sparse_mla reads bf16 rows")
    if not (math.isfinite(scale) and scale >= 0):
        raise ValueError("scale must be finite and not negative")
    _req(q, torch.bfloat16, "q"); _req(seq_of, torch.int32, "seq_of")
    _shape(q, "q", None, None, MLA_DQK)
    T, Hq, _ = q.shape
    nseq, L, _ = cache.shape
    _dims(seq_of, "seq_of", T)
    if out is not None:
        _req(out, torch.bfloat16, "out"); _dims(out, "out", T, Hq, MLA_DV)
    if lse is not None:
        _req(lse, torch.float32, "lse"); _dims(lse, "lse", T, Hq)
    with _on(q, stream, cache, seq_of, per_query, out, lse, workspace) as s:
        if out is None:
            out = q.new_empty((T, Hq, MLA_DV))
        if lse is None and want_lse:
            lse = q.new_empty((T, Hq), dtype=torch.float32)
        ws = workspace
        if ws is None:
            k = per_query.shape[1] if sparse else 0
            ws = torch.empty(nat.workspace_bytes(op, T, Hq, L, 0, k), dtype=torch.uint8, device=q.device)
            ws[:256].zero_()   # the error word; partial results are written before they are read
        head = (_ptr(q), _ptr(cache), KV_FORMS[form], nseq, _seq_stride(cache), L, _ptr(seq_of))
        tail = (float(scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), s)
        if sparse:
            _call("misa_sparse_mla_q", *head, T, Hq, _ptr(per_query), per_query.shape[1], _idx_stride(per_query), *tail)
        else:
            _call("misa_prefix_mla", *head, _ptr(per_query), T, Hq, *tail)
    return out, lse


def sparse_mla_q(q, cache, seq_of, idx, scale: float, out=None, lse=None, want_lse: bool = False, workspace=None,
                 stream=None):
    """misa_sparse_mla_q -> (out [T, Hq, 512] bf16, lse [T, Hq] fp32 or None): q [T,
    Hq, 576] bf16 over the rows idx [T, k] int32 (-1 = empty) of a quantised cache."""
    _req(idx, torch.int32, "idx", contiguous=False)
    _shape(idx, "idx", q.shape[0], None)
    if idx.stride(1) != 1:
        raise ValueError("idx rows must be contiguous")
    return _attend(nat.OP_SPARSE_MLA_Q, q, cache, seq_of, idx, scale, out, lse, want_lse, workspace, stream)


def prefix_mla(q, cache, seq_of, prefix_len, scale: float, out=None, lse=None, want_lse: bool = False,
               workspace=None, stream=None):
    """misa_prefix_mla -> (out [T, Hq, 512] bf16, lse [T, Hq] fp32 or None): q [T,
    Hq, 576] bf16 over the rows below prefix_len [T] int32 of a cache in any form."""
    _req(prefix_len, torch.int32, "prefix_len")
    _dims(prefix_len, "prefix_len", q.shape[0])
    return _attend(nat.OP_PREFIX_MLA, q, cache, seq_of, prefix_len, scale, out, lse, want_lse, workspace, stream)


class LatentCache:
    """The latent caches of nseq sequences with their lengths, and the buffers of
    one batch of T queries: append and attend allocate nothing and can be
    captured in a CUDA graph (lens advances on the device).

    attend and attend_prefix have outputs of their own, which the next call of the
    same one overwrites; out and lse are those of the last call of either."""

    def __init__(self, nseq: int, L: int, form: str, T: int, Hq: int, k: int, device="cuda"):
        self.nseq, self.L, self.form, self.T, self.Hq, self.k = nseq, L, form, T, Hq, k
        self.rows = alloc_kv_cache(nseq, L, form, device)
        self.lens = torch.zeros(nseq, dtype=torch.int32, device=device)
        self._new_lens = torch.empty_like(self.lens)    # append's temporaries
        self._fits, self._also = (torch.empty(nseq, dtype=torch.bool, device=device) for _ in range(2))
        self._listed, self._prefix = ((torch.empty((T, Hq, MLA_DV), dtype=torch.bfloat16, device=device),
                                       torch.empty((T, Hq), dtype=torch.float32, device=device)) for _ in range(2))
        self.out, self.lse = self._listed
        self.ws = nat.alloc_workspace(256, device)
        op = nat.OP_SPARSE_MLA if form == "bf16" else nat.OP_SPARSE_MLA_Q
        self.ws_sparse = nat.alloc_workspace(nat.workspace_bytes(op, T, Hq, L, 0, k), device)
        self.ws_prefix = nat.alloc_workspace(nat.workspace_bytes(nat.OP_PREFIX_MLA, T, Hq, L, 0), device)

    def append(self, rows: torch.Tensor, counts: torch.Tensor | None = None) -> None:
        """Write new rows behind each sequence's last one and advance its length.  A
        sequence whose rows no longer fit (or whose count or length is out of range)
        is left as it was, as misa_append_kv skips it and records it in `ws`."""
        append_kv(self.rows, self.lens, rows, counts=counts, workspace=self.ws)
        n = rows.shape[1]
        lens, new, fits, also = self.lens, self._new_lens, self._fits, self._also
        if counts is None:
            if n <= self.L:
                torch.clamp(lens, 0, self.L - n, out=new)
                torch.eq(new, lens, out=fits)
                lens.add_(fits, alpha=n)
            return
        torch.clamp(counts, 0, n, out=new)
        torch.eq(new, counts, out=fits)
        torch.add(lens, counts, out=new)
        fits.logical_and_(torch.le(new, self.L, out=also))
        fits.logical_and_(torch.ge(new, counts, out=also))   # (a length below zero, or past 2^31, gives less)
        torch.where(fits, new, lens, out=lens)

    def attend(self, q, seq_of, idx, scale: float):
        """Over the tokens the indexer lists -> (out, lse)."""
        self.out, self.lse = self._listed
        if self.form == "bf16":
            with _on(self.rows, None, q, seq_of, idx, self.out, self.lse, self.ws_sparse) as s:
                return nat.sparse_mla(q, self.rows, seq_of, idx, scale, out=self.out, lse=self.lse,
                                      workspace=self.ws_sparse, stream=s)
        return sparse_mla_q(q, self.rows, seq_of, idx, scale, out=self.out, lse=self.lse, workspace=self.ws_sparse)

    def attend_prefix(self, q, seq_of, prefix_len, scale: float):
        """Over the whole prefix -> (out, lse)."""
        self.out, self.lse = self._prefix
        return prefix_mla(q, self.rows, seq_of, prefix_len, scale, out=self.out, lse=self.lse,
                          workspace=self.ws_prefix)
