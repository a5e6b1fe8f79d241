"""bpe_trie_encode_gb300 -- byte-level BPE training and greedy trie encoding on
one GB300 (sm_103a).

The work happens in ``libbpetrie.so`` (hand-written CUDA kernels behind the C
ABI of ``include/bpetrie.h``); this package marshals torch tensors to it.
PyTorch is used only for device memory and streams.

    import torch, bpe_trie_encode_gb300 as bt
    ctx = bt.Context()
    sym = ctx.pretokenize(torch.frombuffer(text, dtype=torch.uint8).cuda())
    merges, final = ctx.train(sym, 4096)
    trie = ctx.trie_build(*bt.vocab_from_merges(merges))
    ids, id_off = ctx.encode(trie, data_u8_cuda, doc_off_i64_cuda)
    uni = ctx.unigram(trie, scores_f64, unk_id, unk_score)       # Viterbi model
    ids, id_off = ctx.unigram_encode(uni, data_u8_cuda, doc_off_i64_cuda)

The output head of a model over the same vocabulary (``examples/generate.py``):

    w8, ws = ctx.head_quantize(weight)                           # once
    x8, xs, stream = ctx.head_norm(hidden, norm_weight, residual)
    logits = ctx.head_logits(x8, xs, w8, ws)
    ids, logprob = ctx.head_sample(logits, u, temperature=0.8, top_p=0.95)
    text = ctx.decode(merges, ids)
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _capi
from ._capi import (BPE_MAX_MERGES, BPE_MERGE_LISTS, BPE_MERGE_LOOKBACK, BPE_MERGE_TILES,  # noqa: F401
                    BPE_MERGE_TWO_PASS, BPE_OPT_LIST_FRONTIER, BPE_OPT_LIST_TAIL,
                    BPE_OPT_CHUNK, BPE_OPT_GRAPH, BPE_OPT_MERGE, BPE_OPT_PERSISTENT, BPE_OPT_PROFILE,
                    BPE_OPT_SPARSE_MERGE, BPE_OPT_TABLE_LOG2, BPE_OPT_TRAIN_WORDS, BPE_OPT_TRIE_LAYOUT,
                    BPE_OPT_UNI_CHUNK, BPE_TRIE_BITMAP, BPE_TRIE_DOUBLE_ARRAY, BPE_WORD_START, BpeError)

__all__ = ["Context", "Trie", "Unigram", "BpeError", "vocab_from_merges", "BPE_WORD_START", "BPE_MAX_MERGES"]


# the current stream's handle without a Stream object around it, where torch has that (2 us of a call's 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need_cuda(t: torch.Tensor, dtype: torch.dtype, name: str, device: torch.device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the context is on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.contiguous()


_HEAD_TYPES = {torch.float32: _capi.BPE_F32, torch.bfloat16: _capi.BPE_BF16, torch.float16: _capi.BPE_F16}
_E4M3 = torch.float8_e4m3fn
_HEAD_MOST = 0x7FFFFFFF   # ctypes cuts what does not fit the library's 32 bits without a word


def _head_place(t, name: str, device: torch.device, dtypes) -> None:
    """The error of a tensor that is not a CUDA tensor of the context's device and of one of the types."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, the context is on {device}")


def _head_matrix(t: torch.Tensor, name: str, device: torch.device, dtypes, shape=None, out: bool = False):
    """(matrix, distance of its rows): a CUDA matrix whose rows are contiguous; an input is copied where they are not."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype not in dtypes:
        _head_place(t, name, device, dtypes)
    size, stride = t.shape, t.stride()
    if len(stride) != 2 or (shape is not None and size != shape):
        raise ValueError(f"{name} must be {'a matrix' if shape is None else tuple(shape)}, got {tuple(size)}")
    if size[0] > _HEAD_MOST or size[1] > _HEAD_MOST:
        raise ValueError(f"{name}: {tuple(size)} has a size above {_HEAD_MOST}")
    if (stride[1] != 1 and size[1] > 1) or (stride[0] < size[1] and size[0] > 1):
        if out:
            raise ValueError(f"{name}: the rows of an output must be contiguous and apart")
        t = t.contiguous()
        return t, t.stride(0)
    return t, stride[0]


def _head_scales(t: torch.Tensor, name: str, device: torch.device, rows: int, blocks: int, out: bool = False):
    """The distances of rows and of blocks.  Scales may lie in any order; those of an output may not share a place."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype is not torch.float32:
        _head_place(t, name, device, (torch.float32,))
    if t.shape != (rows, blocks):
        raise ValueError(f"{name} must be {(rows, blocks)}, got {tuple(t.shape)}")
    s0, s1 = t.stride()
    if out and not (0 < s1 * blocks <= s0 or 0 < s0 * rows <= s1):
        (a, n), (b, m) = sorted(((s0, rows), (s1, blocks)))
        if (n > 1 and a == 0) or (m > 1 and b < (n - 1) * a + 1):
            raise ValueError(f"{name}: the scales of an output must lie apart")
    return s0, s1


def _head_vector(t: torch.Tensor, name: str, device: torch.device, dtype: torch.dtype, rows: int,
                 out: bool = False) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype is not dtype:
        _head_place(t, name, device, (dtype,))
    if t.shape != (rows,):
        raise ValueError(f"{name} must be ({rows},), got {tuple(t.shape)}")
    if rows > 1 and t.stride(0) != 1:
        if out:
            raise ValueError(f"{name}: an output must be contiguous")
        t = t.contiguous()
    return t


def _head_count(k):
    """A number of tokens as the library's 32 bits hold it: none of its vocabularies has as many as the largest."""
    return max(-1, min(k, _HEAD_MOST))


class Trie:
    """A double-array trie uploaded to the GPU (see ``Context.trie_build``)."""

    def __init__(self, handle: int, device: torch.device, n_tok: int):
        self._h = ctypes.c_void_p(handle)
        self.device = device
        self.n_tok = n_tok

    def info(self) -> dict:
        n_nodes, n_slots, max_len = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint32()
        _capi.load().trie_info(self._h, ctypes.byref(n_nodes), ctypes.byref(n_slots), ctypes.byref(max_len))
        return {"n_tok": self.n_tok, "n_nodes": n_nodes.value, "n_slots": n_slots.value,
                "max_token_len": max_len.value}

    def close(self):
        if self._h:
            _capi.load().trie_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Context:
    """A library context on one CUDA device.  Calls are ordered on the torch
    current stream of that device at the time of each call."""

    def __init__(self, device=None):
        if not torch.cuda.is_available():
            raise RuntimeError("bpe_trie_encode_gb300 needs a CUDA GPU")
        self.lib = _capi.load()
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index or 0)
        h = ctypes.c_void_p()
        rc = self.lib.bpe_ctx_create(ctypes.byref(h), self.device.index, ctypes.c_void_p(_stream_ptr(self.device)))
        if rc != 0:
            raise BpeError(rc, "bpe_ctx_create failed")
        self._h = h

    # -- plumbing -----------------------------------------------------------
    def _sync_stream(self):
        self.lib.bpe_ctx_set_stream(self._h, ctypes.c_void_p(_stream_ptr(self.device)))

    def close(self):
        if getattr(self, "_h", None):
            self.lib.bpe_ctx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_option(self, option: int, value: int) -> None:
        _capi.check(self._h, self.lib.bpe_ctx_set_option(self._h, option, value))

    def stats(self) -> dict:
        s = _capi.bpe_stats()
        _capi.check(self._h, self.lib.bpe_last_stats(self._h, ctypes.byref(s)))
        out = {s.k[i].name.decode(): {"launches": s.k[i].launches, "bytes": s.k[i].bytes, "ms": s.k[i].ms}
               for i in range(s.n)}
        out["kernel_launches"] = s.kernel_launches
        return out

    # -- the C ABI --------------------------------------------------------
    def pretokenize(self, data: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """uint8 bytes -> int32 tensor holding the uint32 symbols (bit 16 =
        WORD_START).  Asynchronous on the current stream."""
        data = _need_cuda(data, torch.uint8, "data", self.device)
        n = data.numel()
        if out is None:
            out = torch.empty(n, dtype=torch.int32, device=self.device)
        out = _need_cuda(out, torch.int32, "out", self.device)
        if out.numel() < n:
            raise ValueError("out too small")
        self._sync_stream()
        _capi.check(self._h, self.lib.bpe_pretokenize(self._h, ctypes.c_void_p(data.data_ptr()), n,
                                                      ctypes.c_void_p(out.data_ptr())))
        return out[:n]

    def train(self, symbols: torch.Tensor, n_merges: int, final: bool = True):
        """BPE merge loop.  Returns (merges uint32 [n_done, 4] = (left, right,
        new_id, count), final symbols int32 tensor or None)."""
        symbols = _need_cuda(symbols, torch.int32, "symbols", self.device)
        n = symbols.numel()
        merges = (_capi.bpe_merge * max(n_merges, 1))()
        n_done = ctypes.c_uint32(0)
        n_final = ctypes.c_uint64(0)
        fin = torch.empty(max(n, 1), dtype=torch.int32, device=self.device) if final else None
        self._sync_stream()
        rc = self.lib.bpe_train(self._h, ctypes.c_void_p(symbols.data_ptr() if n else 0), n, n_merges,
                                merges, ctypes.byref(n_done),
                                ctypes.c_void_p(fin.data_ptr()) if fin is not None else None,
                                ctypes.byref(n_final))
        _capi.check(self._h, rc)
        m = np.frombuffer(merges, dtype=np.uint32).reshape(-1, 4)[: n_done.value].copy()
        return m, (fin[: n_final.value] if fin is not None else None)

    def trie_build(self, vocab_bytes, vocab_off) -> Trie:
        """Double-array trie of token strings vocab_bytes[off[t]:off[t+1]]."""
        vb = np.ascontiguousarray(np.frombuffer(bytes(vocab_bytes), dtype=np.uint8)
                                  if isinstance(vocab_bytes, (bytes, bytearray)) else vocab_bytes,
                                  dtype=np.uint8)
        off = np.ascontiguousarray(vocab_off, dtype=np.uint64)
        n_tok = off.size - 1
        h = ctypes.c_void_p()
        _capi.check(self._h, self.lib.trie_build(self._h, ctypes.c_void_p(vb.ctypes.data if vb.size else 0),
                                                 ctypes.c_void_p(off.ctypes.data), n_tok, ctypes.byref(h)))
        return Trie(h.value, self.device, n_tok)

    def encode(self, trie: Trie, data: torch.Tensor, doc_off: torch.Tensor | None = None,
               capacity: int | None = None, ids_out: torch.Tensor | None = None):
        """Greedy longest-match ids.  data: uint8 CUDA tensor; doc_off: int64
        CUDA tensor of n_docs+1 ascending offsets (default: one document).
        Returns (ids int32 [n_ids], id_off int64 [n_docs+1])."""
        data = _need_cuda(data, torch.uint8, "data", self.device)
        if doc_off is None:
            doc_off = torch.tensor([0, data.numel()], dtype=torch.int64, device=self.device)
        doc_off = _need_cuda(doc_off, torch.int64, "doc_off", self.device)
        n_docs = doc_off.numel() - 1
        if ids_out is None:
            cap = data.numel() if capacity is None else capacity
            ids_out = torch.empty(max(cap, 1), dtype=torch.int32, device=self.device)
        else:
            ids_out = _need_cuda(ids_out, torch.int32, "ids_out", self.device)
            cap = ids_out.numel() if capacity is None else min(capacity, ids_out.numel())
        id_off = torch.empty(max(n_docs + 1, 1), dtype=torch.int64, device=self.device)
        n_ids = ctypes.c_uint64(0)
        if data.numel() == 0:   # keep a valid device pointer for empty input
            data = torch.empty(16, dtype=torch.uint8, device=self.device)
        self._sync_stream()
        rc = self.lib.trie_encode(self._h, trie._h, ctypes.c_void_p(data.data_ptr()),
                                  ctypes.c_void_p(doc_off.data_ptr()), max(n_docs, 0),
                                  ctypes.c_void_p(ids_out.data_ptr()), cap,
                                  ctypes.c_void_p(id_off.data_ptr()), ctypes.byref(n_ids))
        if rc == -6:
            raise BpeError(rc, f"{n_ids.value} ids needed, capacity {cap}")
        _capi.check(self._h, rc)
        return ids_out[: n_ids.value], id_off[: n_docs + 1]

    def decode(self, merges, ids: torch.Tensor) -> torch.Tensor:
        """Bytes of ids or symbols (int32 CUDA tensor; WORD_START ignored)
        under the vocabulary of ``merges``: a uint8 CUDA tensor."""
        ids = _need_cuda(ids, torch.int32, "ids", self.device)
        arr, n = _merge_array(merges)
        n_bytes = ctypes.c_uint64(0)
        ptr = ctypes.c_void_p(ids.data_ptr() if ids.numel() else 0)
        self._sync_stream()
        rc = self.lib.bpe_decode(self._h, arr, n, ptr, ids.numel(), None, 0, ctypes.byref(n_bytes))
        if rc not in (0, -6):
            _capi.check(self._h, rc)
        out = torch.empty(max(n_bytes.value, 1), dtype=torch.uint8, device=self.device)
        if ids.numel():
            _capi.check(self._h, self.lib.bpe_decode(self._h, arr, n, ptr, ids.numel(),
                                                     ctypes.c_void_p(out.data_ptr()), out.numel(),
                                                     ctypes.byref(n_bytes)))
        return out[: n_bytes.value]


    def unigram(self, trie: Trie, scores, unk_id: int, unk_score: float) -> "Unigram":
        """A Unigram (Viterbi) model over ``trie``: one f64 score per token
        (host array), the id and score of the <unk> fallback."""
        sc = np.ascontiguousarray(scores, dtype=np.float64)
        h = ctypes.c_void_p()
        _capi.check(self._h, self.lib.unigram_create(self._h, trie._h,
                                                     ctypes.c_void_p(sc.ctypes.data if sc.size else 0),
                                                     sc.size, int(unk_id), float(unk_score), ctypes.byref(h)))
        return Unigram(h.value, self.device, trie)

    def unigram_encode(self, model: "Unigram", data: torch.Tensor, doc_off: torch.Tensor | None = None,
                       capacity: int | None = None, ids_out: torch.Tensor | None = None):
        """Most likely segmentation of each document (Viterbi).  Arguments and
        result as ``encode``."""
        data = _need_cuda(data, torch.uint8, "data", self.device)
        if doc_off is None:
            doc_off = torch.tensor([0, data.numel()], dtype=torch.int64, device=self.device)
        doc_off = _need_cuda(doc_off, torch.int64, "doc_off", self.device)
        n_docs = doc_off.numel() - 1
        if ids_out is None:
            cap = data.numel() if capacity is None else capacity
            ids_out = torch.empty(max(cap, 1), dtype=torch.int32, device=self.device)
        else:
            ids_out = _need_cuda(ids_out, torch.int32, "ids_out", self.device)
            cap = ids_out.numel() if capacity is None else min(capacity, ids_out.numel())
        id_off = torch.empty(max(n_docs + 1, 1), dtype=torch.int64, device=self.device)
        n_ids = ctypes.c_uint64(0)
        if data.numel() == 0:
            data = torch.empty(16, dtype=torch.uint8, device=self.device)
        self._sync_stream()
        rc = self.lib.unigram_encode(self._h, model._h, ctypes.c_void_p(data.data_ptr()),
                                     ctypes.c_void_p(doc_off.data_ptr()), max(n_docs, 0),
                                     ctypes.c_void_p(ids_out.data_ptr()), cap,
                                     ctypes.c_void_p(id_off.data_ptr()), ctypes.byref(n_ids))
        if rc == -6:
            raise BpeError(rc, f"{n_ids.value} ids needed, capacity {cap}")
        _capi.check(self._h, rc)
        return ids_out[: n_ids.value], id_off[: n_docs + 1]

    # -- the output head ------------------------------------------------------
    def head_norm(self, x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                  eps: float = 1e-6, out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                  residual_out: torch.Tensor | None = None):
        """Root-mean-square norm of x + residual, in 8 bits with one scale per
        128 columns.  x, residual: [rows, dim] f32, bf16 or f16; weight: [dim]
        of any of the three.  Returns (x8 float8_e4m3fn [rows, dim], scales f32
        [rows, ceil(dim / 128)], the sum in x's type [rows, dim] or None).  The
        sum is written when a residual is given or residual_out is; it may be x
        or the residual itself.  Asynchronous on the current stream.  Not
        differentiable, like all head_ calls: what they return has no gradient,
        whether the inputs want one or not."""
        dev = self.device
        x, x_stride = _head_matrix(x, "x", dev, _HEAD_TYPES)
        size, dtype = x.shape, x.dtype
        rows, dim = size
        if not isinstance(weight, torch.Tensor) or weight.dtype not in _HEAD_TYPES:
            raise TypeError("weight must be a float32, bfloat16 or float16 tensor")
        weight = _head_vector(weight, "weight", dev, weight.dtype, dim)
        r_ptr, r_stride, ro_ptr, ro_stride = None, 0, None, 0
        if residual is not None:
            residual, r_stride = _head_matrix(residual, "residual", dev, (dtype,), size)
            r_ptr = residual.data_ptr()
            if residual_out is None:
                residual_out = torch.empty(rows, dim, dtype=dtype, device=dev)
        if residual_out is not None:
            residual_out, ro_stride = _head_matrix(residual_out, "residual_out", dev, (dtype,), size, out=True)
            ro_ptr = residual_out.data_ptr()
        if out is None:   # rows start on 16 bytes, which the product reads without a copy
            out = torch.empty(rows, -(-dim // 16) * 16, dtype=_E4M3, device=dev)[:, :dim]
        out, y_stride = _head_matrix(out, "out", dev, (_E4M3,), size, out=True)
        blocks = -(-dim // _capi.BPE_HEAD_BLOCK)
        if scales is None:
            scales = torch.empty(blocks, rows, dtype=torch.float32, device=dev).t()
        s_row, s_block = _head_scales(scales, "scales", dev, rows, blocks, out=True)
        self._sync_stream()
        rc = self.lib.head_norm(self._h, x.data_ptr(), x_stride, _HEAD_TYPES[dtype], weight.data_ptr(),
                                _HEAD_TYPES[weight.dtype], r_ptr, r_stride, rows, dim, eps, ro_ptr, ro_stride,
                                out.data_ptr(), y_stride, scales.data_ptr(), s_row, s_block)
        if rc:
            _capi.check(self._h, rc)
        return out, scales, residual_out

    def head_quantize(self, weight: torch.Tensor):
        """A weight matrix [n_tok, dim] (f32, bf16 or f16) in 8 bits with one
        scale per 128 x 128 block: (w8 float8_e4m3fn [n_tok, dim], its rows
        starting on 16 bytes, ws f32 [ceil(n_tok / 128), ceil(dim / 128)]).
        Not differentiable."""
        weight, stride = _head_matrix(weight, "weight", self.device, _HEAD_TYPES)
        n_tok, dim = weight.shape
        w8 = torch.empty(n_tok, -(-dim // 16) * 16, dtype=_E4M3, device=self.device)[:, :dim]
        ws = torch.empty(-(-n_tok // _capi.BPE_HEAD_BLOCK), -(-dim // _capi.BPE_HEAD_BLOCK), dtype=torch.float32,
                         device=self.device)
        self._sync_stream()
        _capi.check(self._h, self.lib.head_quantize(self._h, weight.data_ptr(), stride,
                                                    _HEAD_TYPES[weight.dtype], n_tok, dim, w8.data_ptr(),
                                                    w8.stride(0), ws.data_ptr(), ws.stride(0)))
        return w8, ws

    def head_logits(self, x8: torch.Tensor, xs: torch.Tensor, w8: torch.Tensor, ws: torch.Tensor,
                    out: torch.Tensor | None = None, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """Logits [rows, n_tok] of 8-bit hidden states x8 [rows, dim] (scales
        xs [rows, ceil(dim / 128)]) and weights w8 [n_tok, dim] (scales ws
        [ceil(n_tok / 128), ceil(dim / 128)]), accumulated in 32 bits and
        rounded once to ``dtype`` (f32, bf16 or f16; ``out``'s when it is
        given).  Scales may have any strides.  Matrices whose rows do not start
        on 16 bytes are copied at each call, to memory that stays with the
        context.  Asynchronous on the current stream.  Not differentiable."""
        dev = self.device
        x8, x_stride = _head_matrix(x8, "x8", dev, (_E4M3,))
        w8, w_stride = _head_matrix(w8, "w8", dev, (_E4M3,))
        rows, dim = x8.shape
        n_tok, w_dim = w8.shape
        if w_dim != dim:
            raise ValueError(f"w8 has {w_dim} columns, x8 {dim}")
        blocks = -(-dim // _capi.BPE_HEAD_BLOCK)
        xs_row, xs_block = _head_scales(xs, "xs", dev, rows, blocks)
        ws_row, ws_block = _head_scales(ws, "ws", dev, -(-n_tok // _capi.BPE_HEAD_BLOCK), blocks)
        if out is None:
            if dtype not in _HEAD_TYPES:
                raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
            out = torch.empty(rows, n_tok, dtype=dtype, device=dev)
        out, out_stride = _head_matrix(out, "out", dev, _HEAD_TYPES, (rows, n_tok), out=True)
        self._sync_stream()
        rc = self.lib.head_logits(self._h, x8.data_ptr(), x_stride, xs.data_ptr(), xs_row, xs_block, w8.data_ptr(),
                                  w_stride, ws.data_ptr(), ws_row, ws_block, rows, n_tok, dim, out.data_ptr(),
                                  out_stride, _HEAD_TYPES[out.dtype])
        if rc:
            _capi.check(self._h, rc)
        return out

    def head_sample(self, logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=None, top_p=None, min_p=None,
                    ids: torch.Tensor | None = None, logprob: torch.Tensor | None = None):
        """One id per row of logits [rows, n_tok] (f32, bf16 or f16), drawn by
        the random numbers u [rows] (f32 in [0, 1)).  temperature, top_p and
        min_p are numbers or f32 [rows] tensors, top_k a number or an int32
        [rows] tensor (None: off; temperature 0: the largest logit).  Returns
        (ids int32 [rows], logprob f32 [rows], the id's log-probability under
        the filtered distribution); a row without a logit above -infinity
        gives -1 and -infinity.  Asynchronous on the current stream."""
        dev = self.device
        logits, stride = _head_matrix(logits, "logits", dev, _HEAD_TYPES)
        rows, n_tok = logits.shape
        u = _head_vector(u, "u", dev, torch.float32, rows)
        if ids is None:
            ids = torch.empty(rows, dtype=torch.int32, device=dev)
        else:
            ids = _head_vector(ids, "ids", dev, torch.int32, rows, out=True)
        if logprob is None:
            logprob = torch.empty(rows, dtype=torch.float32, device=dev)
        else:
            logprob = _head_vector(logprob, "logprob", dev, torch.float32, rows, out=True)
        keep = []   # vectors that had to be copied live until the kernel is queued

        def one(v, name, dtype, off):
            if v is None:
                return off, None
            if not isinstance(v, torch.Tensor):
                return (_head_count(v) if dtype is torch.int32 else v), None
            v = _head_vector(v, name, dev, dtype, rows)
            keep.append(v)
            return off, v.data_ptr()

        t, d_t = one(temperature, "temperature", torch.float32, 1.0)
        k, d_k = one(top_k, "top_k", torch.int32, 0)
        p, d_p = one(top_p, "top_p", torch.float32, 1.0)
        q, d_q = one(min_p, "min_p", torch.float32, 0.0)
        filters = _capi.head_filters(t, k, p, q, d_t, d_k, d_p, d_q)
        self._sync_stream()
        rc = self.lib.head_sample(self._h, logits.data_ptr(), stride, _HEAD_TYPES[logits.dtype], rows, n_tok,
                                  u.data_ptr(), ctypes.byref(filters), ids.data_ptr(), logprob.data_ptr())
        if rc:
            _capi.check(self._h, rc)
        return ids, logprob

    def head_check(self) -> None:
        """Raises BpeError (TIMEOUT), once, when a head_logits of this context
        has given up a wait: some of its logits are NaN.  head_logits and
        head_sample ask the same before they start; a replayed CUDA graph does
        not.  Does not wait: call it after a synchronization."""
        rc = self.lib.head_check(self._h)
        if rc:
            _capi.check(self._h, rc)


class Unigram:
    """A Unigram model on the GPU (see ``Context.unigram``); keeps its trie alive."""

    def __init__(self, handle: int, device: torch.device, trie: Trie):
        self._h = ctypes.c_void_p(handle)
        self.device = device
        self.trie = trie

    def close(self):
        if self._h:
            _capi.load().unigram_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def encode_host(ctx: "Context", trie: "Trie", data, doc_off=None, ids_out=None, id_off_out=None,
                slice_bytes: int = 0):
    """Greedy longest-match ids from host memory (trie_encode_host: the
    copies overlap the encode).  data: uint8 CPU tensor (pinned for overlap);
    doc_off: int64 CPU tensor of n_docs+1 offsets (default: one document).
    Returns (ids int32 CPU tensor, id_off int64 CPU tensor)."""
    if not isinstance(data, torch.Tensor) or data.device.type != "cpu" or data.dtype != torch.uint8:
        raise TypeError("data must be a uint8 CPU tensor")
    if doc_off is None:
        doc_off = torch.tensor([0, data.numel()], dtype=torch.int64)
    doc_off = doc_off.to(torch.int64).contiguous()
    n_docs = doc_off.numel() - 1
    if ids_out is None:
        ids_out = torch.empty(max(data.numel(), 1), dtype=torch.int32, pin_memory=True)
    if id_off_out is None:
        id_off_out = torch.empty(max(n_docs + 1, 1), dtype=torch.int64)
    n = ctypes.c_uint64(0)
    ctx._sync_stream()
    rc = ctx.lib.trie_encode_host(ctx._h, trie._h, ctypes.c_void_p(data.data_ptr() if data.numel() else 0),
                                  ctypes.c_void_p(doc_off.data_ptr()), max(n_docs, 0),
                                  ctypes.c_void_p(ids_out.data_ptr()), ids_out.numel(),
                                  ctypes.c_void_p(id_off_out.data_ptr()), ctypes.byref(n), slice_bytes)
    if rc == -6:
        raise BpeError(rc, f"{n.value} ids needed, capacity {ids_out.numel()}")
    _capi.check(ctx._h, rc)
    return ids_out[: n.value], id_off_out[: n_docs + 1]


class Stream:
    """Streaming encode of one document arriving in slices (trie_stream_*):
    push() returns the ids that no later byte can change; the last push
    returns the rest.  The ids of all pushes, concatenated, equal
    Context.encode on the whole document."""

    def __init__(self, ctx: "Context", trie: Trie):
        self.ctx, self.trie = ctx, trie
        self._h = ctypes.c_void_p()
        _capi.check(ctx._h, ctx.lib.trie_stream_open(ctx._h, trie._h, ctypes.byref(self._h)))

    def push(self, data: torch.Tensor, last: bool = False, ids_out: torch.Tensor | None = None) -> torch.Tensor:
        data = _need_cuda(data, torch.uint8, "data", self.ctx.device)
        cap = data.numel() + self.trie.info()["max_token_len"] + 16   # one id per carried or new byte
        if ids_out is None:
            ids_out = torch.empty(cap, dtype=torch.int32, device=self.ctx.device)
        else:
            ids_out = _need_cuda(ids_out, torch.int32, "ids_out", self.ctx.device)
        n_ids = ctypes.c_uint64(0)
        ptr = data.data_ptr() if data.numel() else 0
        self.ctx._sync_stream()
        rc = self.ctx.lib.trie_stream_push(self._h, ctypes.c_void_p(ptr), data.numel(), 1 if last else 0,
                                           ctypes.c_void_p(ids_out.data_ptr()), ids_out.numel(), ctypes.byref(n_ids))
        if rc == -6:
            raise BpeError(rc, f"{n_ids.value} ids needed, capacity {ids_out.numel()}")
        _capi.check(self.ctx._h, rc)
        return ids_out[: n_ids.value]

    def close(self):
        if self._h:
            self.ctx.lib.trie_stream_close(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _merge_array(merges):
    """(n, 4) uint32 rows (left, right, new_id, count) as a bpe_merge array."""
    m = np.ascontiguousarray(np.asarray(merges, dtype=np.uint32).reshape(-1, 4))
    arr = (_capi.bpe_merge * max(m.shape[0], 1))()
    if m.shape[0]:
        ctypes.memmove(arr, m.ctypes.data, m.nbytes)
    return arr, m.shape[0]


def vocab_from_merges(merges):
    """Token byte strings of ids 0 .. 255 + len(merges), through the library's
    bpe_vocab_from_merges (host only).  Returns (uint8 array, uint64 offsets),
    the layout ``Context.trie_build`` takes."""
    lib = _capi.load()
    arr, n = _merge_array(merges)
    n_bytes = ctypes.c_uint64(0)
    rc = lib.bpe_vocab_from_merges(arr, n, None, 0, None, ctypes.byref(n_bytes))
    if rc not in (0, -6):
        raise BpeError(rc, "bpe_vocab_from_merges: malformed merge table")
    vb = np.empty(max(n_bytes.value, 1), dtype=np.uint8)
    off = np.empty(257 + n, dtype=np.uint64)
    rc = lib.bpe_vocab_from_merges(arr, n, ctypes.c_void_p(vb.ctypes.data), vb.size,
                                   ctypes.c_void_p(off.ctypes.data), ctypes.byref(n_bytes))
    if rc != 0:
        raise BpeError(rc, "bpe_vocab_from_merges failed")
    return vb[: n_bytes.value], off
