"""PuzzleKV page-wise low-rank KV cache compression on GB300 (sm_103a).

Python face of the C ABI in include/puzzlekv.h.  The functions here only
marshal arguments (shapes, dtypes, pointers, the current CUDA stream) into
the CUDA library; PyTorch provides device memory and streams.  Citations name
sections/equations of "PuzzleKV: Page-Wise Low-Rank Decomposition for KV
Cache Compression".
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import BF16, F32, PAGE_DENSE, PAGE_FACTORED, PuzzleKVError, check, last_error, lib  # noqa: F401

_DT = {torch.float32: F32, torch.bfloat16: BF16}
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}


@dataclass(frozen=True)
class StoreConfig:
    num_layers: int
    num_kv_heads: int
    num_q_heads: int
    head_dim: int
    page_size: int
    rank_k: int
    rank_v: int
    sink_tokens: int
    recent_tokens: int
    max_batch: int
    max_tokens_per_seq: int
    kv_dtype: torch.dtype = torch.bfloat16
    factor_int4: bool = False
    rope_theta: float = 0.0  # > 0: keys are given before RoPE with this base and turned at attention

    def c(self) -> _lib.Config:
        c = _lib.Config()
        for name, ctype in _lib.Config._fields_:
            if name == "kv_dtype":
                setattr(c, name, _DT[self.kv_dtype])
            elif ctype is ctypes.c_float:
                setattr(c, name, float(getattr(self, name)))
            else:
                setattr(c, name, _lib.Int32.from_param(int(getattr(self, name))).value)
        return c


def _stream(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, shape, dtype, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


_SEQ_CACHE: dict = {}


def _seq_ids(seq_ids: Sequence[int]):
    key = tuple(int(s) for s in seq_ids)
    arr = _SEQ_CACHE.get(key)
    if arr is None:
        if len(_SEQ_CACHE) > 4096:
            _SEQ_CACHE.clear()
        arr = _SEQ_CACHE[key] = _ints(key, len(key), "seq_ids")
    return arr, len(key)


def _ints(values: Sequence[int], n: int, name: str):
    if len(values) != n:
        raise ValueError(f"{name} must have {n} entries, got {len(values)}")
    v = [int(x) for x in values]
    if v and not (-0x80000000 <= min(v) and max(v) <= 0x7FFFFFFF):  # ctypes would keep the low 32 bits
        raise ValueError(f"{name}: {max(v, key=abs)} does not fit in 32 bits")
    return (ctypes.c_int32 * max(n, 1))(*v)


def query_sizes(cfg: StoreConfig) -> dict:
    """Byte sizes of the dense pool, factor pool, page table and workspace."""
    s = [ctypes.c_size_t() for _ in range(4)]
    c = cfg.c()
    check(lib().puzzlekv_query_sizes(ctypes.byref(c), *[ctypes.byref(x) for x in s]))
    return dict(zip(("dense_pool", "factor_pool", "page_table", "workspace"), (x.value for x in s)))


def classify_pages(T: int, P: int, sink_tokens: int, recent_tokens: int) -> np.ndarray:
    """PAGE_DENSE / PAGE_FACTORED per page of a T-token sequence (host-only)."""
    n = (T + P - 1) // P
    out = (ctypes.c_int32 * max(n, 1))()
    got = lib().puzzlekv_classify_pages(T, P, sink_tokens, recent_tokens, out, n)
    if got != n:
        raise ValueError("bad arguments to classify_pages")
    return np.frombuffer(out, dtype=np.int32, count=n).copy()


def page_storage_ratio(P: int, d: int, rank_k: int, rank_v: int) -> float:
    """(r_K + r_V)(P + d) / (2 P d), eq. (3)."""
    return float(lib().puzzlekv_page_storage_ratio(P, d, rank_k, rank_v))


def factorize_batch(X: torch.Tensor, r: int, out_dtype: torch.dtype = torch.float32, sigma: bool = True,
                    stream: Optional[torch.cuda.Stream] = None):
    """Factorize independent pages X[n, P, d] -> (L[n, P, r], R[n, r, d], sigma[n, P] or None, status[1]).

    ``status`` (int32 on the device) is nonzero if an eigensolve hit its iteration cap.
    """
    if X.dim() != 3:
        raise ValueError("X must be [n, P, d]")
    n, P, d = X.shape
    _need(X, (n, P, d), X.dtype, "X")
    if X.dtype not in _DT:
        raise ValueError("X must be float32 or bfloat16")
    L = torch.empty(n, P, r, dtype=out_dtype, device=X.device)
    R = torch.empty(n, r, d, dtype=out_dtype, device=X.device)
    S = torch.empty(n, P, dtype=torch.float32, device=X.device) if sigma else None
    status = torch.zeros(1, dtype=torch.int32, device=X.device)
    check(lib().puzzlekv_factorize_batch(_ptr(X), _DT[X.dtype], n, P, d, r, _ptr(L), _ptr(R), _DT[out_dtype],
                                         _ptr(S) if S is not None else None, _ptr(status), _stream(stream)))
    return L, R, S, status


def int4_record_bytes(P: int, d: int, rank_k: int, rank_v: int) -> int:
    """Bytes of one INT4 factor record (§4.3) of a store with these shapes."""
    b = ctypes.c_int64()
    check(lib().puzzlekv_int4_record_bytes(P, d, rank_k, rank_v, ctypes.byref(b)))
    return b.value


def factorize_batch_int4(X: torch.Tensor, rank_k: int, rank_v: int, kind: int, absorbed: bool = True,
                         stream: Optional[torch.cuda.Stream] = None):
    """INT4 records of independent bf16 pages X[n, P, d] (§4.3): returns (records uint8
    [n, record_bytes], L~ fp32 [n, P, rp] or None, R~ fp32 [n, rp, d] or None, status[1]);
    kind 0 = key pages at rank_k, 1 = value pages at rank_v."""
    if X.dim() != 3 or X.dtype != torch.bfloat16:
        raise ValueError("X must be bf16 [n, P, d]")
    n, P, d = X.shape
    _need(X, (n, P, d), torch.bfloat16, "X")
    rb = int4_record_bytes(P, d, rank_k, rank_v)
    rp = ((rank_k if kind == 0 else rank_v) + 7) // 8 * 8
    rec = torch.zeros(n, rb, dtype=torch.uint8, device=X.device)
    Lq = torch.empty(n, P, rp, dtype=torch.float32, device=X.device) if absorbed else None
    Rq = torch.empty(n, rp, d, dtype=torch.float32, device=X.device) if absorbed else None
    status = torch.zeros(1, dtype=torch.int32, device=X.device)
    check(lib().puzzlekv_factorize_batch_int4(_ptr(X), n, P, d, rank_k, rank_v, kind, _ptr(rec),
                                              _ptr(Lq) if absorbed else None, _ptr(Rq) if absorbed else None,
                                              _ptr(status), _stream(stream)))
    return rec, Lq, Rq, status


class Store:
    """Paged factor store over four torch-allocated device buffers."""

    def __init__(self, cfg: StoreConfig, device="cuda", stream: Optional[torch.cuda.Stream] = None):
        self.cfg = cfg
        sizes = query_sizes(cfg)
        self.sizes = sizes
        # 256-byte aligned device buffers (the caching allocator aligns to 512)
        self.dense_pool = torch.empty(sizes["dense_pool"], dtype=torch.uint8, device=device)
        self.factor_pool = torch.empty(sizes["factor_pool"], dtype=torch.uint8, device=device)
        self.page_table = torch.empty(sizes["page_table"], dtype=torch.uint8, device=device)
        self.workspace = torch.empty(sizes["workspace"], dtype=torch.uint8, device=device)
        h = ctypes.c_void_p()
        c = cfg.c()
        check(lib().puzzlekv_store_create(ctypes.byref(c), _ptr(self.dense_pool), _ptr(self.factor_pool),
                                          _ptr(self.page_table), _ptr(self.workspace), _stream(stream),
                                          ctypes.byref(h)))
        self._h = h
        self._index = self.dense_pool.device.index

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().puzzlekv_store_destroy(self._h)  # waits for the background stream
            self._h = None
            self._inputs = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def load_prefill(self, seq: int, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """Prefill compression of sequence `seq` from dense k, v [L, H, T, d] (§3.3 ①②③)."""
        c = self.cfg
        T = k.shape[2]
        shape = (c.num_layers, c.num_kv_heads, T, c.head_dim)
        _need(k, shape, c.kv_dtype, "k")
        _need(v, shape, c.kv_dtype, "v")
        check(lib().puzzlekv_load_prefill(self._h, seq, _ptr(k), _ptr(v), T, _stream(stream)))

    def factorize_pages(self, pages: Optional[Sequence[tuple]] = None, stream=None) -> None:
        """Factorize the listed completed pages [(seq, page), ...] of every layer, or
        every eligible page when `pages` is None (§3.3 ③⑤); pages with factors are skipped."""
        if pages is None:
            check(lib().puzzlekv_factorize_pages(self._h, None, None, -1, _stream(stream)))
            return
        n = len(pages)
        seqs, pgs = _ints([b for b, _ in pages], n, "pages"), _ints([p for _, p in pages], n, "pages")
        check(lib().puzzlekv_factorize_pages(self._h, seqs, pgs, n, _stream(stream)))

    def factorize_layer(self, seq: int, layer: int, k: torch.Tensor, v: torch.Tensor, background: bool = True,
                        stream=None) -> None:
        """Prefill compression of one layer from dense k, v [H, T, d] (§3.3 ①②③).  With
        `background`, the factorization runs on the store's internal stream so that the
        caller's later layers overlap it; the store then keeps k and v referenced until
        that stream is past the call (or until wait_background / close)."""
        c = self.cfg
        T = k.shape[1]
        shape = (c.num_kv_heads, T, c.head_dim)
        _need(k, shape, c.kv_dtype, "k")
        _need(v, shape, c.kv_dtype, "v")
        self._release_inputs()
        check(lib().puzzlekv_factorize_layer(self._h, seq, layer, _ptr(k), _ptr(v), T, int(background),
                                             _stream(stream)))
        if background:  # k and v stay referenced until the background stream is past this call
            ev = torch.cuda.Event()
            ev.record(self.background_stream())
            self._inputs.append((ev, k, v))

    def _release_inputs(self) -> None:
        """Drop the references to background prefill inputs the internal stream is done with."""
        inputs = getattr(self, "_inputs", None)
        if inputs is None:
            self._inputs = []
            return
        while inputs and inputs[0][0].query():
            inputs.pop(0)

    def wait_background(self, stream=None) -> None:
        """Order `stream` after all background work queued so far (conversions, layer prefills)."""
        check(lib().puzzlekv_wait_background(self._h, _stream(stream)))
        self._release_inputs()

    def background_stream(self) -> torch.cuda.ExternalStream:
        """The store's internal low-priority stream, as a torch stream object."""
        if getattr(self, "_bg", None) is None:
            h = ctypes.c_void_p()
            check(lib().puzzlekv_background_stream(self._h, ctypes.byref(h)))
            self._bg = torch.cuda.ExternalStream(h.value, device=self.dense_pool.device)
        return self._bg

    def append_token(self, layer: int, k: torch.Tensor, v: torch.Tensor, seq_ids: Sequence[int], stream=None) -> None:
        """Append one token per sequence to `layer`; converts pages leaving the window (§3.3 ⑤)."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        _need(k, (B, c.num_kv_heads, c.head_dim), c.kv_dtype, "k")
        _need(v, (B, c.num_kv_heads, c.head_dim), c.kv_dtype, "v")
        check(lib().puzzlekv_append_token(self._h, layer, _ptr(k), _ptr(v), ids, B, _stream(stream)))

    def decode_attention(self, layer: int, q: torch.Tensor, out: torch.Tensor, seq_ids: Sequence[int],
                         stream=None) -> torch.Tensor:
        """Mixed dense/factorized decode attention of one layer (§3.3 ④, eqs. (4)-(5))."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        _need(q, (B, c.num_q_heads, c.head_dim), c.kv_dtype, "q")
        _need(out, (B, c.num_q_heads, c.head_dim), torch.float32, "out")
        check(lib().puzzlekv_decode_attention(self._h, layer, _ptr(q), _ptr(out), ids, B, _stream(stream)))
        return out

    def decode_step(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                    seq_ids: Sequence[int], stream=None) -> torch.Tensor:
        """Append (k, v) and attend with q in one launch (§3.3 ④⑤); converts the
        page leaving the window first."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        _need(q, (B, c.num_q_heads, c.head_dim), c.kv_dtype, "q")
        _need(k, (B, c.num_kv_heads, c.head_dim), c.kv_dtype, "k")
        _need(v, (B, c.num_kv_heads, c.head_dim), c.kv_dtype, "v")
        _need(out, (B, c.num_q_heads, c.head_dim), torch.float32, "out")
        check(lib().puzzlekv_decode_step(self._h, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), ids, B,
                                         _stream(stream)))
        return out

    def convert_ready_pages(self, stream=None) -> None:
        """Factorize every complete, not yet factorized page of all sequences and
        layers in one batched launch (ahead of its leaving the window)."""
        check(lib().puzzlekv_convert_ready_pages(self._h, _stream(stream)))

    def decode_attention_static_scratch(self, layer: int, q: torch.Tensor, out: torch.Tensor,
                                        seq_ids: Sequence[int], stream=None) -> torch.Tensor:
        """decode_attention with its split-K scratch in the library's static
        device array (no per-call scratch buffer; see include/puzzlekv.h)."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        _need(q, (B, c.num_q_heads, c.head_dim), c.kv_dtype, "q")
        _need(out, (B, c.num_q_heads, c.head_dim), torch.float32, "out")
        check(lib().puzzlekv_decode_attention_static_scratch(self._h, layer, _ptr(q), _ptr(out), ids, B,
                                                             _stream(stream)))
        return out

    def _on(self, stream):
        """Context of a chunk call: the store's device, and `stream` (default: the device's
        current one) as torch's current stream, so that what the call allocates belongs to it."""
        if stream is not None:
            return torch.cuda.stream(stream)
        if torch.cuda.current_device() == self._index:
            return contextlib.nullcontext()
        return torch.cuda.device(self._index)

    def _queue(self, stream) -> ctypes.c_void_p:
        # the raw handle alone: making a Stream object takes longer than a small launch
        return ctypes.c_void_p(stream.cuda_stream if stream is not None
                               else torch._C._cuda_getCurrentRawStream(self._index))

    def _need_here(self, t: torch.Tensor, shape, name: str) -> None:
        _need(t, shape, self.cfg.kv_dtype, name)
        if t.device != self.dense_pool.device:
            raise ValueError(f"{name} is on {t.device}, the store on {self.dense_pool.device}")

    def _scratch(self, nbytes: int) -> torch.Tensor:
        return torch.empty(nbytes, dtype=torch.uint8, device=self.dense_pool.device)

    def chunk_workspace(self, layer: int, seq_ids: Sequence[int], counts: Sequence[int]) -> dict:
        """Workspace bytes of chunk_attention and append_chunk at the present lengths."""
        ids, B = _seq_ids(seq_ids)
        a, b = ctypes.c_size_t(), ctypes.c_size_t()
        check(lib().puzzlekv_chunk_workspace(self._h, layer, ids, _ints(counts, B, "counts"), B, ctypes.byref(a),
                                             ctypes.byref(b)))
        return {"attention": a.value, "append": b.value}

    def chunk_attention(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_ids: Sequence[int],
                        counts: Sequence[int], out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of a chunk of new tokens per sequence over the cache and, causally, the
        chunk (§3.3 ④): q [N, Hq, d], k, v [N, H, d], N = sum(counts), sequences one after another.
        Returns out [N, Hq, d] in kv_dtype; the store is unchanged (append_chunk adds the chunk).
        `out` may be q itself, and shares no memory with another of the tensors.
        `workspace` (uint8, of chunk_workspace's size) is allocated if not given."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        cnt = _ints(counts, B, "counts")
        N = sum(cnt[:B])
        self._need_here(q, (N, c.num_q_heads, c.head_dim), "q")
        self._need_here(k, (N, c.num_kv_heads, c.head_dim), "k")
        self._need_here(v, (N, c.num_kv_heads, c.head_dim), "v")
        with self._on(stream):
            nb = ctypes.c_size_t()
            check(lib().puzzlekv_chunk_workspace(self._h, layer, ids, cnt, B, ctypes.byref(nb), None))
            if out is None:
                out = torch.empty_like(q)
            else:
                self._need_here(out, (N, c.num_q_heads, c.head_dim), "out")
            if N == 0:
                return out
            work = workspace if workspace is not None else self._scratch(nb.value)
            if work.device != self.dense_pool.device or not work.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on the store's device")
            check(lib().puzzlekv_chunk_attention(self._h, layer, _ptr(q), _ptr(k), _ptr(v), _ptr(out), ids, cnt, B,
                                                 _ptr(work), work.numel() * work.element_size(), self._queue(stream)))
        return out

    def append_chunk(self, layer: int, k: torch.Tensor, v: torch.Tensor, seq_ids: Sequence[int],
                     counts: Sequence[int], stream=None) -> None:
        """Append counts[i] tokens to each sequence (empty slots included) of `layer`: k, v
        [N, H, d]; pages that leave the window are factorized (§3.3 ⑤)."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        cnt = _ints(counts, B, "counts")
        N = sum(cnt[:B])
        self._need_here(k, (N, c.num_kv_heads, c.head_dim), "k")
        self._need_here(v, (N, c.num_kv_heads, c.head_dim), "v")
        with self._on(stream):
            nb = ctypes.c_size_t()
            # a chunk of at most a page never outgrows the ring
            if max(cnt[:B], default=0) > c.page_size or N == 0:
                check(lib().puzzlekv_chunk_workspace(self._h, layer, ids, cnt, B, None, ctypes.byref(nb)))
            if N == 0:
                return
            work = self._scratch(nb.value) if nb.value else None
            check(lib().puzzlekv_append_chunk(self._h, layer, _ptr(k), _ptr(v), ids, cnt, B,
                                              _ptr(work) if work is not None else None, nb.value, self._queue(stream)))

    def read_tokens(self, layer: int, seq_ids: Sequence[int], starts: Sequence[int], counts: Sequence[int],
                    stream=None) -> tuple:
        """Rows [starts[i], starts[i] + counts[i]) of each sequence as attention sees them
        (factorized pages as L R): (k, v), each [N, H, d] in kv_dtype."""
        c = self.cfg
        ids, B = _seq_ids(seq_ids)
        st, cnt = _ints(starts, B, "starts"), _ints(counts, B, "counts")
        if any(n < 0 or n > c.max_tokens_per_seq for n in cnt[:B]):  # before anything of that size is allocated
            raise ValueError("counts must be in [0, max_tokens_per_seq]")
        N = sum(cnt[:B])
        with self._on(stream):
            # one row at least, so that an empty read still has a pointer
            k = torch.empty((max(N, 1), c.num_kv_heads, c.head_dim), dtype=c.kv_dtype, device=self.dense_pool.device)
            v = torch.empty_like(k)
            check(lib().puzzlekv_read_tokens(self._h, layer, ids, st, cnt, B, _ptr(k), _ptr(v), self._queue(stream)))
        return (k, v) if N else (k[:0], v[:0])

    def load_factors(self, layer: int, seq: int, page0: int, LK: torch.Tensor, RK: torch.Tensor, LV: torch.Tensor,
                     RV: torch.Tensor, stream=None) -> None:
        """Factors computed elsewhere into the records of pages page0 .. page0 + n - 1: LK [H, n, P, rk],
        RK [H, n, rk, d], LV [H, n, P, rv], RV [H, n, rv, d] in kv_dtype (bf16 and fp32 stores)."""
        c = self.cfg
        if LK.dim() != 4:
            raise ValueError("LK must be [H, n, P, rank_k]")
        H, n, P, d = c.num_kv_heads, LK.shape[1], c.page_size, c.head_dim
        self._need_here(LK, (H, n, P, c.rank_k), "LK")
        self._need_here(RK, (H, n, c.rank_k, d), "RK")
        self._need_here(LV, (H, n, P, c.rank_v), "LV")
        self._need_here(RV, (H, n, c.rank_v, d), "RV")
        with self._on(stream):
            check(lib().puzzlekv_load_factors(self._h, layer, seq, page0, n, _ptr(LK), _ptr(RK), _ptr(LV), _ptr(RV),
                                              self._queue(stream)))

    def copy_sequences(self, src_ids: Sequence[int], dst_ids: Sequence[int], stream=None) -> None:
        """Slot dst_ids[i] becomes what slot src_ids[i] was before the call, all pairs at once
        (forks, reordered beams, compaction); every layer."""
        n = len(dst_ids)
        with self._on(stream):
            check(lib().puzzlekv_copy_sequences(self._h, _ints(src_ids, n, "src_ids"), _ints(dst_ids, n, "dst_ids"), n,
                                                self._queue(stream)))

    def truncate_sequences(self, seq_ids: Sequence[int], lengths: Sequence[int], stream=None) -> None:
        """Cut sequences back to lengths[i] tokens in every layer (0 empties the slot); the pages
        that become dense again must still be in the dense ring."""
        ids, B = _seq_ids(seq_ids)
        with self._on(stream):
            check(lib().puzzlekv_truncate_sequences(self._h, ids, _ints(lengths, B, "lengths"), B, self._queue(stream)))

    def stats(self, seq: int, layer: int) -> dict:
        n = ctypes.c_int32()
        nd, nf, nb = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        check(lib().puzzlekv_store_stats(self._h, seq, layer, ctypes.byref(n), ctypes.byref(nd), ctypes.byref(nf),
                                         ctypes.byref(nb)))
        return {"length": n.value, "dense_pages": nd.value, "factored_pages": nf.value, "bytes_live": nb.value}

    def debug_fail_next_wait(self, where: int, wait_ns: int = 100_000) -> None:
        """Test hook of the failure path: the next decode launch's wait at `where`
        (1 = a unit copy, 2 = the split merge) runs out after wait_ns (see include/puzzlekv.h)."""
        check(lib().puzzlekv_debug_fail_next_wait(self._h, int(where), int(wait_ns)))

    def debug_fail_next_chunk_wait(self, where: int, wait_ns: int = 2_000_000) -> None:
        """The same hook for the chunk and sequence calls: 1 few tokens, 2 staging, 3 attention over the images,
        4 row reads, 5 sequence copies (see include/puzzlekv.h)."""
        check(lib().puzzlekv_debug_fail_next_chunk_wait(self._h, int(where), int(wait_ns)))

    def check_device_status(self, stream=None) -> int:
        """Synchronise and return the status code (raises nothing; OK = 0)."""
        st = lib().puzzlekv_check_device_status(self._h, _stream(stream))
        self._release_inputs()
        return st

    def factorize_counters(self, stream=None) -> tuple:
        """(page jobs, QL rotations) of the store's factorization launches since
        the last call (rotations come only from jobs of rank above P / 2);
        the counters are cleared."""
        jobs, rotations = ctypes.c_int64(0), ctypes.c_int64(0)
        check(lib().puzzlekv_factorize_counters(self._h, _stream(stream), ctypes.byref(jobs), ctypes.byref(rotations)))
        return jobs.value, rotations.value
