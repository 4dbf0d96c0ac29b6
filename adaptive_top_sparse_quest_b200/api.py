"""PyTorch-facing binding of the Twilight sm_100a library.

Every function here only checks tensor dtypes / shapes, allocates outputs with
PyTorch (device memory and streams are the only things PyTorch provides) and
calls the C ABI on the current CUDA stream.  All computation happens in the
CUDA kernels of libtwilight.so.

Method: "Twilight: Adaptive Attention Sparsity with Hierarchical Top-p Pruning"
(arXiv 2502.02770): Quest page pre-selection, top-p pruning of the candidates'
attention weights estimated from a 4-bit key cache (or the 2-bit cache of its
quantisation ablation, KVCache.key_bits = 2), exact sparse attention over the
survivors.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Optional

import torch

from . import _capi
from ._capi import TwKv, TwStep, check

HEAD_DIM = 128
PAGE = 16
INT32_MAX = 2 ** 31 - 1


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _need(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


KEY_BITS = (4, 2)


@dataclasses.dataclass
class KVCache:
    """fp16 K/V in the contiguous [B][Hk][N][128] layout, or a paged pool
    [pages][Hk][16][128] with page_table [B][max_pages].  key_bits is the width
    of the quantised key cache that goes with it (4, or 2)."""
    k: torch.Tensor
    v: Optional[torch.Tensor]
    seq_lens: torch.Tensor
    page_table: Optional[torch.Tensor] = None
    key_bits: int = 4

    def __post_init__(self):
        _need(self.k, torch.float16, "k")
        if self.v is not None:
            _need(self.v, torch.float16, "v")
            if self.v.shape != self.k.shape:
                raise ValueError("k and v must have the same shape")
        _need(self.seq_lens, torch.int32, "seq_lens")
        if self.k.shape[-1] != HEAD_DIM:
            raise ValueError("head_dim must be 128")
        if self.page_table is not None:
            _need(self.page_table, torch.int32, "page_table")
            if self.k.dim() != 4 or self.k.shape[2] != PAGE:
                raise ValueError("paged k must be [pages][Hk][16][128]")
        elif self.k.dim() != 4:
            raise ValueError("contiguous k must be [B][Hk][N][128]")
        if self.key_bits not in KEY_BITS:
            raise ValueError(f"key_bits must be one of {KEY_BITS}")
        self._checked = self.k, self.v, self.seq_lens, self.page_table

    def recheck(self) -> None:
        """Check the tensors again if some have been replaced since."""
        k, v, lens, table = self._checked
        if (self.k is not k or self.v is not v or self.seq_lens is not lens
                or self.page_table is not table):
            self.__post_init__()

    @property
    def code_bytes(self) -> int:
        """Bytes of codes per token row: 128 * key_bits / 8."""
        return HEAD_DIM * self.key_bits // 8

    @property
    def paged(self) -> bool:
        return self.page_table is not None

    @property
    def B(self) -> int:
        return int(self.seq_lens.shape[0])

    @property
    def Hk(self) -> int:
        return int(self.k.shape[1])

    @property
    def N(self) -> int:
        return int(self.page_table.shape[1]) * PAGE if self.paged else int(self.k.shape[2])

    @property
    def max_pages(self) -> int:
        return (self.N + PAGE - 1) // PAGE

    def struct(self) -> TwKv:
        paged = self.paged
        N = self.N
        return TwKv(_ptr(self.k), _ptr(self.v), self.B, self.Hk, N, _ptr(self.seq_lens),
                    _ptr(self.page_table), N // PAGE if paged else 0,
                    self.k.shape[0] if paged else 0, PAGE, HEAD_DIM, self.key_bits)

    def row_shape(self, last: int):
        """Shape of a per-token companion array (codes, scales, zeros)."""
        if self.paged:
            return (self.k.shape[0], self.Hk, PAGE, last)
        return (self.B, self.Hk, self.N, last)

    def meta_shape(self):
        if self.paged:
            return (self.k.shape[0], self.Hk, 2, HEAD_DIM)
        return (self.B, self.Hk, self.max_pages, 2, HEAD_DIM)

    @classmethod
    def from_workload(cls, w, key_bits: int = 4) -> "KVCache":
        return cls(w.k, w.v, w.seq_lens, w.page_table, key_bits)


@dataclasses.dataclass
class Int4Keys:
    """The quantised key cache (4-bit, or 2-bit when its KVCache says so)."""
    codes: torch.Tensor    # uint8  [..][128 * key_bits / 8]
    scales: torch.Tensor   # fp16   [..][4]
    zeros: torch.Tensor    # fp16   [..][4]


def _check_keys(kv: KVCache, keys: Int4Keys) -> None:
    if tuple(keys.codes.shape) != kv.row_shape(kv.code_bytes):
        raise ValueError(f"codes must be {kv.row_shape(kv.code_bytes)} for "
                         f"{kv.key_bits}-bit keys, got {tuple(keys.codes.shape)}")


def quantize_keys(kv: KVCache, out: Optional[Int4Keys] = None, stream=None) -> Int4Keys:
    """Per-token asymmetric key cache (group 32, kv.key_bits wide): tw_quantize_keys."""
    lib = _capi.load()
    if out is None:
        dev = kv.k.device
        out = Int4Keys(torch.zeros(kv.row_shape(kv.code_bytes), dtype=torch.uint8, device=dev),
                       torch.zeros(kv.row_shape(4), dtype=torch.float16, device=dev),
                       torch.zeros(kv.row_shape(4), dtype=torch.float16, device=dev))
    _check_keys(kv, out)
    s = kv.struct()
    check(lib.tw_quantize_keys(ctypes.byref(s), _ptr(out.codes), _ptr(out.scales),
                               _ptr(out.zeros), _stream(stream)), "tw_quantize_keys")
    return out


def page_meta(kv: KVCache, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Quest per-page channel-wise key min / max: tw_page_meta."""
    lib = _capi.load()
    if out is None:
        out = torch.zeros(kv.meta_shape(), dtype=torch.float16, device=kv.k.device)
    s = kv.struct()
    check(lib.tw_page_meta(ctypes.byref(s), _ptr(out), _stream(stream)), "tw_page_meta")
    return out


def append_keys(kv: KVCache, keys: Int4Keys, meta: Optional[torch.Tensor] = None,
                stream=None) -> None:
    """tw_append_keys: quantise the newest token (position seq_lens[b] - 1) of
    every sequence into `keys` and fold it into `meta` (if given).  The caller
    writes that token's K / V rows and raises seq_lens first."""
    lib = _capi.load()
    _check_keys(kv, keys)
    s = kv.struct()
    check(lib.tw_append_keys(ctypes.byref(s), _ptr(keys.codes), _ptr(keys.scales),
                             _ptr(keys.zeros), _ptr(meta), _stream(stream)), "tw_append_keys")


def workspace_bytes(B: int, Hq: int, Hk: int, N: int, capacity: int) -> int:
    lib = _capi.load()
    n = ctypes.c_size_t(0)
    check(lib.tw_workspace_size(B, Hq, Hk, N, capacity, ctypes.byref(n)), "tw_workspace_size")
    return int(n.value)


def new_workspace(B, Hq, Hk, N, capacity, device) -> torch.Tensor:
    """A workspace with its device status word (the first 4 bytes) zeroed."""
    ws = torch.empty(max(workspace_bytes(B, Hq, Hk, N, capacity), 256), dtype=torch.uint8,
                     device=device)
    ws[:256].zero_()
    return ws


def device_status(ws: torch.Tensor) -> int:
    """The workspace's device status word (synchronises): 0, or bit 0 set when a
    bounded wait of the selection kernel gave up (that call's outputs are
    invalid; the C API calls it TW_ERR_TIMEOUT)."""
    return int(ws[:4].view(torch.int32).item())


def budget_pages(budget_tokens: Optional[int], kv: KVCache) -> int:
    return min(budget_tokens // PAGE, kv.max_pages)


def select_pages(q: torch.Tensor, kv: KVCache, meta: torch.Tensor, budget_tokens: int,
                 ws: Optional[torch.Tensor] = None, stream=None):
    """Quest top-K_p pages per (b, KV head): tw_select_pages -> (cand_pages, ncand)."""
    lib = _capi.load()
    _need(q, torch.float16, "q")
    Hq = int(q.shape[1])
    stride = max(1, budget_pages(budget_tokens, kv))
    cand = torch.zeros((kv.B, kv.Hk, stride), dtype=torch.int32, device=q.device)
    ncand = torch.zeros((kv.B, kv.Hk), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = new_workspace(kv.B, Hq, kv.Hk, kv.N, 1, q.device)
    s = kv.struct()
    check(lib.tw_select_pages(_ptr(q), Hq, ctypes.byref(s), _ptr(meta), int(budget_tokens),
                              _ptr(cand), stride, _ptr(ncand), _ptr(ws), ws.numel(),
                              _stream(stream)), "tw_select_pages")
    return cand, ncand


def num_sets(kv: KVCache, Hq: int, group_mode: int) -> int:
    return kv.B * kv.Hk if (group_mode or Hq == kv.Hk) else kv.B * Hq


def topp_prune(q: torch.Tensor, kv: KVCache, keys: Int4Keys, cand: Optional[torch.Tensor],
               ncand: Optional[torch.Tensor], p: float, group_mode: int = 0,
               capacity: Optional[int] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Twilight top-p pruning of the candidates: tw_topp_prune -> (idx, count)."""
    lib = _capi.load()
    _need(q, torch.float16, "q")
    _check_keys(kv, keys)
    Hq = int(q.shape[1])
    stride = int(cand.shape[-1]) if cand is not None else 0
    if capacity is None:
        capacity = min(stride, kv.max_pages) * PAGE if cand is not None else kv.N
        capacity = max(capacity, 1)
    U = num_sets(kv, Hq, group_mode)
    idx = torch.zeros((U, capacity), dtype=torch.int32, device=q.device)
    count = torch.zeros((U,), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = new_workspace(kv.B, Hq, kv.Hk, kv.N, capacity, q.device)
    s = kv.struct()
    check(lib.tw_topp_prune(_ptr(q), Hq, ctypes.byref(s), _ptr(keys.codes), _ptr(keys.scales),
                            _ptr(keys.zeros), _ptr(cand), stride, _ptr(ncand), float(p),
                            int(group_mode), _ptr(idx), capacity, _ptr(count), _ptr(ws),
                            ws.numel(), _stream(stream)), "tw_topp_prune")
    return idx, count


def sparse_decode(q: torch.Tensor, kv: KVCache, idx: torch.Tensor, count: torch.Tensor,
                  group_mode: int = 0, ws: Optional[torch.Tensor] = None, with_lse: bool = True,
                  stream=None):
    """Exact attention over the selected tokens: tw_sparse_decode -> (out, lse)."""
    lib = _capi.load()
    _need(q, torch.float16, "q")
    _need(idx, torch.int32, "idx")
    Hq = int(q.shape[1])
    capacity = int(idx.shape[-1])
    out = torch.empty((kv.B, Hq, HEAD_DIM), dtype=torch.float16, device=q.device)
    lse = torch.empty((kv.B, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    if ws is None:
        ws = new_workspace(kv.B, Hq, kv.Hk, kv.N, capacity, q.device)
    s = kv.struct()
    check(lib.tw_sparse_decode(_ptr(q), Hq, ctypes.byref(s), _ptr(idx), capacity, _ptr(count),
                               int(group_mode), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                               _stream(stream)), "tw_sparse_decode")
    return out, lse


class DecodeStep:
    """Pre-allocated buffers for repeated tw_decode_step calls on one shape.

    budget_tokens None (or <= 0) means base = full attention (every token is a
    candidate); otherwise Quest keeps budget_tokens // 16 pages first.
    append_keys: each call first folds the newest token of every sequence into
    the int4 cache and the page metadata (tw_append_keys inside the step)."""

    def __init__(self, kv: KVCache, keys: Int4Keys, meta: Optional[torch.Tensor], Hq: int,
                 budget_tokens: Optional[int], p: float, group_mode: int = 0,
                 with_lse: bool = True, append_keys: bool = False):
        _check_keys(kv, keys)
        self.kv, self.keys, self.meta = kv, keys, meta
        self.append = bool(append_keys)
        self.Hq = Hq
        self.budget = int(budget_tokens) if budget_tokens and budget_tokens > 0 else 0
        self.p = float(p)
        self.group_mode = int(group_mode)
        dev = kv.k.device
        if self.budget:
            self.cand_stride = max(1, budget_pages(self.budget, kv))
            self.capacity = self.cand_stride * PAGE
        else:
            self.cand_stride = 1
            self.capacity = max(kv.N, 1)
        self.cand = torch.zeros((kv.B, kv.Hk, self.cand_stride), dtype=torch.int32, device=dev)
        self.ncand = torch.zeros((kv.B, kv.Hk), dtype=torch.int32, device=dev)
        U = num_sets(kv, Hq, group_mode)
        self.idx = torch.zeros((U, self.capacity), dtype=torch.int32, device=dev)
        self.count = torch.zeros((U,), dtype=torch.int32, device=dev)
        self.out = torch.zeros((kv.B, Hq, HEAD_DIM), dtype=torch.float16, device=dev)
        self.lse = torch.zeros((kv.B, Hq), dtype=torch.float32, device=dev) if with_lse else None
        self.ws = new_workspace(kv.B, Hq, kv.Hk, kv.N, self.capacity, dev)
        self._q = None
        self._s = None
        self._q_stage = None   # device staging of the query for run_host

    def _struct(self, q: torch.Tensor) -> TwStep:
        if self._s is not None and self._q is q:
            return self._s
        _need(q, torch.float16, "q")
        if tuple(q.shape) != (self.kv.B, self.Hq, HEAD_DIM):
            raise ValueError(f"q must be [{self.kv.B}][{self.Hq}][128]")
        s = TwStep()
        s.q = _ptr(q)
        s.num_q_heads = self.Hq
        s.kv = self.kv.struct()
        s.codes, s.scales, s.zeros = (_ptr(self.keys.codes), _ptr(self.keys.scales),
                                      _ptr(self.keys.zeros))
        s.meta = _ptr(self.meta)
        s.budget_tokens = self.budget
        s.p = self.p
        s.group_mode = self.group_mode
        s.cand_pages, s.cand_stride, s.ncand = _ptr(self.cand), self.cand_stride, _ptr(self.ncand)
        s.idx, s.capacity, s.count = _ptr(self.idx), self.capacity, _ptr(self.count)
        s.out, s.lse = _ptr(self.out), _ptr(self.lse)
        s.ws, s.ws_bytes = _ptr(self.ws), self.ws.numel()
        s.append_keys = 1 if self.append else 0
        self._q, self._s = q, s
        return s

    def __call__(self, q: torch.Tensor, stream=None) -> torch.Tensor:
        lib = _capi.load()
        s = self._struct(q)
        check(lib.tw_decode_step(ctypes.byref(s), _stream(stream)), "tw_decode_step")
        return self.out

    def run_host(self, q_host: torch.Tensor, out_host: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """One step with the query taken from, and the output returned to,
        pinned host memory (tw_decode_step_host): the copies run as kernels of
        the step's launch chain.  q_host / out_host: pinned CPU fp16
        [B][Hq][128].  The step's device q / out buffers serve as staging.
        Synchronise the stream before reading out_host."""
        lib = _capi.load()
        shape = (self.kv.B, self.Hq, HEAD_DIM)
        if out_host is None:
            out_host = torch.empty(shape, dtype=torch.float16).pin_memory()
        for t, name in ((q_host, "q_host"), (out_host, "out_host")):
            if t.dtype != torch.float16 or t.is_cuda or not t.is_pinned() or \
                    not t.is_contiguous() or tuple(t.shape) != shape:
                raise ValueError(f"{name} must be a contiguous pinned CPU fp16 tensor {shape}")
        if self._q_stage is None:
            self._q_stage = torch.empty(shape, dtype=torch.float16, device=self.kv.k.device)
        s = self._struct(self._q_stage)
        check(lib.tw_decode_step_host(ctypes.byref(s), q_host.data_ptr(), out_host.data_ptr(),
                                      _stream(stream)), "tw_decode_step_host")
        return out_host

    def kernel_names(self):
        lib = _capi.load()
        s = self._struct(self._q) if self._q is not None else None
        if s is None:
            raise RuntimeError("call the step once before asking for kernel names")
        n = lib.tw_decode_step_num_kernels(ctypes.byref(s))
        return [lib.tw_decode_step_kernel_name(ctypes.byref(s), i).decode() for i in range(n)]

    def profiled(self, q: torch.Tensor, events, stream=None) -> None:
        """Run one step recording events[0] before and events[i+1] after kernel i."""
        lib = _capi.load()
        s = self._struct(q)
        arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
        check(lib.tw_decode_step_profiled(ctypes.byref(s), arr, len(events), _stream(stream)),
              "tw_decode_step_profiled")


def prepare(w, device=None, key_bits: int = 4):
    """Move a workload to the GPU and build its quantised key cache (key_bits
    wide) and page metadata with the library.  Returns (kv, keys, meta, q)."""
    if device is not None:
        w = w.to(device)
    kv = KVCache.from_workload(w, key_bits)
    keys = quantize_keys(kv)
    meta = page_meta(kv)
    return kv, keys, meta, w.q


# ----------------------------------------------------------------------------- label selector
def label_cache(kv: KVCache, channels: torch.Tensor, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Label cache of the token-level label-channel selector (tw_label_cache):
    the fp16 values of channels[h] (int32 CUDA [Hk][r]) of every key row."""
    lib = _capi.load()
    _need(channels, torch.int32, "channels")
    r = int(channels.shape[-1])
    if tuple(channels.shape) != (kv.Hk, r):
        raise ValueError(f"channels must be [{kv.Hk}][r]")
    if out is None:
        out = torch.zeros(kv.row_shape(r), dtype=torch.float16, device=kv.k.device)
    s = kv.struct()
    check(lib.tw_label_cache(ctypes.byref(s), _ptr(channels), r, _ptr(out), _stream(stream)),
          "tw_label_cache")
    return out


def _check_labels(kv: KVCache, labels: torch.Tensor, channels: torch.Tensor) -> int:
    """Label cache and channels of a KV cache: fp16 rows of r values, int32
    [Hk][r] channels.  Returns r."""
    _need(labels, torch.float16, "labels")
    _need(channels, torch.int32, "channels")
    r = int(channels.shape[-1]) if channels.dim() == 2 else -1
    if tuple(channels.shape) != (kv.Hk, r) or not 1 <= r <= 32:
        raise ValueError(f"channels must be int32 [{kv.Hk}][r] with 1 <= r <= 32")
    if tuple(labels.shape) != kv.row_shape(r):
        raise ValueError(f"labels must be {kv.row_shape(r)}, got {tuple(labels.shape)}")
    return r


def _check_cand_tokens(kv: KVCache, cand: torch.Tensor, ncand: torch.Tensor) -> int:
    """Token candidates [B][Hk][stride] and their counts [B][Hk] (int32).
    Returns stride."""
    _need(cand, torch.int32, "cand")
    _need(ncand, torch.int32, "ncand")
    stride = int(cand.shape[-1]) if cand.dim() == 3 else -1
    if tuple(cand.shape) != (kv.B, kv.Hk, stride) or stride < 1:
        raise ValueError(f"cand must be int32 [{kv.B}][{kv.Hk}][stride]")
    if tuple(ncand.shape) != (kv.B, kv.Hk):
        raise ValueError(f"ncand must be int32 [{kv.B}][{kv.Hk}]")
    return stride


def token_workspace_bytes(B, Hq, Hk, N, cand_stride, capacity, key_bits=4) -> int:
    lib = _capi.load()
    n = ctypes.c_size_t(0)
    check(lib.tw_token_workspace_size(B, Hq, Hk, N, cand_stride, capacity, key_bits,
                                      ctypes.byref(n)), "tw_token_workspace_size")
    return int(n.value)


def _token_ws(kv, Hq, stride, capacity, device):
    n = max(token_workspace_bytes(kv.B, Hq, kv.Hk, kv.N, stride, capacity, kv.key_bits), 256)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()   # the device status word
    return ws


def select_tokens(q: torch.Tensor, kv: KVCache, labels: torch.Tensor, channels: torch.Tensor,
                  budget_tokens: int, ws: Optional[torch.Tensor] = None, stream=None):
    """Token-level label-channel pre-selection (tw_select_tokens) ->
    (cand_tokens [B][Hk][stride], ncand [B][Hk]), stride = min(budget, N)."""
    lib = _capi.load()
    _need(q, torch.float16, "q")
    Hq = int(q.shape[1])
    r = _check_labels(kv, labels, channels)
    stride = max(1, min(int(budget_tokens), kv.N))
    cand = torch.zeros((kv.B, kv.Hk, stride), dtype=torch.int32, device=q.device)
    ncand = torch.zeros((kv.B, kv.Hk), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = _token_ws(kv, Hq, stride, stride, q.device)
    s = kv.struct()
    check(lib.tw_select_tokens(_ptr(q), Hq, ctypes.byref(s), _ptr(labels), _ptr(channels), r,
                               int(budget_tokens), _ptr(cand), stride, _ptr(ncand), _ptr(ws),
                               ws.numel(), _stream(stream)), "tw_select_tokens")
    return cand, ncand


def topp_prune_tokens(q: torch.Tensor, kv: KVCache, keys: Int4Keys, cand: torch.Tensor,
                      ncand: torch.Tensor, p: float, group_mode: int = 0,
                      capacity: Optional[int] = None, ws: Optional[torch.Tensor] = None,
                      stream=None):
    """Twilight top-p over token candidates (tw_topp_prune_tokens) -> (idx, count)."""
    lib = _capi.load()
    _need(q, torch.float16, "q")
    _check_keys(kv, keys)
    Hq = int(q.shape[1])
    stride = _check_cand_tokens(kv, cand, ncand)
    capacity = stride if capacity is None else int(capacity)
    U = num_sets(kv, Hq, group_mode)
    idx = torch.zeros((U, capacity), dtype=torch.int32, device=q.device)
    count = torch.zeros((U,), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = _token_ws(kv, Hq, stride, capacity, q.device)
    s = kv.struct()
    check(lib.tw_topp_prune_tokens(_ptr(q), Hq, ctypes.byref(s), _ptr(keys.codes),
                                   _ptr(keys.scales), _ptr(keys.zeros), _ptr(cand), stride,
                                   _ptr(ncand), float(p), int(group_mode), _ptr(idx), capacity,
                                   _ptr(count), _ptr(ws), ws.numel(), _stream(stream)),
          "tw_topp_prune_tokens")
    return idx, count


class LabelDecodeStep:
    """A decode step with the token-level label-channel base selector:
    tw_select_tokens -> tw_topp_prune_tokens -> tw_sparse_decode on one
    stream with pre-allocated buffers (no host synchronisation)."""

    NAMES = ("select_tokens", "topp_prune_tokens", "sparse_decode")
    LAUNCHES = 2 + 4 + 2   # kernels of the three calls

    def __init__(self, kv: KVCache, keys: Int4Keys, labels: torch.Tensor, channels: torch.Tensor,
                 Hq: int, budget_tokens: int, p: float, group_mode: int = 0,
                 with_lse: bool = True):
        _check_keys(kv, keys)
        _check_labels(kv, labels, channels)
        self.kv, self.keys, self.labels, self.channels = kv, keys, labels, channels
        self.Hq, self.budget, self.p, self.group_mode = Hq, int(budget_tokens), float(p), \
            int(group_mode)
        dev = kv.k.device
        self.stride = max(1, min(self.budget, kv.N))
        self.capacity = self.stride
        self.cand = torch.zeros((kv.B, kv.Hk, self.stride), dtype=torch.int32, device=dev)
        self.ncand = torch.zeros((kv.B, kv.Hk), dtype=torch.int32, device=dev)
        U = num_sets(kv, Hq, group_mode)
        self.idx = torch.zeros((U, self.capacity), dtype=torch.int32, device=dev)
        self.count = torch.zeros((U,), dtype=torch.int32, device=dev)
        self.out = torch.zeros((kv.B, Hq, HEAD_DIM), dtype=torch.float16, device=dev)
        self.lse = torch.zeros((kv.B, Hq), dtype=torch.float32, device=dev) if with_lse else None
        n = max(token_workspace_bytes(kv.B, Hq, kv.Hk, kv.N, self.stride, self.capacity,
                                      kv.key_bits),
                workspace_bytes(kv.B, Hq, kv.Hk, kv.N, self.capacity), 256)
        self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        self.ws[:256].zero_()   # the device status word
        self._kvs = kv.struct()
        self._q_stage = None

    def _calls(self, q: torch.Tensor, stream):
        lib = _capi.load()
        st = _stream(stream)
        kvs, ws, nws = ctypes.byref(self._kvs), _ptr(self.ws), self.ws.numel()
        r = int(self.channels.shape[-1])
        yield lambda: check(lib.tw_select_tokens(
            _ptr(q), self.Hq, kvs, _ptr(self.labels), _ptr(self.channels), r, self.budget,
            _ptr(self.cand), self.stride, _ptr(self.ncand), ws, nws, st), "tw_select_tokens")
        yield lambda: check(lib.tw_topp_prune_tokens(
            _ptr(q), self.Hq, kvs, _ptr(self.keys.codes), _ptr(self.keys.scales),
            _ptr(self.keys.zeros), _ptr(self.cand), self.stride, _ptr(self.ncand), self.p,
            self.group_mode, _ptr(self.idx), self.capacity, _ptr(self.count), ws, nws, st),
            "tw_topp_prune_tokens")
        yield lambda: check(lib.tw_sparse_decode(
            _ptr(q), self.Hq, kvs, _ptr(self.idx), self.capacity, _ptr(self.count),
            self.group_mode, _ptr(self.out), _ptr(self.lse), ws, nws, st), "tw_sparse_decode")

    def __call__(self, q: torch.Tensor, stream=None) -> torch.Tensor:
        _need(q, torch.float16, "q")
        for call in self._calls(q, stream):
            call()
        return self.out

    def kernel_names(self):
        return list(self.NAMES)

    def profiled(self, q: torch.Tensor, events, stream=None) -> None:
        """One step with events[0] before and events[i + 1] after call i."""
        s = torch.cuda.current_stream() if stream is None else stream
        events[0].record(s)
        for i, call in enumerate(self._calls(q, stream)):
            call()
            events[i + 1].record(s)

    def run_host(self, q_host: torch.Tensor, out_host: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """One step from and to pinned host memory (copy-engine transfers)."""
        if out_host is None:
            out_host = torch.empty(tuple(self.out.shape), dtype=torch.float16).pin_memory()
        if self._q_stage is None:
            self._q_stage = torch.empty(tuple(self.out.shape), dtype=torch.float16,
                                        device=self.kv.k.device)
        self._q_stage.copy_(q_host, non_blocking=True)
        self(self._q_stage, stream)
        out_host.copy_(self.out, non_blocking=True)
        return out_host


# ----------------------------------------------------------------------------- serving around the cache
@contextlib.contextmanager
def _on(device: torch.device, stream):
    """Make `device`, and `stream` if one is given, current: what is allocated
    inside belongs to the stream the kernels run on."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device)
        else:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            with torch.cuda.stream(stream):
                yield stream


def _need_on(t: torch.Tensor, dtype, name: str, device, shape=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


# The current stream's handle without a Stream object (3 us of a call's 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Made:
    """Orders calls on any stream behind the making of a step's buffers.  A fill
    of theirs, and work that still uses memory they were given, may be waiting on
    the stream that was current then: a call on another stream waits for what
    that stream held, once.  Not while a call is captured (a graph cannot wait
    for work outside it; torch.cuda.graph synchronises the device first)."""
    __slots__ = ("event", "ordered")

    def __init__(self, device: torch.device):
        s = torch.cuda.current_stream(device)
        self.ordered = {s.cuda_stream}
        # (made inside a capture: the buffers belong to that graph, and so do its calls)
        self.event = None if torch.cuda.is_current_stream_capturing() else s.record_event()

    def wait(self, device: torch.device, stream, handle: int) -> None:
        s = torch.cuda.current_stream(device) if stream is None else stream
        with torch.cuda.stream(s):
            if self.event is None or torch.cuda.is_current_stream_capturing():
                return
        s.wait_event(self.event)
        self.ordered.add(handle)


def _launch(f, where: str, device: torch.device, stream, *args,
            made: Optional[_Made] = None) -> None:
    """f(*args, stream) with the tensors' device current; `stream`, or that
    device's current stream."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    handle = _raw_stream(device.index) if stream is None else stream.cuda_stream
    if made is not None and handle not in made.ordered:
        made.wait(device, stream, handle)
    if torch.cuda.current_device() == device.index:
        status = f(*args, handle)
    else:
        with torch.cuda.device(device):
            status = f(*args, handle)
    if status:
        check(status, where)


class PageTableUpdate:
    """Page tables and slot maps on the GPU from request lengths
    (tw_update_page_table), with output buffers for repeated calls.

    seq_lens [B] are the lengths before the step, page_table [B][W] and the
    stack free_pages [pool pages] are updated in place; the first prefix_len /
    16 entries of every row are the caller's (a shared prefix).  A call takes
    new_lens [B] and num_free [1] (all int32 CUDA tensors) and fills
    seq_lens_out [B] (the lengths reached: a growth that finds no pages is
    refused), num_free_out [1], slots [num_slots] (the cache slot of every new
    token, -1 where there is none) and offsets [B + 1] (a sequence's first
    place in slots).  in_place: seq_lens and num_free take the results
    themselves (the names above are then the same tensors), so that a captured
    call can be replayed step after step.  Calls may come on any stream, one
    after another: they share the output buffers, which are to be kept until
    the last call's work is done."""

    def __init__(self, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 free_pages: torch.Tensor, num_slots: int = 0, prefix_len: int = 0,
                 in_place: bool = False):
        _need(seq_lens, torch.int32, "seq_lens")
        dev = self.device = seq_lens.device
        if seq_lens.dim() != 1 or page_table.dim() != 2 or free_pages.dim() != 1:
            raise ValueError("seq_lens must be [B], page_table [B][W], free_pages [pool pages]")
        B = int(seq_lens.shape[0])
        _need_on(page_table, torch.int32, "page_table", dev, (B, page_table.shape[1]))
        _need_on(free_pages, torch.int32, "free_pages", dev)
        room = PAGE * int(page_table.shape[1])
        if not 0 <= num_slots <= INT32_MAX or free_pages.shape[0] > INT32_MAX:
            raise ValueError("num_slots and the pages of the pool must be 32-bit numbers, not "
                             f"{num_slots} and {free_pages.shape[0]}")
        if prefix_len < 0 or prefix_len % PAGE or prefix_len > room:
            raise ValueError(f"prefix_len must be a multiple of {PAGE} in [0, {room}]")
        self.seq_lens, self.page_table, self.free_pages = seq_lens, page_table, free_pages
        self.prefix_len, self.in_place, self.num_slots = int(prefix_len), bool(in_place), int(num_slots)
        with torch.cuda.device(dev):
            self.seq_lens_out = seq_lens if in_place else torch.empty_like(seq_lens)
            self.num_free_out = None if in_place else seq_lens.new_empty(1)
            self.slots = seq_lens.new_empty(num_slots)   # every call writes all of them
            self.offsets = seq_lens.new_empty(B + 1)
            self._made = _Made(dev)

    def __call__(self, new_lens: torch.Tensor, num_free: torch.Tensor,
                 stream=None) -> "PageTableUpdate":
        lib = _capi.load()
        B, W = self.page_table.shape
        _need_on(new_lens, torch.int32, "new_lens", self.device, (B,))
        _need_on(num_free, torch.int32, "num_free", self.device, (1,))
        if self.in_place:
            self.num_free_out = num_free
        _launch(lib.tw_update_page_table, "tw_update_page_table", self.device, stream,
                B, _ptr(self.seq_lens), _ptr(new_lens), _ptr(self.page_table), W, self.prefix_len,
                _ptr(self.free_pages), self.free_pages.shape[0], _ptr(num_free),
                _ptr(self.num_free_out), _ptr(self.seq_lens_out),
                _ptr(self.slots) if self.num_slots else None, self.num_slots, _ptr(self.offsets),
                made=self._made)
        return self


def update_page_table(seq_lens: torch.Tensor, new_lens: torch.Tensor, page_table: torch.Tensor,
                      free_pages: torch.Tensor, num_free: torch.Tensor, num_slots: int = 0,
                      prefix_len: int = 0, stream=None) -> PageTableUpdate:
    """One PageTableUpdate call with new output buffers: its seq_lens_out,
    num_free_out, slots and offsets are the results."""
    with _on(seq_lens.device, stream):
        u = PageTableUpdate(seq_lens, page_table, free_pages, num_slots, prefix_len)
    return u(new_lens, num_free, stream)


def _token_rows(t: torch.Tensor, name: str, T: int, Hk: int, index: int) -> int:
    """Check new rows [T][Hk][128] (a slice of a wider projection may be given:
    only the last two dimensions must be packed).  Returns the token stride."""
    if t.dtype is not torch.float16 or t.get_device() != index or t.shape != (T, Hk, HEAD_DIM):
        raise ValueError(f"{name} must be fp16 [{T}][{Hk}][128] on the cache's device")
    stride, sh, sd = t.stride()
    if sd != 1 or (sh != HEAD_DIM and Hk > 1):
        raise ValueError(f"{name}: a token's heads must lie side by side")
    width = Hk * HEAD_DIM
    if T <= 1:
        return width
    if stride < width or stride % 8:
        raise ValueError(f"{name}: token stride {stride} must be a multiple of 8, "
                         f"at least {width}")
    return stride


def write_rows(kv: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor,
               keys: Optional[Int4Keys] = None, meta: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """Write new K / V rows [T][Hk][128] to the cache slots slots [T] (int32, -1
    skips) and, in the same pass, quantise the keys into `keys` and fold them
    into `meta` (if given): tw_write_rows."""
    kv.recheck()
    k, v, table = kv.k, kv.v, kv.page_table
    index = k.get_device()
    # (a call for single tokens is as long as these lines: each property is read once)
    def same(t, dtype, shape, name):
        if (t.dtype is not dtype or t.get_device() != index or t.shape != shape
                or not t.is_contiguous()):
            _need_on(t, dtype, name, k.device, shape)

    if v is None or v.get_device() != index:
        raise ValueError(f"the cache needs a v on {k.device}")
    pool, Hk, rows, _ = k.shape
    B = kv.seq_lens.shape[0]
    if table is None:
        if pool < B:
            raise ValueError(f"the cache has {pool} sequences, seq_lens {B}")
        lead, width, pages = (B, Hk, rows), 0, 0
    else:
        lead, width, pages = (pool, Hk, PAGE), table.shape[1], pool
    if slots.dim() != 1:
        raise ValueError("slots must be [T]")
    T = slots.shape[0]
    same(slots, torch.int32, (T,), "slots")
    k_stride = _token_rows(k_new, "k_new", T, Hk, index)
    v_stride = _token_rows(v_new, "v_new", T, Hk, index)
    codes = scales = zeros = mp = None
    if keys is not None:
        c, sc, z = keys.codes, keys.scales, keys.zeros
        if c.shape != lead + (kv.code_bytes,):
            _check_keys(kv, keys)
        same(c, torch.uint8, lead + (kv.code_bytes,), "codes")
        same(sc, torch.float16, lead + (4,), "scales")
        same(z, torch.float16, lead + (4,), "zeros")
        codes, scales, zeros = c.data_ptr(), sc.data_ptr(), z.data_ptr()
    if meta is not None:
        same(meta, torch.float16, kv.meta_shape(), "meta")
        mp = meta.data_ptr()
    if T == 0:
        return
    st = TwKv(k.data_ptr(), v.data_ptr(), B, Hk, width * PAGE if pages else rows,
              kv.seq_lens.data_ptr(), table.data_ptr() if pages else None, width, pages, PAGE,
              HEAD_DIM, kv.key_bits)
    _launch(_capi.load().tw_write_rows, "tw_write_rows", k.device, stream, ctypes.byref(st),
            k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride, slots.data_ptr(), T, codes,
            scales, zeros, mp)


def prefix_workspace_bytes(B: int, Hq: int, Hk: int, prefix_len: int) -> int:
    lib = _capi.load()
    if max(B, Hq, Hk, prefix_len) > INT32_MAX:
        raise ValueError("sizes must be 32-bit numbers")
    n = ctypes.c_size_t(0)
    check(lib.tw_prefix_workspace_size(B, Hq, Hk, prefix_len, ctypes.byref(n)),
          "tw_prefix_workspace_size")
    return int(n.value)


class PrefixDecodeStep:
    """Dense decode attention of a batch whose sequences share their first
    prefix_len tokens (tw_prefix_decode), with pre-allocated outputs `out`
    [B][Hq][128], `lse` [B][Hq] (or None) and workspace for repeated calls.

    The shared tokens are read once, from sequence 0's first pages (or
    contiguous rows).  prefix_len 0 shares nothing: plain dense decode.  A call
    reads the tensors that kv names then; their batch and heads stay.  Calls
    may come on any stream, one after another: they share the outputs and the
    workspace, which are to be kept until the last call's work is done."""

    def __init__(self, kv: KVCache, Hq: int, prefix_len: int, with_lse: bool = True):
        self.kv, self.Hq, self.prefix_len = kv, int(Hq), int(prefix_len)
        dev = kv.k.device
        self._bind()
        with torch.cuda.device(dev):
            self.out = torch.empty((kv.B, Hq, HEAD_DIM), dtype=torch.float16, device=dev)
            self.lse = torch.empty((kv.B, Hq), dtype=torch.float32, device=dev) if with_lse \
                else None
            n = max(prefix_workspace_bytes(kv.B, self.Hq, kv.Hk, self.prefix_len), 256)
            self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
            self.ws[:256].zero_()   # the device status word
            self._made = _Made(dev)
        self._shape = kv.B, kv.Hk, dev

    def _bind(self) -> None:
        """Check the cache's present tensors and take their addresses."""
        kv = self.kv
        kv.recheck()
        if kv.v is None:
            raise ValueError("the cache has no v")
        if self.prefix_len < 0 or self.prefix_len % PAGE or self.prefix_len > kv.N:
            raise ValueError(f"prefix_len must be a multiple of {PAGE} in [0, {kv.N}]")
        dev = kv.k.device
        for t, name in ((kv.v, "v"), (kv.seq_lens, "seq_lens"), (kv.page_table, "page_table")):
            if t is not None and t.device != dev:
                raise ValueError(f"{name} must be on {dev}, got {t.device}")
        shape = (kv.page_table if kv.paged else kv.k).shape
        if shape[0] != kv.B:
            raise ValueError(f"the cache has {shape[0]} sequences, seq_lens {kv.B}")
        self._kvs, self._bound = kv.struct(), (kv.k, kv.v, kv.seq_lens, kv.page_table)

    def __call__(self, q: torch.Tensor, stream=None) -> torch.Tensor:
        lib = _capi.load()
        kv, (k, v, lens, table) = self.kv, self._bound
        if (kv.k is not k or kv.v is not v or kv.seq_lens is not lens
                or kv.page_table is not table):   # the cache has other tensors by now
            if (kv.B, kv.Hk, kv.k.device) != self._shape:
                raise ValueError("the step was made for [B, Hk, device] = "
                                 f"{list(self._shape)}, the cache is "
                                 f"{[kv.B, kv.Hk, kv.k.device]}")
            self._bind()
        _need_on(q, torch.float16, "q", self.kv.k.device, (self.kv.B, self.Hq, HEAD_DIM))
        if self.kv.B == 0:
            return self.out
        _launch(lib.tw_prefix_decode, "tw_prefix_decode", self.kv.k.device, stream,
                _ptr(q), self.Hq, ctypes.byref(self._kvs), self.prefix_len, _ptr(self.out),
                _ptr(self.lse), _ptr(self.ws), self.ws.numel(), made=self._made)
        return self.out


def prefix_decode(q: torch.Tensor, kv: KVCache, prefix_len: int, with_lse: bool = True,
                  stream=None):
    """One PrefixDecodeStep call with new buffers: tw_prefix_decode -> (out, lse)."""
    with _on(kv.k.device, stream):
        step = PrefixDecodeStep(kv, int(q.shape[1]), prefix_len, with_lse)
    return step(q, stream), step.lse
