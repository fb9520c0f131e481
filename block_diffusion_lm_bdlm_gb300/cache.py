"""Python binding of the paged 8-bit cache (the bdlm_cache_* calls of
include/bdlm.h). Argument checks and marshalling only; see the header for the
layout, the mask and what each call leaves undone on an error.

A model that answers block by block uses the calls in this order, for every
block (decode.BlockDecoder does it):

  bdlm_cache_reserve(cache, lens + rows)            once
  bdlm_cache_write(cache, k, v, cu, layer=i)        each layer, each denoising step
  bdlm_cache_attn_fwd(cache, q, cu, B, layer=i)     likewise

Where sequences share pages (bdlm_cache_fork), bdlm_cache_prefixes finds once
per block which do, and bdlm_cache_attn_shared_fwd takes the place of
bdlm_cache_attn_fwd.

Problems found on the device (malformed offsets or tables, too few pages) are
written to the error word of the workspace: pass `workspace` and read it with
bdlm_read_error(workspace), or pass check=True, which synchronises and raises.
"""
from __future__ import annotations

import ctypes
import threading
from contextlib import nullcontext

import torch

from . import BDLM_BF16, BDLM_F32, _bf16_cuda, _CCache, _check, _shape, load_library

PAGE_SIZES = (16, 32, 64, 128)
BDLM_ERR_INVALID_ARG, BDLM_ERR_DEVICE_CHECK = 1, 6


class PageCache:
    """The cache's device tensors, with their sizes:

      k, v             float8_e4m3fn [n_layers, n_pages, Hk, page, d]
      k_scale, v_scale fp32 [n_layers, n_pages, Hk]
      table            int32 [n_seqs, max_pages]
      lens             int32 [n_seqs]

    All contiguous and on one device. The object holds no state of the cache
    itself: table and lens are the truth, and the calls and the program write
    them in stream order. To end sequences, set their lens to 0.

    It keeps one workspace for calls that bring neither workspace nor stream,
    come on the current stream that the first such call came on, are not
    captured into a graph and do not ask for their error word; other calls get
    one of their own.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "table", "lens", "n_layers", "n_pages", "page", "kv_heads",
                 "head_dim", "n_seqs", "max_pages", "device", "index", "pages_bytes", "c", "ref", "home", "scratch", "lock",
                 "need", "need_shared")

    def __init__(self, k, v, k_scale, v_scale, table, lens):
        for nm, t, dt, dims in (("k", k, torch.float8_e4m3fn, 5), ("v", v, torch.float8_e4m3fn, 5),
                                ("k_scale", k_scale, torch.float32, 3), ("v_scale", v_scale, torch.float32, 3),
                                ("table", table, torch.int32, 2), ("lens", lens, torch.int32, 1)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dt or t.dim() != dims \
                    or not t.is_contiguous() or t.numel() == 0:
                raise ValueError(f"{nm} must be a contiguous {dt} CUDA tensor of {dims} dimensions")
            if t.device != k.device:
                raise ValueError(f"{nm} is on {t.device}, k on {k.device}")
        self.n_layers, self.n_pages, self.kv_heads, self.page, self.head_dim = k.shape
        self.n_seqs, self.max_pages = table.shape
        if self.page not in PAGE_SIZES:
            raise ValueError(f"the page size must be one of {PAGE_SIZES}, got {self.page}")
        if self.head_dim not in (64, 128):
            raise ValueError(f"head_dim must be 64 or 128, got {self.head_dim}")
        _shape("v", v, k.shape)
        _shape("k_scale", k_scale, k.shape[:3])
        _shape("v_scale", v_scale, k.shape[:3])
        _shape("lens", lens, (self.n_seqs,))
        self.k, self.v, self.k_scale, self.v_scale, self.table, self.lens = k, v, k_scale, v_scale, table, lens
        self.device, self.index = k.device, k.get_device()
        self.pages_bytes = max(bdlm_cache_pages_workspace_bytes(self.n_pages, self.n_seqs), 256)
        self.c = _CCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(),
                         lens.data_ptr(), self.n_layers, self.n_pages, self.page, self.kv_heads, self.head_dim,
                         self.n_seqs, self.max_pages, 0)
        self.ref = ctypes.byref(self.c)
        self.home, self.scratch, self.lock = None, None, threading.Lock()
        self.need = self.need_shared = None, 0  # (rows, heads) of the last attention call, and the workspace that they need

    @staticmethod
    def empty(n_layers: int, n_pages: int, page: int, kv_heads: int, head_dim: int, n_seqs: int, max_pages: int,
              device="cuda") -> "PageCache":
        """A cache of n_pages free pages and n_seqs empty sequences."""
        codes = [torch.empty((n_layers, n_pages, kv_heads, page, head_dim), dtype=torch.float8_e4m3fn, device=device)
                 for _ in range(2)]
        scales = [torch.ones((n_layers, n_pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        return PageCache(*codes, *scales, torch.zeros((n_seqs, max_pages), dtype=torch.int32, device=device),
                         torch.zeros(n_seqs, dtype=torch.int32, device=device))


def bdlm_cache_write_workspace_bytes() -> int:
    return int(load_library().bdlm_cache_write_workspace_bytes())


def bdlm_cache_attn_fwd_workspace_bytes(total_rows: int, heads: int, kv_heads: int, head_dim: int,
                                        n_seqs: int) -> int:
    return int(load_library().bdlm_cache_attn_fwd_workspace_bytes(total_rows, heads, kv_heads, head_dim, n_seqs))


def bdlm_cache_attn_shared_fwd_workspace_bytes(total_rows: int, heads: int, kv_heads: int, head_dim: int,
                                               n_seqs: int) -> int:
    return int(load_library().bdlm_cache_attn_shared_fwd_workspace_bytes(total_rows, heads, kv_heads, head_dim, n_seqs))


def bdlm_cache_prefixes_workspace_bytes(n_seqs: int) -> int:
    return int(load_library().bdlm_cache_prefixes_workspace_bytes(n_seqs))


def bdlm_cache_pages_workspace_bytes(n_pages: int, n_seqs: int) -> int:
    return int(load_library().bdlm_cache_pages_workspace_bytes(n_pages, n_seqs))


_NULL = nullcontext()


def _on(cache, stream):
    """(handle of the call's stream, context to make the call in): launches go
    to the cache's device, and what the call allocates belongs to the stream
    that uses it."""
    if stream is None:
        here = _NULL if cache.index == torch.cuda.current_device() else torch.cuda.device(cache.index)
        return torch._C._cuda_getCurrentRawStream(cache.index), here
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=cache.device)
    elif stream.device != cache.device:
        raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _workspace(cache, workspace, need, handle, private):
    """The caller's workspace, or one of at least `need` bytes. Calls on one
    stream follow one another, so they may share the cache's; the lock that the
    callers hold keeps the launches of one call together. Whatever may run at
    another time (another stream, a graph that is replayed, an error word that
    is read later: `private`) gets memory of its own."""
    if workspace is None:
        if private or (cache.home is not None and handle != cache.home) or torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=cache.device)
        if cache.scratch is None or cache.scratch.numel() < need:
            cache.home, cache.scratch = handle, torch.empty(need, dtype=torch.uint8, device=cache.device)
        return cache.scratch
    if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous() \
            or workspace.get_device() != cache.index:
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor on the cache's device")
    return workspace


def _ints(name, cache, t, n):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() \
            or t.get_device() != cache.index:
        raise ValueError(f"{name} must be a contiguous int32 tensor of one dimension on the cache's device")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
    return t.data_ptr()


def _layer(cache, layer):
    if not 0 <= layer < cache.n_layers:
        raise ValueError(f"layer {layer} is outside the cache's {cache.n_layers}")


def _read(lib, workspace, handle, where):
    _check(lib.bdlm_read_error(workspace.data_ptr(), handle), where + " (device)")


def _no_rows(cache, cu_rows, workspace, handle, check, where):
    """A call without rows launches none of the library's kernels; the error
    word is what theirs would be: offsets that count any row are malformed."""
    if workspace is None and not check:
        return
    bad = (cu_rows != 0).any().int() * BDLM_ERR_DEVICE_CHECK
    if workspace is not None:
        _workspace(cache, workspace, 256, handle, True)[:256].zero_()[:4].copy_(bad.reshape(1).view(torch.uint8))
    if check:
        _check(int(bad), where + " (device)")


def bdlm_cache_write(cache: PageCache, k_new, v_new, cu_rows, *, layer: int = 0, workspace=None, stream=None,
                     check: bool = False) -> None:
    """Quantise the new key and value rows k_new, v_new [T,Hk,d] (bf16) into
    the pages: rows cu_rows[s] .. cu_rows[s+1]-1 become the last positions of
    sequence s, whose lens already counts them. T may be 0."""
    lib = load_library()
    _bf16_cuda("k_new", k_new)
    _bf16_cuda("v_new", v_new)
    shape = k_new.shape
    if len(shape) != 3 or shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        raise ValueError(f"k_new must be [T, {cache.kv_heads}, {cache.head_dim}], got {tuple(shape)}")
    if v_new.shape != shape:
        raise ValueError(f"v_new must be shaped {tuple(shape)}, got {tuple(v_new.shape)}")
    if k_new.get_device() != cache.index or v_new.get_device() != cache.index:
        raise ValueError("k_new and v_new must be on the cache's device")
    cu = _ints("cu_rows", cache, cu_rows, cache.n_seqs + 1)
    _layer(cache, layer)
    handle, here = _on(cache, stream)
    with here:
        if shape[0] == 0:
            return _no_rows(cache, cu_rows, workspace, handle, check, "bdlm_cache_write")
        with cache.lock:
            ws = _workspace(cache, workspace, 256, handle, check or stream is not None)
            st = lib.bdlm_cache_write(cache.ref, layer, k_new.data_ptr(), v_new.data_ptr(), shape[0], cu, ws.data_ptr(),
                                      ws.numel(), handle)
        _check(st, "bdlm_cache_write")
        if check:
            _read(lib, ws, handle, "bdlm_cache_write")


def bdlm_cache_attn_fwd(cache: PageCache, q, cu_rows, block: int, *, layer: int = 0, q_pos=None,
                        softmax_scale: float = 0.0, out=None, lse=None, workspace=None, stream=None,
                        check: bool = False):
    """Attention of the rows q [T,H,d] (bf16) over the cache under the
    block-causal mask; returns (o [T,H,d], lse [H,T] fp32). o is bf16 unless
    `out` is fp32. With q_pos (int32 [n_seqs], the position of each sequence's
    first row) the rows need not be in the cache, and the result is a partial
    one for bdlm_lse_merge. Rows of q behind cu_rows[-1] are left unwritten. T
    may be 0."""
    return _attn("bdlm_cache_attn_fwd", cache, q, cu_rows, block, None, layer, q_pos, softmax_scale, out, lse, workspace,
                 stream, check)


def bdlm_cache_attn_shared_fwd(cache: PageCache, q, cu_rows, block: int, runs, *, layer: int = 0, q_pos=None,
                               softmax_scale: float = 0.0, out=None, lse=None, workspace=None, stream=None,
                               check: bool = False):
    """bdlm_cache_attn_fwd in which what the sequences of a run share is read
    once: `runs` (int32 [3, n_seqs]) comes from bdlm_cache_prefixes."""
    _plan(cache, runs)
    return _attn("bdlm_cache_attn_shared_fwd", cache, q, cu_rows, block, runs, layer, q_pos, softmax_scale, out, lse,
                 workspace, stream, check)


def _plan(cache, runs):
    if not isinstance(runs, torch.Tensor) or runs.dtype != torch.int32 or not runs.is_contiguous() \
            or runs.get_device() != cache.index or runs.shape != (3, cache.n_seqs):
        raise ValueError(f"runs must be a contiguous int32 tensor [3, {cache.n_seqs}] on the cache's device")


def _attn(name, cache, q, cu_rows, block, runs, layer, q_pos, softmax_scale, out, lse, workspace, stream, check):
    lib = load_library()
    _bf16_cuda("q", q)
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.get_device() != cache.index:
        raise ValueError(f"q must be [T, H, {cache.head_dim}] on the cache's device")
    T, H, d = q.shape
    if H == 0 or H % cache.kv_heads or not 0 < block < 2 ** 31:  # ctypes would take block modulo 2^32
        _check(BDLM_ERR_INVALID_ARG, name)
    cu = _ints("cu_rows", cache, cu_rows, cache.n_seqs + 1)
    pos = None if q_pos is None else _ints("q_pos", cache, q_pos, cache.n_seqs)
    _layer(cache, layer)
    sized, need = cache.need if runs is None else cache.need_shared
    if sized != (T, H):
        need = max(getattr(lib, name + "_workspace_bytes")(T, H, cache.kv_heads, d, cache.n_seqs), 256)
        if runs is None:
            cache.need = (T, H), need
        else:
            cache.need_shared = (T, H), need
    handle, here = _on(cache, stream)
    with here:
        if out is None:
            out = torch.empty_like(q)
        elif out.dtype not in (torch.bfloat16, torch.float32) or out.shape != q.shape or out.device != cache.device \
                or not out.is_contiguous():
            raise ValueError("out must be a contiguous bf16 or fp32 CUDA tensor shaped like q")
        if lse is None:
            lse = torch.empty((H, T), dtype=torch.float32, device=cache.device)
        elif lse.shape != (H, T) or lse.dtype != torch.float32 or lse.device != cache.device \
                or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous fp32 CUDA tensor [H, T]")
        if T == 0:
            _no_rows(cache, cu_rows, workspace, handle, check, name)
            return out, lse
        with cache.lock:
            ws = _workspace(cache, workspace, need, handle, check or stream is not None)
            plan = () if runs is None else (runs.data_ptr(),)
            st = getattr(lib, name)(cache.ref, layer, q.data_ptr(), out.data_ptr(), lse.data_ptr(), T, H, block, cu, pos,
                                    *plan, softmax_scale, BDLM_F32 if out.dtype == torch.float32 else BDLM_BF16,
                                    ws.data_ptr(), ws.numel(), handle)
        _check(st, name)
        if check:
            _read(lib, ws, handle, name)
    return out, lse


def _pages_call(cache, name, args, workspace, stream, check, make=None):
    lib = load_library()
    handle, here = _on(cache, stream)
    with here:
        made = None if make is None else make()
        if made is not None:
            args = (made.data_ptr(),)
        with cache.lock:
            ws = _workspace(cache, workspace, cache.pages_bytes, handle, check or stream is not None)
            st = getattr(lib, name)(cache.ref, *args, ws.data_ptr(), ws.numel(), handle)
        _check(st, name)
        if check:
            _read(lib, ws, handle, name)
    return made


def bdlm_cache_reserve(cache: PageCache, new_lens, *, workspace=None, stream=None, check: bool = False) -> None:
    """Set cache.lens to new_lens (int32 [n_seqs]) and enter free pages for
    the positions gained; pages that shorter lengths give up become free."""
    _pages_call(cache, "bdlm_cache_reserve", (_ints("new_lens", cache, new_lens, cache.n_seqs),), workspace, stream,
                check)


def bdlm_cache_fork(cache: PageCache, parents, children, fork_lens=None, *, workspace=None, stream=None,
                    check: bool = False) -> None:
    """Sequence children[i] (empty) becomes a copy of the first fork_lens[i]
    positions (None: all) of parents[i]: full pages are shared, a partly
    filled last page is copied, in all layers. There may be no forks."""
    n = parents.shape[0] if isinstance(parents, torch.Tensor) and parents.dim() == 1 else None
    args = (_ints("parents", cache, parents, n), _ints("children", cache, children, n),
            None if fork_lens is None else _ints("fork_lens", cache, fork_lens, n), n)
    if n == 0:
        if workspace is not None:
            handle, here = _on(cache, stream)
            with here:
                _workspace(cache, workspace, 256, handle, True)[:256].zero_()
        return
    _pages_call(cache, "bdlm_cache_fork", args, workspace, stream, check)


def bdlm_cache_compact(cache: PageCache, *, workspace=None, stream=None, check: bool = False) -> torch.Tensor:
    """Move the live pages to the front of the pool; returns their number
    (int32 [1], on the device). Pages from there on are free afterwards."""
    return _pages_call(cache, "bdlm_cache_compact", (), workspace, stream, check,
                       make=lambda: torch.zeros(1, dtype=torch.int32, device=cache.device))


def bdlm_cache_prefixes(cache: PageCache, cu_rows, *, total_rows: int | None = None, q_pos=None, out=None, workspace=None,
                        stream=None, check: bool = False) -> torch.Tensor:
    """The runs of sequences that share leading pages (int32 [3, n_seqs]: first
    sequence, number behind the last one, shared positions), for
    bdlm_cache_attn_shared_fwd. They hold for all layers until the table, the
    lengths or the rows change. total_rows bounds the offsets (None: any)."""
    lib = load_library()
    n = cache.n_seqs
    cu = _ints("cu_rows", cache, cu_rows, n + 1)
    pos = None if q_pos is None else _ints("q_pos", cache, q_pos, n)
    if out is not None:
        _plan(cache, out)
    handle, here = _on(cache, stream)
    with here:
        if out is None:
            out = torch.empty((3, n), dtype=torch.int32, device=cache.device)
        with cache.lock:
            ws = _workspace(cache, workspace, 256 + 4 * n, handle, check or stream is not None)
            st = lib.bdlm_cache_prefixes(cache.ref, 2 ** 30 if total_rows is None else total_rows, cu, pos, out.data_ptr(),
                                         ws.data_ptr(), ws.numel(), handle)
        _check(st, "bdlm_cache_prefixes")
        if check:
            _read(lib, ws, handle, "bdlm_cache_prefixes")
    return out
