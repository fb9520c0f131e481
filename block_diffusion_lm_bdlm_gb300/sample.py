"""Python binding of bdlm_sample and bdlm_unmask (include/bdlm.h): from a
denoising step's logits to tokens. Argument checks and marshalling only.

  token, logprob = bdlm_sample(logits, u, temperature=0.8, top_p=0.95)
  tokens, left = bdlm_unmask(tokens, token, logprob, cu_rows, mask_id, n_min=2, threshold=-0.1)

Both run on the current stream (or `stream`) of the device of their tensors.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext

import torch

from . import BDLM_BF16, BDLM_F16, BDLM_F32, _check, _CSampling, SAMPLE_NO_MASK, load_library

_DTYPES = {torch.bfloat16: BDLM_BF16, torch.float16: BDLM_F16, torch.float32: BDLM_F32}
_NULL = nullcontext()


def bdlm_unmask_workspace_bytes() -> int:
    return int(load_library().bdlm_unmask_workspace_bytes())


def _on(device, stream):
    """(handle of the call's stream, context to make the call in)."""
    if stream is None:
        index = device.index
        here = _NULL if index == torch.cuda.current_device() else torch.cuda.device(index)
        return torch._C._cuda_getCurrentRawStream(index), here
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _vector(name, t, dtype, n, index):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() \
            or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of one dimension on cuda:{index}")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return t.data_ptr()


def _either(name, x, dtype, n, index):
    """(pointer, value) of a parameter that is a tensor or one number for all."""
    if isinstance(x, torch.Tensor):
        return _vector(name, x, dtype, n, index), 0
    if dtype == torch.int32:
        if not -2 ** 31 <= int(x) < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits, got {x}")
        return None, int(x)
    return None, float(x)


def bdlm_sample(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, mask_id: int = 0, out=None,
                logprob=None, stream=None, draw_mask: bool = True):
    """Draw a token for each row of logits [rows, vocab] (bf16, fp16 or fp32;
    rows may be strided) with the random numbers u (fp32 [rows], in [0, 1]).
    Returns (token int32 [rows], logprob fp32 [rows]); logprob is that of the
    token under softmax(logits). temperature, top_p, min_p (fp32) and top_k
    (int32) are numbers or tensors [rows]. With `tokens` (int32 [rows]) only
    rows whose token is mask_id are drawn: `out` (which may be tokens itself)
    and `logprob` stay as they were in the others. With draw_mask=False token
    mask_id counts as if its logit were -inf. -1 and -inf stand in rows
    without any logit above -inf. rows may be 0."""
    lib = load_library()
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype not in _DTYPES or logits.dim() != 2:
        raise ValueError("logits must be a bf16, fp16 or fp32 CUDA tensor [rows, vocab]")
    n, vocab = logits.shape
    device, index = logits.device, logits.get_device()
    if vocab == 0 or (vocab > 1 and logits.stride(1) != 1) or (n > 1 and logits.stride(0) < vocab):
        raise ValueError("the logits of a row must be contiguous, at least one, and rows must not overlap")
    if not -2 ** 31 <= int(mask_id) < 2 ** 31:
        raise ValueError(f"mask_id must fit 32 bits, got {mask_id}")
    pu = _vector("u", u, torch.float32, n, index)
    t, t_all = _either("temperature", temperature, torch.float32, n, index)
    k, k_all = _either("top_k", top_k, torch.int32, n, index)
    p, p_all = _either("top_p", top_p, torch.float32, n, index)
    m, m_all = _either("min_p", min_p, torch.float32, n, index)
    now = None if tokens is None else _vector("tokens", tokens, torch.int32, n, index)
    if tokens is not None and (out is None or logprob is None):
        raise ValueError("with tokens, out and logprob hold what the other rows keep: pass them")
    how = _CSampling(t, k, p, m, t_all, k_all, p_all, m_all, 0 if draw_mask else SAMPLE_NO_MASK)
    handle, here = _on(device, stream)
    with here:
        if out is None:
            out = torch.empty(n, dtype=torch.int32, device=device)
        if logprob is None:
            logprob = torch.empty(n, dtype=torch.float32, device=device)
        po, pl = _vector("out", out, torch.int32, n, index), _vector("logprob", logprob, torch.float32, n, index)
        if n == 0:
            return out, logprob
        st = lib.bdlm_sample(logits.data_ptr(), _DTYPES[logits.dtype], n, vocab, max(logits.stride(0), vocab), pu,
                             ctypes.byref(how), now, int(mask_id), po, pl, handle)
        _check(st, "bdlm_sample")
    return out, logprob


def bdlm_unmask(tokens, sampled, logprob, cu_rows, mask_id: int, *, n_min=0, threshold=float("nan"), out=None, left=None,
                workspace=None, stream=None, check: bool = False):
    """Which masked rows (tokens[i] == mask_id) keep their drawn token: those
    whose logprob is at least `threshold` (NaN: none), and at least the n_min
    surest of every sequence; a drawn token below 0, or mask_id itself, is none.
    n_min (int32) and threshold (fp32) are numbers or tensors [n_seqs]. Returns (tokens int32 [T], left int32 [n_seqs]: rows
    still masked); `out` may be tokens itself. Rows behind cu_rows[-1] are left
    unwritten. check=True synchronises and raises on malformed offsets."""
    lib = load_library()
    if not isinstance(tokens, torch.Tensor) or not tokens.is_cuda:
        raise ValueError("tokens must be an int32 CUDA tensor")
    if not -2 ** 31 <= int(mask_id) < 2 ** 31:
        raise ValueError(f"mask_id must fit 32 bits, got {mask_id}")
    device, index, total = tokens.device, tokens.get_device(), tokens.numel()
    pt = _vector("tokens", tokens, torch.int32, None, index)
    ps = _vector("sampled", sampled, torch.int32, total, index)
    pl = _vector("logprob", logprob, torch.float32, total, index)
    pc = _vector("cu_rows", cu_rows, torch.int32, None, index)
    n = cu_rows.numel() - 1
    if n < 1:
        raise ValueError("cu_rows must have at least two entries")
    k, k_all = _either("n_min", n_min, torch.int32, n, index)
    x, x_all = _either("threshold", threshold, torch.float32, n, index)
    if workspace is not None:
        _vector("workspace", workspace, torch.uint8, None, index)
    handle, here = _on(device, stream)
    with here:
        if out is None:
            out = torch.empty_like(tokens)
        if left is None:
            left = torch.empty(n, dtype=torch.int32, device=device)
        po, pn = _vector("out", out, torch.int32, total, index), _vector("left", left, torch.int32, n, index)
        if total == 0:  # no rows: nothing is masked, and offsets that count any are malformed
            left.zero_()
            bad = (cu_rows != 0).any().int() * 6
            if workspace is not None:
                workspace[:256].zero_()[:4].copy_(bad.reshape(1).view(torch.uint8))
            if check:
                _check(int(bad), "bdlm_unmask (device)")
            return out, left
        if workspace is None and check:
            workspace = torch.empty(256, dtype=torch.uint8, device=device)
        ws, size = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
        st = lib.bdlm_unmask(pt, ps, pl, total, pc, n, int(mask_id), k, k_all, x, x_all, po, pn, ws, size, handle)
        _check(st, "bdlm_unmask")
        if check:
            _check(lib.bdlm_read_error(ws, handle), "bdlm_unmask (device)")
    return out, left
