"""The BF16-only paged cache's chunk attention and page copies (oscar_bf16_chunk, oscar_bf16_copy_pages), with
PyTorch tensors."""
from __future__ import annotations

import torch

from . import binding as B
from .pool import HEAD_DIM, _need, _on_current_device, _raw_stream
from .rope import _rows

PAGE = 64


def bf16_chunk_attend(q, k_pages, v_pages, page_table, lengths, cu_tokens, err, workspace=None, out=None):
    """Attention of the last cu_tokens[i+1] - cu_tokens[i] tokens of every sequence over its BF16 pages (their own
    rows among them), causal. q: bf16 [n_tokens, Hq, 128] (tokens may be strided); k_pages, v_pages: bf16
    [n_pages, Hkv, 64, 128]; page_table: int32 [n_seqs, max_pages]; lengths: int32 [n_seqs]; cu_tokens: int32
    [n_seqs + 1]; err: int32 [1], receives DEVERR_* bits. Returns bf16 [n_tokens, Hq, 128]; rows outside every
    sequence are left as they were in `out`."""
    n = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
    stride = _rows(q, n, "q")
    hq, hkv = q.shape[1], k_pages.shape[1] if isinstance(k_pages, torch.Tensor) and k_pages.dim() == 4 else -1
    pages = k_pages.shape[0] if hkv > 0 else -1
    _need(k_pages, torch.bfloat16, (pages, hkv, PAGE, HEAD_DIM), "k_pages")
    _need(v_pages, torch.bfloat16, (pages, hkv, PAGE, HEAD_DIM), "v_pages")
    seqs, width = page_table.shape if isinstance(page_table, torch.Tensor) and page_table.dim() == 2 else (-1, -1)
    _need(page_table, torch.int32, (seqs, width), "page_table")
    _need(lengths, torch.int32, (seqs,), "lengths")
    _need(cu_tokens, torch.int32, (seqs + 1,), "cu_tokens")
    _need(err, torch.int32, (1,), "err")
    lib = B.lib()
    if workspace is None:
        workspace = torch.empty(max(lib.oscar_bf16_chunk_workspace_bytes(hq, hkv, seqs, n), 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((n, hq, HEAD_DIM), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, torch.bfloat16, (n, hq, HEAD_DIM), "out")
    device = q.get_device()
    for t in (k_pages, v_pages, page_table, lengths, cu_tokens, err, workspace, out):
        if t.get_device() != device:
            raise ValueError("pages, tables, workspace and out must be on the device of q")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    B._check("oscar_bf16_chunk", lib.oscar_bf16_chunk(
        hq, hkv, seqs, n, k_pages.data_ptr(), v_pages.data_ptr(), pages, page_table.data_ptr(), width, lengths.data_ptr(),
        cu_tokens.data_ptr(), q.data_ptr(), stride, workspace.data_ptr(), workspace.nbytes, out.data_ptr(), err.data_ptr(),
        _raw_stream()))
    return out


def bf16_copy_pages(k_pages, v_pages, src, dst):
    """Copy pages src[m] of K and V to pages dst[m] (host sequences of ids; no page written twice, nor both read
    and written). k_pages, v_pages: bf16 [n_pages, Hkv, 64, 128], or [layers, n_pages, Hkv, 64, 128] for the same
    copies in every layer."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() not in (4, 5):
        raise ValueError("k_pages must be [n_pages, Hkv, 64, 128] or [layers, n_pages, Hkv, 64, 128]")
    shape = k_pages.shape
    layers = shape[0] if k_pages.dim() == 5 else 1
    pages, hkv = shape[-4], shape[-3]
    _need(k_pages, torch.bfloat16, tuple(shape[:-2]) + (PAGE, HEAD_DIM), "k_pages")
    _need(v_pages, torch.bfloat16, tuple(shape), "v_pages")
    if not _on_current_device(k_pages) or not _on_current_device(v_pages):
        raise ValueError("k_pages and v_pages must be on the current CUDA device")
    B.oscar_bf16_copy_pages(hkv, layers, pages * hkv * PAGE * HEAD_DIM * 2, k_pages, v_pages, pages, src, dst, _raw_stream())
