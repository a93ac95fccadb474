"""The paged key/value cache and the attention of drafted tokens over it.

A decoder keeps the keys and values of its sequences in a pool of pages, appends the next
tokens' and attends with one token, or with a tree of drafted ones, to all of them:

    pool = cache.PagedCache.empty(n_pages, Hkv, 64, torch.float8_e4m3fn, "cuda")
    cache.write(pool, k, v, page_table, start, rope=table)       # rotate, quantise, append
    out, lse = cache.attend(q, pool, page_table, context_lens)   # one token, or a chain of T
    out, lse = cache.attend(q, pool, page_table, context_lens, tree_mask=mask)
    k, v = cache.read(pool, page_table, lens, max_len)           # dense again

Token j of sequence b is slot j % page_size of page ``page_table[b, j // page_size]``.
Pages hold fp32, bf16 or float8 e4m3 with one power-of-two scale per row.  Lengths, page
tables and masks are device tensors and no call reads them on the host, so steps can be
captured in a CUDA graph and replayed while they change.  A page index or a length out of
range is skipped on the device and recorded in the pool's status word (``status``).
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _device, _lib
from . import status as _status_of
from ._views import check_ints, check_positions, float_code, launch, new_like, on_stream, rows

_CODES = {torch.float32: _lib.GQA_F32, torch.bfloat16: _lib.GQA_BF16, torch.float8_e4m3fn: _lib.GQA_E4M3}


class PagedCache:
    """A pool of pages: ``k`` and ``v`` [n_pages, Hkv, page_size, 256] (fp32, bf16 or
    float8_e4m3fn; page_size a power of two in 8 .. 1024; views of other orders of the
    first three dimensions are fine), for e4m3 with ``k_scale`` and ``v_scale``
    [n_pages, Hkv, page_size] fp32.  ``status_word`` (int32 [1], zero at first) receives
    the first device-side error; without one, errors are skipped over unrecorded."""

    def __init__(self, k, v, k_scale=None, v_scale=None, status_word=None):
        code = _CODES.get(k.dtype)
        if code is None or v.dtype != k.dtype:
            raise ValueError("pages must be float32, bfloat16 or float8_e4m3fn, k and v alike")
        if not k.is_cuda or v.device != k.device or k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("k and v must be CUDA tensors [n_pages, Hkv, page_size, 256] of the same strides")
        n, Hkv, page, d = k.shape
        sp, sh, st, sd = k.stride()
        if d != 256 or sd != 1 or n < 1 or Hkv < 1:
            raise ValueError("pages must have contiguous rows of 256 columns")
        if page < 8 or page > 1024 or page & (page - 1):
            raise ValueError("page_size must be a power of two in 8 .. 1024")
        if (sp == 0 and n > 1) or (sh == 0 and Hkv > 1) or st == 0:
            raise ValueError("pages must not overlap")
        if code == _lib.GQA_E4M3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if (t is None or t.dtype != torch.float32 or t.device != k.device or t.shape != (n, Hkv, page)
                        or not t.is_contiguous()):
                    raise ValueError(f"{name} must be a contiguous fp32 tensor [n_pages, Hkv, page_size]")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only float8_e4m3fn pages have scales")
        if status_word is not None:
            check_ints(status_word, (1,), k.device, "status_word")
        self.k, self.v, self.k_scale, self.v_scale, self.status_word = k, v, k_scale, v_scale, status_word
        self.device, self.dtype, self.code, self.Hkv, self.page_size = k.device, k.dtype, code, Hkv, page
        self._struct = _lib.Cache(k.data_ptr(), v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
                                  None if v_scale is None else v_scale.data_ptr(),
                                  None if status_word is None else status_word.data_ptr(), sp, sh, st, n, Hkv, page,
                                  code)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, n_pages, Hkv, page_size, dtype=torch.bfloat16, device="cuda"):
        """A new pool with its scales and its status word."""
        dev = _device(device)
        k, v = (torch.empty((n_pages, Hkv, page_size, 256), dtype=dtype, device=dev) for _ in range(2))
        ks = vs = None
        if dtype == torch.float8_e4m3fn:
            ks, vs = (torch.ones((n_pages, Hkv, page_size), dtype=torch.float32, device=dev) for _ in range(2))
        return cls(k, v, ks, vs, torch.zeros(1, dtype=torch.int32, device=dev))


def status(pool, stream=None) -> int:
    """The pool's first device-side error, or 0 (synchronises ``stream``)."""
    if pool.status_word is None:
        raise ValueError("the pool was made without a status_word")
    return _status_of(pool.status_word, stream)


def _tables(pool, page_table, B):
    if (not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] != B
            or page_table.dtype != torch.int32 or page_table.device != pool.device or not page_table.is_contiguous()):
        raise ValueError(f"page_table must be a contiguous int32 tensor [{B}, max_pages] on {pool.device}")
    return page_table.data_ptr(), page_table.shape[1]


def write(pool, k, v, page_table, start, *, lens=None, rope=None, positions=None, pos_offset=0, stream=None):
    """Appends ``k`` and ``v`` [B, Hkv, L, 256] (fp32 or bf16): token i of sequence b goes to
    place ``start[b] + i``, for i < ``lens[b]`` (default L).  With ``rope`` (a
    ``rotary.Table``) the keys are rotated on the way, at that place plus ``pos_offset``, or
    at ``positions`` (int32, [L] or [B, L]).  e4m3 pages get the row's power-of-two scale
    and its codes.  No two tokens may go to one slot.  Asynchronous on ``stream``."""
    dev = pool.device
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or not isinstance(v, torch.Tensor) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, L, 256]")
    B, Hkv, L, d = k.shape
    code = float_code(k.dtype)
    rk, rv = rows(k, "k", dev, k.dtype), rows(v, "v", dev, k.dtype)
    if Hkv != pool.Hkv:
        raise ValueError(f"k and v have {Hkv} heads, the pool has {pool.Hkv}")
    table, max_pages = _tables(pool, page_table, B)
    check_ints(start, (B,), dev, "start")
    if lens is not None:
        check_ints(lens, (B,), dev, "lens")
    r = None
    if rope is not None:
        positions = check_positions(positions, B, L, dev)
        if positions is not None and pos_offset:
            raise ValueError("pos_offset goes with the tokens' places, not with positions given")
        r = ctypes.byref(rope.struct(dev, positions, int(pos_offset)))
    elif positions is not None or pos_offset:
        raise ValueError("positions and pos_offset need rope")
    launch("gqa_attn_cache_write", dev, stream, pool._ref, ctypes.byref(rk), ctypes.byref(rv), table, max_pages,
           start.data_ptr(), None if lens is None else lens.data_ptr(), B, L, d, code, r)


def read(pool, page_table, lens, max_len, *, dtype=torch.bfloat16, out=None, stream=None):
    """The first ``lens[b]`` tokens of each sequence as dense ``(k, v)`` [B, Hkv, max_len,
    256] of ``dtype``, zeros behind them.  ``out``: a pair of tensors to write.
    Asynchronous on ``stream``."""
    dev = pool.device
    B = page_table.shape[0] if isinstance(page_table, torch.Tensor) and page_table.dim() == 2 else -1
    table, max_pages = _tables(pool, page_table, B)
    check_ints(lens, (B,), dev, "lens")
    max_len = int(max_len)
    if max_len < 0:
        raise ValueError("max_len must not be negative")
    code = float_code(dtype)
    shape = (B, pool.Hkv, max_len, 256)
    if out is None:
        with on_stream(stream):
            out = tuple(torch.empty(shape, dtype=dtype, device=dev) for _ in range(2))
    k, v = out
    for t in (k, v):
        if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"out must be two contiguous {dtype} tensors of shape {shape} on {dev}")
    launch("gqa_attn_cache_read", dev, stream, pool._ref, table, max_pages, lens.data_ptr(), k.data_ptr(), v.data_ptr(),
           B, max_len, 256, code)
    return k, v


@functools.lru_cache(maxsize=1024)
def _tree_bytes(B, Hq, Hkv, T, max_pages, page_size, code, cache_code) -> int:
    return int(_lib.load().gqa_attn_tree_workspace_bytes(B, Hq, Hkv, T, max_pages, page_size, 256, code, cache_code))


def workspace_bytes(B, Hq, T, pool, max_pages, dtype=torch.bfloat16) -> int:
    """Device workspace bytes of one ``attend`` call (0 if the shape is rejected)."""
    return _tree_bytes(B, Hq, pool.Hkv, T, max_pages, pool.page_size, float_code(dtype), pool.code)


def attend(q, pool, page_table, context_lens, *, tree_mask=None, tree_lens=None, out=None, lse=None, workspace=None,
           stream=None):
    """Attention of T drafted tokens ``q`` [B, Hq, T, 256] (fp32 or bf16) per sequence over
    its context of ``context_lens[b]`` tokens and the drafted tokens behind it, all in the
    pool already; ``(out, lse)`` as ``fwd``.  ``tree_mask`` (bool or uint8, [T, T] or [B, T,
    T]): row t sees drafted token u where it is set (its own too has to be); default: a
    chain, u <= t.  ``tree_lens[b]`` < T marks the rows behind it as padding.  A row with no
    visible key gets 0 and -inf.  B and T are at least 1, as in ``fwd``: an empty step is an error
    here, while ``write``, ``read`` and ``rotary.rotate`` do nothing.  Asynchronous on ``stream``."""
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 4):
        raise ValueError("attend takes a 4-d CUDA tensor q")
    dev = pool.device
    B, Hq, T, d = q.shape
    code = float_code(q.dtype)
    rq = rows(q, "q", dev, q.dtype)
    table, max_pages = _tables(pool, page_table, B)
    check_ints(context_lens, (B,), dev, "context_lens")
    if tree_lens is not None:
        check_ints(tree_lens, (B,), dev, "tree_lens")
    mask, mask_sb = None, 0
    if tree_mask is not None:
        if (not isinstance(tree_mask, torch.Tensor) or tree_mask.dtype not in (torch.bool, torch.uint8)
                or tree_mask.device != dev or tree_mask.shape not in ((T, T), (B, T, T))
                or not tree_mask.is_contiguous()):
            raise ValueError(f"tree_mask must be a contiguous bool or uint8 tensor [{T}, {T}] or [{B}, {T}, {T}]")
        mask, mask_sb = tree_mask.data_ptr(), T * T if tree_mask.dim() == 3 else 0
    with on_stream(stream):
        if out is None:
            out = new_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(max(_tree_bytes(B, Hq, pool.Hkv, T, max_pages, pool.page_size, code, pool.code), 256),
                                    dtype=torch.uint8, device=dev)
    if out.shape != q.shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    if lse.shape != (B, Hq, T) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, Hq, T] tensor on q's device")
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    launch("gqa_attn_fwd_tree", dev, stream, ctypes.byref(rq), pool._ref, table, max_pages, context_lens.data_ptr(),
           None if tree_lens is None else tree_lens.data_ptr(), mask, mask_sb, out.data_ptr(), lse.data_ptr(), B, T, d,
           code, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse
