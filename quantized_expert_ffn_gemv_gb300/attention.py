"""Per-head norm + rotation, the quantised paged cache and the attention over
it (include/moe_model.h).

Argument marshalling only.  Shapes, dtypes, strides and devices are checked
here, so a mismatched tensor is a ValueError and never an out-of-bounds device
access; the contents of the batch's index arrays are checked on the device
(``KvCache.check``).  Calls run on ``stream``, or on the current stream of the
tensors' device; tensors they return are allocated there.
"""
import contextlib
import ctypes as C

import numpy as np

from . import moe

BAD_PAGE, BAD_BATCH, TIMEOUT = 1, 2, 4


def _torch():
    import torch
    return torch


_HALF = {}  # torch.bfloat16 / torch.float16 -> the library's code (filled on first use: torch is imported lazily)


def _code(dtype, name):
    if not _HALF:
        torch = _torch()
        _HALF.update({torch.bfloat16: 0, torch.float16: 1})
    code = _HALF.get(dtype)
    if code is None:
        raise ValueError(f"{name}: expected torch.bfloat16 or torch.float16, got {dtype}")
    return code


def _scope(device, stream):
    """Raw stream to launch on, and a context in which `device` is current and allocations belong to the stream."""
    torch = _torch()
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream, torch.cuda.stream(stream)
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        return raw, contextlib.nullcontext()
    return raw, torch.cuda.device(device)


def _on_gpu(t, name, device=None):
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor{'' if device is None else f' on {device}'}, got {t.device}")
    return t.device


def _rows(t, name, shape, dtype, device, out=False):
    """The library's view of a [tokens, heads, D] tensor."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    ts, hs, es = t.stride()
    if es != 1 or (ts | hs) & 7 or t.data_ptr() & 15:
        raise ValueError(f"{name}: heads must be contiguous, strides multiples of 8 elements and data 16-byte aligned")
    if out and ((shape[0] > 1 and ts < shape[2]) or (shape[1] > 1 and hs < shape[2])):
        raise ValueError(f"{name}: rows of an output must not overlap")
    return moe.Heads(t.data_ptr(), ts, hs)


def _out(t, name, shape, dtype, device):
    """An output given by the caller, checked; or a new one."""
    if t is None:
        t = _torch().empty(shape, dtype=dtype, device=device)
    return t, _rows(t, name, shape, dtype, device, True)


def _vector(t, name, dtype, n, device):
    if t is None:
        return None
    if t.dtype != dtype or tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} ({n},), got {t.dtype} {tuple(t.shape)}")
    _on_gpu(t, name, device)
    return t.data_ptr()


def rope_table(n_positions, rot_dim, base, device="cuda"):
    """cos and sin of position * base^(-2 i / rot_dim), angles in 64 bits:
    float32 [n_positions, rot_dim / 2, 2] on `device`."""
    torch = _torch()
    if n_positions < 1 or rot_dim < 16 or rot_dim % 16:
        raise ValueError("n_positions must be positive and rot_dim a positive multiple of 16")
    t = np.empty((n_positions, rot_dim // 2, 2), np.float32)
    moe.check(moe.lib().moe_rope_table(n_positions, rot_dim, base, t.ctypes.data), "moe_rope_table")
    return torch.from_numpy(t).to(device)


def _norm_rope(dtype, dim, device, table, q_weight, k_weight, eps, interleaved, weight_offset):
    torch = _torch()
    n_positions = rot = ptr = 0
    if table is not None:
        if table.dtype != torch.float32 or table.dim() != 3 or table.shape[2] != 2 or not table.is_contiguous():
            raise ValueError("table: expected contiguous float32 [n_positions, rot_dim / 2, 2]")
        _on_gpu(table, "table", device)
        n_positions, rot, ptr = table.shape[0], 2 * table.shape[1], table.data_ptr()
    return moe.NormRope(_vector(q_weight, "q_weight", dtype, dim, device), _vector(k_weight, "k_weight", dtype, dim, device),
                        ptr, n_positions, rot, int(bool(interleaved)), eps, weight_offset)


def qk_norm_rope(q, k, positions, table, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, weight_offset=0.0,
                 q_out=None, k_out=None, stream=None):
    """Per-head RMSNorm and rotation of q [T, n_q, D] and k [T, n_kv, D]
    (bf16 or fp16; views with strides, such as slices of a packed projection,
    are taken as they are).  table: as rope_table gives it, or None for the
    norm alone; positions: int32 [T].  Returns (q_out, k_out); q_out may be q
    and k_out k.  See moe_qk_norm_rope."""
    torch = _torch()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, heads, D]")
    T, nq, dim = q.shape
    nk = k.shape[1]
    dev, dtype = _on_gpu(q, "q"), q.dtype
    code = _code(dtype, "q")
    if table is not None and positions is None:
        raise ValueError("a rotation needs positions")
    desc = _norm_rope(dtype, dim, dev, table, q_weight, k_weight, eps, interleaved, weight_offset)
    qh, kh = _rows(q, "q", (T, nq, dim), dtype, dev), _rows(k, "k", (T, nk, dim), dtype, dev)
    pos = _vector(positions, "positions", torch.int32, T, dev)
    raw, scope = _scope(dev, stream)
    with scope:
        q_out, qo = _out(q_out, "q_out", (T, nq, dim), dtype, dev)
        k_out, ko = _out(k_out, "k_out", (T, nk, dim), dtype, dev)
        moe.check(moe.lib().moe_qk_norm_rope(desc, code, T, dim, nq, qh, qo, nk, kh, ko, pos, raw), "moe_qk_norm_rope")
    return q_out, k_out


class KvBatch:
    """A ragged batch over a cache: block_table int32 [n_seqs, max_pages],
    seq_lens int32 [n_seqs] (positions that hold tokens, new ones included),
    cu_tokens int32 [n_seqs + 1] (rows of the new tokens, from 0), n_tokens
    rows in all (a padded batch may have more than cu_tokens[-1]), at most
    max_tokens of one sequence.  The arrays stay where they are and are read
    when a call runs."""

    def __init__(self, block_table, seq_lens, cu_tokens, n_tokens, max_tokens=None):
        torch = _torch()
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.stride(1) != 1:
            raise ValueError("block_table: expected int32 [n_seqs, max_pages] with contiguous rows")
        n_seqs, max_pages = block_table.shape
        self.device = _on_gpu(block_table, "block_table")
        stride = block_table.stride(0) if n_seqs > 1 else max(block_table.stride(0), max_pages)
        if n_seqs < 1 or max_pages < 1 or stride < max_pages:
            raise ValueError("block_table: rows must not overlap, and there must be a page and a sequence")
        n_tokens = int(n_tokens)
        max_tokens = n_tokens if max_tokens is None else int(max_tokens)
        if n_tokens < 0 or (n_tokens and not 1 <= max_tokens <= n_tokens):
            raise ValueError("max_tokens must lie in 1..n_tokens")
        self._tensors = (block_table, seq_lens, cu_tokens)
        self.n_seqs, self.n_tokens, self.max_tokens = n_seqs, n_tokens, max_tokens
        self.desc = moe.KvBatchDesc(block_table.data_ptr(), _vector(seq_lens, "seq_lens", torch.int32, n_seqs, self.device),
                                    _vector(cu_tokens, "cu_tokens", torch.int32, n_seqs + 1, self.device), n_seqs, stride,
                                    max_pages, n_tokens, max_tokens)


class KvCache:
    """A quantised paged key/value cache: n_pages pages of page_size tokens
    (a multiple of 32), n_kv_heads heads of head_dim (64, 128 or 256)
    elements, 8 or 4 bits with a scale a block of 32.  data: a uint8 CUDA
    tensor of n_pages * page bytes to use as the pool (its layout: moe_model.h),
    or None to allocate one."""

    def __init__(self, n_pages, page_size, n_kv_heads, head_dim, bits=8, device=0, data=None):
        torch = _torch()
        page = int(moe.lib().moe_kv_page_bytes(page_size, n_kv_heads, head_dim, bits))
        if not page or n_pages < 1:
            raise ValueError("page_size a multiple of 32 up to 4096, head_dim 64, 128 or 256, bits 8 or 4, n_pages >= 1")
        self.page_bytes, self.n_pages, self.page_size = page, n_pages, page_size
        self.n_kv_heads, self.head_dim, self.bits = n_kv_heads, head_dim, bits
        if data is None:
            data = torch.empty(n_pages * page, dtype=torch.uint8, device=torch.device("cuda", device))
        elif data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() != n_pages * page or data.data_ptr() & 15:
            raise ValueError(f"data: expected {n_pages * page} contiguous 16-byte aligned uint8")
        self.device = _on_gpu(data, "data")
        self.data = data
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.desc = moe.KvCacheDesc(data.data_ptr(), data.numel(), n_pages, page_size, n_kv_heads, head_dim, bits,
                                    self._status.data_ptr())

    def _io(self, batch, stream):
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        return _scope(self.device, stream)

    def append(self, k, v, batch, stream=None):
        """Quantise the batch's new k, v [n_tokens, n_kv_heads, head_dim] into their pages (moe_kv_append)."""
        shape, dtype = (batch.n_tokens, self.n_kv_heads, self.head_dim), k.dtype
        code = _code(dtype, "k")
        kh, vh = _rows(k, "k", shape, dtype, self.device), _rows(v, "v", shape, dtype, self.device)
        raw, scope = self._io(batch, stream)
        with scope:
            moe.check(moe.lib().moe_kv_append(self.desc, batch.desc, code, kh, vh, raw), "moe_kv_append")

    def append_norm_rope(self, q, k, v, batch, table, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                         weight_offset=0.0, positions=None, q_out=None, stream=None):
        """qk_norm_rope of q and k, and append of the result and v, in one
        pass; positions default to the tokens' places in their sequences.
        Returns q_out (may be q).  See moe_kv_append_norm_rope."""
        torch = _torch()
        dtype, T = q.dtype, batch.n_tokens
        if q.dim() != 3:
            raise ValueError("q must be [n_tokens, heads, head_dim]")
        nq, kv = q.shape[1], (T, self.n_kv_heads, self.head_dim)
        code = _code(dtype, "q")
        desc = _norm_rope(dtype, self.head_dim, self.device, table, q_weight, k_weight, eps, interleaved, weight_offset)
        qh = _rows(q, "q", (T, nq, self.head_dim), dtype, self.device)
        kh, vh = _rows(k, "k", kv, dtype, self.device), _rows(v, "v", kv, dtype, self.device)
        pos = _vector(positions, "positions", torch.int32, T, self.device)
        raw, scope = self._io(batch, stream)
        with scope:
            q_out, qo = _out(q_out, "q_out", (T, nq, self.head_dim), dtype, self.device)
            moe.check(moe.lib().moe_kv_append_norm_rope(self.desc, batch.desc, desc, code, nq, qh, qo, kh, vh, pos, raw),
                      "moe_kv_append_norm_rope")
        return q_out

    def read(self, batch, k_out=None, v_out=None, dtype=None, stream=None):
        """The batch's tokens back from the cache, (k, v) [n_tokens,
        n_kv_heads, head_dim] in dtype (default bf16, or k_out's).  See moe_kv_read."""
        torch = _torch()
        if dtype is None:
            dtype = torch.bfloat16 if k_out is None else k_out.dtype
        shape = (batch.n_tokens, self.n_kv_heads, self.head_dim)
        code = _code(dtype, "dtype")
        raw, scope = self._io(batch, stream)
        with scope:
            k_out, ko = _out(k_out, "k_out", shape, dtype, self.device)
            v_out, vo = _out(v_out, "v_out", shape, dtype, self.device)
            moe.check(moe.lib().moe_kv_read(self.desc, batch.desc, code, ko, vo, raw), "moe_kv_read")
        return k_out, v_out

    def attend(self, q, batch, scale=None, out=None, lse=None, shared_tokens=0, stream=None):
        """Causal attention of the batch's new tokens q [n_tokens, n_q,
        head_dim] over their sequences, the new tokens (append them first)
        included; scale defaults to head_dim ** -0.5.  lse: float32 [n_tokens,
        n_q] to receive the log-sum-exp, or None.  shared_tokens: leading
        positions (a multiple of page_size) whose pages are the same in every
        row of the block table; they are then read once for the whole batch.
        Returns out.  See moe_kv_attend."""
        torch = _torch()
        if q.dim() != 3:
            raise ValueError("q must be [n_tokens, heads, head_dim]")
        dtype, T, nq = q.dtype, batch.n_tokens, q.shape[1]
        shape = (T, nq, self.head_dim)
        code = _code(dtype, "q")
        qh = _rows(q, "q", shape, dtype, self.device)
        lse_ptr = None
        if lse is not None:
            if lse.dtype != torch.float32 or tuple(lse.shape) != (T, nq) or not lse.is_contiguous():
                raise ValueError(f"lse: expected contiguous float32 {(T, nq)}")
            _on_gpu(lse, "lse", self.device)
            lse_ptr = lse.data_ptr()
        raw, scope = self._io(batch, stream)
        with scope:
            out, oh = _out(out, "out", shape, dtype, self.device)
            n = C.c_size_t()
            L = moe.lib()
            moe.check(L.moe_kv_attend_workspace(self.desc, batch.desc, nq, shared_tokens, n), "moe_kv_attend_workspace")
            work = torch.empty(n.value, dtype=torch.uint8, device=self.device)
            moe.check(L.moe_kv_attend(self.desc, batch.desc, code, nq, qh, oh, lse_ptr,
                                      self.head_dim ** -0.5 if scale is None else scale, shared_tokens, work.data_ptr(),
                                      n.value, raw), "moe_kv_attend")
        return out

    def check(self):
        """Synchronise, and raise MoeError if a call found a bad page, a bad
        batch or ran out of a wait since the last check (which clears it)."""
        bits = int(self._status.item())
        if bits:
            self._status.zero_()
            what = [n for b, n in ((BAD_PAGE, "bad page"), (BAD_BATCH, "bad batch"), (TIMEOUT, "timeout")) if bits & b]
            raise moe.MoeError(6 if bits & TIMEOUT else 8, "cache: " + ", ".join(what))
