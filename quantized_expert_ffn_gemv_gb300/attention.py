"""Per-head norm + rotation, the quantised paged cache and the attention over
it (include/moe_model.h).

Argument marshalling only.  Shapes, dtypes, strides and devices are checked
here, so a mismatched tensor is a ValueError and never an out-of-bounds device
access; the contents of the batch's index arrays are checked on the device
(``KvCache.check``).  Calls run on ``stream``, or on the current stream of the
tensors' device; tensors they return are allocated there.  The operators are
forward ones: what they return carries no gradient.

A decode step makes several of these calls a layer, so each function first
offers its arguments to the extension module (csrc/binding.c), which makes
the same checks natively and declines (None) whatever is not the plain case; what
follows it here takes the rest and names what is wrong.
"""
import ctypes as C
import importlib.util
import os

import numpy as np
import torch

from . import build as _build
from . import moe

BAD_PAGE, BAD_BATCH, TIMEOUT = 1, 2, 4

_HALF = {torch.bfloat16: 0, torch.float16: 1}
_i32, _f32 = torch.int32, torch.float32
_heads2, _heads4 = C.c_int64 * 6, C.c_int64 * 12  # two and four moe_heads_t side by side, 24 bytes each
_current_device, _raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


def _load_native():
    """The extension module, bound to the library's functions."""
    if not os.path.exists(_build.BINDING):
        raise RuntimeError(f"extension module not built ({_build.BINDING}); run __graft_entry__.build()")
    spec = importlib.util.spec_from_file_location("moe_binding", _build.BINDING)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    L = moe.lib()
    names = ("moe_qk_norm_rope", "moe_kv_append", "moe_kv_append_norm_rope", "moe_kv_read", "moe_kv_attend_workspace",
             "moe_kv_attend", "moe_sample")
    m.setup(tuple(C.cast(getattr(L, n), C.c_void_p).value for n in names),
            (torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8), torch._C._cuda_getDevice,
            _raw_stream, torch.empty)
    return m


_native_module = None


def _native():
    global _native_module
    if _native_module is None:
        _native_module = _load_native()
    return _native_module


def _code(dtype, name):
    code = _HALF.get(dtype)
    if code is None:
        raise ValueError(f"{name}: expected torch.bfloat16 or torch.float16, got {dtype}")
    return code


def _scope(dev, stream):
    """A context in which device number dev and, when given, the stream are
    current; None when they are already."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        return torch.cuda.stream(stream)
    return None if _current_device() == dev else torch.cuda.device(dev)


def _on_gpu(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    return dev


def _int32(**sizes):
    """The library's sizes are 32-bit, and ctypes would pass on the low bits of a larger one."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name}: {v} is beyond 32 bits")


def _apart(n_tokens, n_heads, dim, ts, hs):
    """No two of the rows share an element (as the library checks it)."""
    if n_tokens < 2 or n_heads < 2:
        return (n_tokens < 2 or ts >= dim) and (n_heads < 2 or hs >= dim)
    (far, n_far), (near, n_near) = sorted(((ts, n_tokens), (hs, n_heads)), reverse=True)
    if near < dim or (n_near - 1) * near + dim <= far:
        return near >= dim
    return all(abs(j * near - i * far) >= dim for j in range(1, n_near) for i in (j * near // far, j * near // far + 1) if 0 < i < n_far)


def _rows(t, name, shape, dtype, dev, out=False):
    """Address and strides of a [tokens, heads, D] tensor, checked."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
        ts, hs, es = t.stride()
        at = t.data_ptr()
        if es != 1 or (ts | hs) & 7 or at & 15:
            raise ValueError(f"{name}: heads must be contiguous, strides multiples of 8 elements and data 16-byte aligned")
        if out and not _apart(*shape, ts, hs):
            raise ValueError(f"{name}: rows of an output must not overlap")
        return at, ts, hs
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{name} must be a CUDA tensor on cuda:{dev}, got {t.device}")


def _vector(t, name, dtype, n, dev):
    """Address of a contiguous [n] tensor, checked; None stays None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == (n,) and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected contiguous {dtype} ({n},) on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def rope_table(n_positions, rot_dim, base, device="cuda"):
    """cos and sin of position * base^(-2 i / rot_dim), angles in 64 bits:
    float32 [n_positions, rot_dim / 2, 2] on `device`."""
    if n_positions < 1 or rot_dim < 16 or rot_dim % 16:
        raise ValueError("n_positions must be positive and rot_dim a positive multiple of 16")
    _int32(n_positions=n_positions, rot_dim=rot_dim)
    t = np.empty((n_positions, rot_dim // 2, 2), np.float32)
    moe.check(moe.lib().moe_rope_table(n_positions, rot_dim, base, t.ctypes.data), "moe_rope_table")
    return torch.from_numpy(t).to(device)


def _norm_rope(dtype, dim, dev, table, q_weight, k_weight, eps, interleaved, weight_offset):
    n_positions = rot = 0
    at = None
    if table is not None:
        shape = table.shape
        if table.dtype is not _f32 or len(shape) != 3 or shape[2] != 2 or not table.is_contiguous():
            raise ValueError("table: expected contiguous float32 [n_positions, rot_dim / 2, 2]")
        if table.get_device() != dev:
            raise ValueError(f"table must be a CUDA tensor on cuda:{dev}, got {table.device}")
        n_positions, rot, at = shape[0], 2 * shape[1], table.data_ptr()
        _int32(n_positions=n_positions, rot_dim=rot)
    return moe.NormRope(_vector(q_weight, "q_weight", dtype, dim, dev), _vector(k_weight, "k_weight", dtype, dim, dev), at,
                        n_positions, rot, 1 if interleaved else 0, eps, weight_offset)


def qk_norm_rope(q, k, positions, table, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, weight_offset=0.0,
                 q_out=None, k_out=None, stream=None):
    """Per-head RMSNorm and rotation of q [T, n_q, D] and k [T, n_kv, D]
    (bf16 or fp16; views with strides, such as slices of a packed projection,
    are taken as they are).  table: as rope_table gives it, or None for the
    norm alone; positions: int32 [T].  Returns (q_out, k_out); q_out may be q
    and k_out k.  See moe_qk_norm_rope."""
    if stream is None:
        r = (_native_module or _native()).qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps, interleaved, weight_offset,
                                                       q_out, k_out)
        if r is not None:
            return r if type(r) is tuple else moe.check(r, "moe_qk_norm_rope")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, heads, D]")
    T, nq, dim = q_shape = q.shape
    nk = k.shape[1]
    _int32(tokens=T, q_heads=nq, k_heads=nk, head_dim=dim)
    k_shape = (T, nk, dim)
    dtype = q.dtype
    code = _code(dtype, "q")
    if table is not None and positions is None:
        raise ValueError("a rotation needs positions")
    dev = _on_gpu(q, "q")
    scope = _scope(dev, stream)
    if scope is not None:
        with scope:
            return qk_norm_rope(q, k, positions, table, q_weight, k_weight, eps, interleaved, weight_offset, q_out, k_out)
    desc = _norm_rope(dtype, dim, dev, table, q_weight, k_weight, eps, interleaved, weight_offset)
    qr, kr = _rows(q, "q", q_shape, dtype, dev), _rows(k, "k", k_shape, dtype, dev)
    pos = _vector(positions, "positions", _i32, T, dev)
    if q_out is None:
        q_out = q.new_empty(q_shape)
    if k_out is None:
        k_out = k.new_empty(k_shape)
    h = _heads4(*qr, *kr, *_rows(q_out, "q_out", q_shape, dtype, dev, True), *_rows(k_out, "k_out", k_shape, dtype, dev, True))
    at = C.addressof(h)
    code = moe.lib().moe_qk_norm_rope(C.addressof(desc), code, T, dim, nq, at, at + 48, nk, at + 24, at + 72, pos, _raw_stream(dev))
    if code:
        moe.check(code, "moe_qk_norm_rope")
    return q_out, k_out


class KvBatch:
    """A ragged batch over a cache: block_table int32 [n_seqs, max_pages],
    seq_lens int32 [n_seqs] (positions that hold tokens, new ones included),
    cu_tokens int32 [n_seqs + 1] (rows of the new tokens, from 0), n_tokens
    rows in all (a padded batch may have more than cu_tokens[-1]), at most
    max_tokens of one sequence (None: n_tokens, which is right for any batch,
    but plans the attention for one long prompt: pass 1 for decode).  The
    arrays stay where they are and are read when a call runs."""

    def __init__(self, block_table, seq_lens, cu_tokens, n_tokens, max_tokens=None):
        if block_table.dim() != 2 or block_table.dtype is not _i32 or block_table.stride(1) != 1:
            raise ValueError("block_table: expected int32 [n_seqs, max_pages] with contiguous rows")
        n_seqs, max_pages = block_table.shape
        dev = _on_gpu(block_table, "block_table")
        stride = block_table.stride(0) if n_seqs > 1 else max(block_table.stride(0), max_pages)
        if n_seqs < 1 or max_pages < 1 or stride < max_pages:
            raise ValueError("block_table: rows must not overlap, and there must be a page and a sequence")
        n_tokens = int(n_tokens)
        max_tokens = n_tokens if max_tokens is None else int(max_tokens)
        if n_tokens < 0 or (n_tokens and not 1 <= max_tokens <= n_tokens):
            raise ValueError("max_tokens must lie in 1..n_tokens")
        _int32(n_tokens=n_tokens, n_seqs=n_seqs, max_pages=max_pages, table_stride=stride)
        self._tensors = (block_table, seq_lens, cu_tokens)
        self.dev, self.n_seqs, self.n_tokens, self.max_tokens = dev, n_seqs, n_tokens, max_tokens
        self.desc = moe.KvBatchDesc(block_table.data_ptr(), _vector(seq_lens, "seq_lens", _i32, n_seqs, dev),
                                    _vector(cu_tokens, "cu_tokens", _i32, n_seqs + 1, dev), n_seqs, stride, max_pages, n_tokens,
                                    max_tokens)
        self._at = C.addressof(self.desc)


class KvCache:
    """A quantised paged key/value cache: n_pages pages of page_size tokens
    (a multiple of 32), n_kv_heads heads of head_dim (64, 128 or 256)
    elements, 8 or 4 bits with a scale a block of 32.  data: a uint8 CUDA
    tensor of n_pages * page bytes to use as the pool (its layout: moe_model.h),
    or None to allocate one."""

    def __init__(self, n_pages, page_size, n_kv_heads, head_dim, bits=8, device=0, data=None):
        _int32(n_pages=n_pages, page_size=page_size, n_kv_heads=n_kv_heads, head_dim=head_dim, bits=bits)
        page = int(moe.lib().moe_kv_page_bytes(page_size, n_kv_heads, head_dim, bits))
        if not page or n_pages < 1:
            raise ValueError("page_size a multiple of 32 up to 4096, head_dim 64, 128 or 256, bits 8 or 4, n_pages >= 1")
        self.page_bytes, self.n_pages, self.page_size = page, n_pages, page_size
        self.n_kv_heads, self.head_dim, self.bits = n_kv_heads, head_dim, bits
        if data is None:
            data = torch.empty(n_pages * page, dtype=torch.uint8, device=torch.device("cuda", device))
        elif data.dtype is not torch.uint8 or not data.is_contiguous() or data.numel() != n_pages * page or data.data_ptr() & 15:
            raise ValueError(f"data: expected {n_pages * page} contiguous 16-byte aligned uint8")
        self.dev = _on_gpu(data, "data")
        self.data = data
        self._status = torch.zeros(1, dtype=_i32, device=data.device)
        self._settle()  # calls on any stream come behind the zeros
        self.desc = moe.KvCacheDesc(data.data_ptr(), data.numel(), n_pages, page_size, n_kv_heads, head_dim, bits,
                                    self._status.data_ptr())
        self._at = C.addressof(self.desc)

    def _enter(self, batch, stream):
        if batch.dev != self.dev:
            raise ValueError(f"the batch is on cuda:{batch.dev}, the cache on cuda:{self.dev}")
        return _scope(self.dev, stream)

    def append(self, k, v, batch, stream=None):
        """Quantise the batch's new k, v [n_tokens, n_kv_heads, head_dim] into their pages (moe_kv_append)."""
        if stream is None and batch.dev == self.dev:
            r = (_native_module or _native()).append(self._at, batch._at, self.dev, k, v)
            if r is not None:
                return moe.check(r, "moe_kv_append") if r else None
        shape, dtype, dev = (batch.n_tokens, self.n_kv_heads, self.head_dim), k.dtype, self.dev
        code = _code(dtype, "k")
        h = _heads2(*_rows(k, "k", shape, dtype, dev), *_rows(v, "v", shape, dtype, dev))
        scope = self._enter(batch, stream)
        if scope is not None:
            with scope:
                return self.append(k, v, batch)
        at = C.addressof(h)
        code = moe.lib().moe_kv_append(self._at, batch._at, code, at, at + 24, _raw_stream(dev))
        if code:
            moe.check(code, "moe_kv_append")

    def append_norm_rope(self, q, k, v, batch, table, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                         weight_offset=0.0, positions=None, q_out=None, stream=None):
        """qk_norm_rope of q and k, and append of the result and v, in one
        pass; positions default to the tokens' places in their sequences.
        Returns q_out (may be q).  See moe_kv_append_norm_rope."""
        if stream is None and batch.dev == self.dev:
            r = (_native_module or _native()).append_norm_rope(self._at, batch._at, self.dev, q, k, v, table, q_weight, k_weight,
                                                               eps, interleaved, weight_offset, positions, q_out)
            if r is not None:
                return moe.check(r, "moe_kv_append_norm_rope") if type(r) is int else r
        if q.dim() != 3:
            raise ValueError("q must be [n_tokens, heads, head_dim]")
        dtype, T, dim, dev = q.dtype, batch.n_tokens, self.head_dim, self.dev
        code = _code(dtype, "q")
        nq = q.shape[1]
        _int32(q_heads=nq)
        q_shape, kv = (T, nq, dim), (T, self.n_kv_heads, dim)
        qr, kr, vr = _rows(q, "q", q_shape, dtype, dev), _rows(k, "k", kv, dtype, dev), _rows(v, "v", kv, dtype, dev)
        scope = self._enter(batch, stream)
        if scope is not None:
            with scope:
                return self.append_norm_rope(q, k, v, batch, table, q_weight, k_weight, eps, interleaved, weight_offset,
                                             positions, q_out)
        desc = _norm_rope(dtype, dim, dev, table, q_weight, k_weight, eps, interleaved, weight_offset)
        pos = _vector(positions, "positions", _i32, T, dev)
        if q_out is None:
            q_out = q.new_empty(q_shape)
        h = _heads4(*qr, *_rows(q_out, "q_out", q_shape, dtype, dev, True), *kr, *vr)
        at = C.addressof(h)
        code = moe.lib().moe_kv_append_norm_rope(self._at, batch._at, C.addressof(desc), code, nq, at, at + 24, at + 48, at + 72,
                                                 pos, _raw_stream(dev))
        if code:
            moe.check(code, "moe_kv_append_norm_rope")
        return q_out

    def read(self, batch, k_out=None, v_out=None, dtype=None, stream=None):
        """The batch's tokens back from the cache, (k, v) [n_tokens,
        n_kv_heads, head_dim] in dtype (default bf16, or k_out's).  See moe_kv_read."""
        if dtype is None:
            dtype = torch.bfloat16 if k_out is None else k_out.dtype
        if stream is None and batch.dev == self.dev:
            r = (_native_module or _native()).read(self._at, batch._at, self.dev, self.data, dtype, k_out, v_out)
            if r is not None:
                return r if type(r) is tuple else moe.check(r, "moe_kv_read")
        code = _code(dtype, "dtype")
        dev, shape = self.dev, (batch.n_tokens, self.n_kv_heads, self.head_dim)
        scope = self._enter(batch, stream)
        if scope is not None:
            with scope:
                return self.read(batch, k_out, v_out, dtype)
        if k_out is None:
            k_out = self.data.new_empty(shape, dtype=dtype)
        if v_out is None:
            v_out = self.data.new_empty(shape, dtype=dtype)
        h = _heads2(*_rows(k_out, "k_out", shape, dtype, dev, True), *_rows(v_out, "v_out", shape, dtype, dev, True))
        at = C.addressof(h)
        code = moe.lib().moe_kv_read(self._at, batch._at, code, at, at + 24, _raw_stream(dev))
        if code:
            moe.check(code, "moe_kv_read")
        return k_out, v_out

    def attend(self, q, batch, scale=None, out=None, lse=None, shared_tokens=0, stream=None):
        """Causal attention of the batch's new tokens q [n_tokens, n_q,
        head_dim] over their sequences, the new tokens (append them first)
        included; scale defaults to head_dim ** -0.5.  lse: float32 [n_tokens,
        n_q] to receive the log-sum-exp, or None.  shared_tokens: leading
        positions (a multiple of page_size) whose pages are the same in every
        row of the block table; they are then read once for the whole batch.
        out may be q.  Returns out.  See moe_kv_attend."""
        if stream is None and batch.dev == self.dev:
            r = (_native_module or _native()).attend(self._at, batch._at, self.dev, self.data, q, scale, out, lse, shared_tokens)
            if r is not None:
                return moe.check(r, "moe_kv_attend") if type(r) is int else r
        if q.dim() != 3:
            raise ValueError("q must be [n_tokens, heads, head_dim]")
        dtype, T, nq, dim, dev = q.dtype, batch.n_tokens, q.shape[1], self.head_dim, self.dev
        shape = (T, nq, dim)
        _int32(q_heads=nq, shared_tokens=shared_tokens)
        code = _code(dtype, "q")
        qr = _rows(q, "q", shape, dtype, dev)
        lse_at = None
        if lse is not None:
            if lse.dtype is not _f32 or lse.shape != (T, nq) or lse.get_device() != dev or not lse.is_contiguous():
                raise ValueError(f"lse: expected contiguous float32 {(T, nq)} on cuda:{dev}")
            lse_at = lse.data_ptr()
        scope = self._enter(batch, stream)
        if scope is not None:
            with scope:
                return self.attend(q, batch, scale, out, lse, shared_tokens)
        if out is None:
            out = q.new_empty(shape)
        h = _heads2(*qr, *_rows(out, "out", shape, dtype, dev, True))
        at = C.addressof(h)
        n = C.c_size_t()
        L = moe.lib()
        status = L.moe_kv_attend_workspace(self._at, batch._at, nq, shared_tokens, C.addressof(n))
        if status:
            moe.check(status, "moe_kv_attend_workspace")
        work = self.data.new_empty(n.value)
        status = L.moe_kv_attend(self._at, batch._at, code, nq, at, at + 24, lse_at, dim ** -0.5 if scale is None else scale,
                                 shared_tokens, work.data_ptr(), n.value, _raw_stream(dev))
        if status:
            moe.check(status, "moe_kv_attend")
        return out

    def _settle(self):
        """Wait for the current stream of the cache's device (a capture runs later, in its own order)."""
        stream = torch.cuda.current_stream(self.dev)
        with torch.cuda.stream(stream):
            if not torch.cuda.is_current_stream_capturing():
                stream.synchronize()

    def check(self):
        """Wait for the device (all its streams), and raise MoeError if a call
        found a bad page, a bad batch or ran out of a wait since the last
        check (which clears it)."""
        torch.cuda.synchronize(self.dev)
        bits = int(self._status.item())
        if bits:
            self._status.zero_()
            self._settle()  # what later calls set on other streams is not cleared
            what = [n for b, n in ((BAD_PAGE, "bad page"), (BAD_BATCH, "bad batch"), (TIMEOUT, "timeout")) if bits & b]
            raise moe.MoeError(6 if bits & TIMEOUT else 8, "cache: " + ", ".join(what))
