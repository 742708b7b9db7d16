"""The Python side of the sequence-side operators without a GPU: what it refuses before the library sees it."""
import ctypes

import pytest
import torch

from quantized_expert_ffn_gemv_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_cuda()
    build.build_binding()


class Fake:
    """What the binding looks at of a CUDA tensor, of any size."""

    def __init__(self, *shape, dtype=torch.bfloat16, stride=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)
        strides = [1]
        for n in shape[:0:-1]:
            strides.insert(0, strides[0] * n)
        self._stride = tuple(stride or strides)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def is_contiguous(self):
        return True


def ints(*shape, **kw):
    return Fake(*shape, dtype=torch.int32, **kw)


def test_sizes_beyond_32_bits_are_refused(monkeypatch):
    """Each of these has low bits that would be a fine size."""
    from quantized_expert_ffn_gemv_gb300 import attention, moe, sampling
    monkeypatch.setattr(attention, "_current_device", lambda: 0)
    big = 2 ** 32
    for bad in (lambda: attention.rope_table(big + 4, 32, 1e4), lambda: attention.KvCache(big + 4, 64, 2, 128),
                lambda: attention.KvCache(4, big + 64, 2, 128), lambda: attention.KvCache(4, 64, 2, big + 128),
                lambda: attention.KvBatch(ints(2, 4), ints(2), ints(3), big + 5, 3),
                lambda: attention.KvBatch(ints(2, 4, stride=(big + 4, 1)), ints(2), ints(3), 5, 3),
                lambda: attention.KvBatch(ints(2, big + 4), ints(2), ints(3), 5, 3),
                lambda: attention.qk_norm_rope(Fake(big + 3, 2, 64), Fake(big + 3, 1, 64), None, None),
                lambda: attention.qk_norm_rope(Fake(3, 2, 64), Fake(3, 1, 64), ints(3), Fake(big + 9, 16, 2, dtype=torch.float32)),
                lambda: sampling.sample(Fake(1, big + 1000), Fake(1, dtype=torch.float32)),
                lambda: sampling.sample(Fake(big + 1, 1000), Fake(big + 1, dtype=torch.float32))):
        with pytest.raises(ValueError, match="beyond 32 bits"):
            bad()
    batch = attention.KvBatch(ints(2, 4), ints(2), ints(3), 5, 3)
    assert (batch.n_tokens, batch.max_tokens, batch.desc.n_tokens, batch.desc.table_stride) == (5, 3, 5, 4)
    cache = attention.KvCache.__new__(attention.KvCache)
    cache.n_kv_heads, cache.head_dim, cache.dev, cache.data = 2, 128, 0, Fake(16, dtype=torch.uint8)
    cache.desc = moe.KvCacheDesc(n_kv_heads=2, head_dim=128)
    cache._at = ctypes.addressof(cache.desc)
    with pytest.raises(ValueError, match="beyond 32 bits"):
        cache.attend(Fake(5, 4, 128), batch, shared_tokens=big + 64)


def collide(T, H, dim, ts, hs):
    """Whether two of the rows share an element, by listing them."""
    starts = sorted(i * ts + j * hs for i in range(T) for j in range(H))
    return any(b - a < dim for a, b in zip(starts, starts[1:]))


def test_rows_of_an_output_that_overlap_are_refused(monkeypatch):
    """Equal strides, or strides whose multiples meet, put two rows in one place: the binding and the library tell every layout
    of small strides apart as a list of the rows does; layouts as views make them are taken."""
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    monkeypatch.setattr(attention, "_current_device", lambda: 0)
    L, at = moe.lib(), 1 << 20
    page = L.moe_kv_page_bytes(64, 3, 64, 8)
    refused = 0
    for T, H in ((1, 3), (2, 3), (5, 3), (4, 1), (7, 2), (1, 1)):
        for ts in range(0, 8 * 64, 32):
            for hs in range(0, 8 * 64, 32):
                bad = collide(T, H, 64, ts, hs)
                assert attention._apart(T, H, 64, ts, hs) != bad, (T, H, ts, hs)
                if not bad:
                    continue
                refused += 1
                heads = (ctypes.c_int64 * 3)(at, ts, hs)
                good = (ctypes.c_int64 * 3)(at, H * 64, 64)
                cache = moe.KvCacheDesc(data=at, data_bytes=page * 8, n_pages=8, page_size=64, n_kv_heads=H, head_dim=64, bits=8, status=at)
                batch = moe.KvBatchDesc(block_table=at, seq_lens=at, cu_tokens=at, n_seqs=1, table_stride=4, max_pages=4, n_tokens=T, max_tokens=T)
                ref = ctypes.byref
                assert L.moe_kv_read(ref(cache), ref(batch), 0, ref(heads), ref(good), None) == 1, (T, H, ts, hs)
                with pytest.raises(ValueError):
                    attention._rows(Fake(T, H, 64, stride=(ts, hs, 1)), "out", (T, H, 64), torch.bfloat16, 0, True)
    assert refused > 100
    for ts, hs in ((8 * 128, 128), (128, 5 * 128), (8 * 256, 256), (1 << 40, 1 << 44)):
        assert attention._rows(Fake(5, 8, 128, stride=(ts, hs, 1)), "out", (5, 8, 128), torch.bfloat16, 0, True) == (at, ts, hs)
