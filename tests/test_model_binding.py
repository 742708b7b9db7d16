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
