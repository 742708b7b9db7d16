"""The cache's status word: calls on other streams, and what a batch's arrays can have wrong."""
import pytest

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000  # cycles, a tenth of a second


def i32(*v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_check_waits_for_calls_on_other_streams():
    """A call still queued on another stream is seen by the check that follows it, and only by that one."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    cache = attention.KvCache(2, 32, 1, 64)
    k = torch.randn(1, 1, 64, device="cuda").bfloat16()
    batch = attention.KvBatch(i32([5]), i32(1), i32(0, 1), 1, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        cache.append(k, k, batch, stream=side)
        with pytest.raises(moe.MoeError, match="bad page"):
            cache.check()
        cache.check()


def test_a_new_cache_is_usable_on_any_stream():
    """The status word's zeros are queued behind other work of the creating stream; a call on a second stream does not lose its flag."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    pool = torch.zeros(2 * 32 * 64 * 3, dtype=torch.uint8, device="cuda")
    k = torch.randn(1, 1, 64, device="cuda").bfloat16()
    batch = attention.KvBatch(i32([5]), i32(1), i32(0, 1), 1, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    cache = attention.KvCache(2, 32, 1, 64, data=pool[:2 * 32 * (128 + 8)])
    cache.append(k, k, batch, stream=side)
    with pytest.raises(moe.MoeError, match="bad page"):
        cache.check()


def test_a_cache_made_inside_a_capture():
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    pool = torch.zeros(2 * 32 * (128 + 8), dtype=torch.uint8, device="cuda")
    k = torch.randn(1, 1, 64, device="cuda").bfloat16()
    batch = attention.KvBatch(i32([1]), i32(1), i32(0, 1), 1, 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache = attention.KvCache(2, 32, 1, 64, data=pool)
        cache.append(k, k, batch)
    g.replay()
    cache.check()
    assert pool.any()
