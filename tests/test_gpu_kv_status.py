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


@pytest.mark.parametrize("cu,lens,rows", [([0, 3, 2], [9, 9], 3), ([0, 2, 5], [9, 9], 4), ([0, -1, 3], [9, 9], 3), ([0, 0, 3, 1, 3], [9] * 4, 3),
                                          ([0, 3, 3], [2, 9], 3), ([0, 3, 6], [9, 9], 6)])
def test_every_call_flags_a_batch_that_cannot_be(cu, lens, rows):
    """Counts that descend, end behind the rows, are negative, exceed the length or max_tokens: append, its fused form, read and
    attend all report them, whichever tokens they find a place for; the pages of others stay as they were."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    n, most = len(lens), 2 if rows == 6 else 3
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    good = attention.KvBatch(table, i32(*[9] * n), i32(*range(n + 1)), n, 1)
    bad = attention.KvBatch(table, i32(*lens), i32(*cu), rows, most)
    cache = attention.KvCache(n + 1, 32, 1, 64)
    cache.data.zero_()
    for batch, fails in ((good, False), (bad, True), (good, False)):
        t = batch.n_tokens
        x = torch.randn(t, 1, 64, device="cuda").bfloat16()
        for call in (lambda: cache.append(x, x, batch), lambda: cache.append_norm_rope(x, x, x, batch, None),
                     lambda: cache.append_norm_rope(x[:, :0], x, x, batch, None), lambda: cache.read(batch), lambda: cache.attend(x, batch)):
            call()
            if fails:
                with pytest.raises(moe.MoeError, match="cache: bad batch:"):
                    cache.check()
            else:
                cache.check()
    assert (cache.data.view(n + 1, -1)[n] == 0).all()


def test_a_batch_of_more_sequences_than_rows():
    """One token, 5,000 sequences: the empty ones are looked at too."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    n = 5000
    cache = attention.KvCache(1, 32, 1, 64)
    x = torch.randn(1, 1, 64, device="cuda").bfloat16()
    table, lens = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    lens[4000] = 1
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[4001:] = 1
    batch = attention.KvBatch(table, lens, cu, 1, 1)
    cache.append(x, x, batch)
    cache.check()
    cu[-1] = 0
    for call in (lambda: cache.append(x, x, batch), lambda: cache.read(batch)):
        call()
        with pytest.raises(moe.MoeError, match="cache: bad batch:"):
            cache.check()
