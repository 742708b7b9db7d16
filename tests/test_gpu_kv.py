"""Per-head norm + rotation and the quantised paged cache against binary64."""
import numpy as np
import pytest

from tests import model_ref as ref
from tests.model_gpu import f64, make_batch, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    import torch
    torch.manual_seed(0)


def types():
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}


def rope_close(got, want, x_pair, dt):
    """Half a step of the output's type relative to the value, and a few fp32
    roundings (mean square, root, weight, two products) of the pair's magnitude: 2^-20."""
    import torch
    tol = torch.finfo(dt).eps / 2 * np.abs(want) * (1 + 2 ** -10) + 2.0 ** -20 * x_pair + 2.0 ** -25
    err = np.abs(got - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,nq,nk,dim,rot,inter,offset", [
    (1, 32, 4, 128, 128, False, 0.0), (7, 5, 1, 64, 32, True, 1.0), (3, 3, 2, 256, 64, False, 1.0), (5, 2, 2, 96, 96, False, 0.0),
    (2, 1, 1, 8, 0, False, 0.0), (4, 2, 1, 40, 16, True, 0.0), (600, 16, 4, 128, 64, False, 0.0), (9, 0, 3, 80, 80, True, 0.0),
    (9, 3, 0, 200, 176, False, 0.0)])
def test_norm_rope(T, nq, nk, dim, rot, inter, offset, dtype):
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    dt = types()[dtype]
    rng = np.random.default_rng(T + dim)
    g = torch.Generator().manual_seed(T * 1000 + dim)
    packed = (torch.randn(T, nq + nk + 1, dim, generator=g) * 3).to(dt).cuda()
    q, k = packed[:, :nq], packed[:, nq:nq + nk]  # strided views
    wq, wk = ((torch.randn(dim, generator=g) * 0.2 + 1 - offset).to(dt).cuda() for _ in range(2))
    pos = torch.from_numpy(rng.integers(0, 5000, T).astype(np.int32)).cuda()
    table = attention.rope_table(5000, rot, 1e6) if rot else None
    qo, ko = attention.qk_norm_rope(q, k, pos, table, wq, wk, interleaved=inter, weight_offset=offset)
    t64 = None if table is None else table.cpu().numpy()
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        want = ref.rms_rope(f64(x), f64(w), offset, 1e-6, t64, pos.cpu().numpy(), inter)
        plain = np.abs(ref.rms_rope(f64(x), f64(w), offset, 1e-6, None, None, inter))
        big = plain.max(-1, keepdims=True) if plain.size else plain
        rope_close(f64(got), want, big, dt)
    # in place, and without weights
    q2, k2 = q.clone(), k.clone()
    a, b = attention.qk_norm_rope(q2, k2, pos, table, interleaved=inter, q_out=q2, k_out=k2)
    assert a is q2 and b is k2
    rope_close(f64(q2), ref.rms_rope(f64(q), None, 0.0, 1e-6, t64, pos.cpu().numpy(), inter), 12.0, dt)


def test_norm_rope_padding_and_far_positions():
    """Negative positions leave rows as they were, positions beyond the table give NaN; others are untouched by either."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    q, k = torch.randn(4, 2, 128).bfloat16().cuda(), torch.randn(4, 1, 128).bfloat16().cuda()
    table = attention.rope_table(10, 64, 1e4)
    pos = torch.tensor([3, -1, 10, 9], dtype=torch.int32).cuda()
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    attention.qk_norm_rope(q, k, pos, table, q_out=qo, k_out=ko)
    good = torch.tensor([3, 0, 0, 9], dtype=torch.int32).cuda()
    a, b = attention.qk_norm_rope(q, k, good, table)
    for got, want in ((qo, a), (ko, b)):
        assert (got[1] == 7).all() and got[2].isnan().all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])


CASES = [(8, 128, 64, 4), (4, 128, 64, 4), (8, 64, 32, 1), (4, 64, 96, 3), (8, 256, 128, 2), (4, 256, 32, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,dim,page,heads", CASES)
def test_append_and_read(bits, dim, page, heads, dtype):
    """What is read back is exactly the blocks' d * q, rounded once to the type; rows behind the last sequence and
    pages of others stay as they were."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    dt = types()[dtype]
    rng = np.random.default_rng(dim + bits)
    news, lens = [1, 5, 0, 70, 33], [1, 64, 200, 70, 100]
    batch, table, n = make_batch(news, lens, page, rng, pad_rows=4, wide=2)
    cache = attention.KvCache(n, page, heads, dim, bits)
    cache.data.fill_(0xA5)
    T = batch.n_tokens
    k, v = (torch.randn(T, heads, 2, dim) * torch.exp(3 * torch.randn(T, heads, 2, 1))).to(dt).cuda().unbind(2)
    k[0, 0, :32] = 0  # a block of zeros
    v[3, 0, 32:64] = 1e-8  # scale below fp16's smallest
    before = cache.data.clone()
    cache.append(k, v, batch)
    cache.check()
    ko, vo = torch.full((T, heads, dim), 9.0, dtype=dt).cuda(), torch.full((T, heads, dim), 9.0, dtype=dt).cuda()
    cache.read(batch, ko, vo)
    cache.check()
    real = sum(news)
    for x, got in ((k, ko), (v, vo)):
        want = torch.from_numpy(ref.held(f64(x[:real]), bits)).to(torch.float32).to(dt)
        have = got[:real].cpu()
        assert ((have == want) | (have.isnan() & want.isnan())).all()  # (a few magnitudes are beyond the cache's range)
        assert (got[real:] == 9).all()
    # bytes of pages that the new tokens do not reach
    touched = {int(table[b, p // page]) for b in range(len(lens)) for p in range(lens[b] - news[b], lens[b])}
    same = (cache.data == before).view(n, -1).all(1).cpu()
    assert all(bool(same[i]) != (i in touched) for i in range(n))


@pytest.mark.parametrize("bits", [8, 4])
def test_non_finite_blocks_read_back_as_nan(bits):
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(1)
    batch, _, n = make_batch([6], [6], 32, rng)
    cache = attention.KvCache(n, 32, 1, 64, bits)
    k = torch.randn(6, 1, 64).bfloat16().cuda()
    k[0, 0, 3], k[1, 0, 40], k[2, 0, 5], k[3, 0, 5], k[4, 0, 63] = float("nan"), float("inf"), 1e30, -65024.0, -float("inf")
    cache.append(k, k, batch)
    ko, vo = cache.read(batch)
    assert torch.equal(ko.isnan(), vo.isnan())
    bad = ko.isnan().view(6, 2, 32)
    assert bad.all(2).eq(bad.any(2)).all()  # whole blocks
    assert bad.any(2).tolist() == [[True, False], [False, True], [True, False], [False, False], [False, True], [False, False]]


@pytest.mark.parametrize("bits,dim", [(8, 128), (4, 256), (4, 64)])
@pytest.mark.parametrize("inter", [False, True])
def test_fused_store_is_the_two_calls(bits, dim, inter):
    """append_norm_rope gives the bits of qk_norm_rope then append; positions default to the cache's."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(dim)
    for news, lens in (([1, 1, 1], [9, 40, 1]), ([300, 2, 150], [300, 7, 500])):
        batch, _, n = make_batch(news, lens, 64, rng, pad_rows=3)
        T, real = batch.n_tokens, sum(news)
        qkv = torch.randn(T, 6 + 2 + 2, dim).bfloat16().cuda()
        q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
        w = (torch.randn(2, dim) * 0.1 + 1).bfloat16().cuda()
        table = attention.rope_table(600, 32, 1e4)
        pos = torch.tensor([p for n_, l in zip(news, lens) for p in range(l - n_, l)] + [-1] * 3, dtype=torch.int32).cuda()
        caches = [attention.KvCache(n, 64, 2, dim, bits) for _ in range(3)]
        for c in caches:
            c.data.zero_()
        qa, ka = attention.qk_norm_rope(q, k, pos, table, w[0], w[1], interleaved=inter)
        caches[0].append(ka, v, batch)
        qb = caches[1].append_norm_rope(q, k, v, batch, table, w[0], w[1], interleaved=inter)
        q2 = q.clone()
        caches[2].append_norm_rope(q2, k, v, batch, table, w[0], w[1], interleaved=inter, positions=pos, q_out=q2)
        assert torch.equal(qa[:real], qb[:real]) and torch.equal(qa[:real], q2[:real]) and torch.equal(q2[real:], q[real:])
        assert torch.equal(caches[0].data, caches[1].data) and torch.equal(caches[0].data, caches[2].data)
        for c in caches:
            c.check()


def test_bad_pages_and_batches_are_flagged_and_skipped():
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    cache = attention.KvCache(3, 32, 1, 64)
    cache.data.zero_()
    k = torch.randn(3, 1, 64).bfloat16().cuda()
    for table, lens, cu in (([[-1], [1], [2]], [1, 1, 1], [0, 1, 2, 3]), ([[3], [1], [2]], [1, 1, 1], [0, 1, 2, 3]),
                            ([[0], [1], [2]], [40, 1, 1], [0, 1, 2, 3])):
        b = attention.KvBatch(torch.tensor(table, dtype=torch.int32).cuda(), i32(*lens), i32(*cu), 3, 1)
        cache.append(k, k, b)
        with pytest.raises(moe.MoeError, match="bad page"):
            cache.check()
        cache.check()  # cleared
        ko, vo = cache.read(b)
        assert ko[0].isnan().all() and vo[0].isnan().all() and not ko[1:].isnan().any()
        with pytest.raises(moe.MoeError):
            cache.check()
    # more new tokens than the sequence is long: the first has no position
    b = attention.KvBatch(torch.tensor([[0]], dtype=torch.int32).cuda(), i32(2), i32(0, 3), 3, 3)
    cache.append(k, k, b)
    with pytest.raises(moe.MoeError, match="bad batch"):
        cache.check()
    ko, _ = cache.read(b)
    assert ko[0].isnan().all() and not ko[1:].isnan().any()
    with pytest.raises(moe.MoeError, match="bad batch"):
        cache.check()


def test_streams_and_graph():
    """On a stream other than the current one, and captured: a replay follows the arrays' new contents."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(3)
    batch, table, n = make_batch([2, 2], [40, 90], 32, rng)
    _, lens_t, _ = batch._tensors
    cache = attention.KvCache(n, 32, 2, 128)
    cache.data.zero_()
    k, v = (torch.randn(4, 2, 128).bfloat16().cuda() for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache.append(k, v, batch, stream=s)
    ko, vo = cache.read(batch, stream=s)
    s.synchronize()
    want = torch.from_numpy(ref.held(f64(k), 8)).float().bfloat16()
    assert torch.equal(ko.cpu(), want)
    graph = torch.cuda.CUDAGraph()
    out_k, out_v = torch.zeros_like(k), torch.zeros_like(v)
    with torch.cuda.graph(graph, stream=s):
        cache.append(k, v, batch)
        cache.read(batch, out_k, out_v)
    k.copy_(torch.randn(4, 2, 128))
    lens_t.sub_(5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_k.cpu(), torch.from_numpy(ref.held(f64(k), 8)).float().bfloat16())
    both = whole(table, lens_t.cpu().numpy())
    full, _ = cache.read(both)
    ends = np.cumsum(lens_t.cpu().numpy())
    assert torch.equal(full[ends[0] - 2:ends[0]], out_k[:2]) and torch.equal(full[ends[1] - 2:ends[1]], out_k[2:])
    cache.check()
