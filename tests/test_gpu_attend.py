"""Attention over the quantised cache against binary64 on the values the cache holds."""
import numpy as np
import pytest

from tests import model_ref as ref
from tests.model_gpu import f64, make_batch, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    import torch
    torch.manual_seed(0)


def fill(cache, table, lens, kv_mul=1.0, dt=None, seed=0):
    """Append random K and V for every position; returns them as float64 per sequence, as held."""
    import torch
    batch = whole(table, lens)
    g = torch.Generator().manual_seed(seed)
    shape = (batch.n_tokens, cache.n_kv_heads, cache.head_dim)
    k, v = ((torch.randn(shape, generator=g) * kv_mul).to(dt or torch.bfloat16).cuda() for _ in range(2))
    if batch.n_tokens:
        cache.append(k, v, batch)
    hk, hv = ref.held(f64(k), cache.bits), ref.held(f64(v), cache.bits)
    at = np.concatenate(([0], np.cumsum(lens)))
    return [(hk[at[i]:at[i + 1]], hv[at[i]:at[i + 1]]) for i in range(len(lens))]


def check(q, out, lse, kv, news, lens, scale, dt, ordinary=False, keys_rounded=False):
    """Per element.  A probability and a value are rounded to fp16 once each (2^-11 of the term; probabilities below
    fp16's normal range, which are held times 2^8, by 2^-33 of the largest), a score is off by delta <= (D / 16 + 4) 2^-21 of the
    sum of its products' magnitudes (fp32 accumulation of D / 16 steps, two scalings, the exponential), which moves a term by
    2 delta relative; then half a step of the output's type.  With more than 64 rows a sequence (32 of heads of 128, 16 of 256), or behind a
    shared prefix, the keys, integer times scale, are rounded to fp16 too: delta grows by 2^-11 of the same sum; with fp16
    activations by 2^-22, a rounding of what that left (and 2^-24 |q| where the rest is subnormal: keys here are not that small),
    and either the probabilities' or the values' rounding is taken up the same way."""
    import torch
    D, at = q.shape[2], 0
    group = q.shape[1] // kv[0][0].shape[1]
    eps = torch.finfo(dt).eps
    keys_rounded = (2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -22) if keys_rounded or max(news) * group > {64: 64, 128: 32, 256: 16}[D] else 0.0
    for (k, v), n, length in zip(kv, news, lens):
        if n == 0:
            continue
        qs, got, got_l = q[at:at + n], out[at:at + n], lse[at:at + n]
        want, want_l = ref.attend(qs, k, v, scale, n)
        mean_abs, _ = ref.attend(qs, k, np.abs(v), scale, n)
        kg, vg = np.repeat(k, group, 1), np.repeat(v, group, 1)
        sums = np.einsum("nhd,lhd->nhl", np.abs(qs), np.abs(kg)).max(-1) * abs(scale) if length else np.zeros(qs.shape[:2])
        delta = ((D / 16 + 4) * 2.0 ** -21 + keys_rounded) * sums
        big = np.abs(vg).max(0)[None] if length else 0.0
        tol = ((2 if dt == torch.bfloat16 else 1) * 2.0 ** -11 + 2.0 ** -18 + 2 * delta[..., None]) * mean_abs * 1.01 + max(length, 1) * 2.0 ** -32 * big
        tol = tol + eps / 2 * (np.abs(want) + tol) + 2.0 ** -25
        err = np.abs(got - want)
        assert (err <= tol).all(), (float((err / tol).max()), n, length)
        if ordinary and length:
            # of the norm: roundings are independent, uniform within half a step (1 / sqrt 3 of it).  Keys move a score by 2^-11 /
            # sqrt 3 of the root of its squared products' sum, which is the queries' size, 2; then P and V (one of them with fp16) and the output
            step = 2.0 ** -11 / 3 ** 0.5
            bound = ((2 * step) ** 2 * (keys_rounded > 2.0 ** -12) + (2 if dt == torch.bfloat16 else 1) * step ** 2 + (eps / 2) ** 2 / 3) ** 0.5
            assert np.linalg.norm(err) <= 1.7 * bound * np.linalg.norm(want), np.linalg.norm(err) / np.linalg.norm(want)
        seen = np.isfinite(want_l)
        assert np.array_equal(seen, np.isfinite(got_l))
        assert (np.abs(got_l - want_l)[seen] <= (delta + 2.0 ** -18)[seen] + 2.0 ** -22 * np.abs(want_l[seen])).all()
        at += n


def run_case(bits, dim, page, hkv, group, news, lens, dtype="bf16", q_mul=2.0, pad=0, kv_mul=1.0, seed=0, scale=None):
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    rng = np.random.default_rng(seed + dim + page)
    batch, table, n = make_batch(news, lens, page, rng, pad_rows=pad, wide=1)
    cache = attention.KvCache(n, page, hkv, dim, bits)
    cache.data.fill_(0xFF)  # NaN scales wherever nothing was written
    kv = fill(cache, table, lens, kv_mul, dt, seed)
    g = torch.Generator().manual_seed(seed + 5)
    T = batch.n_tokens
    q = (torch.randn(T, hkv * group + 1, dim, generator=g) * q_mul).to(dt).cuda()[:, 1:]  # strided
    out = torch.full((T, hkv * group, dim), 5.0, dtype=dt).cuda()
    lse = torch.full((T, hkv * group), 5.0).cuda()
    s = dim ** -0.5 if scale is None else scale
    cache.attend(q, batch, scale=s, out=out, lse=lse)
    cache.check()
    real = sum(news)
    assert (out[real:] == 5).all() and (lse[real:] == 5).all()
    check(f64(q), f64(out), f64(lse), kv, news, lens, s, dt, ordinary=q_mul == 2.0 and kv_mul == 1.0 and scale is None)
    return cache, batch, q, out


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ragged_decode(bits, dim, dtype):
    run_case(bits, dim, 64, 2, 4, [1] * 7, [1, 31, 32, 33, 64, 65, 700], dtype)


@pytest.mark.parametrize("hkv,group", [(1, 1), (3, 5), (2, 16), (1, 17), (1, 40)])
def test_head_layouts(hkv, group):
    run_case(8, 128, 32, hkv, group, [1, 1, 1], [100, 5, 333])


@pytest.mark.parametrize("bits,dim,page", [(8, 128, 32), (4, 128, 96), (8, 256, 160), (4, 64, 128)])
def test_several_tokens_and_none(bits, dim, page):
    """Causal within the new tokens; sequences without new tokens; a padded batch."""
    run_case(bits, dim, page, 2, 3, [2, 0, 5, 1, 4, 9], [2, 10, 5, 64, 200, 37], pad=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,dim,group,n,length", [(8, 128, 8, 90, 90), (4, 128, 2, 300, 517), (8, 64, 1, 130, 131), (4, 256, 4, 77, 400),
                                                     (8, 256, 2, 129, 129), (4, 64, 3, 200, 333), (8, 128, 1, 1, 2500)])
def test_chunks(bits, dim, group, n, length, dtype):
    run_case(bits, dim, 64, 2, group, [n, 1], [length, 3], dtype)


def test_long_context_is_split_and_joined():
    run_case(8, 128, 64, 1, 8, [1], [20011], seed=2)
    run_case(4, 128, 128, 2, 4, [2, 1], [9001, 40], "fp16", seed=3)


@pytest.mark.parametrize("seqs", [1, 130, 300])
def test_many_sequences(seqs):
    rng = np.random.default_rng(seqs)
    run_case(8, 64, 32, 1, 2, [1] * seqs, [int(x) for x in rng.integers(1, 90, seqs)])


@pytest.mark.parametrize("bits,dim", [(8, 128), (4, 256), (8, 64), (4, 128), (8, 256), (4, 64)])
def test_shared_prefix(bits, dim):
    """The hint changes nothing but the order of sums; a sequence may end inside the shared part."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    page, share, hkv, group = 64, 256, 2, 4
    rng = np.random.default_rng(dim)
    lens, news = [257, 500, 100, 256, 0, 256 + 300, 1, 40] + [260 + 13 * i for i in range(14)], [1, 3, 1, 1, 0, 1, 1, 2] + [1] * 14
    batch, table, n = make_batch(news, lens, page, rng, share=share // page, wide=1)
    cache = attention.KvCache(n, page, hkv, dim, bits)
    cache.data.fill_(0xFF)
    kv = []
    prefix = None
    for i, length in enumerate(lens):
        t = torch.Generator().manual_seed(50 + i)
        k, v = (torch.randn(max(length, 1), hkv, dim, generator=t).bfloat16().cuda() for _ in range(2))
        if prefix is None:
            prefix = (k[:share].clone(), v[:share].clone())
        m = min(share, length)
        k[:m], v[:m] = prefix[0][:m], prefix[1][:m]
        if length:
            cache.append(k[:length], v[:length], whole(table[i:i + 1], [length]))
        kv.append((ref.held(f64(k[:length]), bits), ref.held(f64(v[:length]), bits)))
    q = (torch.randn(batch.n_tokens, hkv * group, dim) * 2).bfloat16().cuda()
    for shared in (0, 64, share):
        lse = torch.zeros(batch.n_tokens, hkv * group).cuda()
        out = cache.attend(q, batch, lse=lse, shared_tokens=shared)
        cache.check()
        check(f64(q), f64(out), f64(lse), kv, news, lens, dim ** -0.5, torch.bfloat16, keys_rounded=shared > 0)


def test_shared_prefix_of_a_large_batch():
    """Rows of all sequences fill many row tiles of the shared part."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    page, share, hkv, group, dim, seqs = 32, 320, 1, 5, 128, 77
    rng = np.random.default_rng(4)
    lens = [share + int(x) for x in rng.integers(1, 70, seqs)]
    batch, table, n = make_batch([1] * seqs, lens, page, rng, share=share // page)
    cache = attention.KvCache(n, page, hkv, dim, 8)
    cache.data.fill_(0xFF)
    base = torch.randn(2, share, hkv, dim).bfloat16().cuda()
    kv = []
    for i, length in enumerate(lens):
        own = torch.randn(2, length - share, hkv, dim).bfloat16().cuda()
        k, v = torch.cat((base, own), 1)
        cache.append(k, v, whole(table[i:i + 1], [length]))
        kv.append((ref.held(f64(k), 8), ref.held(f64(v), 8)))
    q = (torch.randn(seqs, hkv * group, dim) * 2).bfloat16().cuda()
    lse = torch.zeros(seqs, hkv * group).cuda()
    out = cache.attend(q, batch, lse=lse, shared_tokens=share)
    cache.check()
    check(f64(q), f64(out), f64(lse), kv, [1] * seqs, lens, dim ** -0.5, torch.bfloat16, keys_rounded=True)


def shared_case(bits, dim, hkv, group, share, seqs, seed=0):
    """Sequences of 1 to share + 70 positions, most longer than share, one to three new tokens each, some none; their first
    pages are the same.  Returns (cache, batch, table, q, kv, news, lens)."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(seed)
    page = 64
    lens = [share + int(x) for x in rng.integers(1, 70, seqs)]
    news = [1] * seqs
    lens[3:8], news[3:8] = [share, 1, share - 5, 0, share + 2], [1, 1, 3, 0, 3]
    news[11], news[20] = 0, 2
    batch, table, n = make_batch(news, lens, page, rng, share=share // page, wide=1)
    cache = attention.KvCache(n, page, hkv, dim, bits)
    cache.data.fill_(0xFF)
    base = torch.randn(2, share, hkv, dim, device="cuda").bfloat16()
    cache.append(base[0], base[1], whole(table[:1], [share]))
    tails = [max(0, x - share) for x in lens]
    own = torch.randn(2, sum(tails), hkv, dim, device="cuda").bfloat16()
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    cu = np.concatenate(([0], np.cumsum(tails)))
    cache.append(own[0], own[1], attention.KvBatch(dev(table.tolist()), dev(lens), dev(cu.tolist()), int(cu[-1]), max(tails)))
    cache.check()
    hb, ho = [ref.held(f64(x), bits) for x in base], [ref.held(f64(x), bits) for x in own]
    kv = [tuple(np.concatenate((hb[j][:min(share, x)], ho[j][cu[i]:cu[i + 1]])) for j in (0, 1)) for i, x in enumerate(lens)]
    q = (torch.randn(batch.n_tokens, hkv * group, dim, device="cuda") * 2).bfloat16()
    return cache, batch, table, q, kv, news, lens


@pytest.mark.parametrize("bits,dim,group,share,seqs", [(8, 128, 2, 1024, 280), (4, 256, 2, 1024, 280), (8, 64, 3, 1920, 180),
                                                       (4, 128, 5, 1984, 160), (8, 256, 1, 576, 500), (4, 64, 2, 1920, 330)])
def test_shared_prefix_read_once(bits, dim, group, share, seqs):
    """Enough reads spared for a pass of its own: a million keys, counted a kv head."""
    import torch
    assert (seqs * 0.9) * share * 4 > 1e6
    cache, batch, _, q, kv, news, lens = shared_case(bits, dim, 4, group, share, seqs)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = cache.attend(q, batch, lse=lse, shared_tokens=share)
    cache.check()
    check(f64(q), f64(out), f64(lse), kv, news, lens, dim ** -0.5, torch.bfloat16, keys_rounded=True)


def test_shared_prefix_captured_and_with_a_bad_page():
    """Replays and a call on another stream agree with the eager call bit for bit; a page out of range makes NaN of what sees it."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import moe
    share = 1024
    cache, batch, table, q, _, news, lens = shared_case(8, 128, 4, 2, share, 280)
    eager = cache.attend(q, batch, shared_tokens=share)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = cache.attend(q, batch, shared_tokens=share, stream=s)
    s.synchronize()
    out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.attend(q, batch, out=out, shared_tokens=share)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager, other) and torch.equal(eager, out) and eager.isfinite().all()
    batch._tensors[0][:, 2] = 2 ** 30  # positions 128 to 191 of all
    bad = cache.attend(q, batch, shared_tokens=share)
    with pytest.raises(moe.MoeError, match="bad page"):
        cache.check()
    at = 0
    for n, length in zip(news, lens):
        if n:
            assert bad[at:at + n].isnan().all() if length > 192 else torch.equal(bad[at:at + n], eager[at:at + n])
        at += n


def test_shared_prefix_with_token_counts_that_decrease():
    """The last sequence's rows would end before they begin: the batch is flagged, the sequences before it that end in time are right."""
    from quantized_expert_ffn_gemv_gb300 import moe
    share = 1024
    cache, batch, _, q, _, news, lens = shared_case(8, 128, 4, 2, share, 280)
    want = cache.attend(q, batch, shared_tokens=share)
    batch._tensors[2][-1] = 40
    got = cache.attend(q, batch, shared_tokens=share)
    with pytest.raises(moe.MoeError, match="bad batch"):
        cache.check()
    assert (got[:40] - want[:40]).abs().max() <= 0.02 * want.abs().max()  # (cut into other parts: each within a bf16 step, 2^-8, and 2^-9)

@pytest.mark.parametrize("n,group", [(1, 4), (3, 2), (100, 2)])
def test_rows_that_see_nothing(n, group):
    """More new tokens than positions: the first rows see nothing, out 0 and lse -infinity; the batch is flagged."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    cache = attention.KvCache(8, 32, 1, 128)
    cache.data.fill_(0xFF)
    length = n // 2
    table = torch.arange(8, dtype=torch.int32).cuda()[None]
    kv = fill(cache, table.cpu().numpy(), [length]) if length else [(np.zeros((0, 1, 128)),) * 2]
    q = torch.randn(n, group, 128).bfloat16().cuda()
    lse = torch.zeros(n, group).cuda()
    out = cache.attend(q, attention.KvBatch(table, i32(length), i32(0, n), n, n), lse=lse)
    with pytest.raises(moe.MoeError, match="bad batch"):
        cache.check()
    empty = n - length
    assert (out[:empty] == 0).all() and (lse[:empty] == -float("inf")).all()
    if length:
        check(f64(q[empty:]), f64(out[empty:]), f64(lse[empty:]), kv, [length], [length], 128 ** -0.5, torch.bfloat16)


def test_scores_out_of_the_ordinary():
    """Queries of bf16's whole range, large and tiny scales, a huge maximum with a flat rest."""
    run_case(8, 128, 64, 1, 4, [1, 2], [70, 300], q_mul=1e-30, scale=1e29)
    run_case(8, 128, 64, 1, 4, [1, 2], [70, 300], q_mul=1e30, scale=1e-31)
    run_case(4, 128, 64, 1, 4, [1, 2], [70, 300], q_mul=30.0)
    run_case(8, 64, 64, 1, 2, [1], [5000], q_mul=0.0)
    run_case(8, 128, 64, 1, 2, [1, 90], [500, 200], kv_mul=3000.0, q_mul=3e-4)


@pytest.mark.parametrize("n", [3, 100])
def test_non_finite_keys_and_values_stay_with_the_rows_that_see_them(n):
    """A NaN among the new tokens' keys or values reaches the rows from its position on and no earlier one."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(9)
    length = n + 20
    batch, table, pages = make_batch([n], [length], 32, rng)
    for kind in ("k", "v"):
        cache = attention.KvCache(pages, 32, 1, 128)
        cache.data.fill_(0xFF)
        k, v = (torch.randn(length, 1, 128).bfloat16().cuda() for _ in range(2))
        bad = length - n + n // 2
        (k if kind == "k" else v)[bad, 0, 70] = float("nan")
        cache.append(k, v, whole(table, [length]))
        q = torch.randn(n, 4, 128).bfloat16().cuda()
        out = cache.attend(q, batch)
        cache.check()
        first = n // 2
        assert torch.isfinite(out[:first]).all()
        assert out[first:].isnan().any(-1).all()
        hk, hv = ref.held(f64(k[:bad]), 8), ref.held(f64(v[:bad]), 8)
        want, _ = ref.attend(f64(q[:first]), hk, hv, 128 ** -0.5, first)
        # two fp16 roundings a term and the output's bf16 one, of magnitudes up to max |v|
        assert np.abs(f64(out[:first]) - want).max() < (2.0 ** -9 + 2.0 ** -8) * np.abs(hv).max()


def test_infinite_and_nan_queries():
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(2)
    batch, table, n = make_batch([4], [50], 32, rng)
    cache = attention.KvCache(n, 32, 1, 64)
    fill(cache, table, [50])
    q = torch.randn(4, 2, 64).bfloat16().cuda()
    clean = cache.attend(q, batch)
    q[1, 0, 3], q[2, 1, 5] = float("nan"), float("inf")
    out = cache.attend(q, batch)
    assert out[1, 0].isnan().all() and out[2, 1].isnan().all()
    keep = torch.ones(4, 2, dtype=torch.bool).cuda()
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("n", [1, 70])
def test_bad_pages_give_nan_rows_and_a_status(n):
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    cache = attention.KvCache(6, 32, 1, 128)
    cache.data.zero_()
    q = torch.randn(2 * n, 2, 128).bfloat16().cuda()
    for bad, length in ((-5, 96), (6, 96), (2, 97)):
        table = torch.tensor([[0, 1, bad], [3, 4, 5]], dtype=torch.int32).cuda()
        b = attention.KvBatch(table, i32(length, 96), i32(0, n, 2 * n), 2 * n, n)
        out = cache.attend(q, b)
        with pytest.raises(moe.MoeError, match="bad page"):
            cache.check()
        assert out[n - 1].isnan().all() and (out[n:] == 0).all()


@pytest.mark.parametrize("news,share", [([1, 1, 1], 0), ([1, 1, 1], 64), ([80, 1, 90], 0)])
def test_graph_replay_two_graphs_and_another_stream(news, share):
    """Captured calls follow the arrays' contents; two graphs replayed in turn and a call on another stream agree with eager
    ones bit for bit."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(6)
    lens = [200, 130, 300]
    batch, table, n = make_batch(news, lens, 64, rng, share=share // 64, extra_pages=4)
    cache = attention.KvCache(n, 64, 2, 128)
    for i in range(3):
        fill(cache, table[i:i + 1], [lens[i]], seed=i)
    lens_t = batch._tensors[1]
    qa, qb = (torch.randn(batch.n_tokens, 8, 128).bfloat16().cuda() for _ in range(2))
    oa, ob = torch.zeros_like(qa), torch.zeros_like(qb)
    eager = [cache.attend(x, batch, shared_tokens=share) for x in (qa, qb)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = cache.attend(qa, batch, shared_tokens=share, stream=s)
    s.synchronize()
    assert torch.equal(other, eager[0])
    graphs = []
    for q, o in ((qa, oa), (qb, ob)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cache.attend(q, batch, out=o, shared_tokens=share)
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, eager[0]) and torch.equal(ob, eager[1])
    lens_t.sub_(3)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, cache.attend(qa, batch, shared_tokens=share)) and not torch.equal(oa, eager[0])
    cache.check()
