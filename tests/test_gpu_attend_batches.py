"""Attention over batches of many sequences: a CTA of either kernel goes through several pieces of work."""
import numpy as np
import pytest

from tests import model_ref as ref
from tests.model_gpu import f64, make_batch, whole
from tests.test_gpu_attend import check, fill, run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    import torch
    torch.manual_seed(0)


def prompts(seqs, seed, most=24, history=90, long=()):
    """(new tokens, lengths) of ragged prompts: one in nine brings none, `long` some of a given size."""
    rng = np.random.default_rng(seed)
    news = [0 if i % 9 == 4 else int(x) for i, x in enumerate(rng.integers(1, most, seqs))]
    for i, n in long:
        news[i] = n
    return news, [n + int(x) for n, x in zip(news, rng.integers(0, history, seqs))]


@pytest.mark.parametrize("bits,dim,group,dtype", [(4, 256, 2, "bf16"), (8, 128, 3, "bf16"), (8, 64, 5, "fp16"), (4, 128, 3, "fp16"), (8, 256, 2, "fp16")])
def test_more_row_tiles_than_ctas(bits, dim, group, dtype):
    """700 sequences of 2 kv heads: nine pieces a CTA, most of fewer than 128 rows, some of several row tiles."""
    news, lens = prompts(700, dim, long=[(50, 100), (51, 61), (300, 150), (699, 90)])
    run_case(bits, dim, 64, 2, group, news, lens, dtype)


@pytest.mark.parametrize("bits,dim,dtype", [(4, 256, "bf16"), (8, 256, "bf16"), (4, 128, "bf16"), (8, 64, "fp16")])
def test_bad_pages_among_many_short_prompts(bits, dim, dtype):
    """Every seventh sequence's only or last page is out of range: the rows that see it are NaN, all others keep their bits."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    seqs, page, group = 700, 32, 4
    rng = np.random.default_rng(dim)
    news = [int(x) for x in rng.integers(1, 28, seqs)]  # one step of keys, one row tile
    news[3], news[10], news[352], news[692] = 60, 64, 40, 64  # rows in a second tile of 128
    lens = [n + (i % 3 == 0) * int(x) for i, (n, x) in enumerate(zip(news, rng.integers(0, 60, seqs)))]
    batch, table, n_pages = make_batch(news, lens, page, rng)
    cache = attention.KvCache(n_pages, page, 2, dim, bits)
    cache.data.fill_(0xFF)
    fill(cache, table, lens, dt=dt)
    q = torch.randn(batch.n_tokens, 2 * group, dim).to(dt).cuda()
    clean = cache.attend(q, batch)
    cache.check()
    assert clean.isfinite().all()
    spoiled, at = torch.zeros(batch.n_tokens, dtype=torch.bool), 0
    for i, (n, length) in enumerate(zip(news, lens)):
        if i % 7 == 3:
            last = (length - 1) // page
            batch._tensors[0][i, last] = -1 if i % 2 else 2 ** 30
            spoiled[at + max(0, n - (length - last * page)):at + n] = True
        at += n
    for _ in range(20):
        got = cache.attend(q, batch)
        with pytest.raises(moe.MoeError, match="bad page"):
            cache.check()
        rows = got.flatten(1).cpu()
        assert rows[spoiled].isnan().all()
        assert torch.equal(rows[~spoiled], clean.flatten(1).cpu()[~spoiled])


@pytest.mark.parametrize("n,dim,bits", [(4, 128, 8), (6, 64, 4), (5, 256, 4), (70, 128, 8), (70, 256, 4)])
def test_a_bad_page_reaches_only_the_rows_that_see_it(n, dim, bits):
    """New tokens on both sides of a page's end: with the second page out of range, or behind the table's width, the rows
    before it keep their bits."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    page, first = 32, n // 2
    start = 3 * page - first  # position of the first new token: `first` of them lie on the third page
    lens = [start + n, start + n + 5]
    rng = np.random.default_rng(n)
    batch, table, n_pages = make_batch([n, n], lens, page, rng)
    cache = attention.KvCache(n_pages, page, 2, dim, bits)
    cache.data.fill_(0xFF)
    kv = fill(cache, table, lens)
    q = torch.randn(2 * n, 4, dim).bfloat16().cuda()
    clean = cache.attend(q, batch)
    cache.check()
    assert clean.isfinite().all()
    bad = table.copy()
    bad[0, 3] = -7
    wide = attention.KvBatch(i32(*bad.tolist()), i32(*lens), i32(0, n, 2 * n), 2 * n, n)
    got = cache.attend(q, wide)
    with pytest.raises(moe.MoeError, match="bad page"):
        cache.check()
    assert torch.equal(got[:first], clean[:first]) and got[first:n].isnan().all() and torch.equal(got[n:], clean[n:])
    narrow = attention.KvBatch(wide._tensors[0][:, :3], i32(*lens), i32(0, n, 2 * n), 2 * n, n)
    lse = torch.zeros(2 * n, 4, device="cuda")
    got = cache.attend(q, narrow, lse=lse)
    with pytest.raises(moe.MoeError, match="bad page"):
        cache.check()
    for b, seen in ((0, first), (1, max(0, first - 5))):
        at = b * n
        assert got[at + seen:at + n].isnan().all() and lse[at + seen:at + n].isnan().all()
        check(f64(q)[at:at + seen], f64(got)[at:at + seen], f64(lse)[at:at + seen], [tuple(x[:3 * page] for x in kv[b])], [seen], [3 * page],
              dim ** -0.5, torch.bfloat16, keys_rounded=n == 70)


def prefix_case(bits, dim, dtype, page, share, seqs, group, hkv=4, tail=70, seed=0):
    """Sequences behind a common prefix, of 1 to 3 new tokens or none, some that end inside it; share is a multiple of the page.
    Returns (cache, batch, table, q, kv, news, lens), kv as held."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    rng = np.random.default_rng(seed)
    lens = [share + int(x) for x in rng.integers(0, tail, seqs)]
    news = [1 + (i % 5 == 2) * 2 for i in range(seqs)]
    lens[2:7], news[2:7] = [share, 1, share - 17, 0, share + 1], [3, 1, 2, 0, 1]
    news[11] = 0
    batch, table, n_pages = make_batch(news, lens, page, rng, share=share // page, wide=1)
    cache = attention.KvCache(n_pages, page, hkv, dim, bits)
    cache.data.fill_(0xFF)
    base = torch.randn(2, share, hkv, dim, device="cuda").to(dt)
    cache.append(base[0], base[1], whole(table[:1], [share]))
    tails = [max(0, x - share) for x in lens]
    own = torch.randn(2, sum(tails), hkv, dim, device="cuda").to(dt)
    cu = np.concatenate(([0], np.cumsum(tails)))
    dev = lambda a: torch.tensor(np.asarray(a).tolist(), dtype=torch.int32, device="cuda")
    cache.append(own[0], own[1], attention.KvBatch(dev(table), dev(lens), dev(cu), int(cu[-1]), max(tails)))
    cache.check()
    hb, ho = [ref.held(f64(x), bits) for x in base], [ref.held(f64(x), bits) for x in own]
    kv = [tuple(np.concatenate((hb[j][:min(share, x)], ho[j][cu[i]:cu[i + 1]])) for j in (0, 1)) for i, x in enumerate(lens)]
    q = (torch.randn(batch.n_tokens, hkv * group, dim, device="cuda") * 2).to(dt)
    assert (seqs - 30) * share * hkv > 1e6  # enough reads spared for a pass of its own
    return cache, batch, table, q, kv, news, lens


def test_a_length_beyond_the_table_behind_a_prefix_that_fills_it():
    """The rows that lie behind the table's last page are NaN, as they are without the hint; the others keep their values."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, moe
    share, seqs, page = 1024, 300, 64
    cache, _, table, _, kv, _, _ = prefix_case(8, 128, "bf16", page, share, seqs, 2)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    lens = [share] * seqs
    lens[5], lens[17], lens[40] = share + 1, share + 40, share + 2  # one new token each, the last two of the fortieth
    news = [1] * seqs
    news[40] = 4
    cu = np.concatenate(([0], np.cumsum(news))).tolist()
    batch = attention.KvBatch(i32(table[:1, :share // page].repeat(seqs, 0).tolist()), i32(lens), i32(cu), cu[-1], 4)
    q = (torch.randn(cu[-1], 8, 128, device="cuda") * 2).bfloat16()
    outs = []
    for shared in (0, share):
        lse = torch.zeros(q.shape[:2], device="cuda")
        outs.append((cache.attend(q, batch, lse=lse, shared_tokens=shared), lse))
        with pytest.raises(moe.MoeError, match="bad page"):
            cache.check()
    beyond = torch.zeros(cu[-1], dtype=torch.bool)
    beyond[[cu[5], cu[17], cu[40] + 2, cu[40] + 3]] = True
    for out, lse in outs:
        assert out.cpu()[beyond].isnan().all() and lse.cpu()[beyond].isnan().all()
        assert out.cpu()[~beyond].isfinite().all()
    # the sequences that fit the table, against binary64
    fit = [i for i in range(seqs) if lens[i] == share]
    rows = np.concatenate([np.arange(cu[i], cu[i + 1]) for i in fit])
    for (out, lse), rounded in zip(outs, (False, True)):
        check(f64(q)[rows], f64(out)[rows], f64(lse)[rows], [kv[2]] * len(fit), [1] * len(fit), [share] * len(fit), 128 ** -0.5,
              torch.bfloat16, keys_rounded=rounded)


@pytest.mark.parametrize("bits,dim,dtype,page,share,seqs,group", [
    (8, 128, "fp16", 64, 1024, 300, 2), (4, 256, "fp16", 32, 992, 320, 2), (8, 256, "fp16", 32, 1056, 300, 1), (4, 64, "fp16", 96, 1056, 290, 3),
    (8, 64, "bf16", 32, 992, 300, 5), (4, 128, "bf16", 32, 1056, 300, 4), (8, 128, "bf16", 96, 1056, 300, 1), (4, 256, "bf16", 32, 1056, 290, 2)])
def test_prefix_pass_of_either_type_and_page(bits, dim, dtype, page, share, seqs, group):
    """A prefix that ends inside a step of 64 keys among them; both types."""
    import torch
    cache, batch, _, q, kv, news, lens = prefix_case(bits, dim, dtype, page, share, seqs, group)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = cache.attend(q, batch, lse=lse, shared_tokens=share)
    cache.check()
    check(f64(q), f64(out), f64(lse), kv, news, lens, dim ** -0.5, q.dtype, keys_rounded=True)


@pytest.mark.parametrize("n", [1, 9])
def test_the_longest_sequence(n):
    """2^31 - 32 positions, all on one page of 32: a softmax over that page's tokens, the sum 2^26 - 1 times as large.  The sums
    of equal terms in fp32 are off by up to half a unit of the running sum a term: of 2^30 where a term is 2^14, 2^-8 of it; and
    the tensor core's accumulator by twice that, as it truncates."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pages, group, dim = 2 ** 26 - 1, 8, 64
    cache = attention.KvCache(1, 32, 1, dim, 4)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    kv = fill(cache, np.zeros((1, 1), np.int32), [32])
    batch = attention.KvBatch(table, i32(32 * pages), i32(0, n), n, n)
    q = torch.randn(n, group, dim, device="cuda").bfloat16()
    lse = torch.zeros(n, group, device="cuda")
    out = cache.attend(q, batch, lse=lse)
    cache.check()
    for i in range(n):  # (that the first of them see eight keys less is 2^-28 of the sum)
        want, want_l = ref.attend(f64(q[i:i + 1]), *kv[0], dim ** -0.5, 1)
        assert np.abs(f64(lse[i:i + 1]) - want_l - np.log(pages)).max() <= 2.0 ** -6
        assert np.abs(f64(out[i:i + 1]) - want).max() <= (2.0 ** -6 + 2.0 ** -8) * np.abs(kv[0][1]).max()


@pytest.mark.parametrize("news,lens", [([1] * 5, [1, 40, 700, 33, 9000]), ([2, 1, 7], [5, 300, 64]), ([300, 2, 90], [300, 1000, 2500])])
def test_out_may_be_q(news, lens):
    """In place, on both kernels, with segments that one CTA finishes and such as are joined: the bits of the other call."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    rng = np.random.default_rng(len(lens))
    batch, table, n_pages = make_batch(news, lens, 64, rng, pad_rows=2)
    cache = attention.KvCache(n_pages, 64, 2, 128, 8)
    fill(cache, table, lens)
    q = torch.randn(batch.n_tokens, 8, 128, device="cuda").bfloat16()
    want, x = q.clone(), q.clone()  # (rows behind the last sequence stay q's)
    cache.attend(q, batch, out=want)
    assert cache.attend(x, batch, out=x) is x
    cache.check()
    assert torch.equal(x, want)


def test_out_may_be_q_behind_a_prefix():
    import torch
    cache, batch, _, q, _, _, _ = prefix_case(8, 128, "bf16", 64, 1024, 300, 2)
    want = cache.attend(q, batch, shared_tokens=1024)
    assert torch.equal(cache.attend(q, batch, out=q, shared_tokens=1024), want)
    cache.check()


@pytest.mark.parametrize("shared", [0, 64])
def test_no_tokens(shared):
    """A call without rows does nothing and gives empty results, whatever the sequences hold."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = attention.KvCache(4, 64, 2, 128)
    cache.data.fill_(3)
    batch = attention.KvBatch(i32([0, 1], [2, 3]), i32(100, 0), i32(0, 0, 0), 0)
    x = torch.empty(0, 2, 128, device="cuda").bfloat16()
    q = torch.empty(0, 8, 128, device="cuda").bfloat16()
    cache.append(x, x, batch)
    assert cache.append_norm_rope(q, x, x, batch, None).shape == q.shape
    assert [t.shape for t in cache.read(batch)] == [x.shape] * 2
    assert cache.attend(q, batch, shared_tokens=shared, lse=torch.empty(0, 8, device="cuda")).shape == q.shape
    assert [t.shape for t in attention.qk_norm_rope(q, x, i32(), None)] == [q.shape, x.shape]
    cache.check()
    assert (cache.data == 3).all()
