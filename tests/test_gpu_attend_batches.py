"""Attention over batches of many sequences: a CTA of either kernel goes through several pieces of work."""
import numpy as np
import pytest

from tests.model_gpu import make_batch
from tests.test_gpu_attend import fill, run_case

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
    fill(cache, table, lens)
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
    got = cache.attend(q, narrow)
    with pytest.raises(moe.MoeError, match="bad page"):
        cache.check()
    for at, seen in ((0, first), (n, max(0, first - 5))):
        rows = got[at:at + n]
        assert rows[seen:].isnan().all()
        # (cut into other parts when shorter: each result within a bf16 step, 2^-8, of the same number)
        assert (rows[:seen].float() - clean[at:at + seen].float()).abs().max() <= 2.0 ** -7 * clean.abs().max() if seen else True
