"""Where top-p cuts does not depend on the launch: a row alone, on eight CTAs, and among many, on one."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def borders(w, per):
    """float32 numbers at and next to the shares of the first `per` prefixes of the weights (in order), each with its neighbours."""
    share = (np.cumsum(w) / w.sum())[:per].astype(np.float32)
    share = share[share < 1]
    return np.concatenate((np.nextafter(share, np.float32(0)), share, np.nextafter(share, np.float32(1))))


@pytest.mark.parametrize("top_k", [420, 0])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_top_p_at_the_borders_alone_and_in_a_batch(top_k, seed):
    """The running sums are integers: wherever top_p's share of the kept mass falls, the same element is the last one kept.  A
    row of 20,000 words alone is spread over eight CTAs and cut from one short list; among 1,200 it has one CTA and goes by
    the histogram of masses.  Nearest float32 numbers to a prefix's share tell sums apart that differ by 2^-30."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import sampling
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(20_000, generator=g) * 2
    w = np.sort(np.exp((z.double() - z.max().double()).numpy()))[::-1]
    p = torch.from_numpy(borders(w[:top_k or None], 400)).cuda()
    n = p.numel()
    rows = z.cuda().expand(n, -1).contiguous()
    u = torch.rand(n, generator=g).cuda()
    k = torch.full((n,), top_k, dtype=torch.int32, device="cuda")
    tok, pr = sampling.sample(rows, u, top_k=k, top_p=p)
    alone = [sampling.sample(rows[i:i + 1], u[i:i + 1], top_k=k[i:i + 1], top_p=p[i:i + 1]) for i in range(n)]
    assert torch.equal(tok, torch.cat([a[0] for a in alone]))
    assert torch.equal(pr, torch.cat([a[1] for a in alone]))


def test_the_cut_follows_top_p():
    """Logits that are multiples of log 2 in fp32 have weights that are powers of two to about 2^-21: a top_p that is 2^-18 above
    or below a prefix's share cuts behind the next element or behind the prefix's own last."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import sampling
    steps = np.repeat(np.arange(12), [1, 3, 2, 5, 1, 7, 30, 2, 64, 100, 3, 9])
    z = torch.from_numpy((-steps * np.log(2.0)).astype(np.float32))
    w = 2.0 ** -steps.astype(np.float64)
    share = np.cumsum(w) / w.sum()
    at = np.arange(len(w) - 1)
    for delta, last in ((-2.0 ** -18, at), (2.0 ** -18, at + 1)):
        p = torch.from_numpy((share[at] + delta).astype(np.float32)).cuda()
        rows = z.cuda().expand(len(at), -1).contiguous()
        u = torch.full((len(at),), 0.99999994, device="cuda")
        tok, pr = sampling.sample(rows, u, top_p=p)
        kept = np.cumsum(w)[last]
        want = np.clip(w[last] / kept, 0, 1)
        # (each share is far above what u leaves over, 2^-24; weights differ from powers of two by what fp32 makes of 11 log 2, 2^-22)
        assert (tok.cpu().numpy() == last).all()
        assert np.allclose(pr.cpu().numpy(), want, rtol=2.0 ** -20)
