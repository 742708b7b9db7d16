"""Sampling against binary64: the kept set's borders, ties, filters, odd rows."""
import numpy as np
import pytest

from tests import model_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    import torch
    torch.manual_seed(0)

TYPES = ["fp32", "bf16", "fp16"]


def dt(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[name]


def run(z, u, temperature=None, top_k=None, top_p=None, min_p=None, **kw):
    import torch
    from quantized_expert_ffn_gemv_gb300 import sampling
    n = z.shape[0]
    f = lambda v, t: None if v is None else torch.as_tensor(np.broadcast_to(np.asarray(v), (n,)).copy()).to(t).cuda()
    tok, p = sampling.sample(z.cuda() if z.device.type == "cpu" else z, f(u, torch.float32), f(temperature, torch.float32),
                             f(top_k, torch.int32), f(top_p, torch.float32), f(min_p, torch.float32), **kw)
    return tok.cpu().numpy(), p.cpu().numpy().astype(np.float64)


def logits(rows, vocab, name, seed, spread=2.0, lead=30):
    import torch
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * spread
    idx = torch.randint(0, vocab, (rows, min(lead, vocab)), generator=g)
    z.scatter_(1, idx, 8 + 2 * torch.randn(idx.shape, generator=g))
    return z.to(dt(name))


def f32(v):
    return float(np.float32(v))


def against(z, u, temperature, top_k, top_p, min_p):
    """Equal tokens, except where u lies within 2^-28 of a border of the running sum (the sums are exact to about 2^-31 a
    weight); probabilities to 2^-22 (a fp32 quotient of rounded operands)."""
    n = z.shape[0]
    tok, p = run(z, u, temperature, top_k, top_p, min_p)
    z64 = z.double().numpy()
    b = lambda v: np.broadcast_to(np.asarray(v), (n,))
    u, temperature, top_k, top_p, min_p = (b(v) for v in (u, temperature, top_k, top_p, min_p))
    for r in range(n):
        args = (f32(temperature[r]), int(top_k[r]), f32(top_p[r]), f32(min_p[r]))
        lo, hi = (ref.sample(z64[r], max(0.0, f32(u[r]) + e), *args)[0] for e in (-2.0 ** -28, 2.0 ** -28))
        want, prob, kept = ref.sample(z64[r], f32(u[r]), *args)
        assert tok[r] in (want, lo, hi), (r, tok[r], want)
        if tok[r] == want:
            assert abs(p[r] - prob) <= 2.0 ** -22 * prob + 2.0 ** -60, (r, p[r], prob)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 4097, 32000, 100_003, 262_144])
def test_plain_and_filtered(vocab, name):
    rng = np.random.default_rng(vocab)
    z = logits(6, vocab, name, vocab)
    u = rng.random(6)
    against(z, u, 1.0, 0, 1.0, 0.0)
    against(z, u, [0.3, 0.7, 1.0, 1.5, 3.0, 1.0], [0, 5, 50, 0, 1000, 2], [0.9, 0.5, 1.0, 0.99, 0.95, 0.999], [0, 0.1, 0.02, 0, 0.3, 0])


@pytest.mark.parametrize("rows", [1, 3, 77, 200])
def test_row_counts(rows):
    rng = np.random.default_rng(rows)
    z = logits(rows, 5003, "fp32", rows)
    against(z, rng.random(rows), rng.uniform(0.2, 2.0, rows), rng.choice([0, 1, 3, 40], rows), rng.choice([1.0, 0.3, 0.9], rows),
            rng.choice([0.0, 0.05], rows))


@pytest.mark.parametrize("top_k,top_p", [(0, 0.4), (0, 0.97), (7, 1.0), (5000, 1.0), (900, 0.6), (19_999, 1.0)])
def test_ties_are_cut_by_index(top_k, top_p):
    """All logits equal, a few values only, and two values: the kept set is decided by the index within a value."""
    import torch
    g = torch.Generator().manual_seed(1)
    n = 20_000
    rows = [torch.zeros(n), torch.randint(0, 4, (n,), generator=g).float(), torch.where(torch.rand(n, generator=g) < 0.001, 3.0, -1.0)]
    z = torch.stack(rows)
    for name in TYPES:
        for u in (0.0, 0.37, 0.9999999):
            against(z.to(dt(name)), u, 1.0, top_k, top_p, 0.0)


def test_flat_bulk_cuts_inside_a_crowded_bin():
    """Broad rows whose cut falls among thousands of nearly equal logits (the finer histograms run)."""
    import torch
    g = torch.Generator().manual_seed(3)
    z = torch.randn(4, 150_000, generator=g) * torch.tensor([[0.01], [0.3], [1.0], [1e-4]])
    for top_k, top_p in ((60_000, 1.0), (0, 0.5), (75_001, 0.7), (149_999, 1.0)):
        against(z, [0.1, 0.5, 0.9, 0.99], 1.0, top_k, top_p, 0.0)


def test_every_token_of_a_small_row_is_hit_in_its_interval():
    """u in the middle of each kept token's interval gives that token: the whole inverse distribution."""
    z = logits(1, 40, "fp32", 5)
    z64 = z.double().numpy()[0]
    for args in ((1.0, 0, 1.0, 0.0), (0.5, 12, 1.0, 0.0), (1.3, 0, 0.8, 0.0), (1.0, 0, 1.0, 0.05), (2.0, 20, 0.9, 0.1)):
        _, _, kept = ref.sample(z64, 0.0, *[f32(a) if i != 1 else a for i, a in enumerate(args)])
        w = np.exp((z64[kept] - z64.max()) / f32(args[0]))
        cum = np.cumsum(w) / w.sum()
        mids = cum - w / w.sum() / 2
        tok, p = run(z.expand(len(kept), 40).contiguous(), mids, *args)
        assert tok.tolist() == kept
        assert np.allclose(p, w / w.sum(), rtol=2 ** -22)


def test_greedy_and_parameters_that_mean_off():
    z = logits(4, 3000, "bf16", 8)
    z[0, 5] = z[0, 2999] = z[0].max() + 1
    best = z.double().numpy().argmax(1)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=nan), dict(top_k=1), dict(top_p=0.0),
               dict(top_p=-1.0), dict(min_p=1.5)):
        tok, p = run(z, 0.77, **kw)
        assert tok.tolist() == best.tolist() and (p == 1).all(), kw
    plain = run(z, 0.77)
    for kw in (dict(top_k=0), dict(top_k=-3), dict(top_k=3000), dict(top_k=99999), dict(top_p=1.0), dict(top_p=2.0), dict(top_p=nan),
               dict(min_p=0.0), dict(min_p=-1.0), dict(min_p=nan), dict(temperature=1.0)):
        got = run(z, 0.77, **kw)
        assert got[0].tolist() == plain[0].tolist() and got[1].tolist() == plain[1].tolist(), kw
    # u is clamped
    assert run(z, nan)[0].tolist() == run(z, 0.0)[0].tolist() == run(z, -1.0)[0].tolist()
    assert run(z, 1.0)[0].tolist() == run(z, inf)[0].tolist() == run(z, 0.99999994)[0].tolist()
    # an infinite temperature is uniform
    tok, p = run(z, 0.5, temperature=inf)
    assert tok.tolist() == [1500] * 4 and np.allclose(p, 1 / 3000, rtol=1e-6)
    # min_p = 1 keeps the ties of the maximum
    assert run(z[:1], 0.6, min_p=1.0)[0].tolist() == [2999] and run(z[:1], 0.4, min_p=1.0)[0].tolist() == [5]


def test_infinities_nan_and_empty_rows():
    import torch
    inf, nan = float("inf"), float("nan")
    z = torch.randn(8, 700)
    z[0, :] = -inf
    z[1, :] = nan
    z[2, 1:] = -inf
    z[3, :650] = -inf
    z[4, [3, 90, 500]] = inf
    z[5, ::2] = nan
    z[6, :] = -inf
    z[6, 699] = -3e38
    z[7, :] = torch.finfo(torch.float32).min
    z[7, 10] = 5.0
    u = np.array([0.5, 0.5, 0.9, 0.9, 0.5, 0.2, 0.3, 0.99])
    for kw in (dict(), dict(top_k=60), dict(top_p=0.9), dict(min_p=0.01), dict(top_k=300, top_p=0.7, temperature=0.8)):
        tok, p = run(z, u, **kw)
        assert tok[0] == tok[1] == -1 and p[0] == p[1] == 0
        full = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, **kw}
        for r in range(2, 8):
            want = ref.sample(z[r].double().numpy(), f32(u[r]), f32(full["temperature"]), full["top_k"], f32(full["top_p"]), f32(full["min_p"]))
            assert tok[r] == want[0], (r, kw)
    assert run(z[4:5], 0.5)[0][0] == 90


@pytest.mark.parametrize("name", TYPES)
def test_rows_at_any_alignment_and_stride(name):
    import torch
    base = logits(5, 9001, name, 11).cuda()
    wide = torch.full((5, 9050), 50.0).to(dt(name)).cuda()
    u = [0.1, 0.3, 0.5, 0.7, 0.9]
    want = run(base, u, top_p=0.9)
    for off in (0, 1, 3, 7, 13):
        wide[:, off:off + 9001] = base
        got = run(wide[:, off:off + 9001], u, top_p=0.9)
        assert got[0].tolist() == want[0].tolist() and got[1].tolist() == want[1].tolist()
        wide.fill_(50.0)


def test_low_temperatures():
    """Most weights vanish; the far end of the histogram collects them."""
    z = logits(5, 50_000, "fp32", 21)
    against(z, [0.0, 0.2, 0.5, 0.8, 0.99], [1e-3, 0.01, 0.05, 0.1, 1e-30], 0, 0.95, 0.0)
    against(z, [0.0, 0.2, 0.5, 0.8, 0.99], [0.02, 0.01, 0.05, 0.1, 0.2], 30_000, 1.0, 0.0)


def test_graph_streams_and_repeat():
    import torch
    from quantized_expert_ffn_gemv_gb300 import sampling
    z = logits(9, 30_001, "fp32", 4).cuda()
    u = torch.rand(9).cuda()
    p = torch.full((9,), 0.9).cuda()
    tok = torch.zeros(9, dtype=torch.int32).cuda()
    pr = torch.zeros(9).cuda()
    want = sampling.sample(z, u, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = sampling.sample(z, u, top_p=p, stream=s)
    s.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        sampling.sample(z, u, top_p=p, tokens=tok, probs=pr)
    u.copy_(torch.rand(9))
    g.replay()
    torch.cuda.synchronize()
    again = sampling.sample(z, u, top_p=p)
    assert torch.equal(tok, again[0]) and torch.equal(pr, again[1])
