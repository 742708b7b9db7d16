"""The sequence-side operators as a model runs them: prefill, then decode steps of one layer around the MoE layer, eager and captured."""
import numpy as np
import pytest

from quantized_expert_ffn_gemv_gb300 import synth
from tests import model_ref as ref
from tests.gpu_common import make_gpu_layer
from tests.model_gpu import f64
from tests.test_gpu_attend import check
from tests.test_gpu_kv import rope_close
from tests.test_gpu_sample import against

pytestmark = pytest.mark.gpu

HQ, HKV, D, VOCAB, PAGE, EPS = 8, 2, 128, 5000, 64, 1e-6
PROMPTS = [37, 1, 130, 64]
KNOBS = dict(temperature=[0.8, 1.0, 0.0, 1.3], top_k=[0, 40, 0, 5], top_p=[0.9, 1.0, 1.0, 0.8], min_p=[0.0, 0.05, 0.0, 0.0])


class Model:
    """One pre-norm layer, an embedding that is also the head, and the state of four sequences."""

    def __init__(self, bits):
        import torch
        from quantized_expert_ffn_gemv_gb300 import attention
        g = torch.Generator().manual_seed(7)
        shape = synth.SMALL
        rand = lambda *s, mul=1.0: (torch.randn(*s, generator=g) * mul).bfloat16().cuda()
        self.H = shape.H
        self.emb = rand(VOCAB, self.H)
        self.w_qkv = rand(self.H, (HQ + 2 * HKV) * D, mul=self.H ** -0.5)
        self.w_o = rand(HQ * D, self.H, mul=(HQ * D) ** -0.5)
        self.wq, self.wk = rand(D, mul=0.1) + 1, rand(D, mul=0.1) + 1
        self.table = attention.rope_table(512, D, 1e6)
        self.layer = make_gpu_layer(synth.make_layer(shape), max_tokens=sum(PROMPTS))
        pages = 4
        self.cache = attention.KvCache(pages * len(PROMPTS), PAGE, HKV, D, bits)
        self.pages = torch.randperm(pages * len(PROMPTS), generator=g).view(len(PROMPTS), pages).int().cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.lens = i32(PROMPTS)
        cu = np.concatenate(([0], np.cumsum(PROMPTS))).tolist()
        self.prefill = attention.KvBatch(self.pages, self.lens, i32(cu), cu[-1], max(PROMPTS))
        self.decode = attention.KvBatch(self.pages, self.lens, i32(list(range(len(PROMPTS) + 1))), len(PROMPTS), 1)
        self.last = torch.tensor(cu[1:], device="cuda") - 1
        self.knobs = [torch.tensor(KNOBS[n], dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda") for n in KNOBS]

    def step(self, ids, batch, u, rows=None):
        """Returns (token, probability, what was seen on the way); rows: the tokens that are sampled from."""
        import torch
        from quantized_expert_ffn_gemv_gb300 import moe, sampling
        x = self.emb[ids]
        T = x.shape[0]
        new = lambda: torch.empty_like(x)
        xhat, x1, xhat1, x2, xhat2 = new(), new(), new(), new(), new()
        moe.residual_rmsnorm(x, None, EPS, None, xhat)
        qkv = (xhat @ self.w_qkv).view(T, HQ + 2 * HKV, D)
        raw, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        q = self.cache.append_norm_rope(raw, k, v, batch, self.table, self.wq, self.wk, eps=EPS)
        o = self.cache.attend(q, batch)
        moe.residual_rmsnorm(x, o.reshape(T, HQ * D) @ self.w_o, EPS, x1, xhat1)
        moe.residual_rmsnorm(x1, self.layer.forward(xhat1), EPS, x2, xhat2)
        logits = (xhat2 if rows is None else xhat2[rows]) @ self.emb.T / 8
        token, p = sampling.sample(logits, u, *self.knobs)
        return token, p, dict(raw=raw, k=k, v=v, q=q, o=o, logits=logits)


@pytest.mark.parametrize("bits", [8, 4])
def test_prefill_and_decode_steps(bits):
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    m = Model(bits)
    rng = np.random.default_rng(bits)
    ids = torch.from_numpy(rng.integers(0, VOCAB, sum(PROMPTS))).cuda()
    lens, kv = [0] * len(PROMPTS), [(np.zeros((0, HKV, D)),) * 2 for _ in PROMPTS]
    batch, news, rows = m.prefill, PROMPTS, m.last
    for step in range(4):
        u = rng.random(len(PROMPTS)).astype(np.float32)
        token, p, seen = m.step(ids, batch, torch.from_numpy(u).cuda(), rows)
        m.cache.check()
        pos = np.concatenate([lens[b] + np.arange(n) for b, n in enumerate(news)])
        want = ref.rms_rope(f64(seen["raw"]), f64(m.wq), 0.0, EPS, m.table.cpu().numpy(), pos, False)
        big = np.abs(ref.rms_rope(f64(seen["raw"]), f64(m.wq), 0.0, EPS, None, None, False)).max(-1, keepdims=True)
        rope_close(f64(seen["q"]), want, big, torch.bfloat16)
        _, kn = attention.qk_norm_rope(seen["raw"], seen["k"], torch.from_numpy(pos.astype(np.int32)).cuda(), m.table, m.wq, m.wk, eps=EPS)
        hk, hv = ref.held(f64(kn), bits), ref.held(f64(seen["v"]), bits)
        at = 0
        for b, n in enumerate(news):
            kv[b] = (np.concatenate((kv[b][0], hk[at:at + n])), np.concatenate((kv[b][1], hv[at:at + n])))
            lens[b] += n
            at += n
        lse = torch.empty(seen["q"].shape[:2], device="cuda")
        again = m.cache.attend(seen["q"], batch, lse=lse)
        assert torch.equal(again, seen["o"])
        check(f64(seen["q"]), f64(seen["o"]), f64(lse), kv, news, lens, D ** -0.5, torch.bfloat16)
        against(seen["logits"].cpu(), u, *(KNOBS[n] for n in ("temperature", "top_k", "top_p", "min_p")))
        z = seen["logits"].double().cpu().numpy()
        assert int(token[2]) == z[2].argmax() and float(p[2]) == 1.0  # the greedy one
        ids, batch, news, rows = token.long(), m.decode, [1] * len(PROMPTS), None
        m.lens.add_(1)


def test_captured_decode_loop_equals_the_eager_one():
    """One captured step that takes its own last tokens, replayed, gives the eager loop's tokens."""
    import torch
    rng = np.random.default_rng(3)
    ids = torch.from_numpy(rng.integers(0, VOCAB, sum(PROMPTS))).cuda()
    us = torch.from_numpy(rng.random((7, len(PROMPTS))).astype(np.float32)).cuda()
    m = Model(8)
    first = m.step(ids, m.prefill, us[0], m.last)[0]
    start, data = m.lens.clone(), m.cache.data.clone()
    eager, token = [], first
    for i in range(1, 7):
        m.lens.add_(1)
        token = m.step(token.long(), m.decode, us[i])[0]
        eager.append(token.clone())
    m.lens.copy_(start)
    m.cache.data.copy_(data)
    cur, u = first.clone(), us[1].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.lens.add_(1)
        cur.copy_(m.step(cur.long(), m.decode, u)[0])
    for i in range(1, 7):
        u.copy_(us[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(cur, eager[i - 1]), i
    m.cache.check()
    assert (m.lens == start + 6).all()
