"""The sequence-side operators without a GPU: page sizes, the rotation table,
refusals of the C calls (each before anything is launched) and of the binding."""
import ctypes as C

import numpy as np
import pytest

from quantized_expert_ffn_gemv_gb300 import build


@pytest.fixture(scope="module")
def moe():
    build.build_cuda()
    from quantized_expert_ffn_gemv_gb300 import moe as m
    return m


INVALID, UNSUPPORTED = 1, 2
ADDR = 1 << 20  # an aligned address that no refused call touches


def test_page_bytes(moe):
    f = moe.lib().moe_kv_page_bytes
    for dim in (64, 128, 256):
        for bits in (8, 4):
            # values and one fp16 scale a block of 32, for K and V
            assert f(64, 3, dim, bits) == 64 * 3 * 2 * (dim * bits // 8 + dim // 32 * 2)
    for bad in ((16, 1, 128, 8), (48, 1, 128, 8), (8192, 1, 128, 8), (64, 0, 128, 8), (64, 1, 96, 8), (64, 1, 128, 6)):
        assert f(*bad) == 0


def test_rope_table_far_positions(moe):
    n, rot, base = 1_000_003, 32, 1e7
    t = np.empty((n, rot // 2, 2), np.float32)
    assert moe.lib().moe_rope_table(n, rot, base, t.ctypes.data) == 0
    import math
    for p in (0, 1, 777_777, 1_000_002):
        for i in (0, 5, 15):
            a = p * base ** (-2.0 * i / rot)
            # half a step of fp32, and the angle's own binary64 rounding (|a| 2^-52, a few roundings)
            tol = 2.0 ** -25 + abs(a) * 2.0 ** -50
            assert abs(t[p, i, 0] - math.cos(a)) <= tol and abs(t[p, i, 1] - math.sin(a)) <= tol
    for bad in ((0, 32, 1e4), (4, 0, 1e4), (4, 24, 1e4), (4, 32, 0.0), (4, 32, float("inf")), (4, 32, float("nan"))):
        assert moe.lib().moe_rope_table(*bad, t.ctypes.data) == INVALID
    assert moe.lib().moe_rope_table(4, 32, 1e4, None) == INVALID


def cache(moe, **kw):
    page = moe.lib().moe_kv_page_bytes(64, 2, 128, 8)
    d = dict(data=ADDR, data_bytes=10 * page, n_pages=10, page_size=64, n_kv_heads=2, head_dim=128, bits=8, status=ADDR)
    d.update(kw)
    return C.byref(moe.KvCacheDesc(**d))


def batch(moe, **kw):
    d = dict(block_table=ADDR, seq_lens=ADDR, cu_tokens=ADDR, n_seqs=3, table_stride=4, max_pages=4, n_tokens=5,
             max_tokens=3)
    d.update(kw)
    return C.byref(moe.KvBatchDesc(**d))


def heads(moe, dim=128, n=2, **kw):
    d = dict(data=ADDR, token_stride=n * dim, head_stride=dim)
    d.update(kw)
    return C.byref((C.c_int64 * 3)(d["data"] or 0, d["token_stride"], d["head_stride"]))  # moe_heads_t


BAD_CACHES = [dict(data=None), dict(data=ADDR + 8), dict(status=None), dict(status=ADDR + 2), dict(n_pages=0), dict(n_pages=11),
              dict(page_size=40), dict(head_dim=96), dict(bits=5), dict(n_kv_heads=0)]
BAD_BATCHES = [dict(block_table=None), dict(seq_lens=None), dict(cu_tokens=None), dict(cu_tokens=ADDR + 1), dict(n_seqs=0),
               dict(n_seqs=65537), dict(table_stride=3), dict(max_pages=0), dict(n_tokens=-1), dict(max_tokens=0),
               dict(max_tokens=6), dict(max_pages=1 << 25, table_stride=1 << 25)]
BAD_HEADS = [dict(data=None), dict(data=ADDR + 8), dict(token_stride=-128), dict(token_stride=260), dict(head_stride=64)]


def test_append_and_read_refuse(moe):
    L = moe.lib()
    h = heads(moe)
    for f in (L.moe_kv_append, L.moe_kv_read):
        for kw in BAD_CACHES:
            assert f(cache(moe, **kw), batch(moe), 0, h, h, None) == INVALID, kw
        for kw in BAD_BATCHES:
            assert f(cache(moe), batch(moe, **kw), 0, h, h, None) == INVALID, kw
        for kw in BAD_HEADS:
            assert f(cache(moe), batch(moe), 0, heads(moe, **kw), h, None) == INVALID, kw
            assert f(cache(moe), batch(moe), 0, h, heads(moe, **kw), None) == INVALID, kw
        assert f(cache(moe), batch(moe), 2, h, h, None) == UNSUPPORTED
        assert f(cache(moe), batch(moe), 3, h, h, None) == INVALID
        assert f(None, batch(moe), 0, h, h, None) == INVALID and f(cache(moe), None, 0, h, h, None) == INVALID
        assert f(cache(moe), batch(moe), 0, None, h, None) == INVALID
        assert f(cache(moe), batch(moe, n_tokens=0, max_tokens=0), 0, h, h, None) == 0  # nothing to do
    # rows of an output may not coincide
    assert L.moe_kv_read(cache(moe), batch(moe), 0, heads(moe, token_stride=0), h, None) == INVALID
    assert L.moe_kv_read(cache(moe), batch(moe), 0, heads(moe, head_stride=0), h, None) == INVALID


def norm(moe, **kw):
    d = dict(q_weight=ADDR, k_weight=ADDR, table=ADDR, n_positions=100, rot_dim=64, interleaved=0, eps=1e-6, weight_offset=0.0)
    d.update(kw)
    return C.byref(moe.NormRope(**d))


def test_norm_rope_refuses(moe):
    L = moe.lib()
    h = heads(moe)

    def call(desc, dtype=0, T=5, dim=128, nq=2, q=h, qo=h, nk=2, k=h, ko=h, pos=ADDR):
        return L.moe_qk_norm_rope(desc, dtype, T, dim, nq, q, qo, nk, k, ko, pos, None)

    bad = [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(weight_offset=float("nan")), dict(q_weight=ADDR + 2),
           dict(k_weight=ADDR + 8), dict(table=None), dict(table=ADDR + 4), dict(n_positions=0), dict(rot_dim=-16),
           dict(rot_dim=24), dict(rot_dim=144)]
    for kw in bad:
        assert call(norm(moe, **kw)) == INVALID, kw
        assert L.moe_kv_append_norm_rope(cache(moe), batch(moe), norm(moe, **kw), 0, 2, h, h, h, h, None, None) == INVALID, kw
    ok = norm(moe)
    assert call(None) == INVALID and call(ok, pos=None) == INVALID and call(ok, pos=ADDR + 1) == INVALID
    assert call(ok, T=-1) == INVALID and call(ok, dim=100) == INVALID and call(ok, dim=264) == INVALID
    assert call(ok, nq=-1) == INVALID and call(ok, nk=-1) == INVALID
    assert call(ok, T=2 ** 31 - 1) == INVALID
    assert call(ok, nq=65535) == UNSUPPORTED and call(ok, nq=1, nk=65535) == UNSUPPORTED
    assert call(ok, dtype=2) == UNSUPPORTED and call(ok, dtype=9) == INVALID
    for kw in BAD_HEADS:
        x = heads(moe, **kw)
        assert call(ok, q=x) == INVALID and call(ok, qo=x) == INVALID and call(ok, k=x) == INVALID and call(ok, ko=x) == INVALID
    assert call(ok, qo=heads(moe, token_stride=0)) == INVALID
    assert call(ok, T=0) == 0 and call(ok, nq=0, nk=0) == 0
    f = L.moe_kv_append_norm_rope
    for kw in BAD_CACHES:
        assert f(cache(moe, **kw), batch(moe), ok, 0, 2, h, h, h, h, None, None) == INVALID, kw
    for kw in BAD_BATCHES:
        assert f(cache(moe), batch(moe, **kw), ok, 0, 2, h, h, h, h, None, None) == INVALID, kw
    assert f(cache(moe), batch(moe), ok, 0, -1, h, h, h, h, None, None) == INVALID
    assert f(cache(moe), batch(moe), ok, 2, 2, h, h, h, h, None, None) == UNSUPPORTED


def test_attend_refuses(moe):
    L = moe.lib()
    h = heads(moe, n=4)

    def call(c=None, b=None, dtype=0, nq=4, q=h, out=h, lse=None, scale=0.1, shared=0, work=ADDR, size=1 << 30):
        return L.moe_kv_attend(c or cache(moe), b or batch(moe), dtype, nq, q, out, lse, scale, shared, work, size, None)

    for kw in BAD_CACHES:
        assert call(c=cache(moe, **kw)) == INVALID, kw
    for kw in BAD_BATCHES:
        assert call(b=batch(moe, **kw)) == INVALID, kw
    assert call(nq=0) == INVALID and call(nq=3) == INVALID and call(nq=-2) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID and call(lse=ADDR + 2) == INVALID
    assert call(shared=-64) == INVALID and call(shared=32) == INVALID and call(shared=5 * 64) == INVALID
    assert call(dtype=2) == UNSUPPORTED and call(dtype=7) == INVALID
    assert call(b=batch(moe, n_tokens=1 << 24, max_tokens=1 << 24)) == UNSUPPORTED
    n = C.c_size_t(5)
    ref = C.byref(n)
    assert L.moe_kv_attend_workspace(cache(moe), batch(moe), 4, 0, None) == INVALID
    assert L.moe_kv_attend_workspace(cache(moe), batch(moe), 3, 0, ref) == INVALID and n.value == 0


def test_sample_refuses(moe):
    L = moe.lib()

    def call(logits=ADDR, dtype=0, rows=4, vocab=1000, stride=1000, u=ADDR, t=None, k=None, p=None, m=None, tok=ADDR, pr=None):
        return L.moe_sample(logits, dtype, rows, vocab, stride, u, t, k, p, m, tok, pr, None)

    for kw in (dict(logits=None), dict(u=None), dict(tok=None), dict(logits=ADDR + 1), dict(dtype=2, logits=ADDR + 2),
               dict(dtype=-1), dict(dtype=3), dict(rows=-1), dict(vocab=0), dict(stride=999), dict(stride=-1), dict(u=ADDR + 2),
               dict(t=ADDR + 1), dict(k=ADDR + 2), dict(p=ADDR + 3), dict(m=ADDR + 2), dict(tok=ADDR + 2), dict(pr=ADDR + 1)):
        assert call(**kw) == INVALID, kw
    assert call(vocab=262145, stride=262145) == UNSUPPORTED
    assert call(rows=0) == 0


def test_binding_refuses_before_the_library(moe, monkeypatch):
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention, sampling
    page = moe.lib().moe_kv_page_bytes(64, 2, 128, 8)

    class Library:  # answers the page size; anything else would be a launch
        moe_kv_page_bytes = moe.lib().moe_kv_page_bytes

        def __getattr__(self, name):
            raise AssertionError(name + " was called")

    attention._native()  # the extension module holds the library's addresses; it declines all of what follows
    monkeypatch.setattr(moe, "lib", lambda: Library())
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    with pytest.raises(ValueError):  # host tensors
        attention.KvBatch(z(2, 4, dt=torch.int32), z(2, dt=torch.int32), z(3, dt=torch.int32), 2)
    with pytest.raises(ValueError):
        attention.KvBatch(z(2, 4, dt=torch.int64), z(2, dt=torch.int32), z(3, dt=torch.int32), 2)
    with pytest.raises(ValueError):
        attention.KvCache(4, 64, 2, 128, data=z(4 * page, dt=torch.uint8))
    with pytest.raises(ValueError):
        attention.KvCache(4, 48, 2, 128)
    with pytest.raises(ValueError):
        attention.qk_norm_rope(z(3, 4, 128), z(3, 2, 128), None, None)
    with pytest.raises(ValueError):
        sampling.sample(z(2, 100), z(2, dt=torch.float32))
    with pytest.raises(ValueError):
        sampling.sample(z(100), z(1, dt=torch.float32))
    c = attention.KvCache.__new__(attention.KvCache)
    c.n_kv_heads, c.head_dim, c.dev = 2, 128, -1
    c.desc, c.data = moe.KvCacheDesc(n_kv_heads=2, head_dim=128), z(16, dt=torch.uint8)
    c._at = C.addressof(c.desc)
    b = attention.KvBatch.__new__(attention.KvBatch)
    b.n_tokens, b.dev = 3, -1
    b.desc = moe.KvBatchDesc(n_tokens=3)
    b._at = C.addressof(b.desc)
    good = z(3, 2, 128)
    bad = [z(2, 2, 128), z(3, 4, 128), z(3, 2, 64), z(3, 2, 128, dt=torch.float16), z(3, 128, 2).transpose(1, 2), z(3, 2, 132)[..., 4:]]
    for x in bad:
        with pytest.raises(ValueError):
            c.append(x, good, b)
        with pytest.raises(ValueError):
            c.append_norm_rope(good, x, good, b, None)
        with pytest.raises(ValueError):
            c.append(good, x, b)
    for x in (z(2, 4, 128), z(3, 4, 64), z(3, 128), z(3, 4, 128, dt=torch.float32), z(3, 4, 132)[..., 4:]):
        with pytest.raises(ValueError):
            c.attend(x, b)
    with pytest.raises(ValueError):
        c.attend(good, b, lse=z(3, 2))
    with pytest.raises(ValueError):
        c.append(z(3, 2, 128, dt=torch.float32), z(3, 2, 128, dt=torch.float32), b)


def test_reference_forms_agree_with_closed_forms():
    """The tests' own binary64 forms: uniform attention is a mean, a rotation keeps norms, greedy is argmax."""
    from tests import model_ref as ref
    rng = np.random.default_rng(0)
    v = rng.standard_normal((5, 1, 64))
    o, lse = ref.attend(np.zeros((2, 3, 64)), rng.standard_normal((5, 1, 64)), v, 1.0, 2)
    assert np.allclose(o[0], v[:4, 0].mean(0)) and np.allclose(o[1], v[:, 0].mean(0)) and np.allclose(lse[1], np.log(5))
    x = rng.standard_normal((2, 3, 64))
    t = np.stack((np.cos(rng.random((4, 16))), np.zeros((4, 16))), -1)
    t[..., 1] = np.sqrt(1 - t[..., 0] ** 2)
    for inter in (False, True):
        y = ref.rms_rope(x, None, 0.0, 0.0, t, np.array([3, 1]), inter)
        assert np.allclose((y * y).mean(-1), 1.0)
    z = rng.standard_normal(50)
    assert ref.sample(z, 0.3, temperature=0.0)[0] == z.argmax()
    assert ref.sample(z, 0.999, top_k=2)[2] == sorted(np.argsort(-z)[:2].tolist())
    h = ref.held(rng.standard_normal((4, 64)), 8)
    assert np.isfinite(h).all()
