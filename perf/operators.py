"""The sequence-side operators of a decode step, as they are timed: per-head
norm + rotation of queries and keys, the quantised paged cache (written and
read back), attention over that cache, and sampling.

``run`` makes one pass: with ``own`` false in elementary torch operations,
with ``own`` true through the package's public calls.  The cache's pages are
bytes of the layout that include/moe_model.h documents, so both forms read and
write the same pool.
"""
import math

import torch

own = False
DEVICE = "cuda"
EPS = 1e-6

def _package():
    from quantized_expert_ffn_gemv_gb300 import attention, sampling
    return attention, sampling


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user, one token: a single decode step's q and k straight from the projection (latency)
        dict(name="rope decode 1", kind="rope", tokens=1, q_heads=32, kv_heads=4, dim=128, rot=128, inter=False, dtype="bf16",
             weight=0.0),
        # a prefill chunk of 4,096 tokens, partial rotation of wide heads, zero-centred norm weights
        dict(name="rope chunk 4096", kind="rope", tokens=4096, q_heads=16, kv_heads=2, dim=256, rot=64, inter=False,
             dtype="bf16", weight=1.0),
        # a ragged batch of 61 sequences written to the cache in the pass that normalises and rotates (interleaved pairs, fp16)
        dict(name="rope store ragged", kind="store", seqs=61, tokens=2387, q_heads=24, kv_heads=8, dim=128, rot=96, inter=True,
             dtype="fp16", weight=0.0, page=64, bits=8, history=500),
        # batched decode: each of 256 sequences appends one token, and reads it back
        dict(name="cache 8-bit decode", kind="cache", seqs=256, tokens=256, kv_heads=4, dim=128, dtype="bf16", page=64, bits=8,
             history=300, back="new"),
        # prefix reuse: a 1,000-token chunk is appended and the whole 33,000-token history comes back for a dense prefill
        dict(name="cache 4-bit history", kind="cache", seqs=2, tokens=2000, kv_heads=8, dim=128, dtype="bf16", page=128, bits=4,
             history=32001, back="all"),
        # one user, 1,000 tokens of context, one new token (latency)
        dict(name="attend decode 1", kind="attend", seqs=1, per_seq=1, shortest=1000, longest=1000, q_heads=32, kv_heads=4, dim=128,
             dtype="bf16", page=64, bits=8, shared=0),
        # a serving batch of 64 very unequal contexts, one token each
        dict(name="attend decode ragged", kind="attend", seqs=64, per_seq=1, shortest=1, longest=24001, q_heads=32, kv_heads=4,
             dim=128, dtype="bf16", page=64, bits=8, shared=0),
        # long contexts in 4 bits, wide heads, 4 tokens checked at once (speculation)
        dict(name="attend 4-bit long", kind="attend", seqs=12, per_seq=4, shortest=60000, longest=131072, q_heads=16, kv_heads=2,
             dim=256, dtype="bf16", page=128, bits=4, shared=0),
        # 48 requests behind one 16k system prompt
        dict(name="attend shared prefix", kind="attend", seqs=48, per_seq=1, shortest=16500, longest=17400, q_heads=32, kv_heads=4,
             dim=128, dtype="bf16", page=64, bits=8, shared=16384),
        # a prefill chunk of 2,048 tokens behind 6,144 cached ones
        dict(name="attend chunk 2048", kind="attend", seqs=1, per_seq=2048, shortest=8192, longest=8192, q_heads=32, kv_heads=4,
             dim=128, dtype="bf16", page=64, bits=8, shared=0),
        # one user's next token from a 151,552-word vocabulary (latency)
        dict(name="sample 1", kind="sample", rows=1, vocab=151552, dtype="bf16", temperature=0.8, top_k=50, top_p=0.95, min_p=0.0,
             mixed=False),
        # a serving batch whose requests each bring their own settings, greedy ones among them
        dict(name="sample 256 mixed", kind="sample", rows=256, vocab=151552, dtype="fp32", temperature=1.0, top_k=0, top_p=0.9,
             min_p=0.02, mixed=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "store", "cache", "attend", "attend", "attend", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    if kind == "rope":
        return dict(kind=kind, tokens=_log_int(rng, 1, 4000), q_heads=kv * group, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4]), inter=rng.random() < 0.3, dtype=dtype, weight=rng.choice([0.0, 1.0]))
    if kind == "store":
        seqs = _log_int(rng, 1, 100)
        return dict(kind=kind, seqs=seqs, tokens=seqs + _log_int(rng, 1, 2000), q_heads=kv * group, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4]), inter=rng.random() < 0.3, dtype=dtype, weight=rng.choice([0.0, 1.0]),
                    page=rng.choice([32, 64, 128]), bits=8, history=_log_int(rng, 1, 2000))
    if kind == "cache":
        seqs = _log_int(rng, 1, 128)
        return dict(kind=kind, seqs=seqs, tokens=seqs + _log_int(rng, 1, 2000), kv_heads=kv, dim=dim, dtype=dtype,
                    page=rng.choice([32, 64, 128]), bits=rng.choice([4, 8]), history=_log_int(rng, 1, max(2, 30000 // seqs)),
                    back=rng.choice(["new", "all"]))
    if kind == "attend":
        form = rng.choice(["decode", "few", "chunk", "shared"])
        seqs = 1 if form == "chunk" else _log_int(rng, 2 if form == "shared" else 1, 48)
        per = 1 if form in ("decode", "shared") else rng.choice([2, 3, 4, 5]) if form == "few" else _log_int(rng, 65, 1500)
        page = rng.choice([32, 64, 128])
        longest = _log_int(rng, per + 1, 6000) if form == "chunk" else _log_int(rng, 64, 500000 // seqs // kv)
        longest = max(longest, per)
        shared = 0
        if form == "shared":
            longest = max(longest, 2 * page)
            shared = page * rng.randint(1, longest // page - 1)
        shortest = max(per, shared, int(longest * rng.random() ** 2))
        return dict(kind=kind, seqs=seqs, per_seq=per, shortest=shortest, longest=longest, q_heads=kv * group, kv_heads=kv, dim=dim,
                    dtype=dtype, page=page, bits=rng.choice([4, 8]), shared=shared)
    return dict(kind="sample", rows=_log_int(rng, 1, 200), vocab=_log_int(rng, 1000, 150000), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                temperature=round(rng.uniform(0.3, 1.5), 2), top_k=rng.choice([0, 0, 1, 20, 100, 1000]),
                top_p=rng.choice([1.0, 0.5, 0.9, 0.95]), min_p=rng.choice([0.0, 0.0, 0.05, 0.1]), mixed=rng.random() < 0.5)


_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _lengths(case):
    """The sequences' cached lengths: spread over the logarithm from the shortest to the longest."""
    n, a, b = case["seqs"], case["shortest"], case["longest"]
    return [b] if n == 1 else [max(a, min(b, int(round(a * (b / a) ** (i / (n - 1)))))) for i in range(n)]


def _news(case):
    """New tokens of each sequence of a ragged append: every one has one at least, the rest grow along the batch."""
    n, total = case["seqs"], case["tokens"]
    extra, tri = total - n, n * (n + 1) // 2
    ends = [extra * ((i + 1) * (i + 2) // 2) // tri for i in range(n)]
    return [1 + e - b for e, b in zip(ends, [0] + ends[:-1])]


def work(case):
    k = case["kind"]
    if k == "rope":
        rows = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        n = rows * case["dim"]
        return {"bytes": 4 * n + case["tokens"] * (4 * case["rot"] + 4), "flops": 8 * n}
    if k == "store":
        t, d = case["tokens"], case["dim"]
        nq, nk = t * case["q_heads"] * d, t * case["kv_heads"] * d
        held = 2 * nk * (case["bits"] / 8 + 1 / 16)
        # q in and out, k and v in, the cache's bytes out, and these read back as values
        return {"bytes": 4 * nq + 4 * nk + held + (held + 4 * nk) + 4 * t * case["rot"], "flops": 8 * (nq + nk)}
    if k == "cache":
        d, heads = case["dim"], case["kv_heads"]
        new = case["tokens"]
        back = new if case["back"] == "new" else new + case["seqs"] * case["history"]
        held = 2 * heads * d * (case["bits"] / 8 + 1 / 16)
        return {"bytes": new * (4 * heads * d + held) + back * (4 * heads * d + held), "flops": 4 * heads * d * (new + back)}
    if k == "attend":
        lens, per, d = _lengths(case), case["per_seq"], case["dim"]
        held = 2 * case["kv_heads"] * d * (case["bits"] / 8 + 1 / 16)
        tokens = case["shared"] + sum(x - case["shared"] for x in lens)
        pairs = sum(per * x - per * (per - 1) // 2 for x in lens)
        return {"bytes": tokens * held + 4 * case["seqs"] * per * case["q_heads"] * d, "flops": 4 * pairs * case["q_heads"] * d}
    return {"bytes": case["rows"] * case["vocab"] * (4 if case["dtype"] == "fp32" else 2), "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------ the cache's pages
# pool: uint8 [pages][kv head][page / 32][tile]; a tile holds 32 tokens of one head:
#   K values [32][R]  K scales fp16 [D/32][32]  V values [32][R]  V scales fp16 [D/32][32]        (R = D * bits / 8 bytes)
# value row r's 16-byte chunk c is stored at chunk c ^ (f(r) & (R / 16 - 1)), f(r) = ((r >> 2 ^ r) & 1) << 2 | (r & 2) | (r >> 2 & 1).

def _row_bytes(dim, bits):
    return dim * bits // 8


def _tile_bytes(dim, bits):
    return 2 * (32 * _row_bytes(dim, bits) + 2 * dim)


def _value_offsets(dim, bits, device):
    """Byte j of row r within a tile's value plane, [32][R]."""
    R = _row_bytes(dim, bits)
    r = torch.arange(32, device=device)[:, None]
    j = torch.arange(R, device=device)[None, :]
    turn = ((((r >> 2) ^ r) & 1) << 2 | (r & 2) | (r >> 2) & 1) & (R // 16 - 1)
    return r * R + (((j >> 4) ^ turn) << 4) + (j & 15)


def _quantise(x, bits):
    """x [..., D] in 32 bits: the bytes that hold it [..., R], and the fp16 scales [..., D / 32]."""
    top, low = (127, -127) if bits == 8 else (7, -8)
    b = x.reshape(*x.shape[:-1], -1, 32)
    d = (b.abs().amax(-1) / top).half()
    d = torch.where(torch.isfinite(d), d, torch.full_like(d, math.nan))
    f = d.float()[..., None]
    q = torch.where(f > 0, torch.clamp(torch.round(b / f), low, top), torch.zeros_like(b))
    u = (q + (128 if bits == 8 else 8)).to(torch.uint8).reshape(x.shape)
    return (u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)), d


def _values(raw, scales, bits):
    """bytes [..., R] and scales [..., D / 32] -> values in 32 bits [..., D]."""
    if bits == 8:
        q = raw.float() - 128
    else:
        q = (torch.stack((raw & 15, raw >> 4), -1).flatten(-2)).float() - 8
    return q * scales.float().repeat_interleave(32, -1)


def _put(state, k, v, rows):
    """Quantise k and v [N][heads][D] and write them at (page, tile, row) of the pool."""
    pool, dim, bits = state["pool"], state["dim"], state["bits"]
    R, nb = _row_bytes(dim, bits), dim // 32
    at = _value_offsets(dim, bits, pool.device)
    page, tile, row = (x[:, None, None] for x in rows)
    head = torch.arange(k.shape[1], device=pool.device)[None, :, None]
    halves = pool.view(torch.float16)
    block = torch.arange(nb, device=pool.device)[None, None, :]
    for x, base in ((k, 0), (v, 32 * R + 2 * dim)):
        raw, d = _quantise(x.float(), bits)
        pool[page, head, tile, base + at[row[:, 0, 0]][:, None, :]] = raw
        halves[page, head, tile, (base + 32 * R) // 2 + block * 32 + row] = d


def _get(state, pages):
    """The values held by `pages` [...]: K and V in 32 bits [..., page size, heads, D]."""
    dim, bits = state["dim"], state["bits"]
    R, nb = _row_bytes(dim, bits), dim // 32
    tiles = state["pool"][pages]  # [..., heads, tiles, bytes]
    at = _value_offsets(dim, bits, tiles.device).reshape(-1)
    halves = tiles.view(torch.float16)
    ks = halves[..., 16 * R:16 * R + dim].unflatten(-1, (nb, 32)).transpose(-1, -2)
    vs = halves[..., 32 * R + dim:32 * R + 2 * dim].unflatten(-1, (nb, 32)).transpose(-1, -2)
    k = _values(tiles[..., :32 * R][..., at].unflatten(-1, (32, R)), ks, bits)
    v = _values(tiles[..., 32 * R + 2 * dim:64 * R + 2 * dim][..., at].unflatten(-1, (32, R)), vs, bits)
    return tuple(x.flatten(-3, -2).transpose(-3, -2) for x in (k, v))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, mul=1.0):
    return (torch.randn(*shape, device=DEVICE, generator=g) * mul).to(dtype)


def _table(positions, rot):
    """cos and sin of position * 10^6^(-2 i / rot), the angles in 64 bits: fp32 [positions][rot / 2][2]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEVICE)
    a = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * torch.exp(-math.log(1e6) * 2 * i / rot)
    return torch.stack((torch.cos(a), torch.sin(a)), -1).float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _cumulative(v):
    return [0] + [sum(v[:i + 1]) for i in range(len(v))]


def _paged(state, case, g, lens, shared=0):
    """A pool whose pages belong to the sequences in mixed order, filled with what was appended before."""
    page, dim, bits, heads = case["page"], case["dim"], case["bits"], case["kv_heads"]
    need = [-(-x // page) for x in lens]
    common = shared // page
    count = sum(x - common for x in need) + common + 1
    order = torch.randperm(count, generator=g, device=DEVICE).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEVICE)
    at = common
    for i, n in enumerate(need):
        table[i, :common] = order[:common]
        table[i, common:n] = order[at:at + n - common]
        at += n - common
    state.update(dim=dim, bits=bits, page=page, heads=heads, pages=count, table=table, lens=_ints(lens), max_len=max(lens))
    state["pool"] = torch.zeros(count, heads, page // 32, _tile_bytes(dim, bits), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 25) // (page * heads * dim))
    for a in range(0, count, step):  # whole pages, a part at a time
        n = min(step, count - a) * page
        slot = torch.arange(a * page, a * page + n, device=DEVICE)
        k = _randn(g, n, heads, dim, dtype=torch.bfloat16)
        v = _randn(g, n, heads, dim, dtype=torch.bfloat16)
        _put(state, k, v, (slot // page, slot % page // 32, slot % 32))


def _places(state, cu, lens, tokens):
    """(page, tile, row) and sequence and position of each new token."""
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = lens.long()[seq] - cu.long()[seq + 1] + t
    page = state["table"].long()[seq, pos // state["page"]]
    off = pos % state["page"]
    return (page, off // 32, off % 32), seq, pos


def prepare(case, seed):
    g, s = _generator(seed), {"kind": case["kind"], "case": case}
    if case["kind"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        # a broad bulk and a few dozen words far above it, as a language model's head gives
        z = _randn(g, rows, vocab, mul=2.0)
        lead = torch.randint(0, vocab, (rows, 40), generator=g, device=DEVICE)
        z.scatter_(1, lead, 9 + 2 * torch.randn(rows, 40, generator=g, device=DEVICE))
        s["logits"] = z.to(_TYPES[case["dtype"]])
        s["u"] = torch.rand(rows, generator=g, device=DEVICE)
        i = torch.arange(rows, device=DEVICE)
        s["temperature"] = torch.full((rows,), case["temperature"], device=DEVICE)
        s["top_k"] = torch.full((rows,), case["top_k"], dtype=torch.int32, device=DEVICE)
        s["top_p"] = torch.full((rows,), case["top_p"], device=DEVICE)
        s["min_p"] = torch.full((rows,), case["min_p"], device=DEVICE)
        if case["mixed"]:
            s["temperature"] = torch.where(i % 8 == 3, torch.zeros_like(s["u"]), s["temperature"] * (0.75 + 0.125 * (i % 5)))
            s["top_k"] = torch.where(i % 3 == 1, torch.full_like(s["top_k"], 40), s["top_k"])
            s["top_p"] = torch.where(i % 5 == 2, torch.ones_like(s["u"]), s["top_p"])
        return s
    heads, dim, kind = case["kv_heads"], case["dim"], case["kind"]
    dt = _TYPES[case["dtype"]]
    if kind in ("rope", "store"):
        t, hq = case["tokens"], case["q_heads"]
        # q, k and v as the projection leaves them: one row of heads a token
        qkv = _randn(g, t, hq + 2 * heads, dim, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
        off = case["weight"]
        s["wq"], s["wk"] = (_randn(g, dim, mul=0.1).add_(1 - off).to(dt) for _ in range(2))
    if kind == "rope":
        s["positions"] = torch.randint(0, 32768, (t,), generator=g, device=DEVICE, dtype=torch.int32)
        s["angles"] = _table(32768, case["rot"])
    if kind in ("store", "cache"):
        new = _news(case)
        lens = [case["history"] + n for n in new]
        _paged(s, case, g, lens)
        s["cu"] = _ints(_cumulative(new))
        s["max_new"], s["tokens"] = max(new), case["tokens"]
        if kind == "store":
            s["angles"] = _table(max(lens), case["rot"])
            back = new
        else:
            s["k"], s["v"] = (_randn(g, case["tokens"], heads, dim, dtype=dt) for _ in range(2))
            back = new if case["back"] == "new" else lens
        s["cu_back"], s["back"], s["max_back"] = _ints(_cumulative(back)), sum(back), max(back)
    if kind == "attend":
        lens = _lengths(case)
        _paged(s, case, g, lens, case["shared"])
        n = case["per_seq"]
        s["cu"] = _ints([n * i for i in range(len(lens) + 1)])
        s["max_new"], s["tokens"] = n, n * len(lens)
        # queries a few times longer than the keys: attention that has its favourites
        s["q"] = _randn(g, s["tokens"], case["q_heads"], dim, dtype=dt, mul=2.5)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _norm_rope(x, weight, case, angles):
    """x [T][heads][D], angles [T][rot / 2][2]: in 32 bits, rounded once to x's type."""
    f = x.float()
    f = f / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS) * (weight.float() + case["weight"])
    rot = case["rot"]
    c, s = angles[:, None, :, 0], angles[:, None, :, 1]
    if case["inter"]:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, f[..., rot:]), -1).to(x.dtype)


def _read_plain(state, cu, tokens):
    (page, tile, row), _, _ = _places(state, cu, state["lens"], tokens)
    off = tile * 32 + row
    k, v = _get(state, state["table"].long())  # [seqs, pages, page size, heads, D]
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = state["lens"].long()[seq] - cu.long()[seq + 1] + t
    dt = _TYPES[state["case"]["dtype"]]
    return tuple(x[seq, pos // state["page"], off].to(dt) for x in (k, v))


def _run_plain(s):
    case = s["case"]
    kind = s["kind"]
    if kind == "rope":
        a = s["angles"][s["positions"].long()]
        return {"q": _norm_rope(s["q"], s["wq"], case, a), "k": _norm_rope(s["k"], s["wk"], case, a)}
    if kind in ("store", "cache"):
        rows, _, pos = _places(s, s["cu"], s["lens"], s["tokens"])
        out, k = {}, s["k"]
        if kind == "store":
            a = s["angles"][pos]
            out["q"], k = _norm_rope(s["q"], s["wq"], case, a), _norm_rope(s["k"], s["wk"], case, a)
        _put(s, k, s["v"], rows)
        out["k"], out["v"] = _read_plain(s, s["cu_back"], s["back"])
        return out
    if kind == "attend":
        n, seqs, heads, dim = case["per_seq"], case["seqs"], s["heads"], s["dim"]
        group = case["q_heads"] // heads
        k, v = (x.flatten(1, 2).transpose(1, 2) for x in _get(s, s["table"].long()))  # [seqs, heads, L, D]
        q = s["q"].float().view(seqs, n, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(seqs, heads, n * group, dim)
        z = q @ k.transpose(-1, -2) * dim ** -0.5
        pos = s["lens"].long()[:, None] - n + torch.arange(n, device=DEVICE)  # [seqs, n]
        hidden = torch.arange(z.shape[-1], device=DEVICE) > pos.repeat_interleave(group, 1)[..., None]
        z = z.masked_fill_(hidden[:, None], -math.inf)
        p = torch.exp(z - z.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        return {"o": o.view(seqs, heads, n, group, dim).permute(0, 2, 1, 3, 4).reshape(seqs * n, heads * group, dim).to(s["q"].dtype)}
    # sampling, in 64 bits: sums are compared with each other
    z = s["logits"].double()
    order = torch.sort(z, dim=-1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    top = order.values[:, :1]
    w = torch.where(t > 0, torch.exp((order.values - top) / torch.where(t > 0, t, torch.ones_like(t))), (order.values == top).double())
    rank = torch.arange(z.shape[1], device=DEVICE)[None]
    most = torch.where(t[:, 0] > 0, torch.where(s["top_k"] > 0, s["top_k"], z.shape[1]), 1)[:, None]
    w = torch.where(rank < most, w, torch.zeros_like(w))
    before = torch.cumsum(w, -1)
    total = before[:, -1:].clone()
    before -= w
    p = s["top_p"].double()[:, None]
    keep = (rank < most) & ((p >= 1) | (before < p * total) | (rank == 0)) & ((w >= s["min_p"].double()[:, None]) | (rank == 0))
    w = torch.where(keep, w, torch.zeros_like(w))
    kept = torch.zeros_like(w).scatter_(1, order.indices, w)
    sums = torch.cumsum(kept, -1)
    token = (sums <= s["u"].double()[:, None] * sums[:, -1:]).sum(-1, keepdim=True).clamp_(max=z.shape[1] - 1)
    return {"token": token[:, 0].to(torch.int32), "p": (kept.gather(1, token) / sums[:, -1:])[:, 0].float()}


def _handles(s):
    """What a program that serves a model keeps: the cache over its pool, and the batch's tables."""
    if "cache" not in s:
        attention, _ = _package()
        s["cache"] = attention.KvCache(s["pages"], s["page"], s["heads"], s["dim"], s["bits"], data=s["pool"])
        s["batch"] = attention.KvBatch(s["table"], s["lens"], s["cu"], s["tokens"], s["max_new"])
        if "cu_back" in s:
            s["batch_back"] = attention.KvBatch(s["table"], s["lens"], s["cu_back"], s["back"], s["max_back"])
    return s["cache"], s["batch"]


def _run_own(s):
    attention, sampling = _package()
    case, kind = s["case"], s["kind"]
    if kind == "rope":
        q, k = attention.qk_norm_rope(s["q"], s["k"], s["positions"], s["angles"], s["wq"], s["wk"], eps=EPS,
                                      interleaved=case["inter"], weight_offset=case["weight"])
        return {"q": q, "k": k}
    if kind in ("store", "cache"):
        cache, batch = _handles(s)
        out = {}
        if kind == "store":
            out["q"] = cache.append_norm_rope(s["q"], s["k"], s["v"], batch, s["angles"], s["wq"], s["wk"], eps=EPS,
                                              interleaved=case["inter"], weight_offset=case["weight"])
        else:
            cache.append(s["k"], s["v"], batch)
        out["k"], out["v"] = cache.read(s["batch_back"], dtype=_TYPES[case["dtype"]])
        return out
    if kind == "attend":
        cache, batch = _handles(s)
        return {"o": cache.attend(s["q"], batch, shared_tokens=case["shared"])}
    token, p = sampling.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    return {"token": token, "p": p}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows(state, pages):
    """K and V of whole pages [...] in 64 bits, [..., page size, heads, D], byte by byte from the pages' layout."""
    dim, bits, page, heads = state["dim"], state["bits"], state["page"], state["heads"]
    R = dim * bits // 8
    tile = 64 * R + 4 * dim
    off = torch.arange(page, device=DEVICE)[:, None, None]
    head = torch.arange(heads, device=DEVICE)[None, :, None]
    d = torch.arange(dim, device=DEVICE)[None, None, :]
    row = off % 32
    start = (head * (page // 32) + off // 32) * tile
    byte = d * bits // 8
    turn = torch.tensor([0, 4, 2, 6, 5, 1, 7, 3], device=DEVICE)[row % 8]
    at = row * R + ((byte // 16) ^ (turn % (R // 16))) * 16 + byte % 16
    flat = state["pool"].view(state["pages"], -1)
    got = []
    for base in (0, 32 * R + 2 * dim):
        scale = base + 32 * R + 2 * ((d // 32) * 32 + row)
        u = flat[pages][..., (start + base + at).reshape(-1)].long()
        if bits == 4:
            u = (u >> (4 * (d % 2)).expand(page, heads, dim).reshape(-1)) % 16
        sc = flat.view(torch.float16)[pages][..., ((start + scale) // 2).reshape(-1)].double()
        got.append(((u - (128 if bits == 8 else 8)).double() * sc).unflatten(-1, (page, heads, dim)))
    return got


def _exact_held(x, bits):
    """What the cache holds of x [..., D], in 64 bits."""
    top = 127 if bits == 8 else 7
    b = x.double().unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1, keepdim=True) / top).to(torch.float16).double()
    q = torch.clamp(torch.round(b / torch.where(d > 0, d, torch.ones_like(d))), -127 if bits == 8 else -8, top)
    return (q * d).flatten(-2)


def _exact_norm_rope(x, weight, case, angles):
    f = x.double()
    f = f * torch.rsqrt(f.pow(2).sum(-1, keepdim=True) / f.shape[-1] + EPS) * (weight.double() + case["weight"])
    h = case["rot"] // 2
    z = torch.view_as_complex(angles.double())[:, None]
    first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["inter"] else (slice(0, h), slice(h, 2 * h))
    turned = torch.complex(f[..., first], f[..., second]) * z
    f[..., first], f[..., second] = turned.real, turned.imag
    return f


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        a = s["angles"][s["positions"].long()]
        return {"q": _exact_norm_rope(s["q"], s["wq"], case, a), "k": _exact_norm_rope(s["k"], s["wk"], case, a)}
    if kind in ("store", "cache"):
        new = _news(case)
        k, out, dt = s["k"], {}, _TYPES[case["dtype"]]
        if kind == "store":
            pos = torch.cat([torch.arange(case["history"], case["history"] + n, device=DEVICE) for n in new])
            out["q"] = _exact_norm_rope(s["q"], s["wq"], case, s["angles"][pos])
            k = _exact_norm_rope(s["k"], s["wk"], case, s["angles"][pos]).to(dt)  # held from the values as they are passed on
        k, v = _exact_held(k, case["bits"]), _exact_held(s["v"], case["bits"])
        if case.get("back") == "all":
            parts, at = ([], []), 0
            for i, n in enumerate(new):
                pages = s["table"][i, :-(-(case["history"] + n) // case["page"])].long()
                for part, old, x in zip(parts, _exact_rows(s, pages), (k, v)):
                    part += [old.flatten(0, 1)[:case["history"]], x[at:at + n]]
                at += n
            k, v = (torch.cat(p) for p in parts)
        out["k"], out["v"] = k, v
        return out
    if kind == "attend":
        n, heads = case["per_seq"], case["kv_heads"]
        rows = []
        for i, length in enumerate(_lengths(case)):
            pages = s["table"][i, :-(-length // case["page"])].long()
            k, v = (x.flatten(0, 1)[:length].transpose(0, 1) for x in _exact_rows(s, pages))  # [heads, L, D]
            q = s["q"][n * i:n * i + n].double().unflatten(1, (heads, -1)).permute(1, 2, 0, 3)  # [heads, group, n, D]
            z = torch.einsum("hgnd,hld->hgnl", q, k) / math.sqrt(case["dim"])
            seen = torch.ones(n, length, dtype=torch.bool, device=DEVICE).tril(length - n)
            p = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
            rows.append(torch.einsum("hgnl,hld->nhgd", p, v).flatten(1, 2))
        return {"o": torch.cat(rows)}
    if case["rows"] * case["vocab"] > 50_000_000:
        return None
    import numpy as np
    z, u = s["logits"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    temperature, top_k, top_p, min_p = (s[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p"))
    tokens, ps = [], []
    for r in range(case["rows"]):
        order = np.argsort(-z[r], kind="stable")
        if temperature[r] <= 0:
            tokens.append(int(order[0]))
            ps.append(1.0)
            continue
        order = order[:int(top_k[r])] if top_k[r] > 0 else order
        w = np.exp((z[r, order] - z[r, order[0]]) / temperature[r])
        before = np.concatenate(([0.0], np.cumsum(w)))
        n = len(w) if top_p[r] >= 1 else max(1, int(np.sum(before[:-1] < top_p[r] * before[-1])))
        n = max(1, min(n, int(np.sum(w >= min_p[r]))))
        kept = np.sort(order[:n])
        w = np.exp((z[r, kept] - z[r, order[0]]) / temperature[r])
        at = min(int(np.searchsorted(np.cumsum(w), u[r] * w.sum(), side="right")), n - 1)
        tokens.append(int(kept[at]))
        ps.append(float(w[at] / w.sum()))
    return {"token": torch.tensor(tokens, dtype=torch.int32), "p": torch.tensor(ps, dtype=torch.float64)}
