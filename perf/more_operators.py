"""Attention with a sliding window and sinks, the append with per-head norms, and page copies, as cases to measure.

Four operators over paged caches of 16-token blocks:

* ``decode``: one query token a request. The token at position i sees the keys j <= i with j > i - W (the
  window) or j < S (the sinks). Caches of bf16 values, or of E4M3 codes with one scale for K and one for V
  (``tensor``).
* ``extend``: several new tokens a request over a cache and over themselves, under the same mask; without a
  cache (``kind`` none) whole prompts.
* ``append``: every head of the queries and new keys divided by its root mean square and multiplied by a
  weight, rotated by its position, and keys and values appended to the cache (``block``: E4M3 codes with a
  scale for each block and KV head, which grows with what is appended).
* ``copy``: pages of a pool copied onto other pages of it, in every layer.

``run`` computes them in plain torch operations, or through the package's calls where ``own`` is set.
"""
import math

import torch

own = False

BS = 16          # tokens of a cache block
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
MAX_POS = 131072

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")


# ---- the cases -----------------------------------------------------------------------------------

def listed():
    return [
        # a handful of short sequences under a narrow window: latency
        dict(name="decode_few", op="decode", kind="bf16", R=4, lo=16, hi=200, Hq=8, Hkv=2, d=64, W=64, S=4, freed=False),
        # a decode step of 256 sequences, 16 query heads a KV head, a window shorter than the sequences
        dict(name="decode_batch", op="decode", kind="bf16", R=256, lo=2000, hi=3000, Hq=64, Hkv=4, d=128, W=1024, S=4,
             freed=False),
        # long sequences whose pages between the sinks and the window were given back; an 8-bit cache
        dict(name="decode_long_fp8", op="decode", kind="tensor", R=24, lo=30000, hi=100000, Hq=64, Hkv=8, d=128, W=4096,
             S=64, freed=True),
        # the check of a few drafted tokens for each sequence
        dict(name="extend_draft", op="extend", kind="bf16", R=32, nlo=4, nhi=4, lo=1000, hi=4000, Hq=64, Hkv=8, d=128,
             W=1024, S=4, freed=False),
        # chunks of prompts over what earlier chunks left, under a narrow window
        dict(name="extend_chunks", op="extend", kind="bf16", R=8, nlo=301, nhi=512, lo=4000, hi=32000, Hq=64, Hkv=8, d=128,
             W=128, S=16, freed=True),
        # the last chunk of one very long prompt over an 8-bit cache
        dict(name="extend_long_fp8", op="extend", kind="tensor", R=1, nlo=2048, nhi=2048, lo=100000, hi=100000, Hq=64,
             Hkv=8, d=128, W=4096, S=128, freed=True),
        # whole prompts: the window bounds what would be quadratic
        dict(name="prefill_prompts", op="extend", kind="none", R=3, nlo=4000, nhi=10007, lo=0, hi=0, Hq=64, Hkv=8, d=128,
             W=4096, S=0, freed=False),
        # one token of one sequence: what the append's call costs
        dict(name="append_one", op="append", kind="bf16", R=1, new=1, lo=100, hi=100, pad=0, Hq=8, Hkv=2, d=64, rot=64,
             inter=False, w32=False),
        # the append of a decode step: one token for each of 250 sequences, in a batch padded to 256
        dict(name="append_decode_step", op="append", kind="block", R=250, new=1, lo=2000, hi=3000, pad=6, Hq=64, Hkv=4,
             d=128, rot=128, inter=False, w32=False),
        # a whole prompt of 10,000 tokens
        dict(name="append_prompt", op="append", kind="bf16", R=1, new=10000, lo=0, hi=0, pad=0, Hq=64, Hkv=8, d=128,
             rot=128, inter=False, w32=False),
        # four samples fork from each of three sequences: their last, partly filled pages, in every layer
        dict(name="copy_fork", op="copy", kind="bf16", L=32, n=12, fan=4, nb=48, Hkv=2, d=64),
        # a pool is compacted: the pages of a 6,400-token prompt move down, in 20 layers
        dict(name="copy_compact", op="copy", kind="bf16", L=20, n=400, fan=1, nb=900, Hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "extend", "append", "copy"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128])
    if op == "copy":
        kind = rng.choice(["bf16", "tensor", "block"])
        d = 128 if kind == "block" else d
        page = 2 * BS * Hkv * d * (2 if kind == "bf16" else 1)
        L = _log_int(rng, 1, 80)
        n = _log_int(rng, 1, max(1, min(2000, int(3e8 / (L * page)))))
        return dict(op=op, kind=kind, L=L, n=n, fan=rng.choice([1, 1, 2, 7]), nb=2 * n + rng.randint(1, n + 5), Hkv=Hkv, d=d)
    G = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        kind = rng.choice(["bf16", "tensor", "block"])
        d = 128 if kind == "block" else d
        new = rng.choice([1, 1, _log_int(rng, 2, 4000)])
        R = _log_int(rng, 1, max(1, min(256, 10000 // new)))
        lo = min(rng.choice([0, _log_int(rng, 1, 4000)]), 400000 // R)
        hi = lo + _log_int(rng, 1, max(1, min(2000, 400000 // R))) - 1
        Hq = min(64, Hkv * G)
        return dict(op=op, kind=kind, R=R, new=new, lo=lo, hi=hi, pad=rng.choice([0, 0, rng.randint(1, 9)]), Hq=Hq - Hq % Hkv,
                    Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, 32]), inter=rng.random() < 0.4, w32=rng.random() < 0.4)
    W, S = _log_int(rng, 1, 8192), rng.choice([0, rng.randint(1, 16), _log_int(rng, 1, 300)])
    if op == "decode":
        kind = rng.choice(["bf16", "tensor"])
        d = 128 if kind == "tensor" else d
        R = _log_int(rng, 1, 512)
        most = int(2.5e8 / (R * Hkv * d * 4))  # visible tokens a sequence
        W = min(W, max(1, most))
        freed = rng.random() < 0.5
        hi = _log_int(rng, 1, 100000 if freed else max(1, min(100000, 4 * most)))
        return dict(op=op, kind=kind, R=R, lo=max(1, int(hi * rng.choice([1.0, rng.random()]))), hi=hi, Hq=Hkv * G, Hkv=Hkv,
                    d=d, W=W, S=S, freed=freed)
    kind = rng.choice(["none", "bf16", "bf16", "tensor"])
    d = 128 if kind == "tensor" else d
    R = _log_int(rng, 1, 24)
    nhi = _log_int(rng, 1, max(1, min(6000, 20000 // R)))
    nhi = max(1, min(nhi, int(6e11 / (4.0 * Hkv * G * d * R * (W + S)))))
    hi = 0 if kind == "none" else _log_int(rng, 1, 32000)
    return dict(op=op, kind=kind, R=R, nlo=max(1, int(nhi * rng.choice([1.0, rng.random()]))), nhi=nhi,
                lo=int(hi * rng.choice([1.0, rng.random()])), hi=hi, Hq=Hkv * G, Hkv=Hkv, d=d, W=W, S=S,
                freed=rng.random() < 0.5)


def _spread(lo, hi, n):
    """n lengths spread evenly over [lo, hi]."""
    return [lo + ((hi - lo) * (2 * i + 1) + n) // (2 * n) for i in range(n)]


def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    if op == "copy":
        page = 2 * BS * Hkv * d * (2 if case["kind"] == "bf16" else 1) + (8 * Hkv if case["kind"] == "block" else 0)
        sources = (case["n"] + case["fan"] - 1) // case["fan"]
        return {"bytes": case["L"] * page * (case["n"] + sources) + 8 * case["n"], "flops": 0}
    R, Hq = case["R"], case["Hq"]
    if op == "append":
        T, rot = R * case["new"], case["rot"]
        by = 2 * T * Hq * d * 2 + T * rot * 4 + 16 * T + T * Hkv * d * (2 + 2 + 2)
        by += 2 * T * Hkv * d * (2 if case["kind"] == "bf16" else 1) + 2 * d * (4 if case["w32"] else 2)
        return {"bytes": by, "flops": T * (Hq + Hkv) * (3 * rot + 4 * d)}
    W, S, ctx = case["W"], case["S"], _spread(case["lo"], case["hi"], R)
    token = 2 * Hkv * d * (2 if case["kind"] == "bf16" else 1)
    if op == "decode":
        seen = sum(min(c, S + W) for c in ctx)
        return {"bytes": seen * token + seen // 4 + 2 * R * Hq * d * 2 + 4 * R * Hq, "flops": 4 * Hq * d * seen}
    new = _spread(case["nlo"], case["nhi"], R)
    T = sum(new)
    cached = sum(min(c, S + W - 1) for c in ctx)
    m = S + W  # keys of the rows that have as many
    pairs = 0
    for c, n in zip(ctx, new):
        short = min(n, max(0, m - c))  # rows that see every key up to their own
        pairs += short * c + short * (short + 1) // 2 + (n - short) * m
    return {"bytes": cached * token + cached // 4 + T * (2 * Hq * d * 2 + 2 * Hkv * d * 2 + 4 * Hq), "flops": 4 * Hq * d * pairs}


# ---- the inputs ----------------------------------------------------------------------------------

def _generators(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    dg = torch.Generator(device=DEV)
    dg.manual_seed(seed + 1)
    return g, dg


def _tables(kept, most, g):
    """Block tables [R, most]: request r's logical blocks kept[r] hold pages of a shuffled pool 1.2 times as large as
    needed, the others -1 (pages that were given back)."""
    nb = max(1, math.ceil(1.2 * sum(len(k) for k in kept)))
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    t = torch.full((len(kept), max(1, most)), -1, dtype=torch.int32)
    at = 0
    for r, k in enumerate(kept):
        t[r, torch.tensor(k, dtype=torch.int64)] = perm[at:at + len(k)]
        at += len(k)
    return t, nb


def _codes(x):
    return x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _cache(nb, Hkv, d, kind, dg):
    """One of K and V: [nb, 16, Hkv, d] of normal values (E4M3 codes of them at a scale of 1 / 64)."""
    out = torch.empty((nb, BS, Hkv, d), dtype=torch.bfloat16 if kind == "bf16" else torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (BS * Hkv * d))
    for s in range(0, nb, step):
        x = torch.randn(out[s:s + step].shape, generator=dg, device=DEV)
        out[s:s + step] = x.to(torch.bfloat16) if kind == "bf16" else _codes(x * 64.0)
    return out


def _block_cache(nb, Hkv, d, dg):
    """Codes and scales [nb, Hkv] (powers of two, as appends leave them) of values whose size differs from block to block."""
    x = torch.randn((nb, BS, Hkv, d), generator=dg, device=DEV)
    x *= torch.exp(0.4 * torch.randn((nb, 1, Hkv, 1), generator=dg, device=DEV))
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(1, 3)) / 448.0)))
    return _codes(x / s[:, None, :, None]), s


def _rope_table(rot):
    """[MAX_POS, rot] fp32: the cosines of rot / 2 frequencies, then the sines."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(MAX_POS, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g, dg = _generators(seed)
    op, kind, Hkv, d = case["op"], case["kind"], case["Hkv"], case["d"]
    st = dict(case=case)
    if op == "copy":
        L, n, nb = case["L"], case["n"], case["nb"]
        ids = torch.randperm(nb, generator=g).to(torch.int32)
        sources = (n + case["fan"] - 1) // case["fan"]
        st.update(src=ids[:sources].repeat_interleave(case["fan"])[:n].to(DEV), dst=ids[sources:sources + n].to(DEV))
        if kind == "block":
            made = [(*_block_cache(nb, Hkv, d, dg), *_block_cache(nb, Hkv, d, dg)) for _ in range(L)]
            st.update(kc=[m[0] for m in made], vc=[m[2] for m in made], ks=[m[1] for m in made], vs=[m[3] for m in made])
        else:
            st.update(kc=[_cache(nb, Hkv, d, kind, dg) for _ in range(L)], vc=[_cache(nb, Hkv, d, kind, dg) for _ in range(L)])
        return st
    R, Hq = case["R"], case["Hq"]
    ctx = _spread(case["lo"], case["hi"], R)
    ctx = [ctx[i] for i in torch.randperm(R, generator=g).tolist()]

    def normal(*shape):
        return torch.randn(shape, generator=dg, device=DEV).to(torch.bfloat16)

    if op == "append":
        new = case["new"]
        kept = [range((c + new + BS - 1) // BS) for c in ctx]
        table, nb = _tables(kept, max(len(k) for k in kept), g)
        pos = torch.cat([torch.arange(c, c + new) for c in ctx])
        req = torch.arange(R).repeat_interleave(new)
        slot = table[req, pos // BS].long() * BS + pos % BS
        T = R * new
        # rows behind the batch's tokens (a batch padded to a fixed size): slot -1
        slot = torch.cat([slot, torch.full((case["pad"],), -1)])
        pos = torch.cat([pos, torch.zeros(case["pad"], dtype=torch.int64)])
        Tp = T + case["pad"]
        wt = torch.float32 if case["w32"] else torch.bfloat16
        # projections differ in size from head to head before the norm
        q = (torch.randn((Tp, Hq, d), generator=dg, device=DEV) * torch.exp(torch.randn((1, Hq, 1), generator=dg, device=DEV)))
        k = (torch.randn((Tp, Hkv, d), generator=dg, device=DEV) * torch.exp(torch.randn((1, Hkv, 1), generator=dg, device=DEV)))
        st.update(T=T, q=q.to(torch.bfloat16), k=k.to(torch.bfloat16), v=normal(Tp, Hkv, d), pos=pos.to(DEV), slot=slot.to(DEV),
                  qw=(1.0 + 0.3 * torch.randn(d, generator=dg, device=DEV)).to(wt),
                  kw=(1.0 + 0.3 * torch.randn(d, generator=dg, device=DEV)).to(wt), rope=_rope_table(case["rot"]),
                  q_out=torch.zeros((Tp, Hq, d), dtype=torch.bfloat16, device=DEV),
                  k_out=torch.zeros((Tp, Hkv, d), dtype=torch.bfloat16, device=DEV))
        if kind == "block":
            kc, ks = _block_cache(nb, Hkv, d, dg)
            vc, vs = _block_cache(nb, Hkv, d, dg)
            st.update(kc=kc, vc=vc, ks=ks, vs=vs)
        else:
            st.update(kc=_cache(nb, Hkv, d, kind, dg), vc=_cache(nb, Hkv, d, kind, dg))
            if kind == "tensor":
                st.update(ks=5.0 / 448.0, vs=4.5 / 448.0)
        return st
    new = [1] * R if op == "decode" else _spread(case["nlo"], case["nhi"], R)
    new = [new[i] for i in torch.randperm(R, generator=g).tolist()]
    total = ctx if op == "decode" else [c + n for c, n in zip(ctx, new)]
    T = sum(new)
    st.update(new=new, ctx=ctx, q=normal(T, Hq, d), lens=torch.tensor(total, dtype=torch.int32, device=DEV), max_len=max(total),
              out=torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=DEV),
              lse=torch.zeros((T, Hq), dtype=torch.float32, device=DEV))
    if kind != "none":
        W, S = case["W"], case["S"]
        kept = []
        for n, t in zip(new, total):
            first = max(0, t - n - W + 1) // BS  # the first page of the window of the first new token
            blocks = range((t + BS - 1) // BS)
            kept.append([b for b in blocks if b >= first or b * BS < S] if case["freed"] else list(blocks))
        table, nb = _tables(kept, max((t + BS - 1) // BS for t in total), g)
        st.update(table=table.to(DEV), kc=_cache(nb, Hkv, d, kind, dg), vc=_cache(nb, Hkv, d, kind, dg))
        if kind == "tensor":
            st.update(ks=1.0 / 64.0, vs=1.0 / 64.0)
    if op == "extend":
        cu = torch.zeros(R + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(new).cumsum(0)
        st.update(k_new=normal(T, Hkv, d), v_new=normal(T, Hkv, d), cu=cu.to(DEV), max_new=max(new))
    else:
        # the scratch that a program keeps for its decode calls (more than any shape here asks for)
        st["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return st


# ---- one pass ------------------------------------------------------------------------------------

def _values(st, name, pages):
    """fp32 rows of the cache `name` at pages (any shape of block numbers and offsets: [..., Hkv, d])."""
    x = st[name + "c"][pages]
    return x.view(E4M3).float() * st[name + "s"] if x.dtype is torch.uint8 else x.float()


def _attend(q, k, v, seen):
    """q [R, I, Hkv, G, d], k, v [R, M, Hkv, d] fp32, seen [R, I, M] -> out [R, I, Hkv, G, d], lse [R, I, Hkv, G]."""
    R, I, H, G, d = q.shape
    x = q.permute(0, 2, 3, 1, 4).reshape(R, H, G * I, d)
    s = torch.matmul(x, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d)).view(R, H, G, I, -1)
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min_(-1e30)  # (rows of padding see nothing)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, H, G * I, -1), v.transpose(1, 2)).view(R, H, G, I, d) / l
    return o.permute(0, 3, 1, 2, 4), (m + torch.log(l))[..., 0].permute(0, 3, 1, 2)


def _plain_decode(st):
    case, q, lens = st["case"], st["q"], st["lens"].long()
    R, Hq, d = q.shape
    W, S = min(case["W"], st["max_len"]), min(case["S"], st["max_len"])
    # the visible positions of each request: the sinks, then the window behind them
    j = torch.arange(min(S + W, st["max_len"]), device=q.device)[None]
    first = torch.clamp(lens - W, min=S)[:, None]
    pos = torch.where(j < S, j, first + j - S)
    seen = pos < lens[:, None]
    pos = torch.where(seen, pos, lens[:, None] - 1)
    pages = (st["table"].long().gather(1, pos // BS), pos % BS)
    o, z = _attend(q.float().view(R, 1, case["Hkv"], -1, d), _values(st, "k", pages), _values(st, "v", pages), seen[:, None])
    return o.reshape(R, Hq, d).to(torch.bfloat16), z.reshape(R, Hq)


def _plain_extend(st):
    case, q = st["case"], st["q"]
    T, Hq, d = q.shape
    R, Hkv, W, S = case["R"], case["Hkv"], min(case["W"], st["max_len"]), min(case["S"], st["max_len"])
    start = st["cu"][:-1].long()[:, None]
    n = (st["cu"][1:] - st["cu"][:-1]).long()[:, None]
    total = st["lens"].long()[:, None]
    c = total - n
    out, lse = torch.empty_like(q), torch.empty_like(st["lse"])
    step = int(max(16, min(st["max_new"], 3e8 / (R * Hq * (S + W)))))
    for a in range(0, st["max_new"], step):  # the scores of all rows at once would not fit
        i = a + torch.arange(min(step, st["max_new"] - a), device=q.device)[None]
        at = c + i  # positions of the queries
        # positions that some row of these may see: the sinks, then what the windows reach
        j = torch.arange(S + W - 1 + i.shape[1], device=q.device)[None]
        pos = torch.where(j < S, j, torch.clamp(c + a - W + 1, min=S) + j - S)
        k_at, q_at = pos[:, None, :], at[:, :, None]
        seen = (k_at <= q_at) & ((k_at > q_at - W) | (k_at < S)) & (k_at < total[:, :, None]) & (i < n)[:, :, None]
        pos = torch.where(seen.any(1), pos, total - 1)
        rows = start + (pos - c).clamp(min=0)
        k, v = st["k_new"][rows].float(), st["v_new"][rows].float()
        if case["kind"] != "none":
            cached = (pos < c)[:, :, None, None]
            p = torch.where(pos < c, pos, 0)
            page = st["table"].long().gather(1, p // BS).clamp_(min=0)
            k = torch.where(cached, _values(st, "k", (page, p % BS)), k)
            v = torch.where(cached, _values(st, "v", (page, p % BS)), v)
        rows = start + torch.minimum(i, n - 1)
        o, z = _attend(q[rows].float().view(R, -1, Hkv, Hq // Hkv, d), k, v, seen)
        live = (i < n).reshape(-1)
        rows = rows.reshape(-1)[live]
        out[rows] = o.reshape(-1, Hq, d)[live].to(torch.bfloat16)
        lse[rows] = z.reshape(-1, Hq)[live]
    return out, lse


def _normed(x, w):
    return x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * w.float()


def _rotate(x, cos, sin, inter):
    """x [T, H, d] fp32 with its first 2 n dims rotated; cos, sin [T, n]."""
    n = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    w, rest = x[..., :2 * n], x[..., 2 * n:]
    if inter:
        a, b = w[..., 0::2], w[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)
    a, b = w[..., :n], w[..., n:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def _append_scaled(x, slot, codes, scales):
    """Append rows x [T, H, d] (fp32) at `slot` to E4M3 codes with a power-of-two scale a block and head."""
    nb, _, H, d = codes.shape
    blk, off = slot // BS, slot % BS
    amax = torch.zeros((nb, H), device=x.device).index_reduce(0, blk, x.abs().amax(-1), "amax")
    first = torch.full((nb,), BS, dtype=torch.int64, device=x.device).index_reduce(0, blk, off, "amin")
    a, old, f = amax[blk], scales[blk], first[blk]
    m, e = torch.frexp(a)                      # a = m 2^e, 0.5 <= m < 1, and 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    need = ((torch.where(a > 0, e, -64).clamp(-64, 120) + 127) << 23).to(torch.int32).view(torch.float32)
    s = torch.where((f == 0)[:, None], need, torch.maximum(old, need))
    # the rows that were there, at the new scale
    was = codes[blk]
    now = _codes(was.view(E4M3).float() * (old / s)[:, None, :, None])
    keep = (torch.arange(BS, device=x.device)[None] < f[:, None])[:, :, None, None]
    codes[blk] = torch.where(keep, now, was)
    codes.view(nb * BS, H, d)[slot] = _codes(x * (1.0 / s)[:, :, None])
    scales[blk] = s


def _plain_append(st):
    case, T = st["case"], st["T"]
    slot, pos = st["slot"][:T], st["pos"][:T]
    cs = st["rope"][pos]
    cos, sin = cs[:, :cs.shape[1] // 2], cs[:, cs.shape[1] // 2:]
    q = _rotate(_normed(st["q"][:T].float(), st["qw"]), cos, sin, case["inter"])
    k = _rotate(_normed(st["k"][:T].float(), st["kw"]), cos, sin, case["inter"])
    st["q_out"][:T] = q.to(torch.bfloat16)
    st["k_out"][:T] = k.to(torch.bfloat16)
    kc, vc, v = st["kc"], st["vc"], st["v"][:T]
    if case["kind"] == "block":
        _append_scaled(k, slot, kc, st["ks"])
        _append_scaled(v.float(), slot, vc, st["vs"])
    elif case["kind"] == "tensor":
        inv = [float(1.0 / torch.tensor(s, dtype=torch.float32)) for s in (st["ks"], st["vs"])]
        kc.view(-1, *kc.shape[2:])[slot] = _codes(k * inv[0])
        vc.view(-1, *vc.shape[2:])[slot] = _codes(v.float() * inv[1])
    else:
        kc.view(-1, *kc.shape[2:])[slot] = k.to(torch.bfloat16)
        vc.view(-1, *vc.shape[2:])[slot] = v


def _shown(x):
    """A cache as the values that it holds (codes: the E4M3 numbers)."""
    return x.view(E4M3) if x.dtype is torch.uint8 else x


def _appended(st):
    """What an append leaves: the rotated rows and the cache."""
    T = st["T"]
    r = dict(q=st["q_out"][:T], k=st["k_out"][:T], k_cache=_shown(st["kc"]), v_cache=_shown(st["vc"]))
    if st["case"]["kind"] == "block":
        r.update(k_scale=st["ks"], v_scale=st["vs"])
    return r


def _pools(st):
    """Every layer's pool."""
    r = dict(k=[_shown(x) for x in st["kc"]], v=[_shown(x) for x in st["vc"]])
    if "ks" in st:
        r.update(k_scale=st["ks"], v_scale=st["vs"])
    return r


def run(state):
    st = state
    case = st["case"]
    op = case["op"]
    if own:
        import paged_kv_attention_reshape_gb300 as pkv
        scales = dict(k_scale=st["ks"], v_scale=st["vs"]) if "ks" in st else {}
        if op == "copy":
            if "layers" not in st:
                st["layers"] = pkv.CacheLayers(st["kc"], st["vc"], st.get("ks"), st.get("vs"))
            pkv.kv_block_copy(st["layers"], st["src"], st["dst"])
            return _pools(st)
        if op == "append":
            pkv.kv_append(st["q"], st["k"], st["v"], st["pos"], st["slot"], st["kc"], st["vc"], st["rope"],
                          interleaved=case["inter"], q_norm=st["qw"], k_norm=st["kw"], norm_eps=EPS, q_out=st["q_out"],
                          k_out=st["k_out"], **scales)
            return _appended(st)
        mask = dict(window=case["W"], sinks=case["S"])
        if op == "decode":
            return pkv.paged_decode_attn(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["max_len"], out=st["out"],
                                         lse=st["lse"], workspace=st["ws"], **scales, **mask)
        if case["kind"] == "none":
            return pkv.varlen_prefill_attn(st["q"], st["k_new"], st["v_new"], st["cu"], st["max_new"], out=st["out"],
                                           lse=st["lse"], **mask)
        return pkv.extend_attn(st["q"], st["k_new"], st["v_new"], st["cu"], st["lens"], st["kc"], st["vc"], st["table"],
                               st["max_new"], st["max_len"], out=st["out"], lse=st["lse"], **scales, **mask)
    if op == "copy":
        src, dst = st["src"].long(), st["dst"].long()
        for pages in st["kc"] + st["vc"] + st.get("ks", []) + st.get("vs", []):  # a tensor of its own each
            pages[dst] = pages[src]
        return _pools(st)
    if op == "append":
        _plain_append(st)
        return _appended(st)
    return _plain_decode(st) if op == "decode" else _plain_extend(st)


# ---- from the definition, in 64 bits -------------------------------------------------------------

def _grid(x):
    """The nearest E4M3 number (ties to even), saturated at 448, of doubles."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 4).clamp(min=-9))
    return torch.copysign(torch.round(a / step) * step, x)


def _turn(x, p, st):
    """x [T, H, d] doubles at positions p, by complex numbers."""
    rot = st["rope"].shape[1]
    t = st["rope"][p].double()
    z = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
    w = x[..., :rot]
    if st["case"]["inter"]:
        w = torch.view_as_real(torch.view_as_complex(w.reshape(*w.shape[:-1], rot // 2, 2).contiguous()) * z).flatten(-2)
    else:
        y = torch.complex(w[..., :rot // 2].contiguous(), w[..., rot // 2:].contiguous()) * z
        w = torch.cat([y.real, y.imag], -1)
    return torch.cat([w, x[..., rot:]], -1)


def _exact_append(st):
    T, kind, new = st["T"], st["case"]["kind"], st["case"]["new"]
    slot, pos = st["slot"][:T], st["pos"][:T]
    q, k = (_turn(x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * st[n + "w"].double(), pos, st)
            for n, x in (("q", st["q"][:T].double()), ("k", st["k"][:T].double())))
    r = dict(q=q, k=k)
    for name, x in (("k", k), ("v", st["v"][:T].double())):
        cache = st[name + "c"]
        if kind == "bf16":
            c = cache.double()
            c.view(-1, *c.shape[2:])[slot] = x
        elif kind == "tensor":
            c = cache.view(E4M3).double()
            c.view(-1, *c.shape[2:])[slot] = _grid(x / st[name + "s"])
        else:
            c, s = cache.view(E4M3).double(), st[name + "s"].double()
            # every token's run: the tokens of its request in its block; its first and its last one
            i = torch.arange(T, device=x.device)
            req, at = i // new, pos % BS
            lo = torch.maximum(i - at, req * new)
            j = lo[:, None] + torch.arange(BS, device=x.device)
            same = (j < (req[:, None] + 1) * new) & (j - i[:, None] < (BS - at)[:, None])
            rows = x.abs().amax(-1)[j.clamp(max=T - 1)] * same[:, :, None]
            a = rows.amax(1)
            need = torch.exp2(torch.ceil(torch.log2(a / 448.0)).clamp(-64, 120))
            f = pos[lo] % BS
            b = slot // BS
            s1 = torch.where((f == 0)[:, None], need, torch.maximum(s[b], need))
            was = c[b]
            now = _grid(was * (s[b] / s1)[:, None, :, None])
            c[b] = torch.where((torch.arange(BS, device=x.device)[None] < f[:, None])[:, :, None, None], now, was)
            c.view(-1, *c.shape[2:])[slot] = _grid(x / s1[:, :, None])
            s[b] = s1
            r[name + "_scale"] = s
        r[name + "_cache"] = c
    return {n: r[n] for n in ("q", "k", "k_cache", "v_cache", "k_scale", "v_scale") if n in r}


def _exact_attention(st):
    case = st["case"]
    R, Hq, Hkv, d, W, S = (case[n] for n in ("R", "Hq", "Hkv", "d", "W", "S"))
    G = Hq // Hkv
    T = st["q"].shape[0]
    out = torch.empty((T, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.empty((T, Hq), dtype=torch.float64, device=DEV)
    row0 = 0
    for r in range(R):
        n = st["new"][r]
        total = int(st["lens"][r])
        c = total if case["op"] == "decode" else total - n  # keys that the cache holds
        for a in range(0, n, 512):
            z = min(n, a + 512)
            at = torch.arange(total - n + a, total - n + z, device=DEV)
            low = max(0, int(at[0]) - W + 1)
            j = torch.arange(low, int(at[-1]) + 1, device=DEV)
            j = torch.cat([torch.arange(min(S, low), device=DEV), j])
            hide = (j[None] > at[:, None]) | ((j[None] <= at[:, None] - W) & (j[None] >= S))
            old, young = j[j < c], j[j >= c]
            rows = slice(row0 + a, row0 + z)
            for h in range(Hkv):
                hq = slice(h * G, (h + 1) * G)
                k, v = [], []
                if case["kind"] != "none":
                    b = st["table"][r].long()[old // BS]
                    for name, to in (("k", k), ("v", v)):
                        x = st[name + "c"][b, old % BS, h]
                        to.append(x.view(E4M3).double() * st[name + "s"] if case["kind"] == "tensor" else x.double())
                if case["op"] == "extend":
                    k.append(st["k_new"][row0 + young - c, h].double())
                    v.append(st["v_new"][row0 + young - c, h].double())
                x = torch.einsum("tgd,jd->tgj", st["q"][rows, hq].double(), torch.cat(k)) / math.sqrt(d)
                x.masked_fill_(hide[:, None, :], -math.inf)
                y = torch.logsumexp(x, -1)
                lse[rows, hq] = y
                out[rows, hq] = torch.einsum("tgj,jd->tgd", torch.exp(x - y[..., None]), torch.cat(v))
        row0 += n
    return out, lse


def exact(case, seed):
    if work(case)["flops"] > 3e12:
        return None  # too long in 64 bits
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "copy":
        # page i of a pool is what page `of[i]` was
        of = torch.arange(case["nb"], device=DEV)
        of[st["dst"].long()] = st["src"].long()
        return {k: [x.double().index_select(0, of) for x in v] for k, v in _pools(st).items()}
    return _exact_attention(st)
