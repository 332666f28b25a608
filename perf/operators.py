"""The block-scaled 8-bit KV cache: its append call and the attentions that read it, as cases to measure.

Three operators over a paged cache of 16-token blocks:

* ``append``: rotate the queries and the new keys by their positions and append the new keys and
  values to the cache. Cache kinds: ``bf16``; ``tensor`` (E4M3 codes, one scale for all of K and one
  for all of V); ``block`` (E4M3 codes, one fp32 scale for each block and KV head, which grows with
  what is appended); ``latent`` (one bf16 row a token that stands for keys and values, rotated in its
  tail only).
* ``decode``: one query token a request over a ``block`` cache.
* ``extend``: several new tokens a request over a ``block`` cache, and causally over themselves.

``run`` computes them in plain torch operations, or through the package's calls where ``own`` is set.
"""
import math

import torch

own = False

BS = 16          # tokens of a cache block
D = 128          # head width of the 8-bit attentions
E4M3 = torch.float8_e4m3fn
MAX_POS = 131072

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")


# ---- the cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one token of one small sequence: what the call costs when there is nothing to move
        dict(name="append_one", op="append", kind="bf16", R=1, new=1, lo=100, hi=100, pad=0, Hq=8, Hkv=2, d=64, rot=64,
             inter=False),
        # the append of a decode step: one token for each of 250 sequences, in a batch padded to 256
        dict(name="append_decode_step", op="append", kind="block", R=250, new=1, lo=2000, hi=3000, pad=6, Hq=64, Hkv=4,
             d=128, rot=128, inter=False),
        # chunks of several prompts that start inside a block; a rotation of half of the head, in pairs
        dict(name="append_chunks_tensor", op="append", kind="tensor", R=8, new=509, lo=4001, hi=32001, pad=0, Hq=64,
             Hkv=8, d=128, rot=64, inter=True),
        # the latent row of a layer whose keys and values share it: 64 rotated dims after 512 others
        dict(name="append_latent", op="append", kind="latent", R=128, new=1, lo=10000, hi=11000, pad=0, Hq=16, Hkv=1,
             d=576, rot=64, inter=True),
        # a whole prompt of 10,000 tokens into the block-scaled cache
        dict(name="append_prompt", op="append", kind="block", R=1, new=10000, lo=0, hi=0, pad=0, Hq=64, Hkv=8, d=128,
             rot=128, inter=False),
        # a handful of short sequences: latency
        dict(name="decode_few", op="decode", R=4, lo=16, hi=200, Hq=8, Hkv=2, qs=1.0),
        # a decode step of 256 sequences, 16 query heads a KV head
        dict(name="decode_batch", op="decode", R=256, lo=2000, hi=3000, Hq=64, Hkv=4, qs=1.0),
        # the decode half of a mixed step: very different lengths, 8 query heads a KV head
        dict(name="decode_ragged", op="decode", R=192, lo=1000, hi=8000, Hq=64, Hkv=8, qs=3.0),
        # one long sequence alone: the split of one context over the whole GPU
        dict(name="decode_long", op="decode", R=1, lo=100003, hi=100003, Hq=64, Hkv=8, qs=1.0),
        # the check of a few drafted tokens for each sequence
        dict(name="extend_draft", op="extend", R=32, new=4, lo=1000, hi=4000, Hq=64, Hkv=8, qs=1.0),
        # chunks of prompts over what earlier chunks left in the cache
        dict(name="extend_chunks", op="extend", R=8, new=512, lo=4000, hi=32000, Hq=64, Hkv=8, qs=1.0),
        # the last chunk of one very long prompt
        dict(name="extend_long", op="extend", R=1, new=2048, lo=100000, hi=100000, Hq=64, Hkv=8, qs=2.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "extend"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        kind = rng.choice(["bf16", "tensor", "block", "block", "latent"])
        new = rng.choice([1, 1, _log_int(rng, 2, 4000)])
        R = _log_int(rng, 1, max(1, min(256, 10000 // new)))
        lo = rng.choice([0, _log_int(rng, 1, 4000)])
        lo = min(lo, 400000 // R)
        hi = lo + _log_int(rng, 1, max(1, min(2000, 400000 // R))) - 1
        d = 576 if kind == "latent" else 128 if kind == "block" else rng.choice([64, 128])
        rot = 64 if kind == "latent" else rng.choice([d, d, d // 2, 32])
        if kind == "latent":
            Hkv, Hq = 1, 16 * rng.choice([1, 2, 4, 8]) if new == 1 else 16
        else:
            Hq = min(64, Hkv * G)
            Hq -= Hq % Hkv
        return dict(op=op, kind=kind, R=R, new=new, lo=lo, hi=hi, pad=rng.choice([0, 0, rng.randint(1, 9)]), Hq=Hq,
                    Hkv=Hkv, d=d, rot=rot, inter=rng.random() < 0.4)
    qs = rng.choice([1.0, 1.0, 3.0])
    if op == "decode":
        R = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, max(1, min(100000, 6_000_000 // (R * Hkv))))
        lo = max(1, int(hi * rng.choice([1.0, rng.random()])))
        return dict(op=op, R=R, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, qs=qs)
    R = _log_int(rng, 1, 24)
    new = _log_int(rng, 1, 700)
    most = 2e12 / (4.0 * Hkv * G * D * R * new)
    hi = _log_int(rng, 1, max(1, min(32000, int(most))))
    lo = rng.choice([hi, int(hi * rng.random())])
    return dict(op=op, R=R, new=new, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, qs=qs)


def _spread(lo, hi, n):
    """n lengths spread evenly over [lo, hi]."""
    return [lo + ((hi - lo) * (2 * i + 1) + n) // (2 * n) for i in range(n)]


def _contexts(case):
    return _spread(case["lo"], case["hi"], case["R"])


def work(case):
    R, Hq, Hkv = case["R"], case["Hq"], case["Hkv"]
    ctx = _contexts(case)
    blocks = sum((c + BS - 1) // BS for c in ctx)
    if case["op"] == "append":
        T, d, rot = R * case["new"], case["d"], case["rot"]
        kind = case["kind"]
        by = 2 * T * Hq * d * 2 + T * rot * 4 + 16 * T
        if kind == "latent":
            by += T * d * 2 * 3
        else:
            by += T * Hkv * d * (2 + 2 + 2) + 2 * T * Hkv * d * (2 if kind == "bf16" else 1)
        return {"bytes": by, "flops": 3 * T * (Hq + Hkv) * rot}
    cache = 2 * sum(ctx) * Hkv * D + 8 * blocks * Hkv + 4 * blocks
    if case["op"] == "decode":
        return {"bytes": cache + 2 * R * Hq * D * 2 + 4 * R * Hq, "flops": 4 * Hq * D * sum(ctx)}
    n = case["new"]
    pairs = sum(n * c + n * (n + 1) // 2 for c in ctx)
    return {"bytes": cache + R * n * (2 * Hq * D * 2 + 2 * Hkv * D * 2 + 4 * Hq), "flops": 4 * Hq * D * pairs}


# ---- the inputs ----------------------------------------------------------------------------------

def _generators(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    dg = torch.Generator(device=DEV)
    dg.manual_seed(seed + 1)
    return g, dg


def _tables(need, g):
    """Block tables [R, most] over a shuffled pool 1.2 times as large as needed."""
    nb = max(1, math.ceil(1.2 * sum(need)))
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    t = torch.zeros((len(need), max([1] + need)), dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = perm[at:at + n]
        at += n
    return t, nb


def _block_cache(nb, Hkv, dg, pow2):
    """Codes [nb, 16, Hkv, 128] and scales [nb, Hkv] of normal values whose size differs from block to block."""
    codes = torch.empty((nb, BS, Hkv, D), dtype=torch.uint8, device=DEV)
    scales = torch.empty((nb, Hkv), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (BS * Hkv * D))
    for s in range(0, nb, step):
        e = min(nb, s + step)
        x = torch.randn((e - s, BS, Hkv, D), generator=dg, device=DEV)
        x *= torch.exp(0.4 * torch.randn((e - s, 1, Hkv, 1), generator=dg, device=DEV))
        sc = x.abs().amax(dim=(1, 3)) / 448.0
        if pow2:
            sc = torch.exp2(torch.ceil(torch.log2(sc)))
        scales[s:e] = sc
        codes[s:e] = (x / sc[:, None, :, None]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
    return codes, scales


def _rope_table(rot):
    """[MAX_POS, rot] fp32: the cosines of rot / 2 frequencies, then the sines."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(MAX_POS, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g, dg = _generators(seed)
    R, Hq, Hkv = case["R"], case["Hq"], case["Hkv"]
    ctx = _contexts(case)
    ctx = [ctx[i] for i in torch.randperm(R, generator=g).tolist()]
    new = case.get("new", 1)

    def normal(*shape):
        return torch.randn(shape, generator=dg, device=DEV).to(torch.bfloat16)

    st = dict(case=case)
    if case["op"] == "append":
        d, kind = case["d"], case["kind"]
        table, nb = _tables([(c + new + BS - 1) // BS for c in ctx], g)
        pos = torch.cat([torch.arange(c, c + new) for c in ctx])
        req = torch.arange(R).repeat_interleave(new)
        slot = table[req, pos // BS].long() * BS + pos % BS
        T = R * new
        # rows behind the batch's tokens (a batch padded to a fixed size): slot -1
        slot = torch.cat([slot, torch.full((case["pad"],), -1)])
        pos = torch.cat([pos, torch.zeros(case["pad"], dtype=torch.int64)])
        Tp = T + case["pad"]
        st.update(T=T, q=normal(Tp, Hq, d), k=normal(Tp, Hkv, d), v=normal(Tp, Hkv, d) if kind != "latent" else None,
                  pos=pos.to(DEV), slot=slot.to(DEV), rope=_rope_table(case["rot"]), off=512 if kind == "latent" else 0,
                  q_out=torch.zeros((Tp, Hq, d), dtype=torch.bfloat16, device=DEV),
                  k_out=torch.zeros((Tp, Hkv, d), dtype=torch.bfloat16, device=DEV))
        if kind == "block":
            # what earlier appends left: scales that are powers of two
            kc, ks = _block_cache(nb, Hkv, dg, True)
            vc, vs = _block_cache(nb, Hkv, dg, True)
            st.update(kc=kc, vc=vc, ks=ks, vs=vs)
        elif kind == "tensor":
            st.update(kc=torch.randint(0, 120, (nb, BS, Hkv, d), dtype=torch.uint8, generator=dg, device=DEV),
                      vc=torch.randint(0, 120, (nb, BS, Hkv, d), dtype=torch.uint8, generator=dg, device=DEV),
                      ks=5.0 / 448.0, vs=4.5 / 448.0)
        else:
            st.update(kc=normal(nb, BS, Hkv, d), vc=normal(nb, BS, Hkv, d) if kind == "bf16" else None)
        return st
    if case["op"] == "decode":
        n_new, total = 1, [max(c, 1) for c in ctx]
    else:
        n_new, total = new, [c + new for c in ctx]
    T = R * n_new
    table, nb = _tables([(t + BS - 1) // BS for t in total], g)
    kc, ks = _block_cache(nb, Hkv, dg, False)
    vc, vs = _block_cache(nb, Hkv, dg, False)
    q = (torch.randn((T, Hq, D), generator=dg, device=DEV) * case["qs"]).to(torch.bfloat16)
    st.update(ctx=ctx, total=total, q=q, table=table.to(DEV), lens=torch.tensor(total, dtype=torch.int32, device=DEV),
              kc=kc, vc=vc, ks=ks, vs=vs, out=torch.zeros_like(q),
              lse=torch.zeros((T, Hq), dtype=torch.float32, device=DEV), max_len=max(total))
    if case["op"] == "extend":
        st.update(k_new=normal(T, Hkv, D), v_new=normal(T, Hkv, D),
                  cu=torch.arange(0, T + 1, n_new, dtype=torch.int32, device=DEV))
    else:
        # the scratch that a program keeps for its decode calls (more than any shape here asks for)
        st["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return st


# ---- one pass ------------------------------------------------------------------------------------

def _rotate(x, cos, sin, off, inter):
    """x [T, H, d] fp32 with dims off .. off + 2 n - 1 rotated; cos, sin [T, n]."""
    n = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    w = x[..., off:off + 2 * n]
    if inter:
        a, b = w[..., 0::2], w[..., 1::2]
        y[..., off:off + 2 * n:2] = a * c - b * s
        y[..., off + 1:off + 2 * n:2] = b * c + a * s
    else:
        a, b = w[..., :n], w[..., n:]
        y[..., off:off + n] = a * c - b * s
        y[..., off + n:off + 2 * n] = b * c + a * s
    return y


def _codes(x):
    return x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _inverse(scale):
    """1 / scale in 32 bits."""
    return float(1.0 / torch.tensor(scale, dtype=torch.float32))


def _append_scaled(x, slot, codes, scales):
    """Append rows x [T, H, d] (fp32) at `slot` to E4M3 codes with a power-of-two scale a block and head."""
    T = x.shape[0]
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
    q = _rotate(st["q"][:T].float(), cos, sin, st["off"], case["inter"])
    k = _rotate(st["k"][:T].float(), cos, sin, st["off"], case["inter"])
    st["q_out"][:T] = q.to(torch.bfloat16)
    st["k_out"][:T] = k.to(torch.bfloat16)
    kc, vc = st["kc"], st["vc"]
    if case["kind"] == "block":
        _append_scaled(k, slot, kc, st["ks"])
        _append_scaled(st["v"][:T].float(), slot, vc, st["vs"])
    elif case["kind"] == "tensor":
        kc.view(-1, *kc.shape[2:])[slot] = _codes(k * _inverse(st["ks"]))
        vc.view(-1, *vc.shape[2:])[slot] = _codes(st["v"][:T].float() * _inverse(st["vs"]))
    else:
        kc.view(-1, *kc.shape[2:])[slot] = k.to(torch.bfloat16)
        if vc is not None:
            vc.view(-1, *vc.shape[2:])[slot] = st["v"][:T]


def _gathered(codes, scales, table):
    """[R, H, n * 16, 128] fp32 values of the blocks in table [R, n]."""
    x = codes[table].view(E4M3).float() * scales[table][:, :, None, :, None]
    R, n, _, H, d = x.shape
    return x.reshape(R, n * BS, H, d).transpose(1, 2)


def _plain_decode(st):
    q, lens = st["q"].float(), st["lens"]
    R, Hq, d = q.shape
    Hkv = st["kc"].shape[2]
    t = st["table"].long()
    k = _gathered(st["kc"], st["ks"], t)
    s = torch.matmul(q.view(R, Hkv, Hq // Hkv, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    s = s.masked_fill((torch.arange(s.shape[-1], device=q.device)[None] >= lens[:, None])[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gathered(st["vc"], st["vs"], t)) / l
    return o.reshape(R, Hq, d).to(torch.bfloat16), (m + torch.log(l)).reshape(R, Hq)


def _plain_extend(st):
    n, Hkv = st["case"]["new"], st["case"]["Hkv"]
    q, kn, vn = st["q"], st["k_new"], st["v_new"]
    Hq = q.shape[1]
    G = Hq // Hkv
    out, lse = torch.empty_like(q), torch.empty_like(st["lse"])
    i = torch.arange(n, device=q.device)
    for r, c in enumerate(st["ctx"]):  # requests of very different contexts, one after another
        rows = slice(r * n, (r + 1) * n)
        t = st["table"][r:r + 1, :(c + BS - 1) // BS].long()
        k = torch.cat([_gathered(st["kc"], st["ks"], t)[0, :, :c], kn[rows].transpose(0, 1).float()], 1)
        x = q[rows].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        s = torch.matmul(x, k.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).view(Hkv, G, n, c + n)
        s[..., c:] = s[..., c:].masked_fill(i[None, :] > i[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        v = torch.cat([_gathered(st["vc"], st["vs"], t)[0, :, :c], vn[rows].transpose(0, 1).float()], 1)
        o = torch.matmul(p.view(Hkv, G * n, c + n), v).view(Hkv, G, n, D) / l
        out[rows] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(torch.bfloat16)
        lse[rows] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(n, Hq)
    return out, lse


def _appended(st):
    """What an append leaves: the rotated rows and the cache, codes as the E4M3 numbers they stand for."""
    kind, T = st["case"]["kind"], st["T"]
    r = dict(q=st["q_out"][:T], k=st["k_out"][:T])
    if kind in ("bf16", "latent"):
        r.update(k_cache=st["kc"], v_cache=st["vc"])
    else:
        r.update(k_cache=st["kc"].view(E4M3), v_cache=st["vc"].view(E4M3))
    if kind == "block":
        r.update(k_scale=st["ks"], v_scale=st["vs"])
    return r


def run(state):
    st = state
    op = st["case"]["op"]
    if own:
        import paged_kv_attention_reshape_gb300 as pkv
        if op == "append":
            more = dict(k_scale=st["ks"], v_scale=st["vs"]) if "ks" in st else {}
            pkv.kv_append(st["q"], st["k"], st["v"], st["pos"], st["slot"], st["kc"], st["vc"], st["rope"],
                          rope_offset=st["off"], interleaved=st["case"]["inter"], q_out=st["q_out"], k_out=st["k_out"],
                          **more)
            return _appended(st)
        if op == "decode":
            return pkv.paged_decode_attn(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["max_len"], out=st["out"],
                                         lse=st["lse"], workspace=st["ws"], k_scale=st["ks"], v_scale=st["vs"])
        return pkv.extend_attn(st["q"], st["k_new"], st["v_new"], st["cu"], st["lens"], st["kc"], st["vc"], st["table"],
                               st["case"]["new"], st["max_len"], out=st["out"], lse=st["lse"], k_scale=st["ks"],
                               v_scale=st["vs"])
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
    rot, off = st["rope"].shape[1], st["off"]
    t = st["rope"][p].double()
    z = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
    w = x[..., off:off + rot]
    if st["case"]["inter"]:
        w = torch.view_as_real(torch.view_as_complex(w.reshape(*w.shape[:-1], rot // 2, 2).contiguous()) * z).flatten(-2)
    else:
        y = torch.complex(w[..., :rot // 2].contiguous(), w[..., rot // 2:].contiguous()) * z
        w = torch.cat([y.real, y.imag], -1)
    return torch.cat([x[..., :off], w, x[..., off + rot:]], -1)


def _exact_append(st):
    T, kind, new = st["T"], st["case"]["kind"], st["case"]["new"]
    slot, pos = st["slot"][:T], st["pos"][:T]
    q, k = (_turn(st[n][:T].double(), pos, st) for n in ("q", "k"))
    r = dict(q=q, k=k)
    for name, x in (("k", k), ("v", None if st["v"] is None else st["v"][:T].double())):
        cache = st[name + "c"]
        if x is None:
            r[name + "_cache"] = None
            continue
        if kind in ("bf16", "latent"):
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
    return r


def exact(case, seed):
    if case["op"] == "extend" and work(case)["flops"] > 4e12:
        return None  # too long in 64 bits
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    Hkv, n = case["Hkv"], case.get("new", 1) if case["op"] == "extend" else 1
    Hq = case["Hq"]
    out = torch.empty((case["R"] * n, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((case["R"] * n, Hq), dtype=torch.float64, device=DEV)
    for r, L in enumerate(st["total"]):
        c = L if case["op"] == "decode" else L - n
        j = torch.arange(c, device=DEV)
        b = st["table"][r].long()[j // BS]
        for h in range(Hkv):
            hq = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k = st["kc"].view(E4M3)[b, j % BS, h].double() * st["ks"][b, h].double()[:, None]
            v = st["vc"].view(E4M3)[b, j % BS, h].double() * st["vs"][b, h].double()[:, None]
            if case["op"] == "extend":
                k = torch.cat([k, st["k_new"][r * n:(r + 1) * n, h].double()])
                v = torch.cat([v, st["v_new"][r * n:(r + 1) * n, h].double()])
            x = torch.einsum("tgd,jd->tgj", st["q"][r * n:(r + 1) * n, hq].double(), k) / math.sqrt(D)
            if case["op"] == "extend":
                i = torch.arange(n, device=DEV)
                x[:, :, c:] += torch.where(i[None, :] > i[:, None], -math.inf, 0.0)[:, None, :]
            z = torch.logsumexp(x, -1)
            lse[r * n:(r + 1) * n, hq] = z
            out[r * n:(r + 1) * n, hq] = torch.einsum("tgj,jd->tgd", torch.exp(x - z[..., None]), v)
    return out, lse
