"""A windowed model's serving steps as an engine makes them, two layers on one pool of blocks: prompts in chunks (append with
norms and rotation, windowed extend), pages given back as they slide out, sequences forked with a copy of their last block in
every layer, decode steps of all of them. Every attention is compared with a dense softmax in 64 bits over
the keys as they were appended, kept apart from the pool; the appended rows with the formula."""
import math

import pytest
import torch

from test_append_norm import close, formula, rope_table
from test_window import U, seen_mask

BS, HQ, HKV, D, L = 16, 8, 2, 128, 2
WINDOW, SINKS, EPS = 50, 6, 1e-5


class Engine:
    """A pool of blocks, its free list, and the sequences: block numbers (-1: given back) and what was appended."""

    def __init__(self, kind, blocks=64):
        import paged_kv_attention_reshape_gb300 as pkv
        self.kind, self.g = kind, torch.Generator().manual_seed(11)
        bf = kind == "bf16"
        new = lambda: torch.full((blocks, BS, HKV, D), math.nan if bf else 0x7F, dtype=torch.bfloat16 if bf else torch.uint8, device="cuda")
        self.k, self.v = [new() for _ in range(L)], [new() for _ in range(L)]
        if not bf:
            for c in self.k + self.v:
                c.fill_(0x7F)  # NaN codes
        self.scales = {} if bf else dict(k_scale=0.03, v_scale=0.02)
        self.free = torch.randperm(blocks, generator=self.g).tolist()
        self.layers = pkv.CacheLayers(self.k, self.v)
        self.table = rope_table(D, 1000).cuda()
        self.w = [(1 + 0.2 * torch.randn(D, generator=self.g)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.seqs = []  # dict(blocks, n, k [L] of [n, HKV, D] doubles, v)

    def add(self):
        self.seqs.append(dict(blocks=[], n=0, k=[torch.zeros(0, HKV, D, dtype=torch.float64)] * L,
                              v=[torch.zeros(0, HKV, D, dtype=torch.float64)] * L))
        return len(self.seqs) - 1

    def fork(self, i):
        """Full blocks are shared, the last, partly filled one is copied in every layer."""
        import paged_kv_attention_reshape_gb300 as pkv
        s = self.seqs[i]
        t = dict(blocks=list(s["blocks"]), n=s["n"], k=list(s["k"]), v=list(s["v"]))
        if s["n"] % BS:
            t["blocks"][-1] = self.free.pop()
            ids = lambda x: torch.tensor([x, -1], dtype=torch.int32, device="cuda")
            pkv.kv_block_copy(self.layers, ids(s["blocks"][-1]), ids(t["blocks"][-1]))
        self.seqs.append(t)
        return len(self.seqs) - 1

    def step(self, batch):
        """batch: (sequence, new tokens); one append and one attention a layer."""
        import paged_kv_attention_reshape_gb300 as pkv
        T = sum(n for _, n in batch)
        pos, slot, cu = [], [], [0]
        for i, n in batch:
            s = self.seqs[i]
            while len(s["blocks"]) * BS < s["n"] + n:
                s["blocks"].append(self.free.pop())
            p = range(s["n"], s["n"] + n)
            pos += p
            slot += [s["blocks"][x // BS] * BS + x % BS for x in p]
            cu.append(cu[-1] + n)
            # pages that no later row sees are given back
            low = s["n"] - WINDOW + 1
            for b in range(len(s["blocks"])):
                if b * BS >= SINKS and b * BS + BS - 1 < low:
                    s["blocks"][b] = -1
        width = max(len(self.seqs[i]["blocks"]) for i, _ in batch)
        table = torch.tensor([self.seqs[i]["blocks"] + [-1] * (width - len(self.seqs[i]["blocks"])) for i, _ in batch],
                             dtype=torch.int32, device="cuda")
        lens = torch.tensor([self.seqs[i]["n"] + n for i, n in batch], dtype=torch.int32, device="cuda")
        pos, slot = torch.tensor(pos, device="cuda"), torch.tensor(slot, device="cuda")
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for layer in range(L):
            q, k, v = (torch.randn((T, h, D), generator=self.g).to(torch.bfloat16).cuda() for h in (HQ, HKV, HKV))
            kc, vc = self.k[layer], self.v[layer]
            qo, ko = pkv.kv_append(q, k, v, pos, slot, kc, vc, self.table, q_norm=self.w[0], k_norm=self.w[1], norm_eps=EPS,
                                   **self.scales)
            for got, x, w in ((qo, q, self.w[0]), (ko, k, self.w[1])):
                close(got, *formula(x, w, pos, self.table, 0, False))
            mask = dict(window=WINDOW, sinks=SINKS, **self.scales)
            longest, most = int(lens.max()), max(n for _, n in batch)
            if most == 1:
                out, lse = pkv.paged_decode_attn(qo, kc, vc, table, lens, longest, **mask)
            else:
                out, lse = pkv.extend_attn(qo, ko, v, cu, lens, kc, vc, table, most, longest, **mask)
            self.verify(layer, batch, qo.cpu(), ko.cpu(), v.cpu(), slot.cpu(), out.cpu(), lse.cpu(), most == 1)
        for i, n in batch:
            self.seqs[i]["n"] += n

    def stored(self, cache, slot, scale):
        rows = cache.view(-1, HKV, D)[slot.cuda()].cpu()
        return rows.double() if self.kind == "bf16" else rows.view(torch.float8_e4m3fn).float().double() * scale

    def verify(self, layer, batch, q, k, v, slot, out, lse, decode):
        at = 0
        for i, n in batch:
            s, rows = self.seqs[i], slice(at, at + n)
            kept = [self.stored(c[layer], slot[rows], self.scales.get(x, 1.0))
                    for c, x in ((self.k, "k_scale"), (self.v, "v_scale"))]
            own = kept if decode else (k[rows].double(), v[rows].double())  # (an extend takes its new rows as they come)
            keys, vals = torch.cat([s["k"][layer], own[0]]), torch.cat([s["v"][layer], own[1]])
            c = s["n"]
            seen = seen_mask(torch.arange(c, c + n), torch.arange(c + n), WINDOW, SINKS)
            scale = 1.0 / math.sqrt(D)
            for h in range(HQ):
                x, kh, vh = q[rows, h].double(), keys[:, h // (HQ // HKV)], vals[:, h // (HQ // HKV)]
                z = (x @ kh.T * scale).masked_fill(~seen, -math.inf)
                mag = (x.abs() @ kh.abs().T * scale).masked_fill(~seen, 0).amax(-1)
                want = torch.logsumexp(z, -1)
                p = torch.exp(z - want[:, None])
                # the bounds of test_window.py, the 8-bit cache's terms included
                e = 2.0 ** -16 * mag + 2.0 ** -20 * (1 + want.abs()) + 2.0 ** -21 * scale * x.abs().max() * kh.abs().sum(-1).max()
                tol = U * (p @ vh).abs() + (U + 2 * e[:, None] + 2.0 ** -11 + (c + n) * 2.0 ** -23) * (p @ vh.abs()) \
                    + 2.0 ** -22 * (seen.double() @ vh.abs())
                assert torch.all((out[rows, h].double() - p @ vh).abs() <= tol)
                assert torch.all((lse[rows, h].double() - want).abs() <= e)
            s["k"][layer] = torch.cat([s["k"][layer], kept[0]])
            s["v"][layer] = torch.cat([s["v"][layer], kept[1]])
            at += n


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "tensor"])
def test_serving(kind):
    import paged_kv_attention_reshape_gb300 as pkv
    eng = Engine(kind)
    a, b = eng.add(), eng.add()
    eng.step([(a, 37), (b, 3)])
    eng.step([(a, 60), (b, 64)])          # b's first chunk behind it: a second one over a cache
    forks = [eng.fork(a) for _ in range(3)] + [eng.fork(b)]
    everyone = [a, b] + forks
    for _ in range(3):                    # the forks part: each appends its own tokens behind the copied block
        eng.step([(i, 1) for i in everyone])
    eng.step([(i, 1 + 5 * (i % 3)) for i in everyone])
    late = eng.fork(forks[0])             # of a sequence whose early pages are gone
    eng.step([(i, 1) for i in everyone + [late]])
    assert pkv.device_errors() == 0
    assert any(-1 in s["blocks"] for s in eng.seqs)
