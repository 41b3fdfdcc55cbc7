"""Inputs and fp64 references of the paged-cache, tree-attention and log-probability tests."""
import math
import random

import torch

HALF_BF16 = 2.0 ** -8        # the largest relative error of one rounding to bf16
HALF_E4M3 = 2.0 ** -4        # ... to E4M3 (normal numbers)
F32 = 2.0 ** -24


class Paged:
    """A paged cache and a batch over it. Slots that no sequence owns hold NaN (E4M3: the
    NaN code), pages are handed out in random order and one page belongs to nobody."""

    def __init__(self, n, ctx, n_kv, d, page=16, kv="bf16", layout="hnd", seed=0, device="cuda", rows=None, extra_pages=0,
                 k_scale=0.0625, v_scale=0.04, layers=None):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.n, self.ctx, self.n_kv, self.d, self.page, self.kv = n, ctx, n_kv, d, page, kv
        B = len(n)
        per = [-(-(a + c) // page) for a, c in zip(n, ctx)]
        self.width = max(per + [1]) + extra_pages
        self.pages = sum(per) + 1
        order = torch.randperm(self.pages, generator=g, device=device)
        table = torch.full((B, self.width), -7, dtype=torch.int32)      # entries behind the last page are not read
        at = 0
        for b, p in enumerate(per):
            table[b, :p] = order[at:at + p].cpu().int()
            at += p
        self.table = table.to(device)
        starts = [0]
        for a in n:
            starts.append(starts[-1] + a)
        self.starts, self.T = starts, starts[-1] if rows is None else rows
        self.q_start = torch.tensor(starts, dtype=torch.int32, device=device)
        self.ctx_len = torch.tensor(ctx, dtype=torch.int32, device=device)
        self.f8 = kv == "e4m3"
        self.ks, self.vs = (k_scale, v_scale) if self.f8 else (1.0, 1.0)
        lead = () if layers is None else (layers,)
        inner = (n_kv, page, d) if layout == "hnd" else (page, n_kv, d)
        shape = (*lead, self.pages, *inner) if layout != "interleaved" else (*lead, self.pages, 2, n_kv, page, d)
        if layout == "interleaved":                                     # K and V of a page in one allocation
            both = self._fresh(shape, g, device)
            self.k, self.v = both.select(-4, 0), both.select(-4, 1)
        else:
            self.k, self.v = self._fresh(shape, g, device), self._fresh(shape, g, device)
            if layout == "nhd":
                self.k, self.v = self.k.transpose(-3, -2), self.v.transpose(-3, -2)
        self.blank_unowned()

    def _fresh(self, shape, g, device):
        x = torch.randn(shape, generator=g, device=device)
        if self.f8:
            return (x / 0.05).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return x.to(torch.bfloat16)

    def blank_unowned(self):
        nan = 0x7F if self.f8 else math.nan
        own = torch.zeros(self.pages, self.page, dtype=torch.bool, device=self.k.device)
        for b in range(len(self.n)):
            pg, sl = self.slots(b)
            own[pg, sl] = True
        gone = ~own
        for t in (self.k, self.v):
            if t.dim() == 4:
                t.permute(0, 2, 1, 3)[gone] = nan
            else:
                t.permute(1, 3, 0, 2, 4)[gone] = nan

    def slots(self, b, upto=None):
        i = torch.arange(self.ctx[b] + self.n[b] if upto is None else upto, device=self.k.device)
        return self.table[b].long()[i // self.page], i % self.page

    def values(self, t):
        return t.view(torch.float8_e4m3fn).double() if self.f8 else t.double()

    def keys(self, b, h):
        """fp64 K, V [len, d] of a sequence and kv head."""
        pg, sl = self.slots(b)
        return self.values(self.k[pg, h, sl]) * self.ks, self.values(self.v[pg, h, sl]) * self.vs

    def handles(self, m, max_new=None):
        return (m.make_kv_cache(self.k, self.v, self.ks, self.vs),
                m.make_kv_batch(self.q_start, self.ctx_len, self.table, max(self.n + [0]) if max_new is None else max_new))


def tree_sets(n, seed):
    """Ancestor-or-self sets (whole numbers) of a random tree of n nodes, parents first."""
    r = random.Random(seed)
    sets = []
    for i in range(n):
        p = r.randrange(-1, i) if i else -1
        sets.append((sets[p] if p >= 0 else 0) | 1 << i)
    return sets


def mask_tensor(sets, words, device="cuda"):
    def signed(w):
        return w - (1 << 64) if w >= 1 << 63 else w
    return torch.tensor([[signed(w >> 64 * j & (1 << 64) - 1) for j in range(words)] for w in sets], dtype=torch.int64,
                        device=device).reshape(len(sets), words)


def seen_matrix(P, b, sets=None):
    n, ctx = P.n[b], P.ctx[b]
    seen = torch.ones(n, ctx + n, dtype=torch.bool, device=P.k.device)
    if sets is None:
        seen[:, ctx:] = torch.ones(n, n, dtype=torch.bool, device=P.k.device).tril()
    else:
        rows = sets[P.starts[b]:P.starts[b] + n]
        seen[:, ctx:] = torch.tensor([[w >> j & 1 for j in range(n)] for w in rows], dtype=torch.bool,
                                     device=P.k.device).reshape(n, n)
    return seen


def attention_ref(P, q, n_q, sets=None, scale=None, hide=None):
    """fp64 out [T, n_q, d], lse [T, n_q] of the rows that belong to a sequence, and the
    largest errors that the arithmetic allows (tol_out, tol_lse):
      scores are fp32 dots of d terms, |ds| <= (d + 4) 2^-24 sum |q||k| scale =: e;
      p is rounded to 16 bits (2^-8 at most, relative) and carries the score's error
      (e^{2e} - 1 <= 4e with the maximum's own error) and 2^-18 for exp2 and the sums;
      out is rounded once: 2^-8 of itself."""
    d = P.d
    scale = 1 / math.sqrt(d) if scale is None else scale
    T = P.T
    out = torch.zeros(T, n_q, d, dtype=torch.float64, device=q.device)
    lse = torch.full((T, n_q), -math.inf, dtype=torch.float64, device=q.device)
    to, tl = torch.zeros_like(out), torch.zeros_like(lse)
    G = n_q // P.n_kv
    for b in range(len(P.n)):
        if P.n[b] == 0:
            continue
        r0, r1 = P.starts[b], P.starts[b + 1]
        seen = seen_matrix(P, b, sets)
        if hide is not None:
            seen = seen & ~hide[b][None, :]
        for h in range(P.n_kv):
            K, V = P.keys(b, h)
            for g in range(G):
                qq = q[r0:r1].view(r1 - r0, n_q, d)[:, h * G + g].double()
                x = (qq @ K.T) * scale
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, 1)
                p = torch.where(seen, torch.exp(x - z[:, None]), torch.zeros_like(x))
                p = torch.where(torch.isinf(z)[:, None] & (z < 0)[:, None], torch.zeros_like(p), p)
                # what a row does not see contributes nothing, infinities and NaN among it
                Vv = torch.where(torch.isfinite(V), V, torch.zeros_like(V))
                o = p @ Vv
                bad = (~torch.isfinite(V)).double()
                if bool(bad.any()):
                    hit = (seen.double() @ bad) > 0                      # rows that see a value without a number
                    o = torch.where(hit, torch.full_like(o, math.nan), o)
                out[r0:r1, h * G + g] = o
                lse[r0:r1, h * G + g] = z
                Kf = torch.where(torch.isfinite(K), K, torch.zeros_like(K))
                e = (d + 4) * F32 * abs(scale) * torch.where(seen, qq.abs() @ Kf.abs().T, torch.zeros_like(x)).amax(1)
                e = e + F32 * 4 * torch.nan_to_num(x.abs(), posinf=0.0, neginf=0.0).amax(1)
                to[r0:r1, h * G + g] = HALF_BF16 * o.abs() + (HALF_BF16 + 4 * e + 2.0 ** -18)[:, None] * (p @ Vv.abs())
                tl[r0:r1, h * G + g] = 2 * e + 2.0 ** -18 + 4 * F32 * torch.nan_to_num(z.abs(), posinf=0.0)
    return out, lse, to, tl
