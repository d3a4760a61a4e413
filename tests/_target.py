"""Inputs and 64-bit references of the target's side of a step, shared by its tests."""
import math

import numpy as np
import torch

import speculative_decoding_03_gb300 as ds

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tree_parents(n, g):
    """A random tree of n tokens (list), nearer parents likelier."""
    u = torch.rand(n, generator=g, device="cuda").tolist()
    return [-1] + [min(i - 1, int(i * math.sqrt(u[i]))) for i in range(1, n)]


def depths(parents):
    d = []
    for i, p in enumerate(parents):
        d.append(0 if p < 0 else d[p] + 1)
    return d


def sees(parents, i):
    s = []
    while i >= 0:
        s.append(i)
        i = parents[i]
    return s


class Batch:
    """Requests with counts and lengths, padded or packed, chains or trees, and their pages."""

    def __init__(self, counts, lengths, page, seed=0, packed=False, tree=False, N=None, spare=2, extra_rows=3,
                 room=0):
        g = gen(seed)
        self.counts, self.lengths, self.page = list(counts), list(lengths), page
        self.B, self.N = len(counts), N or max(max(counts), 1)
        self.trees = [tree_parents(n, g) if tree else list(range(-1, n - 1)) for n in counts]
        if packed:
            self.first = np.concatenate([[0], np.cumsum(counts)]).astype(int).tolist()
            self.rows = self.first[-1] + extra_rows
            self.lead = (self.rows,)
            self.kw = dict(starts=i32(self.first), nodes=self.N)
        else:
            self.first = [b * self.N for b in range(self.B)]
            self.rows = self.B * self.N
            self.lead = (self.B, self.N)
            self.kw = dict(counts=i32(self.counts))
        self.live = [(b, i, self.first[b] + i) for b in range(self.B) for i in range(counts[b])]
        if tree:
            p = torch.full((self.rows,), -7, dtype=torch.int32)       # rows of no token hold anything
            for b, i, row in self.live:
                p[row] = self.trees[b][i]
            self.kw["parents"] = p.cuda().view(self.lead)
        each = [-(-(l + n + room) // page) for l, n in zip(lengths, counts)]
        self.max_pages = max(max(each), 1)
        self.n_pages = sum(each) + spare
        order = torch.rand(self.n_pages, generator=g, device="cuda").argsort().tolist()
        table = np.full((self.B, self.max_pages), -5, dtype=np.int32)   # entries without a slot hold anything
        at = 0
        for b, k in enumerate(each):
            table[b, :k] = order[at:at + k]
            at += k
        self.table = table
        self.pages, self.lens = torch.from_numpy(table).cuda(), i32(self.lengths)

    def place(self, b, slots):
        slots = np.asarray(slots)
        return (torch.from_numpy(self.table[b, slots // self.page].astype(np.int64)).cuda(),
                torch.from_numpy((slots % self.page).astype(np.int64)).cuda())

    def live_rows(self):
        return torch.tensor([row for _, _, row in self.live], dtype=torch.long, device="cuda")


def new_cache(batch, heads, D, dtype, seed=1, layers=0, order="slots", fill=float("nan")):
    """k, v [(layers,) pages, page, heads, D] of ``fill`` (NaN: nothing may read what was not written)."""
    shape = ((layers,) if layers else ()) + ((batch.n_pages, batch.page, heads, D) if order == "slots"
                                             else (batch.n_pages, heads, batch.page, D))
    kv = [torch.full(shape, fill, dtype=dtype, device="cuda") for _ in range(2)]
    return [t if order == "slots" else t.transpose(-3, -2) for t in kv]


def fill_cache(batch, k, v, seed=2, tokens=True):
    """Random values in every slot in use (and the step's tokens' slots)."""
    g = gen(seed)
    for b in range(batch.B):
        end = batch.lengths[b] + (batch.counts[b] if tokens else 0)
        if end:
            page, line = batch.place(b, np.arange(end))
            for t in (k, v):
                t[page, line] = torch.randn((end,) + t.shape[2:], generator=g, device="cuda").to(t.dtype)


def attention_reference(batch, q, k, v, scale):
    """(out, lse, spread) in 64 bits for the live rows: spread is sum p |v| (per element), and the
    largest sum |q k| scale of a row."""
    Hkv, D = k.shape[-2:]
    qf = q.reshape(batch.rows, q.shape[-2], D)
    out, lse, spread, size = [], [], [], []
    for b in range(batch.B):
        n, l = batch.counts[b], batch.lengths[b]
        if not n:
            continue
        page, line = batch.place(b, np.arange(l + n))
        kk, vv = k[page, line].double(), v[page, line].double()
        mask = torch.zeros(n, l + n, dtype=torch.bool)
        mask[:, :l] = True
        for i in range(n):
            mask[i, [l + a for a in sees(batch.trees[b], i)]] = True
        mask = mask.cuda()[:, None, None]
        x = qf[batch.first[b]:batch.first[b] + n].double().view(n, Hkv, -1, D)
        s = torch.einsum("nhgd,lhd->nhgl", x, kk) * scale
        s = torch.where(mask, s, -math.inf)
        p = torch.softmax(s, -1)
        vis = torch.where(mask, 1.0, 0.0)
        o = torch.stack([torch.einsum("hgl,lhd->hgd", p[i], torch.where(mask[i, 0, 0][:, None, None], vv, 0.0))
                         for i in range(n)])
        a = torch.stack([torch.einsum("hgl,lhd->hgd", p[i], torch.where(mask[i, 0, 0][:, None, None], vv, 0.0).abs())
                         for i in range(n)])
        big = torch.einsum("nhgd,lhd->nhgl", x.abs(), torch.nan_to_num(kk).abs()) * scale * vis
        out.append(o.reshape(n, -1, D))
        lse.append(torch.logsumexp(s, -1).reshape(n, -1))
        spread.append(a.reshape(n, -1, D))
        size.append(big.amax(-1).reshape(n, -1))
    return torch.cat(out), torch.cat(lse), torch.cat(spread), torch.cat(size)


def attention_tolerance(batch, ref, spread, size, v, dtype):
    """Of every output: its own rounding; the probabilities' rounding (half a step each, against
    sum p |v|); the scores' fp32 sums over D (2^-23 a term of sum |q k|) and their exponent (2^-22 and
    2^-23 of the score), twice, for numerator and denominator; the products' and sums' fp32
    accumulation over the slots; in fp16 half of 2^-24 a slot where p is below its normal range (the
    sum is at least 1)."""
    u, D, L = HALF[dtype], ref.shape[-1], max(batch.lengths) + batch.N
    rel = u + 2 * (size * (D + 4) * 2.0 ** -23 + 2.0 ** -21)[..., None] + (L / 8 + 64) * 2.0 ** -23
    tol = u * ref.abs() + spread * rel * (1 + u)
    if dtype is torch.float16:
        tol = tol + L * 2.0 ** -25 * float(torch.nan_to_num(v.float()).abs().max()) + 2.0 ** -25
    return tol


def verify_reference(batch, p, tokens, uniforms, q=None):
    """accept_len, path, out_tokens, n_out by the definition, request by request."""
    B, N, V = batch.B, batch.N, p.shape[-1]
    P = p.reshape(batch.rows, V).float().cpu().numpy().astype(np.float64)
    Q = None if q is None else q.reshape(batch.rows, V).float().cpu().numpy().astype(np.float64)
    tok, u = tokens.reshape(-1).cpu().numpy(), uniforms.reshape(-1).cpu().numpy().astype(np.float64)
    out = dict(accept_len=np.zeros(B, np.int32), path=np.full((B, N), -1, np.int32),
               out_tokens=np.full((B, N), -1, np.int32), n_out=np.zeros(B, np.int32))
    for b in range(B):
        n, f = batch.counts[b], batch.first[b]
        if not n:
            continue
        at, r, s, a = 0, P[f].copy(), 1.0, 0
        for i in range(1, n):
            if batch.trees[b][i] != at:
                continue
            x = tok[f + i]
            if x < 0 or x >= V:
                continue
            if u[f + i] * (1.0 if Q is None else Q[f + at, x]) * s < r[x]:
                out["path"][b, a], out["out_tokens"][b, a] = i, x
                a, at, r, s = a + 1, i, P[f + i].copy(), 1.0
            elif Q is None:
                s -= r[x]
                r[x] = 0.0
            else:
                r = np.maximum(r - s * Q[f + at], 0.0).astype(np.float32).astype(np.float64)
                s = float(np.float32(r.sum()))
        if not r.sum() > 0:
            r = P[f + at]
        up_to = np.cumsum(r)
        if up_to[-1] > 0:
            out["out_tokens"][b, a] = min(int(np.searchsorted(up_to, u[f] * up_to[-1], side="right")),
                                          int(np.nonzero(r > 0)[0][-1]))
        out["accept_len"][b], out["n_out"][b] = a, a + 1
    return out


def workspace(batch=None, q_heads=1, heads=1, D=128):
    return ds.Workspace.of_bytes(256 if batch is None else
                                 ds.tree_attention_workspace_bytes(batch.B, batch.N, q_heads, heads, D))
