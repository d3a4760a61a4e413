"""The target's side of a step as it is used: steps after one another, captured and replayed, on
other streams and with bad tables, and the forms that the kernels choose by size and layout."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")
if torch.cuda.is_available():
    from _target import (HALF, Batch, attention_reference, attention_tolerance, fill_cache, gen, i32, new_cache,
                         verify_reference, workspace)

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEVICE_CHECK = 5


def check_rows(batch, q, k, v, out, live=None):
    ref, _, spread, size = attention_reference(batch, q, k, v, q.shape[-1] ** -0.5)
    tol = attention_tolerance(batch, ref, spread, size, v, q.dtype)
    err = (out.reshape((batch.rows,) + out.shape[-2:])[batch.live_rows()].double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()


# ------------------------------------------------------------- forms chosen by size

PARTS = [
    # counts, lengths, page, q_heads, heads, D
    ([1], [3000], 16, 4, 1, 128),             # 24 parts of a row block, joined by the last of them
    ([1], [3100], 16, 4, 1, 128),             # 25: joined by a kernel of their own
    ([2, 1, 0], [2000, 900, 64], 32, 16, 8, 64),
    ([16], [127], 16, 1, 1, 64),              # two tiles
    ([16], [112], 16, 1, 1, 64),              # a tile that is full: nothing to join
    ([4, 4], [5000, 130], 64, 8, 2, 64),      # 16 rows, 78 parts
    ([17], [2500], 128, 1, 1, 128),           # 17 rows
    ([33, 64], [700, 2100], 16, 2, 2, 128),
    ([64, 3], [4000, 10], 256, 16, 2, 64),    # 512 rows in blocks of 128
    ([40], [9000], 32, 4, 2, 64),             # many parts of 80 rows
    ([8, 3], [7000, 2000], 16, 8, 2, 128),    # and of 32
    ([5] * 33, [40 * i for i in range(33)], 16, 6, 3, 64),       # more requests than a warp looks at
]


@pytest.mark.parametrize("case", PARTS, ids=[f"{i}" for i in range(len(PARTS))])
def test_attention_in_parts(case):
    """Right whatever the parts, and the same bits from call to call on one workspace."""
    counts, lengths, page, Hq, Hkv, D = case
    batch = Batch(counts, lengths, page, seed=21, tree=True)
    k, v = new_cache(batch, Hkv, D, BF16)
    fill_cache(batch, k, v)
    q = torch.randn(batch.lead + (Hq, D), generator=gen(22), device="cuda").to(BF16)
    ws, cache = workspace(batch, Hq, Hkv, D), ds.PagedCache(k, v)
    first = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, out=torch.zeros_like(q), **batch.kw)
    check_rows(batch, q, k, v, first)
    for _ in range(20):
        again = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, out=torch.zeros_like(q), **batch.kw)
        assert torch.equal(again, first)
    assert ws.status() == 0


@pytest.mark.parametrize("page,rows", [(16, 3), (64, 40), (256, 7)])
@pytest.mark.parametrize("layout", ["apart", "in line", "heads first", "one head", "one page"])
def test_attention_layouts_of_a_cache(layout, page, rows):
    """Heads of 128 in lines of their own, side by side, one after the other; tiles that end inside a
    page and pages inside a tile."""
    heads = 1 if layout == "one head" else 3
    lengths = [5, 0] if layout == "one page" else [333, 130]
    if layout == "one page":
        batch = Batch([min(rows, 10)], [2], 16 if page == 16 else page, seed=23, spare=0)
    else:
        batch = Batch([rows, 1], lengths, page, seed=23, tree=rows < 30)
    if layout == "heads first":
        k, v = new_cache(batch, heads, 128, F16, order="heads")
    elif layout == "apart":
        k, v = (t[..., :128] for t in new_cache(batch, heads, 192, F16))
    else:
        k, v = new_cache(batch, heads, 128, F16)
    fill_cache(batch, k, v)
    q = torch.randn(batch.lead + (2 * heads, 128), generator=gen(24), device="cuda").to(F16)
    ws = workspace(batch, 2 * heads, heads)
    out = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, **batch.kw)
    check_rows(batch, q, k, v, out)
    assert ws.status() == 0


@pytest.mark.parametrize("B", [1, 31, 32, 33, 1500])
def test_append_finds_packed_rows(B):
    """Requests of 0, 1 and 2 tokens, far fewer than the bound on them, in a padded batch."""
    rng = np.random.default_rng(B)
    counts = rng.integers(0, 3, B).tolist()
    counts[-1] = 1
    batch = Batch(counts, rng.integers(0, 40, B).tolist(), 16, packed=True, extra_rows=9, N=5000)
    k, v = (torch.randn(batch.rows, 2, 16, generator=gen(25 + i), device="cuda").to(BF16) for i in range(2))
    kc, vc = new_cache(batch, 2, 16, BF16, fill=7.0)
    want_k, want_v = kc.clone(), vc.clone()
    slots = np.array([(b, batch.lengths[b] + i) for b, i, _ in batch.live])
    page = torch.from_numpy(batch.table[slots[:, 0], slots[:, 1] // 16].astype(np.int64)).cuda()
    line = torch.from_numpy(slots[:, 1] % 16).cuda()
    rows = batch.live_rows()
    want_k[page, line], want_v[page, line] = k[rows], v[rows]
    ws = workspace()
    ds.cache_append(ds.PagedCache(kc, vc), k, v, batch.pages, batch.lens, ws, **batch.kw)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and ws.status() == 0


def test_append_turns_at_far_positions():
    """Positions up to 2^29 and frequencies of every size against pi to 60 places.  A pair (1, 0) becomes
    (cos, sin): off by 2^-21 in fp32 and half a step of fp16."""
    getcontext().prec = 60
    tau = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    freq = torch.tensor([1.0, 0.1, 3.7e-5, 1.1e-9, -0.3, 25.0, 1e-42, 0.0], device="cuda")
    for length in (0, 1, 12345, (1 << 24) + 1, (1 << 29) + 77):
        table = torch.zeros(1, length // 256 + 1, dtype=torch.int32, device="cuda")
        k, v = (torch.zeros(1, 256, 1, 16, dtype=F16, device="cuda") for _ in range(2))
        x = torch.zeros(1, 1, 1, 16, dtype=F16, device="cuda")
        x[..., :8] = 1.0
        ws = workspace()
        out = ds.cache_append(ds.PagedCache(k, v), x, x, table, i32([length]), ws, q=x, inv_freq=freq)
        assert ws.status() == 0 and torch.equal(k[0, length % 256, 0], out[0, 0, 0])
        for j, f in enumerate(freq.double().tolist()):
            angle = float(Decimal(length) * Decimal(f) % tau)
            for got, want in ((out[0, 0, 0, j], math.cos(angle)), (out[0, 0, 0, 8 + j], math.sin(angle))):
                assert abs(got.item() - want) <= 2.0 ** -21 + 2.0 ** -11 * abs(want) + 2.0 ** -25, (length, f)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_of_a_frequency_that_is_none(bad):
    freq = torch.tensor([1.0] * 8, device="cuda")
    freq[3] = bad
    k, v = (torch.zeros(1, 16, 1, 16, dtype=BF16, device="cuda") for _ in range(2))
    x = torch.ones(1, 1, 1, 16, dtype=BF16, device="cuda")
    out = ds.cache_append(ds.PagedCache(k, v), x, x, i32([[0]]), i32([5]), workspace(), q=x, inv_freq=freq)[0, 0, 0]
    wrong = torch.tensor([j % 8 == 3 for j in range(16)], device="cuda")
    assert torch.isnan(out[wrong]).all() and torch.isfinite(out[~wrong]).all()
    assert torch.equal(v[0, 5, 0], x[0, 0, 0])


# ---------------------------------------------------------------------- steps in a row

class Steps:
    """A batch of requests through steps of a drafted tree: what a program keeps between calls."""

    def __init__(self, B=5, N=7, lengths=(0, 15, 100, 250, 31), packed=False, room=40):
        self.batch = Batch([(3 * b) % N + 1 for b in range(B)], list(lengths), 16, seed=31, packed=packed, tree=True, N=N,
                           room=room)
        self.k, self.v = new_cache(self.batch, 2, 64, BF16, layers=2)
        for t in (0, 1):
            fill_cache(self.batch, self.k[t], self.v[t], seed=32 + t, tokens=False)
        self.cache = ds.PagedCache(self.k, self.v)
        self.ws = ds.Workspace.of_bytes(ds.tree_attention_workspace_bytes(B, N, 6, 2, 64))
        self.inv = (1e4 ** -(torch.arange(0, 64, 2, device="cuda") / 64.0)).float()
        lead, rows, V = self.batch.lead, self.batch.rows, 50
        g = gen(34)
        make = lambda *s: torch.randn(lead + s, generator=g, device="cuda").to(BF16)  # noqa: E731
        self.x = [(make(6, 64), make(2, 64), make(2, 64)) for _ in range(2)]
        self.out = [torch.zeros(lead + (6, 64), dtype=BF16, device="cuda") for _ in range(2)]
        self.q = [torch.zeros(lead + (6, 64), dtype=BF16, device="cuda") for _ in range(2)]
        self.p = torch.softmax(2 * torch.randn(rows, V, generator=g, device="cuda"), 1)
        order = self.p.argsort(1, descending=True)
        tokens = torch.zeros(rows, dtype=torch.int32)
        for b, i, row in self.batch.live:             # (siblings differ)
            up = self.batch.trees[b][i]
            if up >= 0:
                tokens[row] = order[self.batch.first[b] + up, sum(t == up for t in self.batch.trees[b][:i])]
        self.tokens = tokens.cuda()
        self.u = torch.rand(rows, generator=g, device="cuda") * 0.3
        shaped = lambda t: t.view(lead + t.shape[1:])  # noqa: E731
        self.verify_args = (shaped(self.p), shaped(self.tokens), shaped(self.u))
        B, N = self.batch.B, self.batch.N
        self.answer = {"accept_len": i32([0] * B), "path": i32([[0] * N] * B), "out_tokens": i32([[0] * N] * B),
                       "n_out": i32([0] * B)}

    def run(self, stream=None):
        b, kw = self.batch, self.batch.kw
        for t in (0, 1):
            q, k, v = self.x[t]
            ds.cache_append(self.cache, k, v, b.pages, b.lens, self.ws, q=q, q_out=self.q[t], inv_freq=self.inv, layer=t,
                            stream=stream, **kw)
            ds.tree_attention(self.q[t], self.cache, b.pages, b.lens, self.ws, out=self.out[t], layer=t, stream=stream, **kw)
        ds.tree_verify(*self.verify_args, self.ws, out=self.answer, stream=stream, **kw)
        ds.cache_keep(self.cache, b.pages, b.lens, self.answer["path"], self.answer["accept_len"], self.ws, stream=stream)

    def state(self):
        return [self.k, self.v, *self.out, *self.q, *self.answer.values()]


@pytest.mark.parametrize("packed", [False, True])
def test_steps_in_a_row(packed):
    """Two steps of two layers: each attends to what it should, and what the first accepted is what the
    second sees, slot by slot."""
    s = Steps(packed=packed)
    b = s.batch
    for _ in range(2):
        before = [s.k.clone(), s.v.clone()]
        lengths = list(b.lengths)
        s.run()
        assert s.ws.status() == 0
        want = verify_reference(b, s.p, s.tokens, s.u)
        for key, value in want.items():
            np.testing.assert_array_equal(s.answer[key].cpu().numpy(), value, err_msg=key)
        # the step's tokens again, without keeping: the cache that the attention saw
        full = [t.clone() for t in before]
        cache = ds.PagedCache(*full)
        for t in (0, 1):
            ds.cache_append(cache, s.x[t][1], s.x[t][2], b.pages, b.lens, s.ws, inv_freq=s.inv, layer=t, **b.kw)
            check_rows(b, s.q[t], full[0][t], full[1][t], s.out[t])
        for r in range(b.B):
            a = int(want["accept_len"][r])
            if a:
                src = b.place(r, [lengths[r] + int(x) for x in want["path"][r, :a]])
                dst = b.place(r, [lengths[r] + 1 + j for j in range(a)])
                for t in (0, 1):
                    for now, old in zip((s.k, s.v), full):
                        assert torch.equal(now[t][dst], old[t][src])
            if lengths[r]:
                src = b.place(r, np.arange(lengths[r]))
                assert torch.equal(s.k[:, src[0], src[1]], before[0][:, src[0], src[1]])
            b.lengths[r] += 1 + a
        assert want["accept_len"].max() > 0
        b.lens.copy_(i32(b.lengths))


def test_captured_steps_share_a_workspace_and_replay_on_new_inputs():
    """Two captured steps on one workspace, replayed in turn, after the lengths and queries have changed."""
    one, two = Steps(), Steps(lengths=(3, 0, 64, 200, 129))
    two.ws = one.ws
    start = [[t.clone() for t in s.state()] for s in (one, two)]
    graphs = []
    for s in (one, two):
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn in range(3):
        for s, g, old in zip((one, two), graphs, start):
            for t, o in zip(s.state(), old):
                t.copy_(o)
            if turn:
                s.batch.lens.copy_(i32([max(0, x - turn) for x in s.batch.lengths]))
                s.x[0][0].mul_(0.5)
            s.run()
            want = [t.clone() for t in s.state()]
            for t, o in zip(s.state(), old):
                t.copy_(o)
            g.replay()
            for t, w in zip(s.state(), want):
                assert torch.equal(torch.nan_to_num(t.float()), torch.nan_to_num(w.float()))
    assert one.ws.status() == 0


def test_two_streams_at_once():
    """Steps on two streams with a workspace each, against the same on one."""
    lone = [Steps(), Steps(lengths=(3, 0, 64, 200, 129))]
    both = [Steps(), Steps(lengths=(3, 0, 64, 200, 129))]
    for s in lone:
        s.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, stream in zip(both, streams):
            s.run(stream)
    torch.cuda.synchronize()
    for a, b in zip(lone, both):
        assert b.ws.status() == 0
        for x, y in zip(a.out, b.out):
            assert torch.equal(x, y)
        for key in a.answer:
            assert torch.equal(a.answer[key], b.answer[key])


# -------------------------------------------------------------- bad tables, nothing to do

BAD = [
    # what the second of three requests has, and whether the first and third are still whole
    dict(counts=[3, 9, 2]), dict(counts=[3, -1, 2]), dict(lengths=[20, -1, 5]), dict(lengths=[20, 1 << 30, 5]),
    dict(page=-1), dict(page=1 << 20), dict(parent=3), dict(parent=-2),
]


@pytest.mark.parametrize("bad", BAD, ids=[str(b) for b in BAD])
@pytest.mark.parametrize("wide", [False, True])
def test_bad_tables_are_reported(bad, wide):
    batch = Batch([3, 4, 2], [20, 40, 5], 16, tree=True, N=4)
    Hq, Hkv = (64, 1) if wide else (4, 2)
    k, v = new_cache(batch, Hkv, 64, BF16, fill=0.0)
    fill_cache(batch, k, v)
    q = torch.randn(3, 4, Hq, 64, generator=gen(41), device="cuda").to(BF16)
    ws = workspace(batch, Hq, Hkv, 64)
    good = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, out=torch.full_like(q, 5.0), **batch.kw)
    pages, lens, kw = batch.pages.clone(), batch.lens, dict(batch.kw)
    kw["counts"] = i32(bad.get("counts", batch.counts))
    lens = i32(bad.get("lengths", batch.lengths))
    if "page" in bad:
        pages[1, 1] = bad["page"]
    if "parent" in bad:
        kw["parents"] = kw["parents"].clone()
        kw["parents"][1, 2] = bad["parent"]
    got = ds.tree_attention(q, ds.PagedCache(k, v), pages, lens, ws, out=torch.full_like(q, 5.0), **kw)
    assert ws.status() == DEVICE_CHECK and ws.status() == 0
    assert torch.equal(got[0, :3], good[0, :3]) and torch.equal(got[2, :2], good[2, :2])
    assert (got[0, 3:] == 5.0).all() and (got[2, 2:] == 5.0).all()
    if "counts" in bad or "lengths" in bad:
        assert (got[1] == 5.0).all()
    # the same tables for the other calls
    x = torch.ones(3, 4, Hkv, 64, dtype=BF16, device="cuda")
    kc, vc = k.clone(), v.clone()
    inv = torch.ones(32, device="cuda")
    ds.cache_append(ds.PagedCache(kc, vc), x, x, pages, lens, ws, inv_freq=inv, **kw)
    if "page" not in bad:
        assert ws.status() == DEVICE_CHECK
    page, line = batch.place(0, [20, 21, 22])
    assert (vc[page, line] == 1.0).all()
    if "counts" in bad or "parent" in bad:
        p = torch.softmax(torch.randn(3, 4, 40, generator=gen(42), device="cuda"), -1)
        ds.tree_verify(p, i32([[0] * 4] * 3), torch.rand(3, 4, generator=gen(43), device="cuda"), ws, **kw)
        assert ws.status() == DEVICE_CHECK


def test_starts_that_descend_are_reported():
    batch = Batch([3, 4, 2], [20, 40, 5], 16, packed=True)
    k, v = new_cache(batch, 1, 64, BF16, fill=0.0)
    x = torch.ones(batch.rows, 1, 64, dtype=BF16, device="cuda")
    ws = workspace(batch, 1, 1, 64)
    for starts in ([0, 3, 2, 9], [0, 3, 7, 1 << 20], [-4, 3, 7, 9]):
        kw = dict(batch.kw, starts=i32(starts))
        ds.cache_append(ds.PagedCache(k, v), x, x, batch.pages, batch.lens, ws, **kw)
        assert ws.status() == DEVICE_CHECK
        ds.tree_attention(x, ds.PagedCache(k, v), batch.pages, batch.lens, ws, **kw)
        assert ws.status() == DEVICE_CHECK


@pytest.mark.parametrize("packed", [False, True])
def test_nothing_to_do(packed):
    """No requests, and requests without tokens: nothing is written."""
    batch = Batch([0, 0], [3, 0], 16, packed=packed, N=4)
    k, v = new_cache(batch, 2, 64, BF16, fill=3.0)
    q = torch.ones(batch.lead + (4, 64), dtype=BF16, device="cuda")
    x = q[..., :2, :].contiguous()
    ws = workspace(batch, 4, 2, 64)
    cache = ds.PagedCache(k, v)
    out, q_out = torch.full_like(q, 5.0), torch.full_like(q, 5.0)
    ds.cache_append(cache, x, x, batch.pages, batch.lens, ws, q=q, q_out=q_out, **batch.kw)
    ds.tree_attention(q, cache, batch.pages, batch.lens, ws, out=out, **batch.kw)
    p = torch.ones(batch.lead + (9,), device="cuda")
    got = ds.tree_verify(p, torch.zeros(batch.lead, dtype=torch.int32, device="cuda"), torch.zeros(batch.lead, device="cuda"), ws,
                         **batch.kw)
    assert (got["n_out"] == 0).all() and (got["path"] == -1).all() and (got["out_tokens"] == -1).all()
    ds.cache_keep(cache, batch.pages, batch.lens, got["path"], got["accept_len"], ws)
    assert (out == 5.0).all() and (q_out == 5.0).all() and (k == 3.0).all() and (v == 3.0).all() and ws.status() == 0
    none = dict(starts=i32([0]), nodes=4) if packed else {}
    lead = (0,) if packed else (0, 4)
    e = torch.zeros(lead + (4, 64), dtype=BF16, device="cuda")
    empty = torch.zeros(0, batch.max_pages, dtype=torch.int32, device="cuda")
    ds.tree_attention(e, cache, empty, i32([]), ws, **none)
    ds.cache_append(cache, e[..., :2, :], e[..., :2, :], empty, i32([]), ws, **none)
    assert ws.status() == 0


# ------------------------------------------------------------------ refusals from Python

def _refused():
    t = lambda *shape, dtype=BF16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    k = t(3, 16, 2, 64)
    good = dict(cache=ds.PagedCache(k, t(3, 16, 2, 64)), k=t(2, 4, 2, 64), v=t(2, 4, 2, 64), pages=i32([[0, 1], [2, 1]]),
                lengths=i32([0, 0]), ws=ds.Workspace.of_bytes(ds.tree_attention_workspace_bytes(2, 4, 4, 2, 64)),
                q=t(2, 4, 4, 64), q_out=t(2, 4, 4, 64))
    attend = {a: good[a] for a in ("cache", "pages", "lengths", "ws", "q")} | dict(out=t(2, 4, 4, 64))
    verify = dict(p=torch.full((2, 4, 9), 1 / 9, device="cuda"), tokens=i32([[0] * 4] * 2), ws=good["ws"],
                  uniforms=torch.zeros(2, 4, device="cuda"),
                  out={a: i32([0, 0]) for a in ("accept_len", "n_out")} | {a: i32([[0] * 4] * 2) for a in ("path", "out_tokens")})
    keep = dict(cache=good["cache"], pages=good["pages"], lengths=good["lengths"], path=i32([[-1] * 4] * 2),
                accept_len=i32([0, 0]), ws=good["ws"])
    wide, cpu = t(2, 4, 4, 128), torch.zeros(2, dtype=torch.int32)
    return [
        (ds.cache_append, good, [
            dict(k=t(2, 4, 2, 64, dtype=F16)), dict(k=t(2, 4, 3, 64)), dict(v=t(2, 3, 2, 64)), dict(v=t(2, 4, 2, 32)),
            dict(q=t(2, 4, 4, 64).transpose(0, 1)), dict(q=wide[..., ::2]), dict(q_out=t(2, 4, 5, 64)), dict(q=None),
            dict(pages=i32([0, 1])), dict(pages=i32([[0, 1]])), dict(lengths=cpu), dict(lengths=i32([0, 0, 0])),
            dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(counts=i32([1])), dict(starts=i32([0, 1, 2])),
            dict(parents=i32([[0] * 4])), dict(inv_freq=t(8)), dict(inv_freq=t(33, dtype=F32)), dict(inv_freq=t(4, dtype=F32)),
            dict(q_weight=t(32, dtype=F32)), dict(eps=-1.0), dict(eps=math.nan), dict(layer=1), dict(layer=-1),
            dict(nodes=3, starts=i32([0, 1, 2]), counts=i32([1, 1])), dict(k=good["k"].cpu())]),
        (ds.tree_attention, attend, [
            dict(q=t(2, 4, 3, 64)), dict(q=t(2, 4, 4, 64, dtype=F16)), dict(out=t(2, 4, 2, 64)), dict(out=wide[..., ::2]),
            dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(lse=t(2, 4, dtype=F32)), dict(lse=t(2, 4, 4)),
            dict(ws=ds.Workspace.of_bytes(256)), dict(parents=i32([[0] * 4])), dict(pages=good["pages"].t()), dict(layer=7),
            dict(counts=torch.zeros(4, dtype=torch.int32, device="cuda")[::2])]),
        (ds.tree_verify, verify, [
            dict(p=t(2, 4, 9, dtype=torch.float64)), dict(p=t(8, 9, dtype=F32)), dict(q=t(2, 4, 9)), dict(q=t(2, 4, 8, dtype=F32)),
            dict(tokens=i32([0] * 7)), dict(tokens=t(2, 4, dtype=F32)), dict(uniforms=t(2, 4)),
            dict(out=verify["out"] | dict(path=i32([[0] * 3] * 2))), dict(out=verify["out"] | dict(n_out=cpu))]),
        (ds.cache_keep, keep, [
            dict(path=i32([0] * 8)), dict(path=i32([[0] * 4])), dict(accept_len=cpu), dict(accept_len=i32([0])),
            dict(pages=i32([[0, 1]])), dict(path=i32([[0] * 65] * 2))]),
    ]


def test_calls_refuse_from_python():
    """Every bad argument raises, on the current stream and on a given one, and nothing is written."""
    for call, good, bads in _refused():
        ws = good["ws"]
        for bad in bads:
            for stream in (None, torch.cuda.current_stream()):
                tensors = [x for x in (good | bad).values() if torch.is_tensor(x)]
                before = [x.clone() for x in tensors]
                with pytest.raises((ValueError, ds.DSparkError)):
                    call(**(good | bad), stream=stream)
                assert all(torch.equal(x, y) for x, y in zip(tensors, before))
        for stream in (None, torch.cuda.current_stream()):
            call(**good, stream=stream)                    # and what is good is taken
        assert ws.status() == 0, call


def test_strided_rows_and_forms_of_arguments():
    """Rows inside a wider projection (two and one leading dimensions), whole numbers for floats, and no
    outputs: as with contiguous rows and outputs that are given."""
    batch = Batch([3, 2], [20, 7], 16)
    k, v = new_cache(batch, 2, 64, BF16, fill=0.0)
    fill_cache(batch, k, v)
    cache, ws = ds.PagedCache(k, v), workspace(batch, 4, 2, 64)
    wide = torch.randn(2, 3, 10, 64, generator=gen(51), device="cuda").to(BF16)
    q = wide[:, :, 3:7]
    want = ds.tree_attention(q.contiguous(), cache, batch.pages, batch.lens, ws, out=torch.zeros_like(q.contiguous()), scale=1.0,
                             **batch.kw)
    for out in (None, torch.zeros(2, 3, 6, 64, dtype=BF16, device="cuda")[:, :, 1:5]):
        got = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, out=out, scale=1, **batch.kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1, :2], want[1, :2])
    flat = wide.view(6, 10, 64)[:, 3:7]
    got = ds.tree_attention(flat, cache, batch.pages, batch.lens, ws, starts=i32([0, 3, 5]), nodes=3, scale=1.0)
    alone = ds.tree_attention(wide[:1, :, 3:7], cache, batch.pages[:1], batch.lens[:1], ws, scale=1.0)
    assert torch.equal(got[:3], want[0]) and torch.equal(got[3:5], want[1, :2]) and torch.equal(alone[0], want[0])
    assert ws.status() == 0
