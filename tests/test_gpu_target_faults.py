"""The target's side of a step on what only the device sees to be wrong, and on values that are not
finite: what is reported, what still is answered, and that nothing else changes."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")
from speculative_decoding_03_gb300 import target  # noqa: E402
if torch.cuda.is_available():
    from _target import Batch, attention_tolerance, fill_cache, gen, i32, new_cache, sees, workspace

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEVICE_CHECK = 5


def noise(t, seed):
    """Random values in every element of t."""
    return t.copy_(torch.randn(t.shape, generator=gen(seed), device="cuda"))


# ------------------------------------------------------------------------- appending

STARTS = [
    # starts of 3 requests, and the rows (of request, place) that are certainly its own
    ([0, 3, 2, 9], {0: (0, 0), 1: (0, 1), 4: (2, 2), 8: (2, 6)}),
    ([0, 1 << 30, 2, 9], {}),
    ([5, 2, 7, 9], {7: (2, 0), 8: (2, 1)}),
    ([9, 5, 1, 3], {}),
    ([0, 3, -(1 << 31), 9], {}),
    ([0, 3, (1 << 31) - 1, 9], {0: (0, 0), 2: (0, 2)}),
]


@pytest.mark.parametrize("starts,own", STARTS, ids=[str(s[0]) for s in STARTS])
def test_append_of_starts_that_descend(starts, own):
    """A row whose request begins behind it counts as none: nothing is written in front of a request's
    tokens, nor for a request whose rows are refused."""
    batch = Batch([3, 7, 9], [20, 40, 5], 16, packed=True, N=9)
    rows = 16
    k, v = (noise(t, 60 + j) for j, t in enumerate(new_cache(batch, 2, 64, BF16, fill=0.0)))
    want_k, want_v = k.clone(), v.clone()
    x = torch.randn(rows, 8, 64, generator=gen(62), device="cuda").to(BF16)
    q, new_k, new_v = x[:, :4], x[:, 4:6], x[:, 6:]
    q_out = torch.full((rows, 4, 64), 5.0, dtype=BF16, device="cuda")
    ws = workspace()
    ds.cache_append(ds.PagedCache(k, v), new_k, new_v, batch.pages, batch.lens, ws, q=q, q_out=q_out, starts=i32(starts),
                    nodes=9)
    assert ws.status() == DEVICE_CHECK and ws.status() == 0
    good = [b for b in range(3) if 0 <= starts[b] <= starts[b + 1] <= rows and starts[b + 1] - starts[b] <= 9]
    may = torch.zeros(rows, dtype=torch.bool, device="cuda")   # rows of a request that is none of the bad
    free_k = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    for b in good:
        may[starts[b]:starts[b + 1]] = True
        page, line = batch.place(b, [batch.lengths[b] + i for i in range(min(starts[b + 1] - starts[b], batch.counts[b]))])
        free_k[page, line] = True
    assert torch.equal(k[~free_k], want_k[~free_k]) and torch.equal(v[~free_k], want_v[~free_k])
    assert (q_out[~may] == 5.0).all()
    for row, (b, i) in own.items():
        page, line = batch.place(b, [batch.lengths[b] + i])
        assert torch.equal(k[page, line][0], new_k[row]) and torch.equal(v[page, line][0], new_v[row])
        assert torch.equal(q_out[row], q[row])


# --------------------------------------------------------------------------- keeping

def kept(batch, k, v, paths):
    """What ``cache_keep`` leaves of [layers, ...] caches, for paths {request: [(j, place), ..]}."""
    want = [k.clone(), v.clone()]
    for b, moves in paths.items():
        for j, node in moves:
            src, dst = batch.place(b, [batch.lengths[b] + node]), batch.place(b, [batch.lengths[b] + 1 + j])
            for new, old in zip(want, (k, v)):
                new[:, dst[0], dst[1]] = old[:, src[0], src[1]]
    return want


def test_keep_of_requests_whose_pages_are_full():
    """A request without tokens whose pages are full is not looked at; one that accepts all it has
    room for is kept, and one that accepts more is not."""
    batch = Batch([0, 4, 0, 4], [32, 28, 32, 29], 16, N=6, spare=4)
    assert batch.max_pages == 3
    pages = batch.pages[:, :2].contiguous()                   # room for 32 slots of each
    k, v = (noise(t, 63 + j) for j, t in enumerate(new_cache(batch, 2, 64, BF16, layers=2)))
    ws, cache = workspace(), ds.PagedCache(k, v)
    path = i32([[-1] * 6, [1, 3, -1, -1, -1, -1], [-1] * 6, [-1] * 6])
    want = kept(batch, k, v, {1: [(1, 3)]})
    ds.cache_keep(cache, pages, batch.lens, path, i32([0, 2, 0, 0]), ws)
    assert ws.status() == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    want = kept(batch, k, v, {1: [(0, 2)]})
    path = i32([[1] + [-1] * 5, [2] + [-1] * 5, [-1] * 6, [1, 2, 3, -1, -1, -1]])
    ds.cache_keep(cache, pages, batch.lens, path, i32([1, 1, 0, 3]), ws)
    assert ws.status() == DEVICE_CHECK and ws.status() == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


BAD_KEEPS = [
    # what the second of three requests has, and its moves that are still made
    (dict(accept=-1), []), (dict(accept=8), []), (dict(accept=1 << 30), []), (dict(length=-1), []),
    (dict(length=(1 << 31) - 1), []), (dict(length=1 << 20), []),
    (dict(path=[3, 1, 6]), [(0, 3), (2, 6)]), (dict(path=[3, -1, 6]), [(0, 3), (2, 6)]),
    (dict(path=[3, 8, 6]), [(0, 3), (2, 6)]), (dict(path=[0, 5, 6]), [(1, 5), (2, 6)]),
    (dict(path=[3, 1 << 30, 6]), [(0, 3), (2, 6)]),
    (dict(path=[3, 7, 5]), [(0, 3), (2, 5)]),                  # a slot behind the table's last page
    (dict(page=-1), []), (dict(page=1 << 20), []),
]


@pytest.mark.parametrize("bad,moves", BAD_KEEPS, ids=[str(b[0]) for b in BAD_KEEPS])
def test_keep_of_what_is_out_of_range(bad, moves):
    """What is refused of one request is reported and moves nothing; the rest moves as ever."""
    batch = Batch([8, 7, 8], [20, 25, 5], 16, N=8)
    k, v = (noise(t, 65 + j) for j, t in enumerate(new_cache(batch, 2, 64, BF16, layers=2)))
    path = np.full((3, 8), -1, np.int32)
    path[0, :2], path[2, :3] = [2, 5], [3, 4, 7]
    mine = bad.get("path", [3, 5, 6])
    path[1, :len(mine)] = mine
    accept, lengths, pages = [2, bad.get("accept", 3), 3], [20, bad.get("length", 25), 5], batch.pages.clone()
    if "page" in bad:
        pages[1, 1] = bad["page"]                              # slots 16 to 31: all of its tokens'
    want = kept(batch, k, v, {0: [(0, 2), (1, 5)], 1: moves, 2: [(0, 3), (1, 4), (2, 7)]})
    ws = workspace()
    ds.cache_keep(ds.PagedCache(k, v), pages, i32(lengths), i32(path.tolist()), i32(accept), ws)
    assert ws.status() == DEVICE_CHECK and ws.status() == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


# ---------------------------------------------------------------------- verification

def rejected(dtype, V=3001, B=4, N=4, seed=70):
    """Requests whose children, siblings of one root, are all rejected; p, q, tokens, u, parents."""
    g = gen(seed)
    p = torch.softmax(torch.randn(B, N, V, generator=g, device="cuda"), -1)
    q = torch.softmax(torch.randn(B, N, V, generator=g, device="cuda"), -1)
    tokens = i32([[0, 7, 8, 9]] * B)
    p[:, 0, 7:10] = 0.0
    parents = i32([[-1, 0, 0, 0]] * B)
    u = torch.full((B, N), 0.5, device="cuda")
    return p.to(dtype), q.to(dtype), tokens, u, parents


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("where", ["p", "q", "p at a child", "q at a child", "p is infinite", "both infinite"])
@pytest.mark.parametrize("children", [1, 3])
def test_verify_reports_what_is_not_finite(dtype, where, children):
    """A NaN, or an infinite probability, in the row that a request draws from is reported and gives no
    token, whatever was rejected before; the other requests are answered as ever."""
    p, q, tokens, u, parents = rejected(dtype, V=40000 if children == 1 else 3001)     # by clusters, by a CTA
    counts = i32([1 + children] * 4)
    ws = workspace()
    want = {}
    for drawn in (True, False):
        want[drawn] = ds.tree_verify(p, tokens, u, ws, q=q if drawn else None, counts=counts, parents=parents)
        assert ws.status() == 0 and (want[drawn]["n_out"] == 1).all() and (want[drawn]["out_tokens"][:, 0] >= 0).all()
    at = 7 if "child" in where else 2500
    if where.startswith(("p", "both")):
        p[2, 0, at] = math.inf if "infinite" in where else math.nan
    if where.startswith(("q", "both")):
        q[2, 0, at] = math.inf if "infinite" in where else math.nan
    for drawn in (True, False):
        if not drawn and where.startswith("q"):
            continue
        got = ds.tree_verify(p, tokens, u, ws, q=q if drawn else None, counts=counts, parents=parents)
        assert ws.status() == DEVICE_CHECK and ws.status() == 0
        assert got["out_tokens"][2].tolist() == [-1] * 4 and got["accept_len"][2] == 0
        for key, value in want[drawn].items():
            others = torch.tensor([0, 1, 3], device="cuda")
            assert torch.equal(got[key][others], value[others]), key


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_reads_no_more_than_it_answers_from(drawn):
    """NaN in rows of tokens that are not reached, and in a row all of whose probability is left."""
    p, q, tokens, u, parents = rejected(F32)
    p[:, 0, 7] = 0.9                                           # the first child is accepted
    p[:, 2:], q[:, 2:] = math.nan, math.nan
    p[:, 0, 2500], q[:, 0, 2500] = math.nan, math.nan
    ws = workspace()
    got = ds.tree_verify(p, tokens, u, ws, q=q if drawn else None, parents=parents)
    assert ws.status() == 0 and (got["accept_len"] == 1).all() and (got["path"][:, 0] == 1).all()
    assert (got["out_tokens"][:, :2] >= 0).all()


@pytest.mark.parametrize("given", [[], ["path"], ["accept_len", "out_tokens"], ["n_out", "path", "accept_len", "out_tokens"]])
@pytest.mark.parametrize("on_stream", [False, True])
def test_verify_makes_the_outputs_that_it_lacks(given, on_stream):
    """A dict of some of the outputs is filled: what it holds is written, what it lacks is made."""
    p, q, tokens, u, parents = rejected(F32)
    stream = torch.cuda.current_stream() if on_stream else None
    want = ds.tree_verify(p, tokens, u, workspace(), q=q, parents=parents)
    mine = {key: torch.full_like(want[key], -9) for key in given}
    out = dict(mine)
    if given == ["path"]:
        out["n_out"] = None
    got = ds.tree_verify(p, tokens, u, workspace(), q=q, parents=parents, out=out, stream=stream)
    assert got is out and set(got) == set(want)
    assert all(got[key] is t for key, t in mine.items())
    for key, value in want.items():
        assert torch.equal(got[key], value), key


# -------------------------------------------------------------------------- attention

def attention_without(batch, q, k, v, scale, gone):
    """(out, lse, spread, size) of the live rows in 64 bits, where the slots gone[b] count as none."""
    Hkv, D = k.shape[-2:]
    flat = q.reshape(batch.rows, q.shape[-2], D)
    parts = []
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
        mask[:, [s for s in gone.get(b, []) if s < l + n]] = False
        mask = mask.cuda()[:, None, None]
        x = flat[batch.first[b]:batch.first[b] + n].double().view(n, Hkv, -1, D)
        s = torch.where(mask, torch.einsum("nhgd,lhd->nhgl", x, kk) * scale, -math.inf)
        p = torch.nan_to_num(torch.softmax(s, -1))            # (a row of no slots: zeroes)
        o, a = torch.einsum("nhgl,lhd->nhgd", p, vv), torch.einsum("nhgl,lhd->nhgd", p, vv.abs())
        big = (torch.einsum("nhgd,lhd->nhgl", x.abs(), kk.abs()) * scale).amax(-1)
        parts.append((o.reshape(n, -1, D), torch.logsumexp(s, -1).reshape(n, -1), a.reshape(n, -1, D), big.reshape(n, -1)))
    return [torch.cat(t) for t in zip(*parts)]


GONE = [
    # counts, lengths, page, q_heads, heads, D, and the pages of each request that are none
    ([3, 4], [100, 20], 16, 4, 2, 128, {0: [0, 3]}),          # up to 16 rows a key head: a lone tile
    ([3, 4], [700, 20], 16, 4, 2, 64, {0: [1, 40], 1: [1]}),  # parts, and the tokens' own page
    ([1], [3000], 16, 4, 1, 128, {0: [0, 50, 100, 187]}),     # parts joined by the last
    ([1], [3100], 256, 4, 1, 128, {0: [0, 5]}),               # and by a kernel; tiles that hold nothing
    ([12, 9], [300, 0], 32, 8, 2, 128, {0: [2, 9], 1: [0]}),  # up to 64 rows
    ([12], [2000], 128, 3, 1, 64, {0: [0, 1, 15]}),
    ([40, 17], [260, 129], 64, 8, 2, 128, {0: [0, 4], 1: [1]}),       # more, in two row blocks
    ([33], [3000], 16, 4, 1, 64, {0: [0, 1, 2, 3, 4, 5, 6, 7, 9, 100]}),
    ([5, 2], [40, 0], 16, 2, 1, 64, {0: [0, 1, 2], 1: [0]}),  # no page at all
    ([20, 2], [40, 0], 16, 16, 2, 128, {0: [0, 1, 2, 3], 1: [0]}),
]


@pytest.mark.parametrize("case", GONE, ids=[f"{i}" for i in range(len(GONE))])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_of_pages_that_are_none(case, dtype):
    """Slots on a page outside the cache take no part: the others are attended to as without them, in
    outputs and sums, and rows with nothing left get zeroes and -inf."""
    counts, lengths, page, Hq, Hkv, D, pages_gone = case
    batch = Batch(counts, lengths, page, seed=80, tree=True)
    k, v = new_cache(batch, Hkv, D, dtype)
    fill_cache(batch, k, v)
    pages = batch.pages.clone()
    gone = {b: [s for i in at for s in range(page * i, page * (i + 1))] for b, at in pages_gone.items()}
    for b, at in pages_gone.items():
        for j, i in enumerate(at):
            pages[b, i] = (-1, batch.n_pages, -(1 << 31), (1 << 31) - 1)[j % 4]
    q = torch.randn(batch.lead + (Hq, D), generator=gen(81), device="cuda").to(dtype)
    out, lse = torch.full_like(q, 5.0), torch.full(batch.lead + (Hq,), 5.0, device="cuda")
    ws = workspace(batch, Hq, Hkv, D)
    ds.tree_attention(q, ds.PagedCache(k, v), pages, batch.lens, ws, out=out, lse=lse, **batch.kw)
    assert ws.status() == DEVICE_CHECK and ws.status() == 0
    ref, ref_lse, spread, size = attention_without(batch, q, k, v, D ** -0.5, gone)
    rows = batch.live_rows()
    tol = attention_tolerance(batch, ref, spread, size, v, dtype)
    assert ((out.view(batch.rows, Hq, D)[rows].double() - ref).abs() <= tol).all()
    got, none = lse.view(batch.rows, Hq)[rows].double(), torch.isinf(ref_lse)
    assert torch.equal(got == -math.inf, none)
    bound = size * (D + 4) * 2.0 ** -23 + (max(lengths) / 32 + 128) * 2.0 ** -23 + torch.nan_to_num(ref_lse).abs() * 2.0 ** -22
    assert ((got - ref_lse).abs() <= bound)[~none].all()


# rows a key head (12 tokens' query heads): up to 16 and 64 rows, and one and two blocks of 128
GROUPS = [1, 2, 8, 16]


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [0, 120, 500, 2500])        # the last two shared out in parts
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_of_values_and_keys_that_are_not_finite(group, D, length, bad):
    """A token's value that is not finite reaches the rows that see the token and no others, by every
    kernel and through the joining of parts; so does its key."""
    batch = Batch([12], [length], 16, seed=11, tree=True)
    k, v = new_cache(batch, 2, D, BF16)
    fill_cache(batch, k, v)
    clean = v.clone()
    page, line = batch.place(0, [length + 3])
    v[page, line, 1, 5] = bad                                 # token 3's value of head 1, two elements
    v[page, line, 1, D - 1] = bad
    q = torch.randn(1, 12, 2 * group, D, generator=gen(9), device="cuda").to(BF16)
    ws = workspace(batch, 2 * group, 2, D)
    cache = ds.PagedCache(k, v)
    out = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, **batch.kw)
    hit = torch.tensor([3 in sees(batch.trees[0], i) for i in range(12)], device="cuda")
    assert hit.any() and not hit.all()
    seen = torch.zeros_like(out, dtype=torch.bool)
    seen[0, :, group:, 5] = hit[:, None]
    seen[0, :, group:, D - 1] = hit[:, None]
    got = out[seen]
    assert torch.isnan(got).all() if math.isnan(bad) else (got == bad).all()
    v.copy_(clean)
    want = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, **batch.kw)
    assert torch.isfinite(want).all() and torch.equal(out[~seen], want[~seen])
    # two tokens' values that are opposite infinities, where both are seen
    if math.isinf(bad):
        v[page, line, 1, 5] = bad
        root = batch.place(0, [length])
        v[root[0], root[1], 1, 5] = -bad
        out = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, **batch.kw)
        assert torch.isnan(out[0, hit][:, group:, 5]).all() and (out[0, ~hit][:, group:, 5] == -bad).all()
        v.copy_(clean)
    k[page, line, 1, 5] = bad
    out = ds.tree_attention(q, cache, batch.pages, batch.lens, ws, **batch.kw)
    reach = torch.zeros_like(seen)
    reach[0, :, group:] = hit[:, None, None]
    assert torch.equal(out[~reach], want[~reach])
    if math.isnan(bad):
        assert torch.isnan(out[reach]).all()
    assert ws.status() == 0


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [300, 2500])
def test_attention_of_queries_that_are_not_finite(group, D, length):
    """A query head of NaN gives NaN of its own row alone."""
    batch = Batch([12], [length], 16)
    k, v = new_cache(batch, 2, D, F16)
    fill_cache(batch, k, v)
    q = torch.randn(1, 12, 2 * group, D, generator=gen(1), device="cuda").to(F16)
    ws = workspace(batch, 2 * group, 2, D)
    want = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, **batch.kw)
    q[0, 7, group, D - 2] = math.nan
    out = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, **batch.kw)
    other = torch.ones_like(out, dtype=torch.bool)
    other[0, 7, group] = False
    assert torch.isnan(out[0, 7, group]).all() and torch.isfinite(want).all()
    assert torch.equal(out[other], want[other]) and ws.status() == 0


# --------------------------------------------------------- calls that are checked in Python

def test_calls_without_the_module(monkeypatch, tmp_path):
    """Where the module of the checks in C is not there the calls give the same bits."""
    batch = Batch([3, 7, 0], [20, 45, 5], 16, N=7, tree=True)
    g = gen(90)
    x = torch.randn(batch.lead + (8, 64), generator=g, device="cuda").to(BF16)
    p = torch.softmax(2 * torch.randn(batch.lead + (301,), generator=g, device="cuda"), -1)
    tokens, u = p.argmax(-1).to(torch.int32), torch.rand(batch.lead, generator=g, device="cuda")

    def step():
        k, v = new_cache(batch, 2, 64, BF16, fill=0.0)
        fill_cache(batch, k, v, tokens=False)
        cache, ws = ds.PagedCache(k, v), workspace(batch, 4, 2, 64)
        q = torch.zeros_like(x[..., :4, :])
        out, lse = torch.zeros_like(q), torch.zeros(batch.lead + (4,), device="cuda")
        answer = {key: torch.zeros(shape, dtype=torch.int32, device="cuda")
                  for key, shape in (("accept_len", 3), ("path", (3, 7)), ("out_tokens", (3, 7)), ("n_out", 3))}
        ds.cache_append(cache, x[..., 4:6, :], x[..., 6:, :], batch.pages, batch.lens, ws, q=x[..., :4, :], q_out=q, **batch.kw)
        ds.tree_attention(q, cache, batch.pages, batch.lens, ws, out=out, lse=lse, **batch.kw)
        ds.tree_verify(p, tokens, u, ws, out=answer, **batch.kw)
        ds.cache_keep(cache, batch.pages, batch.lens, answer["path"], answer["accept_len"], ws)
        assert ws.status() == 0
        return [k, v, q, out, lse, *answer.values()]

    want = step()
    assert target._calls() is not target._Unchecked
    monkeypatch.setattr(target._build, "CALLS", str(tmp_path / "none.so"))
    target._calls.cache_clear()
    try:
        got = step()
        assert target._calls() is target._Unchecked
    finally:
        target._calls.cache_clear()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
