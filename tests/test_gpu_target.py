"""The target's side of a step on the GPU against 64-bit references: appending to a paged cache,
attention of drafted tokens over it, verification from given numbers, keeping the accepted."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")
if torch.cuda.is_available():
    from _target import (HALF, Batch, attention_reference, attention_tolerance, depths, fill_cache, gen, i32,
                         new_cache, verify_reference, workspace)

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# ----------------------------------------------------------------------------- append

def append_reference(batch, x, weight, inv_freq, interleaved, eps):
    """(x', bound of what fp32 may be off before the rounding) of the live rows in 64 bits."""
    x = x.reshape((batch.rows,) + x.shape[-2:])[batch.live_rows()].double()
    D = x.shape[-1]
    off = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
        off = x.abs() * (D / 2 + 8) * 2.0 ** -24          # the mean's sum halves in the root
    if inv_freq is not None:
        h = inv_freq.numel()
        pos = torch.tensor([batch.lengths[b] + depths(batch.trees[b])[i] for b, i, _ in batch.live],
                           dtype=torch.float64, device="cuda")
        ang = pos[:, None, None] * inv_freq.double()
        c, s = ang.cos(), ang.sin()
        lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
        a, d = x[..., lo].clone(), x[..., hi].clone()
        oa, od = off[..., lo].clone(), off[..., hi].clone()
        x[..., lo], x[..., hi] = a * c - d * s, d * c + a * s
        # cos and sin to 2^-21 (the angle's last rounding and the functions'), two products and a sum
        more = (a.abs() + d.abs()) * 2.0 ** -20 + oa + od
        off[..., lo] = more
        off[..., hi] = more
    return x, off


APPENDS = [
    # counts, lengths, page, q_heads, heads, D, R, interleaved, norm, tree, packed, dtype
    ([1], [0], 16, 1, 1, 16, 16, False, False, False, False, BF16),
    ([1, 3, 2], [5, 0, 31], 16, 4, 2, 64, 64, False, True, True, True, F16),
    ([0, 7, 0, 64], [9, 1000, 2, 17], 32, 8, 8, 128, 128, False, False, True, False, BF16),
    ([5, 6], [250, 3], 256, 7, 1, 96, 32, True, True, True, True, BF16),
    ([16, 1], [1000000, 77], 256, 12, 4, 256, 256, True, False, False, False, F16),
    ([300, 41], [0, 129], 64, 28, 4, 128, 64, True, False, False, True, F16),
    ([2, 2], [15, 16], 128, 32, 8, 128, 0, False, True, False, False, BF16),
    ([3], [40], 16, 0, 3, 32, 32, False, False, False, True, BF16),
    ([4, 4], [40, 41], 16, 2, 2, 128, 0, False, False, True, True, F16),
]


@pytest.mark.parametrize("case", APPENDS, ids=[f"{i}" for i in range(len(APPENDS))])
def test_append(case):
    counts, lengths, page, Hq, Hkv, D, R, inter, norm, tree, packed, dtype = case
    batch = Batch(counts, lengths, page, seed=3, packed=packed, tree=tree)
    g = gen(4)
    qkv = torch.randn(batch.lead + (Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
    q = qkv[..., :Hq, :] if Hq else None
    k, v = qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
    kc, vc = new_cache(batch, Hkv, D, dtype, fill=7.0)
    kc0, vc0 = kc.clone(), vc.clone()
    inv = (1e4 ** -(torch.arange(0, R, 2, device="cuda").double() / R)).float() if R else None
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")) for _ in range(2)) if norm else (None, None)
    ws = workspace()
    out = torch.full(batch.lead + (Hq, D), 3.0, dtype=dtype, device="cuda") if Hq else None
    got = ds.cache_append(ds.PagedCache(kc, vc), k, v, batch.pages, batch.lens, ws, q=q, q_out=out, inv_freq=inv,
                          interleaved=inter, q_weight=wq if Hq else None, k_weight=wk, eps=1e-5, **batch.kw)
    assert got is out and ws.status() == 0
    rows = batch.live_rows()

    def close(y, x, weight):
        ref, off = append_reference(batch, x, weight, inv, inter, 1e-5)
        tol = HALF[dtype] * (ref.abs() + off) + off + 2.0 ** -25
        assert ((y.double() - ref).abs() <= tol).all()

    if Hq:
        flat = out.view((batch.rows,) + out.shape[-2:])
        close(flat[rows], q, wq)
        rest = torch.ones(batch.rows, dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert (flat[rest] == 3.0).all()
    at = [batch.place(b, [batch.lengths[b] + i]) for b, i, _ in batch.live]
    page_at, line_at = torch.cat([a[0] for a in at]), torch.cat([a[1] for a in at])
    close(kc[page_at, line_at], k, wk)
    vc0[page_at, line_at] = v.reshape((batch.rows,) + v.shape[-2:])[rows]
    assert torch.equal(vc, vc0)
    kc0[page_at, line_at] = kc[page_at, line_at]
    assert torch.equal(kc, kc0)                              # other slots as they were


def test_append_in_place_other_layouts_and_layers():
    """Queries over themselves; pages whose heads come before their slots; one layer of three."""
    batch = Batch([3, 0, 2], [30, 4, 0], 16, packed=True)
    g = gen(5)
    k, v = (torch.randn(batch.rows, 2, 64, generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(batch.rows, 4, 64, generator=g, device="cuda").to(BF16)
    inv = (1e4 ** -(torch.arange(0, 64, 2, device="cuda") / 64.0)).float()
    plain = new_cache(batch, 2, 64, BF16, fill=0.0)
    ref_q = ds.cache_append(ds.PagedCache(*plain), k, v, batch.pages, batch.lens, workspace(), q=q, inv_freq=inv, **batch.kw)
    kc, vc = new_cache(batch, 2, 64, BF16, layers=3, order="heads", fill=0.0)
    before = kc.clone()
    mine = q.clone()
    got = ds.cache_append(ds.PagedCache(kc, vc), k, v, batch.pages, batch.lens, workspace(), q=mine, q_out=mine,
                          inv_freq=inv, layer=1, **batch.kw)
    rows = batch.live_rows()
    assert got is mine and torch.equal(mine[rows], ref_q[rows]) and torch.equal(mine[-3:], q[-3:])
    assert torch.equal(kc[1], plain[0]) and torch.equal(vc[1], plain[1])
    assert torch.equal(kc[0], before[0]) and torch.equal(kc[2], before[2])


# -------------------------------------------------------------------------- attention

ATTENDS = [
    # counts, lengths, page, q_heads, heads, D, tree, packed, dtype
    ([1], [0], 16, 1, 1, 64, False, False, BF16),
    ([1], [0], 16, 8, 1, 128, False, False, F16),
    ([1, 1, 1, 1, 1], [127, 128, 126, 1, 255], 16, 4, 2, 128, False, True, BF16),
    ([2, 5, 0, 3], [126, 127, 40, 0], 32, 8, 8, 64, True, True, F16),
    ([64, 1, 64], [100, 0, 63], 16, 2, 2, 128, True, False, BF16),       # a tree past its tile's end
    ([64, 33], [300, 1], 64, 8, 1, 128, True, True, BF16),               # 512 rows: four row blocks
    ([17, 16, 15], [1000, 999, 1001], 128, 16, 2, 64, True, False, F16),
    ([64, 64], [64, 0], 256, 7, 7, 128, False, False, F16),
    ([8], [20001], 256, 32, 8, 128, False, False, BF16),                 # shared out over the CTAs
    ([7, 7], [9001, 5], 16, 5, 5, 64, True, True, BF16),
    ([4] * 300, [(37 * i) % 260 for i in range(300)], 16, 4, 2, 64, True, True, BF16),   # more requests than threads
]


@pytest.mark.parametrize("case", ATTENDS, ids=[f"{i}" for i in range(len(ATTENDS))])
def test_attention(case):
    counts, lengths, page, Hq, Hkv, D, tree, packed, dtype = case
    batch = Batch(counts, lengths, page, seed=6, packed=packed, tree=tree)
    k, v = new_cache(batch, Hkv, D, dtype)                    # NaN wherever there is no token
    fill_cache(batch, k, v)
    g = gen(7)
    q = torch.randn(batch.lead + (Hq, D), generator=g, device="cuda").to(dtype)
    out = torch.full_like(q, 5.0)
    lse = torch.full(batch.lead + (Hq,), 5.0, device="cuda")
    ws = workspace(batch, Hq, Hkv, D)
    got = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, out=out, lse=lse, **batch.kw)
    assert got is out and ws.status() == 0
    check_attention(batch, q, k, v, D ** -0.5, out, lse)


def check_attention(batch, q, k, v, scale, out, lse=None, fill=5.0):
    ref, ref_lse, spread, size = attention_reference(batch, q, k, v, scale)
    tol = attention_tolerance(batch, ref, spread, size, v, q.dtype)
    rows = batch.live_rows()
    flat = out.reshape((batch.rows,) + out.shape[-2:])
    err = (flat[rows].double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    rest = torch.ones(batch.rows, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert (flat[rest] == fill).all()
    if lse is not None:
        fl = lse.view(batch.rows, -1)
        # the scores' sums and exponents as above, the sum's fp32 additions, the logarithm's own
        bound = size * (q.shape[-1] + 4) * 2.0 ** -23 + (max(batch.lengths) / 32 + 128) * 2.0 ** -23 + ref_lse.abs() * 2.0 ** -22
        assert ((fl[rows].double() - ref_lse).abs() <= bound).all()
        assert (fl[rest] == fill).all()


def test_attention_scores_that_rise():
    """Scores that rise along the cache by hundreds: the running maximum is raised tile after tile."""
    batch = Batch([3], [1500], 16)
    k, v = new_cache(batch, 1, 64, BF16)
    fill_cache(batch, k, v)
    page, line = batch.place(0, np.arange(1503))
    k[page, line] = (torch.arange(1503, device="cuda").float()[:, None, None] * 0.01).expand(1503, 1, 64).to(BF16)
    q = torch.ones(1, 3, 2, 64, device="cuda").to(BF16)
    q[:, 1] = -1.0                                            # and falls for another token
    ws = workspace(batch, 2, 1, 64)
    out = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, scale=0.7, **batch.kw)
    check_attention(batch, q, k, v, 0.7, out)


def test_attention_other_layouts():
    """Queries inside a wider projection, outputs with a stride, heads before slots, a layer."""
    batch = Batch([5, 9], [200, 77], 32, tree=True)
    k3, v3 = new_cache(batch, 2, 128, F16, layers=2, order="heads")
    fill_cache(batch, k3[1], v3[1])
    g = gen(8)
    q = torch.randn(2, 9, 12, 128, generator=g, device="cuda").to(F16)[:, :, 2:10]
    out = torch.full((2, 9, 10, 128), 5.0, device="cuda").to(F16)[:, :, 1:9]
    ws = workspace(batch, 8, 2)
    ds.tree_attention(q, ds.PagedCache(k3, v3), batch.pages, batch.lens, ws, out=out, layer=1, **batch.kw)
    check_attention(batch, q, k3[1], v3[1], 128 ** -0.5, out)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lengths", [[120], [500], [0]])
def test_attention_values_not_finite_stay_where_they_are_seen(bad, lengths):
    batch = Batch([12], lengths, 16, seed=11, tree=True)
    k, v = new_cache(batch, 2, 128, BF16)
    fill_cache(batch, k, v)
    page, line = batch.place(0, [lengths[0] + 3])
    v[page, line, 1, 5] = bad                                 # token 3's value of head 1, one element
    g = gen(9)
    q = torch.randn(1, 12, 4, 128, generator=g, device="cuda").to(BF16)
    ws = workspace(batch, 4, 2)
    out = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, **batch.kw)
    from _target import sees
    hit = torch.tensor([3 in sees(batch.trees[0], i) for i in range(12)], device="cuda")
    seen = torch.zeros_like(out, dtype=torch.bool)
    seen[0, :, 2:, 5] = hit[:, None]
    assert hit.any() and not hit.all()
    assert torch.isfinite(out[~seen]).all()
    got = out[seen]
    assert torch.isnan(got).all() if math.isnan(bad) else (got == bad).all()
    # keys that are not finite reach the tokens that see them, and no others
    v[page, line, 1, 5] = 0.0
    k[page, line, 1, 5] = bad
    out = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, ws, **batch.kw)
    reach = torch.zeros_like(seen)
    reach[0, :, 2:] = hit[:, None, None]
    assert torch.isfinite(out[~reach]).all() and ws.status() == 0


def test_attention_of_a_query_that_is_not_finite():
    batch = Batch([6], [300], 16)
    k, v = new_cache(batch, 1, 64, BF16)
    fill_cache(batch, k, v)
    q = torch.randn(1, 6, 2, 64, generator=gen(1), device="cuda").to(BF16)
    q[0, 2, 1, 7] = math.nan
    out = ds.tree_attention(q, ds.PagedCache(k, v), batch.pages, batch.lens, workspace(batch, 2, 1, 64), **batch.kw)
    assert torch.isnan(out[0, 2, 1]).all() and torch.isfinite(out[0, 2, 0]).all()
    assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[0, 3:]).all()


def test_attention_in_a_cache_of_more_than_32_bits():
    """Slots whose offsets pass 2^31 elements and 2^32 bytes, in keys and in values."""
    batch = Batch([2], [2049], 256, spare=0)
    each = 256 * 8 * 128
    pages = (1 << 32) // each + 16
    k, v = (torch.zeros(pages, 256, 8, 128, dtype=BF16, device="cuda") for _ in range(2))
    batch.table = (batch.table + pages - batch.n_pages).astype(np.int32)
    batch.pages = torch.from_numpy(batch.table).cuda()
    new_k, new_v = (torch.randn(1, 2, 8, 128, generator=gen(3), device="cuda").to(BF16) for _ in range(2))
    fill_cache(batch, k, v, tokens=False)
    cache = ds.PagedCache(k, v)
    ws = workspace(batch, 8, 8)
    ds.cache_append(cache, new_k, new_v, batch.pages, batch.lens, ws)
    page, line = batch.place(0, [2049, 2050])
    assert torch.equal(k[page, line], new_k[0]) and torch.equal(v[page, line], new_v[0])
    q = torch.randn(1, 2, 8, 128, generator=gen(2), device="cuda").to(BF16)
    out = ds.tree_attention(q, cache, batch.pages, batch.lens, ws)
    check_attention(batch, q, k, v, 128 ** -0.5, out)
    ds.cache_keep(cache, batch.pages, batch.lens, i32([[1, -1]]), i32([1]), ws)
    assert torch.equal(k[page, line], new_k[0]) and ws.status() == 0


# ----------------------------------------------------------------------- verification

def distributions(batch, V, dtype, seed, near=0.6, sharp=2.0):
    g = gen(seed)
    z = torch.randn(batch.rows, V, generator=g, device="cuda") * sharp
    q = torch.softmax(z, 1)
    p = torch.softmax(z + near * torch.randn(batch.rows, V, generator=g, device="cuda"), 1)
    tokens = torch.zeros(batch.rows, dtype=torch.int32, device="cuda")
    draws = torch.multinomial(q, 64, replacement=True, generator=g)
    for b, i, row in batch.live:
        if i and batch.trees[b][i] >= 0:
            tokens[row] = draws[batch.first[b] + batch.trees[b][i], i].to(torch.int32)
    u = torch.rand(batch.rows, generator=g, device="cuda")
    return p.to(dtype), q.to(dtype), tokens, u


def check_verify(batch, p, tokens, u, q, ws=None, **more):
    ws = ws or workspace()
    shaped = lambda t: None if t is None else t.view(batch.lead + t.shape[1:])  # noqa: E731
    got = ds.tree_verify(shaped(p), shaped(tokens), shaped(u), ws, q=shaped(q), **batch.kw, **more)
    ref = verify_reference(batch, p, tokens, u, q)
    for key, want in ref.items():
        np.testing.assert_array_equal(got[key].cpu().numpy(), want, err_msg=key)
    return got, ws


VERIFIES = [
    # counts, V, dtype, points, tree, packed
    ([1], 8, F32, False, False, False),
    ([8], 151936, F32, False, False, False),
    ([6] * 40, 1003, F32, False, False, False),
    ([1, 6, 0, 3, 17], 32768, BF16, False, False, True),
    ([16] * 24, 999, F32, False, True, False),
    ([64, 64, 5], 4099, F16, False, True, True),
    ([16, 1, 9] * 20, 8000, BF16, True, True, True),
    ([64] * 3, 50001, F32, True, True, False),
    ([5] * 700, 257, F16, True, False, False),
    ([9] * 33, 1, F32, False, True, False),
]


@pytest.mark.parametrize("case", VERIFIES, ids=[f"{i}" for i in range(len(VERIFIES))])
@pytest.mark.parametrize("near", [0.3, 3.0])
def test_verify(case, near):
    counts, V, dtype, points, tree, packed = case
    batch = Batch(counts, [0] * len(counts), 16, seed=12, packed=packed, tree=tree)
    p, q, tokens, u = distributions(batch, V, dtype, 13, near)
    _, ws = check_verify(batch, p, tokens, u, None if points else q)
    assert ws.status() == 0


def test_verify_strided_and_misaligned_rows():
    batch = Batch([4, 7, 7], [0] * 3, 16, tree=True)
    p, q, tokens, u = distributions(batch, 1501, F32, 14)
    wide_p, wide_q = torch.zeros(batch.rows, 1600, device="cuda"), torch.zeros(batch.rows, 1507, device="cuda")
    wide_p[:, 3:1504], wide_q[:, 2:1503] = p, q
    shaped = lambda t: t.view(batch.lead + t.shape[1:])  # noqa: E731
    got = ds.tree_verify(wide_p.view(3, 7, 1600)[..., 3:1504], shaped(tokens), shaped(u), workspace(),
                         q=wide_q.view(3, 7, 1507)[..., 2:1503], **batch.kw)
    for key, want in verify_reference(batch, p, tokens, u, q).items():
        np.testing.assert_array_equal(got[key].cpu().numpy(), want, err_msg=key)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_ends(dtype):
    """Uniform numbers at both ends, distributions of a single token, a residual of nothing, equal
    children, and rows with nothing to draw from."""
    batch = Batch([3] * 8, [0] * 8, 16, N=3)
    V = 5000
    p, q, tokens, u = distributions(batch, V, dtype, 15)
    u.zero_()
    u[3:6] = 1.0 - 2.0 ** -24
    p[6:9], q[6:9] = 0.0, 0.0
    p[6:9, V - 1] = 1.0
    q[6:9, 0] = 1.0
    tokens[6:9] = 0                                            # rejected; only the last token is left
    q[9:12] = p[9:12]                                          # always accepted
    p[12:15] = q[12:15] * 0.5                                  # nothing is left of p after a rejection
    u[12:15] = 0.9
    p[15:18, 100:], p[18:21, :4900] = 0.0, 0.0                 # mass at one end only
    u[15:21] = 0.999
    check_verify(batch, p, tokens, u, q)
    got, ws = check_verify(batch, p, tokens, u, None)
    assert ws.status() == 0
    p[0:3] = 0.0
    got, ws = check_verify(batch, p, tokens, u, None)
    assert got["out_tokens"][0, 0] == -1 and got["n_out"][0] == 1 and ws.status() == 5


def test_verify_equal_children_and_siblings():
    """Children that name the same token: a second point mass has nothing left; a second draw is
    tried against what the first left."""
    batch = Batch([5] * 64, [0] * 64, 16)
    batch.trees = [[-1, 0, 0, 0, 0]] * 64
    batch.kw["parents"] = i32(batch.trees)
    p, q, tokens, u = distributions(batch, 300, F32, 16, near=2.0)
    tokens.view(64, 5)[:, 2] = tokens.view(64, 5)[:, 1]
    check_verify(batch, p, tokens, u, q)
    check_verify(batch, p, tokens, u, None)


@pytest.mark.parametrize("points", [False, True])
def test_verify_is_lossless(points):
    """The first token of the answer is distributed as p, whatever the tree: 60000 requests with three
    children each; every frequency within five standard deviations."""
    B, V = 60000, 6
    g = gen(17)
    p0 = torch.tensor([0.35, 0.05, 0.2, 0.1, 0.25, 0.05], device="cuda")
    q0 = torch.tensor([0.1, 0.3, 0.25, 0.05, 0.1, 0.2], device="cuda")
    parents = i32([[-1, 0, 0, 0]]).expand(B, 4).contiguous()
    p, q = p0.expand(B, 4, V).contiguous(), q0.expand(B, 4, V).contiguous()
    if points:
        tokens = i32([0, 1, 4, 2]).expand(B, 4).contiguous()
    else:
        tokens = torch.multinomial(q0, 4 * B, replacement=True, generator=g).view(B, 4).to(torch.int32)
    u = torch.rand(B, 4, generator=g, device="cuda")
    out = ds.tree_verify(p, tokens, u, workspace(), q=None if points else q, parents=parents)
    f = torch.bincount(out["out_tokens"][:, 0].long(), minlength=V).double() / B
    assert ((f - p0.double()).abs() <= 5 * (p0.double() * (1 - p0.double()) / B).sqrt()).all()


# ---------------------------------------------------------------------------- keeping

@pytest.mark.parametrize("heads,D,page,layers,order", [(2, 64, 16, 3, "slots"), (8, 128, 16, 2, "heads"),
                                                        (1, 16, 256, 1, "slots"), (20, 256, 32, 0, "slots")])
def test_keep(heads, D, page, layers, order):
    counts = [64, 1, 9, 5, 16, 2]
    batch = Batch(counts, [0, 5, 250, 31, 16, 1], page, N=64)
    k, v = new_cache(batch, heads, D, BF16, layers=layers, order=order)
    g = gen(18)
    for t in (k, v):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    paths = [list(range(1, 64, 2)), [], [8], [1, 2, 3, 4], [2, 3, 9, 15], [1]]
    path = np.full((6, 64), -1, np.int32)
    for b, s in enumerate(paths):
        path[b, :len(s)] = s
    want = [k.clone(), v.clone()]
    for b, s in enumerate(paths):
        if s:
            src, dst = batch.place(b, [batch.lengths[b] + a for a in s]), batch.place(b, [batch.lengths[b] + 1 + j for j in range(len(s))])
            for t, o in zip(want, (k, v)):
                if layers:
                    t[:, dst[0], dst[1]] = o[:, src[0], src[1]]
                else:
                    t[dst] = o[src]
    ws = workspace()
    ds.cache_keep(ds.PagedCache(k, v), batch.pages, batch.lens, torch.from_numpy(path).cuda(), i32([len(s) for s in paths]), ws)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and ws.status() == 0
