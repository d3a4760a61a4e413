"""The calls on rows of logits and of tables against their formulas in 64 bits: types, odd
lengths, strides and bases off 16-byte borders, ties, masked and empty rows, one row and
many, and gradients also against differences.

Tolerances.  A softmax sum of at most 9001 terms is formed by lanes that add at most 36 terms
each (512 lanes a CTA) and a tree of 10: under 50 roundings of 2^-24, 3e-6 relative; an
exponential adds 2^-22, and its argument's rounding |z - m| 2^-23 <= 5e-6 for terms that
matter (e^-40 at most beside them).  So sums agree within 1e-5 relative (SUM), logarithms of
them within 1e-5 absolute (20011 terms: the lanes of 2 to 8 CTAs, no more each).  An output of 16 bits is rounded once more, by half a step of its
type.  Longer rows (one case) have 8 CTAs and 125 terms a lane: the same bound."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")

SUM = 1e-5
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
NEG = -math.inf


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture
def ws():
    w = ds.Workspace.of_bytes(256)
    yield w
    assert w.status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def half_step(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def close(got, want, rtol=SUM, atol=SUM):
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= atol + rtol * want.abs())
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off; first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()}")


def logits(n, V, dtype, seed, layout="packed"):
    z = (torch.randn(n, V, generator=gen(seed), device="cuda") * 3).to(dtype)
    if layout == "packed":
        return z
    # rows `pad` apart in a larger buffer whose first row starts off a 16-byte border
    pad, first = {"strided": (24, 0), "odd": (13, 3)}[layout]
    buf = torch.zeros(n * (V + pad) + first, dtype=dtype, device="cuda")
    out = buf[first:].view(n, V + pad)[:, :V]
    out.copy_(z)
    return out


# --------------------------------------------------------------------- token_logprobs

def ref_logprobs(z, tokens, top):
    z = z.double()
    n, V = z.shape
    m = z.amax(1)
    e = torch.where(z == NEG, torch.zeros_like(z), (z - m[:, None]).exp())
    s = e.sum(1)
    d = torch.where(e > 0, z - m[:, None], torch.zeros_like(z))
    out = dict(row_max=m, row_sumexp=s, entropy=s.log() - (e * d).sum(1) / s)
    y = tokens.long().clamp(min=0)
    zy = z.gather(1, y[:, None])
    at = torch.arange(V, device=z.device)
    out["logprob"] = zy[:, 0] - m - s.log()
    out["rank"] = 1 + ((z > zy) | ((z == zy) & (at < y[:, None]))).sum(1)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    ids = torch.full((n, top), -1, device=z.device)
    ids[:, :order.shape[1]] = order
    lp = torch.full((n, top), NEG, device=z.device, dtype=torch.float64)
    lp[:, :order.shape[1]] = z.gather(1, order) - m[:, None] - s.log()[:, None]
    out["top_ids"], out["top_logprobs"] = ids, lp
    off = tokens < 0
    for key, fill in dict(row_max=NEG, row_sumexp=0, entropy=0, logprob=0, rank=0, top_ids=-1, top_logprobs=NEG).items():
        out[key][off] = fill
    return out


def check_logprobs(z, tokens, top, ws):
    got = ds.token_logprobs(z, tokens, top, ws)
    ref = ref_logprobs(z, tokens, top)
    torch.cuda.synchronize()
    assert torch.equal(got["row_max"].double(), ref["row_max"])
    assert torch.equal(got["rank"].long(), ref["rank"])
    close(got["row_sumexp"], ref["row_sumexp"])
    close(got["logprob"], ref["logprob"])
    close(got["entropy"], ref["entropy"], atol=3 * SUM)        # a mean of |z - m| of up to 3 here
    if top:
        assert torch.equal(got["top_ids"].long(), ref["top_ids"])
        close(got["top_logprobs"], ref["top_logprobs"])
    return got


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
@pytest.mark.parametrize("n,V,top", [(1, 1, 1), (3, 7, 2), (2, 8, 8), (5, 1000, 20), (4, 1000, 128),
                                     (1, 9001, 5), (3, 9001, 128), (700, 515, 1), (2, 4099, 0), (2, 100, 128),
                                     (3, 20011, 64)])
def test_logprobs(dtype, layout, n, V, top, ws):
    z = logits(n, V, dtype, 1, layout)
    tokens = torch.randint(0, V, (n,), generator=gen(2), device="cuda", dtype=torch.int32)
    if n > 2:
        tokens[1] = -1
    check_logprobs(z, tokens, top, ws)


def test_logprobs_many_rows_of_one_cta_and_long_rows(ws):
    for n, V, dtype in ((1300, 20011, torch.bfloat16), (9, 151936, torch.float32), (1, 600001, torch.float32)):
        z = logits(n, V, dtype, 3)
        tokens = torch.randint(0, V, (n,), generator=gen(4), device="cuda", dtype=torch.int32)
        got = ds.token_logprobs(z, tokens, 33, ws)
        ref = ref_logprobs(z, tokens, 33)
        assert torch.equal(got["top_ids"].long(), ref["top_ids"])
        assert torch.equal(got["rank"].long(), ref["rank"])
        close(got["logprob"], ref["logprob"], atol=3 * SUM)
        close(got["entropy"], ref["entropy"], atol=9 * SUM)


@pytest.mark.parametrize("n", [3000, 70000])
def test_logprobs_few_answers_among_many_rows(n, ws):
    """Long rows, nearly all without a token, below and above the number of rows that are dealt
    by their tokens."""
    V = 33000
    z = torch.empty(n, V, dtype=torch.bfloat16, device="cuda").normal_(0, 3, generator=gen(16))
    tokens = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    at = torch.randperm(n, generator=gen(17), device="cuda")[:40]
    tokens[at] = torch.randint(0, V, (40,), generator=gen(18), device="cuda", dtype=torch.int32)
    got = ds.token_logprobs(z, tokens, 7, ws)
    ref = ref_logprobs(z[at], tokens[at], 7)
    for key in ("top_ids", "rank"):
        assert torch.equal(got[key][at].long(), ref[key])
    for key in ("logprob", "top_logprobs", "row_sumexp"):
        close(got[key][at], ref[key], atol=3 * SUM)
    off = tokens < 0
    assert (got["logprob"][off] == 0).all() and (got["rank"][off] == 0).all() and (got["top_ids"][off] == -1).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [1000, 9001, 40000])
def test_logprobs_ties_and_orders(dtype, V, ws):
    """Rows that put every element at the bound: equal, ascending, descending and two-valued."""
    at = torch.arange(V, device="cuda")
    rows = torch.stack([torch.zeros(V, device="cuda"), at / V * 8, 8 - at / V * 8, (at % 3 == 1) * 2.0,
                        torch.full((V,), torch.finfo(dtype).min, device="cuda"), -0.0 * (at % 2)])
    tokens = torch.tensor([V // 2, V - 1, 0, 1, 3, V - 2], dtype=torch.int32, device="cuda")
    z = rows.to(dtype)
    got = ds.token_logprobs(z, tokens, 100, ws)
    ref = ref_logprobs(z, tokens, 100)
    assert torch.equal(got["top_ids"].long(), ref["top_ids"])
    assert torch.equal(got["rank"].long(), ref["rank"])
    close(got["logprob"], ref["logprob"], atol=3 * SUM)
    close(got["entropy"], ref["entropy"], atol=12 * SUM)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("V", [1000, 9001])
def test_logprobs_masked_logits(dtype, V, ws):
    z = logits(6, V, dtype, 5)
    z[0, 10:] = NEG                                    # ten alternatives left
    z[1, :] = NEG                                      # none
    z[2, 1::2] = torch.finfo(dtype).min
    z[3, V - 1] = math.nan
    z[4, 0] = math.inf
    z[5, :] = NEG
    z[5, V - 3] = -2.0                                 # one
    tokens = torch.tensor([3, 5, 4, 6, 7, V - 3], dtype=torch.int32, device="cuda")
    got = ds.token_logprobs(z, tokens, 20, ws)
    ref = ref_logprobs(z[[0, 2, 5]], tokens[[0, 2, 5]], 20)
    for key in ("top_ids", "rank"):
        assert torch.equal(got[key][[0, 2, 5]].long(), ref[key])
    for key in ("logprob", "top_logprobs", "row_sumexp"):
        close(got[key][[0, 2, 5]], ref[key])
    close(got["entropy"][[0, 2, 5]], ref["entropy"], atol=3 * SUM)
    assert got["logprob"][1] == NEG and got["entropy"][1] == 0 and got["row_max"][1] == NEG
    assert got["row_sumexp"][1] == 0 and (got["top_logprobs"][1] == NEG).all()
    for r in (3, 4):
        assert all(got[k][r].isnan().all() for k in ("logprob", "entropy", "top_logprobs", "row_sumexp"))
        assert got["rank"][r] == 0 and (got["top_ids"][r] == -1).all()


def test_logprobs_of_a_step_reads_no_row_without_a_token(ws):
    """Target rows [B, gamma + 1, V] and out_tokens as a verification leaves them: NaN in the
    rows past the answer touches nothing; without tokens every row is used."""
    B, g1, V = 3, 4, 1000
    T = logits(B * g1, V, torch.float32, 6).view(B, g1, V)
    out_tokens = torch.tensor([[5, 6, -1, -1], [7, -1, -1, -1], [1, 2, 3, 999]], dtype=torch.int32, device="cuda")
    clean = T.clone()
    T[out_tokens < 0] = math.nan
    got = ds.token_logprobs(T, out_tokens, 4, ws)
    ref = ref_logprobs(clean.view(-1, V), out_tokens.view(-1), 4)
    assert got["logprob"].shape == (B, g1) and got["top_ids"].shape == (B, g1, 4)
    close(got["logprob"].view(-1), ref["logprob"])
    assert torch.equal(got["top_ids"].view(-1, 4).long(), ref["top_ids"])
    every = ds.token_logprobs(clean, None, 4, ws)
    assert "logprob" not in every and "rank" not in every
    ref = ref_logprobs(clean.view(-1, V), torch.zeros(B * g1, device="cuda"), 4)
    assert torch.equal(every["top_ids"].view(-1, 4).long(), ref["top_ids"])
    close(every["entropy"].view(-1), ref["entropy"], atol=3 * SUM)


def test_bad_tokens_are_reported():
    w = ds.Workspace.of_bytes(256)
    z = logits(3, 1000, torch.float32, 7)
    tokens = torch.tensor([1, 1000, -2], dtype=torch.int32, device="cuda")
    got = ds.token_logprobs(z, tokens, 2, w)
    assert w.status() == 5 and w.status() == 0
    assert got["rank"].tolist()[1:] == [0, 0] and (got["top_ids"][1:] == -1).all()
    d = ds.token_logprobs_grad(z, tokens, got["row_max"], got["row_sumexp"], got["entropy"],
                               torch.ones(3, device="cuda"), None, w)
    assert w.status() == 5 and (d[1:] == 0).all() and (d[0] != 0).any()


def ref_logprobs_grad(z, tokens, gl, gh):
    z = z.double()
    p = torch.softmax(z, 1)
    logp = torch.log_softmax(z, 1)
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    H = -plogp.sum(1, keepdim=True)
    d = -gl[:, None].double() * p - gh[:, None].double() * (plogp + p * H)
    d.scatter_add_(1, tokens.long().clamp(min=0)[:, None], gl[:, None].double())
    d[tokens < 0] = 0
    return d


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
@pytest.mark.parametrize("out", ["new", "in place", "off by one"])
@pytest.mark.parametrize("n,V", [(1, 1), (3, 7), (4, 1000), (2, 9001)])
def test_logprobs_grad(dtype, layout, out, n, V, ws):
    z = logits(n, V, dtype, 8, layout)
    if V > 100:
        z[0, 50:60] = NEG
    tokens = torch.randint(0, V, (n,), generator=gen(9), device="cuda", dtype=torch.int32)
    if V > 100:
        tokens[0] = 3
    if n > 2:
        tokens[1] = -1
        z[1, 0] = math.nan
    st = ds.token_logprobs(z, tokens, 0, ws)
    gl, gh = (torch.randn(n, generator=gen(10 + i), device="cuda") for i in range(2))
    ref = ref_logprobs_grad(torch.where(tokens[:, None] < 0, torch.zeros_like(z), z), tokens, gl, gh)
    buf = None
    if out == "in place":
        buf = z
    elif out == "off by one":
        buf = torch.empty(n * (V + 1) + 1, dtype=dtype, device="cuda")[1:].view(n, V + 1)[:, :V]
    got = ds.token_logprobs_grad(z, tokens, st["row_max"], st["row_sumexp"], st["entropy"], gl, gh, ws, buf)
    # p within SUM relative, times a factor of at most |gl| + |gh| (|log p| + H) < 3 + 3 * 20
    close(got, ref, rtol=4 * SUM + half_step(dtype), atol=4 * SUM)


def test_logprobs_grad_against_differences(ws):
    n, V, h = 4, 300, 1e-2
    z = logits(n, V, torch.float32, 11)
    tokens = torch.tensor([0, 5, 299, 17], dtype=torch.int32, device="cuda")
    gl, gh = (torch.randn(n, generator=gen(12 + i), device="cuda") for i in range(2))
    st = ds.token_logprobs(z, tokens, 0, ws)
    d = ds.token_logprobs_grad(z, tokens, st["row_max"], st["row_sumexp"], st["entropy"], gl, gh, ws)
    way = torch.randn(n, V, generator=gen(14), device="cuda")
    way /= way.norm(dim=1, keepdim=True)

    def f(x):
        o = ds.token_logprobs(x, tokens, 0, ws)
        return gl * o["logprob"] + gh * o["entropy"]
    got = (f(z + h * way) - f(z - h * way)) / (2 * h)
    # h^2 times a third derivative of order 10, and two roundings of the values over 2 h
    close(got, (d * way).sum(1), rtol=0, atol=5e-3)


def test_one_upstream_gradient_and_empty_rows(ws):
    z = logits(3, 1000, torch.float32, 15)
    z[2] = NEG
    tokens = torch.tensor([3, 4, 5], dtype=torch.int32, device="cuda")
    st = ds.token_logprobs(z, tokens, 0, ws)
    one, zero = torch.ones(3, device="cuda"), torch.zeros(3, device="cuda")
    a = ds.token_logprobs_grad(z, tokens, st["row_max"], st["row_sumexp"], None, one, None, ws)
    close(a[:2], ref_logprobs_grad(z[:2], tokens[:2], one[:2], zero[:2]))
    b = ds.token_logprobs_grad(z, tokens, st["row_max"], st["row_sumexp"], st["entropy"], None, one, ws)
    close(b[:2], ref_logprobs_grad(z[:2], tokens[:2], zero[:2], one[:2]), atol=4 * SUM)
    assert (a[2] == 0).all() and (b[2] == 0).all()


# ------------------------------------------------------------------------------ distill

def ref_distill(z, ids, t, labels, w, g, tau, kl, tv, ce):
    x = z.double() / tau
    logq = torch.log_softmax(x, 1)
    n, V = z.shape
    on = (ids >= 0) & (ids < V)
    at = torch.where(on, ids, 0).long()
    tt = torch.where(on, t.double() / tau, NEG)
    some = (tt > NEG).any(1, keepdim=True)
    p = torch.where(some, torch.softmax(torch.where(some, tt, 0.0), 1), 0.0) * on
    lq = logq.gather(1, at)
    q = torch.where(on & some, lq.exp(), 0.0)
    KL = torch.where(p > 0, p * (p.clamp(min=1e-300).log() - lq), 0.0).sum(1)
    TV = (p - q).clamp(min=0).sum(1)
    y = labels.long()
    named = (y >= 0).double()
    yl = logq.gather(1, y.clamp(min=0)[:, None])[:, 0]
    terms = torch.zeros(n, dtype=torch.float64, device="cuda")
    if kl:
        terms = terms + kl * KL
    if tv:
        terms = terms + tv * TV
    if ce:
        terms = terms - ce * torch.where(named > 0, yl, 0.0)
    a = torch.zeros_like(p)
    if kl:
        a = a + kl * p
    a = a + tv * q * (q < p)
    tgt = torch.zeros_like(logq)
    tgt.scatter_add_(1, at, a * on)
    tgt.scatter_add_(1, y.clamp(min=0)[:, None], (ce * named)[:, None])
    d = (logq.exp() * tgt.sum(1, keepdim=True) - tgt) * (g.double() * w.double() / tau)[:, None]
    live = w != 0
    dead = ~live | (~some[:, 0] & (named == 0))
    d[dead] = 0
    loss = torch.where(dead, 0.0, terms * w.double())
    return dict(loss=loss, accept=torch.where(dead, 0.0, torch.minimum(p, q).sum(1)), d_logits=d)


def teacher(n, V, K, seed, z=None):
    """Distinct ids in random order with holes, and log probabilities."""
    g = gen(seed)
    ids = torch.rand(n, V, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32)
    if ids.shape[1] < K:
        ids = torch.cat([ids, torch.full((n, K - ids.shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    t = torch.randn(n, K, generator=g, device="cuda") * 2 - 5
    ids[torch.rand(n, K, generator=g, device="cuda") < 0.1] = -1
    return ids.contiguous(), t


def check_distill(z, ids, t, labels, w, g, ws, out=None, tol=1.0, **kw):
    full = dict(temperature=1.0, kl=1.0, tv=0.0, ce=0.0) | kw
    zero = torch.where(w[:, None] != 0, z, torch.zeros_like(z))
    ref = ref_distill(zero, ids, t, labels, w, g, full["temperature"], full["kl"], full["tv"], full["ce"])
    alone = ds.distill_loss(z, ids, t, ws, labels, w, **full)
    buf = None if out is None else dict(loss=torch.empty_like(w), accept=torch.empty_like(w), d_logits=out)
    got = ds.distill_loss_grad(z, ids, t, ws, labels, w, g, out=buf, **full)
    for o in (alone, got):
        # log q to SUM (twice: the argument is divided by the temperature), weights up to 3
        close(o["loss"], ref["loss"], rtol=2 * SUM, atol=6 * SUM * tol)
        close(o["accept"], ref["accept"], rtol=2 * SUM, atol=2 * SUM)
    scale = (g * w).abs().max().item() / full["temperature"]
    close(got["d_logits"], ref["d_logits"], rtol=2 * SUM * tol + half_step(z.dtype), atol=2 * SUM * scale * tol)
    return got


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
@pytest.mark.parametrize("n,V,K", [(1, 1, 1), (3, 7, 3), (4, 8, 128), (16, 1000, 8), (2, 9001, 128), (5, 9001, 33),
                                   (3, 20011, 64)])
@pytest.mark.parametrize("terms", [dict(kl=1.0), dict(kl=0.0, tv=0.9, ce=0.1), dict(kl=0.5, tv=0.3, ce=0.2, temperature=2.0)],
                         ids=["kl", "tv+ce", "all"])
def test_distill(dtype, layout, n, V, K, terms, ws):
    z = logits(n, V, dtype, 20, layout)
    ids, t = teacher(n, V, K, 21)
    labels = torch.randint(-1, V, (n,), generator=gen(22), device="cuda", dtype=torch.int32)
    w = torch.rand(n, generator=gen(23), device="cuda") + 0.5
    g = torch.randn(n, generator=gen(24), device="cuda")
    if n > 2:
        w[1] = 0
        z[1, 0] = math.nan                             # a masked row is not read
        labels[2] = ids[2, 0]                          # the label among the teacher's entries
    check_distill(z, ids, t, labels, w, g, ws, **terms)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("out", ["in place", "off by one"])
@pytest.mark.parametrize("n,V", [(3, 1000), (2, 9001), (400, 257), (2, 20011)])
def test_distill_output_buffers(dtype, out, n, V, ws):
    z = logits(n, V, dtype, 30)
    ids, t = teacher(n, V, 16, 31)
    labels = torch.randint(0, V, (n,), generator=gen(32), device="cuda", dtype=torch.int32)
    w = torch.ones(n, device="cuda")
    w[0] = 0
    g = torch.ones(n, device="cuda")
    if out == "in place":
        want = check_distill(z.clone(), ids, t, labels, w, g, ws, kl=0.9, ce=0.1)["d_logits"]
        got = ds.distill_loss_grad(z, ids, t, ws, labels, w, g, kl=0.9, ce=0.1,
                                   out=dict(loss=torch.empty_like(w), accept=torch.empty_like(w), d_logits=z))
        assert got["d_logits"].data_ptr() == z.data_ptr() and torch.equal(z, want)
    else:
        buf = torch.empty(n * (V + 1) + 1, dtype=dtype, device="cuda")[1:].view(n, V + 1)[:, :V]
        check_distill(z, ids, t, labels, w, g, ws, out=buf, kl=0.9, ce=0.1)


def test_distill_rows_beyond_shared_memory(ws):
    """Rows longer than eight CTAs hold (1.7 MB): their rest is read twice."""
    n, V = 2, 500003
    z = logits(n, V, torch.float32, 33)
    ids, t = teacher(n, V, 64, 34)
    ids[0, 0], ids[0, 1] = V - 1, 0
    labels = torch.tensor([499999, -1], dtype=torch.int32, device="cuda")
    one = torch.ones(n, device="cuda")
    check_distill(z, ids, t, labels, one, one, ws, tol=3.0, kl=0.7, tv=0.2, ce=0.1)


def test_distill_many_rows(ws):
    n, V = 900, 20008
    z = logits(n, V, torch.bfloat16, 35)
    ids, t = teacher(n, V, 20, 36)
    labels = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    w = torch.exp(-(torch.arange(n, device="cuda") % 5) / 4.0)
    check_distill(z, ids, t, labels, w, torch.ones(n, device="cuda"), ws, tol=2.0)


def test_distill_rows_with_nothing_to_learn(ws):
    n, V, K = 6, 1000, 4
    z = logits(n, V, torch.float32, 37)
    ids, t = teacher(n, V, K, 38)
    ids[ids < 0] = 5
    ids[0] = -1                                        # no entry, no label
    t[1] = NEG                                         # entries without weight, a label
    t[2, 1] = NEG                                      # one entry without weight
    t[3] = NEG                                         # entries without weight, no label
    ids[4, 1] = ids[4, 0]                              # an id twice
    z[5, ids[5, 0].item()] = NEG                       # the student gives an entry probability 0
    labels = torch.tensor([-1, 7, -1, -1, 9, -1], dtype=torch.int32, device="cuda")
    one = torch.ones(n, device="cuda")
    got = check_distill(z, ids, t, labels, one, one, ws, kl=0.5, ce=0.5)
    assert (got["d_logits"][[0, 3]] == 0).all() and (got["loss"][[0, 3]] == 0).all()
    assert got["loss"][5] == math.inf and got["d_logits"][5].isfinite().all()
    check_distill(z, ids, t, labels, one, one, ws, kl=0.0, tv=1.0)


def test_distill_labels_alone_and_no_gradient_of_masked_values(ws):
    n, V = 3, 1000
    z = logits(n, V, torch.bfloat16, 39)
    labels = torch.tensor([1, 2, -1], dtype=torch.int32, device="cuda")
    w = torch.tensor([1.0, 0.0, 1.0], device="cuda")
    z[1] = math.nan
    got = ds.distill_loss_grad(z, None, None, ws, labels, w, kl=0.0, ce=1.0)
    ref = -torch.log_softmax(z[0].double(), 0)[1]
    close(got["loss"][:1], ref[None])
    assert got["loss"][1] == 0 and got["loss"][2] == 0 and (got["accept"] == 0).all()
    assert (got["d_logits"][1:] == 0).all()
    z[0, 5] = math.nan                                 # in a live row it shows
    assert ds.distill_loss(z, None, None, ws, labels, w, kl=0.0, ce=1.0)["loss"][0].isnan()


@pytest.mark.parametrize("terms", [dict(), dict(kl=0.0, tv=1.0), dict(kl=0.0, tv=0.5, ce=0.5)], ids=["kl", "tv", "tv+ce"])
def test_distill_shows_nan_and_inf(terms, ws):
    """A NaN or +inf in a live row, or a NaN from the teacher, reaches loss, acceptance and
    gradient; other rows are untouched."""
    n, V, K = 4, 1000, 8
    z = logits(n, V, torch.float32, 45)
    ids, t = teacher(n, V, K, 46)
    ids[ids < 0] = 999
    labels = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    clean = ds.distill_loss_grad(z, ids, t, ws, labels, **terms)
    z[1, 77], z[2, 78] = math.nan, math.inf
    t[3, 2] = math.nan
    got = ds.distill_loss_grad(z, ids, t, ws, labels, **terms)
    for key in got:
        assert torch.equal(got[key][0], clean[key][0])
        assert got[key][1:3].isnan().all()
    assert got["loss"][3].isnan() and got["accept"][3].isnan()


def test_distill_against_differences(ws):
    n, V, K, h = 4, 300, 10, 1e-2
    z = logits(n, V, torch.float32, 40)
    ids, t = teacher(n, V, K, 41)
    labels = torch.tensor([0, 5, -1, 17], dtype=torch.int32, device="cuda")
    w = torch.tensor([1.0, 0.5, 2.0, 0.0], device="cuda")
    kw = dict(temperature=1.5, kl=0.6, tv=0.5, ce=0.3)
    d = ds.distill_loss_grad(z, ids, t, ws, labels, w, **kw)["d_logits"]
    way = torch.randn(n, V, generator=gen(42), device="cuda")
    way /= way.norm(dim=1, keepdim=True)
    f = lambda x: ds.distill_loss(x, ids, t, ws, labels, w, **kw)["loss"]  # noqa: E731
    # as above; a total variation term's corner within h adds at most h times its slope's jump
    close((f(z + h * way) - f(z - h * way)) / (2 * h), (d * way).sum(1), rtol=0, atol=1e-2)


def test_distill_reports_bad_ids():
    w = ds.Workspace.of_bytes(256)
    z = logits(2, 1000, torch.float32, 43)
    ids, t = teacher(2, 1000, 4, 44)
    ids[:] = torch.tensor([[1, 2, 1000, 4], [1, 2, 3, 4]], dtype=torch.int32)
    got = ds.distill_loss_grad(z, ids, t, w)
    assert w.status() == 5
    ids[0, 2] = -1
    want = ds.distill_loss_grad(z, ids, t, w)
    assert w.status() == 0 and all(torch.equal(got[k], want[k]) for k in want)
    ds.distill_loss(z, ids, t, w, torch.tensor([1000, 0], dtype=torch.int32, device="cuda"))
    assert w.status() == 5


# -------------------------------------------------------------------------------- embed

@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, None), (torch.bfloat16, None), (torch.float16, None),
                                             (torch.bfloat16, torch.float32), (torch.float16, torch.float32)], ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
@pytest.mark.parametrize("n,V,D", [(0, 5, 8), (1, 1, 1), (7, 100, 17), (33, 1000, 256), (5, 40, 2560), (3, 9, 4099)])
def test_embed(dtype, out_dtype, layout, n, V, D, ws):
    W = logits(V, D, dtype, 50, layout)
    ids = torch.randint(0, V, (n,), generator=gen(51), device="cuda", dtype=torch.int32)
    if n > 2:
        ids[1] = -1
    got = ds.embed(W, ids, ws, 0.7, dtype=out_dtype)
    ref = 0.7 * W[ids.long().clamp(min=0)].double()
    ref[ids < 0] = 0
    # the scale rounded to fp32, the product rounded, and the store
    close(got, ref, rtol=2 ** -23 + half_step(out_dtype or dtype), atol=1e-7)


def test_embed_nd_ids_and_bad_ids():
    w = ds.Workspace.of_bytes(256)
    W = logits(10, 16, torch.float32, 52)
    W[3] = math.nan
    ids = torch.tensor([[0, 10], [-5, 2]], dtype=torch.int32, device="cuda")
    got = ds.embed(W, ids, w)
    assert w.status() == 5 and got.shape == (2, 2, 16)
    assert torch.equal(got[0, 0], W[0]) and torch.equal(got[1, 1], W[2])
    assert (got[0, 1] == 0).all() and (got[1, 0] == 0).all()


def ids_of(kind, n, V, seed):
    g = gen(seed)
    if kind == "same":
        ids = torch.full((n,), V // 2, dtype=torch.int32, device="cuda")
    elif kind == "uniform":
        ids = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    else:                                              # a few tokens hold most positions
        u = torch.rand(n, generator=g, device="cuda")
        ids = (V * u ** 6).to(torch.int32).clamp(max=V - 1)
    if kind != "same":
        ids[torch.rand(n, generator=g, device="cuda") < 0.05] = -1
    return ids


def ref_embed_grad(d_out, ids, V, scale):
    d = torch.zeros(V + 1, d_out.shape[1], dtype=torch.float64, device="cuda")
    a = torch.zeros_like(d)
    at = torch.where(ids < 0, V, ids).long()
    d.index_add_(0, at, d_out.double())
    a.index_add_(0, at, d_out.double().abs())
    return scale * d[:V], abs(scale) * a[:V]


def check_embed_grad(d_out, ids, V, out=None, dtype=None, accumulate=False):
    n, D = d_out.shape
    w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(n, V, D))
    ref, size = ref_embed_grad(d_out, ids, V, 0.7)
    start = None
    if accumulate:
        start = out.clone()
        ref = ref + start.double()
        size = size + start.double().abs()
    got = ds.embed_grad(d_out, ids, V, w, 0.7, out, accumulate, dtype)
    assert w.status() == 0
    # fp32 sums of up to n terms in some order: at most (n + 3) roundings of the absolute sum
    off = (got.double() - ref).abs()
    bound = (n + 3) * 2.0 ** -24 * size + half_step(got.dtype) * ref.abs() * 1.001 + 1e-7 * half_step(got.dtype)
    assert (off <= bound).all(), f"off by {(off - bound).max().item():.3g}"
    rows = torch.zeros(V, dtype=torch.bool, device="cuda")
    rows[ids[ids >= 0].long()] = True
    if accumulate:
        assert torch.equal(got[~rows], start[~rows])
    else:
        assert (got[~rows] == 0).all()
        again = ds.embed_grad(d_out, ids, V, w, 0.7, None, False, dtype)
        assert torch.equal(again, got)                 # the same bits
    return got


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, None), (torch.bfloat16, None), (torch.float16, None),
                                             (torch.bfloat16, torch.float32), (torch.float16, torch.float32)], ids=str)
@pytest.mark.parametrize("kind", ["uniform", "uneven", "same"])
@pytest.mark.parametrize("n,V,D", [(0, 5, 8), (1, 1, 1), (9, 100, 17), (64, 10, 8), (1000, 300, 256), (8192, 50, 16),
                                   (8193, 1000, 24), (30000, 300000, 8), (20000, 513, 33), (2049, 70, 40),
                                   (140000, 5000, 16), (700, 50, 2560), (3000, 300000, 8)])
def test_embed_grad(dtype, out_dtype, kind, n, V, D):
    d_out = logits(n, D, dtype, 60)
    check_embed_grad(d_out, ids_of(kind, n, V, 61), V, dtype=out_dtype)


@pytest.mark.parametrize("kind", ["uniform", "uneven", "same"])
def test_embed_grad_many_positions_of_a_large_table(kind):
    """Zeroes enough to hide one cluster's sort of several tiles a CTA."""
    n, V, D = 17000, 70000, 256
    check_embed_grad(logits(n, D, torch.float32, 58), ids_of(kind, n, V, 59), V)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided", "odd"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,V,D", [(500, 40, 64), (9000, 700, 72)])
def test_embed_grad_layouts(dtype, layout, accumulate, n, V, D):
    d_out = logits(n, D, dtype, 62, layout)
    out = logits(V, D, dtype, 63, layout)
    check_embed_grad(d_out, ids_of("uneven", n, V, 64), V, out=out, accumulate=accumulate)


def test_embed_grad_leaves_the_padding_between_rows(ws):
    V, D = 20, 10
    buf = torch.full((V, 16), 7.0, device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(3, V, D))
    ds.embed_grad(torch.ones(3, D, device="cuda"), ids, V, w, out=buf[:, :D])
    assert (buf[0, :D] == 3).all() and (buf[1:, :D] == 0).all() and (buf[:, D:] == 7).all()


def test_embed_grad_reports_bad_ids():
    for n in (50, 9000):
        d_out = logits(n, 8, torch.float32, 65)
        ids = ids_of("uniform", n, 30, 66)
        w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(n, 30, 8))
        want = ds.embed_grad(d_out, torch.where(torch.arange(n, device="cuda") == 7, -1, ids).to(torch.int32), 30, w)
        assert w.status() == 0
        ids[7] = 30
        got = ds.embed_grad(d_out, ids, 30, w)
        assert w.status() == 5 and torch.equal(got, want)


def test_embed_grad_is_embeds_gradient(ws):
    """<d_out, embed(dW)> = <embed_grad(d_out), dW> for any dW: the lookup is linear."""
    V, D, n = 200, 48, 900
    ids = ids_of("uneven", n, V, 67)
    d_out = torch.randn(n, D, generator=gen(68), device="cuda")
    way = torch.randn(V, D, generator=gen(69), device="cuda")
    w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(n, V, D))
    left = (ds.embed(way, ids, ws, 1.5).double() * d_out.double()).sum()
    right = (ds.embed_grad(d_out, ids, V, w, 1.5).double() * way.double()).sum()
    size = (ds.embed(way, ids, ws, 1.5).double() * d_out.double()).abs().sum()
    assert abs(left - right) <= 1e-5 * size


# ------------------------------------------------------------- streams, graphs, refusals

def test_on_another_stream_and_in_a_graph():
    n, V = 8, 5000
    z = logits(n, V, torch.float32, 70)
    ids, t = teacher(n, V, 8, 71)
    tokens = torch.randint(0, V, (n,), generator=gen(72), device="cuda", dtype=torch.int32)
    d_e = torch.randn(n, 64, generator=gen(73), device="cuda")
    w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(n, V, 64))

    def all_calls(stream=None):
        lp = ds.token_logprobs(z, tokens, 5, w, stream=stream)
        dz = ds.token_logprobs_grad(z, tokens, lp["row_max"], lp["row_sumexp"], lp["entropy"], lp["logprob"],
                                    None, w, stream=stream)
        di = ds.distill_loss_grad(z, ids, t, w, stream=stream)
        dw = ds.embed_grad(d_e, tokens, V, w, stream=stream)
        return [*lp.values(), dz, *di.values(), dw, ds.embed(dw, tokens, w, 2.0, stream=stream)]

    want = [x.clone() for x in all_calls()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = all_calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_calls()
    for x in got:
        x.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and w.status() == 0


def test_python_refusals(ws):
    z = logits(4, 100, torch.float32, 74)
    i32 = torch.zeros(4, dtype=torch.int32, device="cuda")
    ids, t = teacher(4, 100, 3, 75)
    refused = [
        lambda: ds.token_logprobs(z.double(), i32, 1, ws),
        lambda: ds.token_logprobs(z.cpu(), i32, 1, ws),
        lambda: ds.token_logprobs(z.t(), i32, 1, ws),
        lambda: ds.token_logprobs(z, i32.long(), 1, ws),
        lambda: ds.token_logprobs(z, i32[:3], 1, ws),
        lambda: ds.token_logprobs(z, i32.cpu(), 1, ws),
        lambda: ds.token_logprobs(z.view(2, 2, 100).transpose(0, 1), i32, 1, ws),
        lambda: ds.token_logprobs(z, i32, 2, ws, out=dict(ds.token_logprobs(z, i32, 1, ws))),
        lambda: ds.token_logprobs_grad(z, i32, z[:, 0], z[:, 1], None, None, None, ws),
        lambda: ds.distill_loss(z, ids.long(), t, ws),
        lambda: ds.distill_loss(z, ids, t[:, :2], ws),
        lambda: ds.distill_loss(z, ids, t.half(), ws),
        lambda: ds.distill_loss_grad(z, ids, t, ws, out=dict(loss=z[:, 0].contiguous(), accept=z[:, 0].contiguous(),
                                                             d_logits=z.half())),
        lambda: ds.embed(z, i32.long(), ws),
        lambda: ds.embed(z[0], i32, ws),
        lambda: ds.embed(z, i32, ws, out=z[:3]),
        lambda: ds.embed_grad(z, i32[:2], 10, ws),
        lambda: ds.embed_grad(z, i32, 10, ws, accumulate=True),
        lambda: ds.embed_grad(z, i32, 10, ws, out=z),
        lambda: ds.embed_grad_workspace_bytes(4, 0, 8),
    ]
    for call in refused:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ds.token_logprobs(z, i32, 129, ws), lambda: ds.distill_loss(z, ids, t, ws, temperature=0.0),
                 lambda: ds.embed(z.half(), i32, ws, dtype=torch.bfloat16),
                 lambda: ds.embed_grad(z, i32, 10, ws)):           # a workspace of 256 bytes is too small
        with pytest.raises(ds.DSparkError):
            call()
    assert ds.token_logprobs(z[:0], i32[:0], 3, ws)["top_ids"].shape == (0, 3)
