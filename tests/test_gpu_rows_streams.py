"""Long rows by the persistent clusters, many to a cluster, against the formulas in 64 bits: every
buffer and barrier is used again several times, with CTAs of a row on 1, 2, 4 and 8 SMs, masked
rows in the middle of the stream, and rows whose end takes another path than their neighbours'.

Paths.  Rows of up to 4096 16-byte chunks (``token_logprobs``; 2048 for the distillation) go to a
CTA each; these cases are longer.  A GB300 holds 304, 152, 74 and 36 clusters of 1, 2, 4 and 8
CTAs; each case says how many CTAs a row has there and how many rows a cluster.

Tolerances.  A thread adds its elements in batches of 16 or 32 (two sums of two lanes: 4 or 8
additions, one to join them), then batch to batch, lane to lane, over the warp (5) and over the
cluster (at most 7): 19 batches of 16 for a row of 600001 over 8 CTAs of 256 threads, and at most
4 of a chunk each at its part's end, so under 45 roundings of 2^-24 = 2.7e-6 relative.  An
exponential adds 2^-22, its argument's rounding |z - m| 2^-23 <= 5e-6 for terms that matter.  So
sums agree within 1e-5 relative (SUM of test_gpu_rows), their logarithms within 1e-5; an entropy
subtracts a mean of |z - m| (at most 8 here) of the same accuracy.  Values of 16 bits are rounded
once more."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")

from test_gpu_rows import NEG, SUM, close, gen, half_step, ref_distill  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture
def ws():
    w = ds.Workspace.of_bytes(256)
    yield w
    assert w.status() == 0


def in_chunks(n, V, f):
    """{key: rows} of f(rows) over slices of about 32 M elements."""
    step = max(1, (1 << 25) // V)
    parts = [f(slice(i, min(n, i + step))) for i in range(0, n, step)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def long_logits(n, V, dtype, seed):
    z = torch.empty(n, V, dtype=dtype, device="cuda")
    return z.normal_(0, 3, generator=gen(seed))


# --------------------------------------------------------------------- token_logprobs

def ref_rows(z, y, top):
    """Every output for finite tokens y, ties to the lowest index."""
    f = z.float()
    z = z.double()
    n, V = z.shape
    m = z.amax(1)
    some = m > NEG
    d = torch.where(z > NEG, z - torch.where(some, m, 0.0)[:, None], NEG)
    e = d.exp()
    s = e.sum(1)
    logs = s.log()
    zy = z.gather(1, y[:, None])
    at = torch.arange(V, device=z.device)
    out = dict(row_max=m, row_sumexp=s)
    out["entropy"] = torch.where(some, logs - (e * torch.where(e > 0, d, 0.0)).sum(1) / s, 0.0)
    out["logprob"] = torch.where(some, zy[:, 0] - m - logs, NEG)
    out["rank"] = 1 + ((z > zy) | ((z == zy) & (at < y[:, None]))).sum(1)
    bits = f.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) + (V - 1 - at)
    ids = V - 1 - (key.topk(top, 1).values & 0xFFFFFFFF)
    out["top_ids"] = ids
    out["top_logprobs"] = torch.where(some[:, None], z.gather(1, ids) - m[:, None] - logs[:, None], NEG)
    return out


MOST = 64


@pytest.mark.parametrize("n,V,dtype", [
    (2500, 17000, torch.float32),      # 1 CTA a row, 8 rows a cluster
    (3000, 40000, torch.float16),      # 1, 10
    (1536, 129280, torch.float32),     # 2, 10
    (750, 600001, torch.bfloat16),     # 4, 10, two pieces a maximum, rows off 16-byte borders
    (400, 600001, torch.float32),      # 8, 11
], ids=str)
def test_logprobs_many_rows_a_cluster(n, V, dtype, ws):
    z = long_logits(n, V, dtype, 200)
    y = torch.randint(0, V, (n,), generator=gen(201), device="cuda")
    # rows whose end is longer than their neighbours': equal, ascending, few logits, none
    at = torch.arange(V, device="cuda")
    z[11::97] = 0.5
    z[23::97] = (at / V * 8).to(dtype)
    z[37::97, 10:] = NEG
    z[38::97] = NEG
    ref = in_chunks(n, V, lambda i: ref_rows(z[i], y[i], MOST))
    z[50::97, V // 3], z[51::97, V - 1] = math.nan, math.inf
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[50::97] = bad[51::97] = True
    used = torch.rand(n, generator=gen(202), device="cuda") < 0.7
    used[:2] = False
    every = torch.ones_like(used)

    def check(got, rows, top, tokens):
        want = {k: v.clone() for k, v in ref.items() if tokens or k not in ("logprob", "rank")}
        if top:
            want["top_ids"], want["top_logprobs"] = want["top_ids"][:, :top], want["top_logprobs"][:, :top]
        else:
            del want["top_ids"], want["top_logprobs"]
        for key, v in want.items():
            v[bad] = {"rank": 0, "top_ids": -1}.get(key, math.nan)
            v[~rows] = {"rank": 0, "top_ids": -1, "row_max": NEG, "top_logprobs": NEG}.get(key, 0)
        assert set(got) == set(want)
        skip = bad & rows                              # (row_max: the largest number that is one)
        assert torch.equal(got["row_max"].double()[~skip], want["row_max"][~skip])
        close(got["row_sumexp"], want["row_sumexp"])
        close(got["entropy"], want["entropy"], atol=9 * SUM)
        if tokens:
            assert torch.equal(got["rank"].long(), want["rank"])
            close(got["logprob"], want["logprob"], atol=3 * SUM)
        if top:
            assert torch.equal(got["top_ids"].long(), want["top_ids"])
            close(got["top_logprobs"], want["top_logprobs"], atol=3 * SUM)

    tokens = torch.where(used, y, -1).to(torch.int32)
    check(ds.token_logprobs(z, tokens, MOST, ws), used, MOST, True)
    check(ds.token_logprobs(z, tokens, 0, ws), used, 0, True)
    check(ds.token_logprobs(z, y.to(torch.int32), 5, ws), every, 5, True)
    check(ds.token_logprobs(z, None, 33, ws), every, 33, False)


# ------------------------------------------------------------------------------ distill

@pytest.mark.parametrize("n,V,dtype", [
    (2800, 20001, torch.float32),      # 1 CTA a row, 9 rows a cluster, rows off 16-byte borders
    (1400, 40000, torch.float32),      # 2, 9
    (1400, 80001, torch.float16),      # 2, 9, rows off 16-byte borders
    (640, 160000, torch.bfloat16),     # 4, 9
    (320, 129280, torch.float32),      # 8, 9
    (300, 500003, torch.float32),      # 8, 8, the rest of a row read twice, off 16-byte borders
], ids=str)
@pytest.mark.parametrize("out", ["new", "in place", "off by one"])
def test_distill_many_rows_a_cluster(n, V, dtype, out, ws):
    K = 40
    g = gen(210)
    z = long_logits(n, V, dtype, 211)
    first = torch.randint(0, V, (n, 1), generator=g, device="cuda")
    ids = ((first + torch.arange(K, device="cuda") * (V // K)) % V).to(torch.int32)   # over all of the row
    ids[torch.rand(n, K, generator=g, device="cuda") < 0.1] = -1
    t = torch.randn(n, K, generator=g, device="cuda") * 2 - 5
    labels = torch.randint(-1, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(n, generator=g, device="cuda") + 0.5
    w[torch.rand(n, generator=g, device="cuda") < 0.25] = 0
    w[0], w[-1] = 0, 0
    d_loss = torch.randn(n, generator=g, device="cuda")
    # rows that end in their own way, in the middle of the stream
    rows = lambda i: torch.arange(i, n, 41, device="cuda")  # noqa: E731
    ids[rows(3)], labels[rows(3)] = -1, -1                  # nothing to learn
    t[rows(5)], labels[rows(5)] = NEG, -1                   # entries without weight
    ids[rows(7)], labels[rows(7)] = -1, 11                  # the label alone
    d_loss[rows(9)] = 0
    ids[rows(11), 0], ids[rows(11), 1], ids[rows(11), 2] = V - 1, 0, V - 1     # an id twice
    ids[rows(13), 5], labels[rows(13)] = 77, 77             # the label among the entries
    ids[rows(15), 6] = 78
    z[rows(15), 78] = NEG                                   # the student gives an entry probability 0
    z[rows(17), V // 2] = math.nan
    z[rows(19), V - 1] = math.inf
    for r in (3, 5, 7, 9, 11, 13, 15, 17, 19, 21):
        w[rows(r)[0]] = 1.0
    kw = dict(temperature=1.5, kl=0.5, tv=0.3, ce=0.2)
    # (rows of weight 0 hold NaN: they are not read)
    clean = z.clone()
    z[w == 0] = math.nan
    clean[w == 0] = 0
    ref = in_chunks(n, V, lambda i: ref_distill(clean[i], ids[i], t[i], labels[i], w[i], d_loss[i], 1.5, 0.5, 0.3, 0.2))
    t[rows(21)] = math.nan                                  # a teacher without a number
    for key, v in ref.items():
        dark = rows(21)
        v[dark[w[dark] != 0]] = math.nan
    alone = ds.distill_loss(z, ids, t, ws, labels, w, **kw)
    buf = None
    if out == "in place":
        buf = {"d_logits": z}
    elif out == "off by one":
        buf = {"d_logits": torch.empty(n * (V + 1) + 1, dtype=dtype, device="cuda")[1:].view(n, V + 1)[:, :V]}
    got = ds.distill_loss_grad(z, ids, t, ws, labels, w, d_loss, out=buf, **kw)
    for o in (alone, got):
        # log q to SUM, weights up to 1.5, values up to 30
        close(o["loss"], ref["loss"], rtol=2 * SUM, atol=6 * SUM)
        close(o["accept"], ref["accept"], rtol=2 * SUM, atol=2 * SUM)
    # d_loss times the weight: 8 at most; a value of 0 by a row with nothing to learn
    scale = (d_loss * w).abs().max().item()
    step = max(1, (1 << 25) // V)
    for i in range(0, n, step):
        close(got["d_logits"][i:i + step], ref["d_logits"][i:i + step], rtol=2 * SUM + half_step(dtype),
              atol=2 * SUM * scale)
    for r in (3, 5):
        live = rows(r)[w[rows(r)] != 0]
        assert len(live) and (got["d_logits"][live] == 0).all() and (got["loss"][live] == 0).all()
    zero = w == 0
    assert (got["d_logits"][zero] == 0).all() and (got["loss"][zero] == 0).all() and (got["accept"][zero] == 0).all()
