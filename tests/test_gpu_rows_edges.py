"""The calls on rows of logits and of tables at the edges of what they take.  Tolerances as in
test_gpu_rows."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")

from test_gpu_rows import SUM, close, logits, ref_distill, teacher  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture
def ws():
    w = ds.Workspace.of_bytes(256)
    yield w
    assert w.status() == 0


def ones(n):
    return torch.ones(n, device="cuda")


# ------------------------------------------------------------------------------ no rows

@pytest.mark.parametrize("lead", [(0,), (0, 4)])
def test_distill_of_no_rows(lead, ws):
    z = torch.empty(lead + (1000,), device="cuda")
    ids = torch.empty(lead + (8,), dtype=torch.int32, device="cuda")
    t = torch.empty(lead + (8,), device="cuda")
    alone = ds.distill_loss(z, ids, t, ws, labels=ids[..., 0].contiguous(), weights=t[..., 0].contiguous())
    both = ds.distill_loss_grad(z, ids, t, ws, d_loss=t[..., 0].contiguous())
    assert alone["loss"].shape == alone["accept"].shape == both["loss"].shape == lead
    assert both["d_logits"].shape == z.shape


@pytest.mark.parametrize("dtype,out_dtype,D", [(torch.float32, None, 512), (torch.float32, None, 516),
                                               (torch.float32, None, 2560), (torch.bfloat16, None, 1032),
                                               (torch.bfloat16, torch.float32, 2561), (torch.float16, None, 4096)], ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided"])
def test_embed_grad_of_no_positions(dtype, out_dtype, D, layout):
    """Zeroes the table's gradient, rows of every width; adds nothing to one that is given."""
    V, pad = 300, {"packed": 0, "strided": 8}[layout]
    w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(0, V, D))
    d_out = torch.empty(0, D, dtype=dtype, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    buf = torch.full((V, D + pad), 7.0, dtype=out_dtype or dtype, device="cuda")
    ds.embed_grad(d_out, ids, V, w, out=buf[:, :D], accumulate=True)
    assert (buf == 7).all()
    ds.embed_grad(d_out, ids, V, w, out=buf[:, :D])
    assert (buf[:, :D] == 0).all() and (buf[:, D:] == 7).all()
    assert w.status() == 0


# ----------------------------------------------------------------- teachers without a number

TERMS = [dict(), dict(kl=0.0, tv=1.0), dict(kl=0.0, tv=0.5, ce=0.5), dict(kl=0.3, tv=0.3, ce=0.4)]


@pytest.mark.parametrize("terms", TERMS, ids=["kl", "tv", "tv+ce", "all"])
@pytest.mark.parametrize("V", [1000, 20008])           # a CTA a row; rows cut over a cluster
@pytest.mark.parametrize("K", [1, 8, 40])
@pytest.mark.parametrize("labelled", [False, True])
def test_distill_shows_a_teacher_without_a_number(K, V, terms, labelled, ws):
    """A NaN or +inf among the logits of a row's entries reaches its loss, acceptance and whole
    gradient, whatever the other entries are; absent entries and rows of weight 0 are not read,
    and other rows are untouched."""
    n = 7
    z = logits(n, V, torch.float32, 100)
    ids, t = teacher(n, V, K, 101)
    ids = torch.where(ids < 0, V - 1, ids)
    if K > 1:
        ids[4, 1] = -1
    labels = torch.full((n,), 5 if labelled else -1, dtype=torch.int32, device="cuda")
    w = ones(n)
    w[5] = 0
    clean = ds.distill_loss_grad(z, ids, t, ws, labels, w, **terms)
    bad = t.clone()
    bad[1] = math.nan                                  # every entry
    bad[2] = -math.inf
    bad[2, K - 1] = math.nan                           # beside entries of probability 0
    bad[3, 0] = math.inf
    if K > 1:
        bad[4, 1] = math.nan                           # an absent entry
    bad[5] = math.nan                                  # a row of weight 0
    bad[6, K // 2] = math.nan                          # beside ordinary entries
    got = ds.distill_loss_grad(z, ids, bad, ws, labels, w, **terms)
    alone = ds.distill_loss(z, ids, bad, ws, labels, w, **terms)
    for key in got:
        for row in (0, 4, 5):
            assert torch.equal(got[key][row], clean[key][row]), (key, row)
        for row in (1, 2, 3, 6):
            assert got[key][row].isnan().all(), (key, row)
    for key in alone:
        assert torch.equal(alone[key].isnan(), got[key].isnan())


@pytest.mark.parametrize("V", [1000, 20008])
def test_distill_of_labels_alone_beside_a_teacher_without_a_number(V, ws):
    """With the label's term alone the teacher enters the acceptance only."""
    z = logits(2, V, torch.float32, 102)
    ids, t = teacher(2, V, 8, 103)
    labels = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    clean = ds.distill_loss_grad(z, ids, t, ws, labels, kl=0.0, ce=1.0)
    t[1] = math.nan
    got = ds.distill_loss_grad(z, ids, t, ws, labels, kl=0.0, ce=1.0)
    assert torch.equal(got["loss"], clean["loss"]) and torch.equal(got["d_logits"], clean["d_logits"])
    assert got["accept"][0] == clean["accept"][0] and got["accept"][1].isnan()


# ---------------------------------------------------------------------- small temperatures

@pytest.mark.parametrize("V", [1000, 20008])
@pytest.mark.parametrize("shift", [-5.0, 0.0, 5.0])
def test_distill_at_a_temperature_near_zero(shift, V, ws):
    """Only differences of the teacher's logits count: at 1e-38 both distributions are their
    largest logit, whatever the logits' sign, although a logit over the temperature is
    beyond fp32."""
    n, K = 4, 8
    z = logits(n, V, torch.float32, 104)
    ids = z.topk(K, 1).indices.to(torch.int32)
    t = -0.5 * torch.arange(K, device="cuda").repeat(n, 1) + shift
    got = ds.distill_loss_grad(z, ids, t, ws, temperature=1e-38, kl=1.0, tv=1.0)
    assert (got["accept"] == 1).all() and (got["loss"] == 0).all() and (got["d_logits"] == 0).all()


@pytest.mark.parametrize("V", [1000, 20008])
def test_distill_takes_logits_far_from_zero(V, ws):
    """t / temperature rounded before the maximum is subtracted would be off by |t / temperature|
    2^-24 = 2.6e-4 here, ten times the tolerance."""
    n, K = 5, 33
    z = logits(n, V, torch.float32, 105)
    ids, t = teacher(n, V, K, 106)
    t += 3000.0
    labels = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    kw = dict(temperature=0.7, kl=0.5, tv=0.3, ce=0.2)
    got = ds.distill_loss_grad(z, ids, t, ws, labels, ones(n), **kw)
    ref = ref_distill(z, ids, t, labels, ones(n), ones(n), 0.7, 0.5, 0.3, 0.2)
    close(got["loss"], ref["loss"], rtol=2 * SUM, atol=6 * SUM)
    close(got["accept"], ref["accept"], rtol=2 * SUM, atol=2 * SUM)
    close(got["d_logits"], ref["d_logits"], rtol=2 * SUM, atol=2 * SUM / 0.7)


# -------------------------------------------------------------------- partly given outputs

def test_distill_makes_the_outputs_that_are_not_given(ws):
    n, V, K = 3, 1000, 8
    z = logits(n, V, torch.float32, 107)
    ids, t = teacher(n, V, K, 108)
    want = ds.distill_loss_grad(z, ids, t, ws)
    got = ds.distill_loss_grad(z, ids, t, ws, out={"d_logits": z})
    assert got["d_logits"] is z and set(got) == {"loss", "accept", "d_logits"}
    assert all(torch.equal(got[k], want[k]) for k in want)
    loss = torch.empty(n, device="cuda")
    z = logits(n, V, torch.float32, 107)
    got = ds.distill_loss(z, ids, t, ws, out={"loss": loss})
    assert got["loss"] is loss and torch.equal(loss, want["loss"]) and torch.equal(got["accept"], want["accept"])


# --------------------------------------------------------------------- what accept stands for

@pytest.mark.parametrize("K", [4, 32, 128])
@pytest.mark.parametrize("V,spread", [(1000, 3.0), (20008, 1.0)])
def test_accept_is_off_by_no_more_than_the_mass_left_out(K, V, spread, ws):
    """With a teacher's top log probabilities: accept against sum min(p, q) over the vocabulary."""
    n = 16
    T = logits(n, V, torch.float32, 109) * spread / 3
    z = logits(n, V, torch.float32, 110) * spread / 3 + T
    top = ds.token_logprobs(T, None, K, ws)
    got = ds.distill_loss(z, top["top_ids"], top["top_logprobs"], ws)["accept"].double()
    p, q = torch.softmax(T.double(), 1), torch.softmax(z.double(), 1)
    left = 1 - top["top_logprobs"].double().exp().sum(1)
    off = (got - torch.minimum(p, q).sum(1)).abs()
    assert (off <= left + 4 * SUM).all() and (left > 0).any()
