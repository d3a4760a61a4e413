"""The operators that train the draft head and report on its tokens: cases and plain forms.

  logprobs       log probabilities of given tokens, entropy, rank and top alternatives of rows
                 of logits (``token_logprobs``), and the gradient of the first two
                 (``token_logprobs_grad``)
  distill        distillation of the student's logits from a teacher's top logits: loss and
                 expected acceptance (``distill_loss``), or both with the gradient
                 (``distill_loss_grad``)
  embed          embedding lookup with scaling (``embed``) and its gradient, summed over the
                 occurrences of every token (``embed_grad``)

A case names its operator in "op" and its direction in "form".  ``run`` makes one pass: the
plain form in torch (``own`` false), or the framework's calls (``own`` true).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
#: The most that a pass over logits moves: the largest listed case's bytes.
MOST_BYTES = 1.30e9


# ------------------------------------------------------------------------------- cases

def _logprobs(name, rows, kept, V, top, dtype, form="forward"):
    return dict(name=name, op="logprobs", form=form, rows=rows, kept=kept, V=V, top=top, dtype=dtype)


def _distill(name, rows, kept, V, top, dtype, form="gradient", temperature=1.0, kl=1.0, tv=0.0, ce=0.0):
    return dict(name=name, op="distill", form=form, rows=rows, kept=kept, V=V, top=top, dtype=dtype,
                temperature=temperature, kl=kl, tv=tv, ce=ce)


def _embed(name, n, V, D, dtype, form="forward", zipf=1.0, scale=1.0):
    return dict(name=name, op="embed", form=form, n=n, V=V, D=D, dtype=dtype, zipf=zipf, scale=scale)


def listed():
    return [
        # one answered token of one request, with the 20 alternatives a client may ask for
        _logprobs("logprobs_one_row", 1, 1, 151936, 20, "bf16"),
        # a verified step of 32 requests, 8 target rows each, half of them answered with a token
        _logprobs("logprobs_step", 256, 128, 151936, 20, "f32"),
        # the teacher's side of training: every target row of 256 requests, top 64 logits kept
        _logprobs("logprobs_teacher", 1536, 1536, 129280, 64, "f32"),
        # gradient of log probability and entropy for the drafted tokens of 256 requests
        _logprobs("logprobs_grad", 1280, 1152, 129280, 0, "bf16", form="gradient"),
        # the smallest training call: 4 requests of 4 positions; total variation and labels
        _distill("distill_tiny", 16, 14, 1000, 8, "f32", kl=0.0, tv=0.9, ce=0.1),
        # 256 requests of 5 positions in 32 bits
        _distill("distill_block", 1280, 1216, 129280, 64, "f32", kl=0.9, ce=0.1),
        # 128 requests of 15 positions in 16 bits, softened by a temperature
        _distill("distill_long_block", 1920, 1824, 151936, 32, "bf16", temperature=2.0),
        # evaluation (the loss alone) on an odd vocabulary: rows start off 16-byte borders
        _distill("distill_eval", 224, 200, 99991, 20, "bf16", form="forward", kl=0.9, ce=0.1),
        # the predecessors of one drafted position of 32 requests
        _embed("embed_step", 32, 151936, 256, "bf16", scale=16.0),
        # the tokens of a prompt batch, rows of the hidden size
        _embed("embed_prompt", 16384, 151936, 2560, "bf16", scale=0.5),
        # the draft head's table: 256 requests of 5 positions
        _embed("embed_grad_head", 1280, 129280, 256, "f32", form="gradient", scale=16.0),
        # a training batch of the hidden size, tokens as uneven as text
        _embed("embed_grad_batch", 32768, 151936, 2560, "bf16", form="gradient"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.randrange(6)
    dtype = rng.choice(("f32", "bf16", "f16"))
    if kind < 4:
        V = _log_uniform(rng, 1000, 152000)
        # widths as vocabularies have them, mostly multiples of 8, and odd ones
        V = V // 8 * 8 if rng.random() < 0.6 else V | 1
        passes = 2 if kind in (1, 3) else 1
        most = int(MOST_BYTES / (passes * V * SIZES[dtype]))
        rows = _log_uniform(rng, 1, min(2048, most))
        kept = rows - int(rows * rng.choice((0.0, 0.1, 0.5)))
        if kind == 0:
            return {k: v for k, v in _logprobs("", rows, kept, V, rng.choice((0, 1, 5, 20, 33, 64, 128)), dtype).items() if k != "name"}
        if kind == 1:
            return {k: v for k, v in _logprobs("", rows, kept, V, 0, dtype, "gradient").items() if k != "name"}
        top = rng.choice((1, 8, 20, 32, 64, 100, 128))
        # the total variation's gradient jumps where p = q: few entries are near that border
        tv = 0.9 if rows * top <= 1000 and rng.random() < 0.5 else 0.0
        case = _distill("", rows, kept, V, top, dtype, "gradient" if kind == 3 else "forward",
                        rng.choice((1.0, 1.0, 0.7, 2.0)), rng.choice((0.9, 1.0)) - tv, tv, rng.choice((0.0, 0.1)))
    else:
        V = _log_uniform(rng, 1000, 152000)
        D = _log_uniform(rng, 16, 4096)
        D = D // 16 * 16 if rng.random() < 0.7 else D | 1
        V = min(V, int(4e8 / D))
        n = _log_uniform(rng, 1, min(65536, int(1e8 / D)))
        case = _embed("", n, V, D, dtype, "gradient" if kind == 5 else "forward", rng.choice((0.0, 1.0, 1.3)),
                      rng.choice((1.0, 0.5, 16.0)))
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------------------ inputs

def _chosen(rows, kept, g):
    """A mask of ``rows`` entries, ``kept`` of them true."""
    return torch.rand(rows, generator=g, device="cuda").argsort().argsort() < kept


def _logits(rows, V, g):
    """Logits as the synthetic workloads have them: N(0, 3^2), one in a hundred raised by 8."""
    z = torch.randn(rows, V, generator=g, device="cuda").mul_(3.0)
    return z.add_(torch.rand(rows, V, generator=g, device="cuda").lt_(0.01), alpha=8.0)


def _sampled(z, g):
    """One token of each row, drawn from softmax(z)."""
    u = torch.rand(z.shape, generator=g, device="cuda").clamp_(min=1e-12)
    return u.log_().neg_().log_().neg_().add_(z).argmax(1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "embed":
        n, V, D, dtype = case["n"], case["V"], case["D"], TYPES[case["dtype"]]
        # token frequencies by rank: 1 / rank^zipf, the ranks dealt over the table at random
        p = (1.0 + torch.arange(V, device="cuda", dtype=torch.float64)).pow_(-case["zipf"])
        p = p[torch.rand(V, generator=g, device="cuda").argsort()].cumsum_(0)
        u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64).mul_(p[-1])
        ids = torch.searchsorted(p, u).clamp_(max=V - 1).to(torch.int32)
        s["ids"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, -1, ids).contiguous()  # padding
        if case["form"] == "forward":
            s["W"] = torch.randn(V, D, generator=g, device="cuda").mul_(0.02).to(dtype)
        else:
            s["d_out"] = torch.randn(n, D, generator=g, device="cuda").mul_(1e-2).to(dtype)
        return s
    rows, V, top, dtype = case["rows"], case["V"], case["top"], TYPES[case["dtype"]]
    kept = _chosen(rows, case["kept"], g)
    z = _logits(rows, V, g)
    tokens = _sampled(z, g)
    if case["op"] == "logprobs":
        s["logits"] = z.to(dtype)
        s["tokens"] = torch.where(kept, tokens, -1)
        if case["form"] == "gradient":
            zd = s["logits"].double()
            s["row_max"] = zd.amax(1)
            e = (zd - s["row_max"][:, None]).exp_()
            total = e.sum(1)
            s["entropy"] = (total.log() - e.mul_(zd.sub_(s["row_max"][:, None])).sum(1) / total).float()
            s["row_max"], s["row_sumexp"] = s["row_max"].float(), total.float()
            s["d_logprob"] = torch.randn(rows, generator=g, device="cuda")
            s["d_entropy"] = torch.randn(rows, generator=g, device="cuda").mul_(0.01)
        return s
    t = z + torch.randn(rows, V, generator=g, device="cuda")  # the teacher's own logits
    t, ids = torch.log_softmax(t, 1).topk(min(top, V), 1)
    s["teacher_logits"] = t.contiguous()
    s["teacher_ids"] = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < 0.01, -1, ids).to(torch.int32)
    s["labels"] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.05, -1, tokens).to(torch.int32)
    # weights that fall over the positions of a block, 0 where a position is padding
    s["weights"] = torch.exp(-(torch.arange(rows, device="cuda") % 5) / 4.0) * kept
    s["logits"] = z.to(dtype)
    return s


# ------------------------------------------------------------------------- plain forms

def _plain_logprobs(s):
    c = s["case"]
    z, tokens = s["logits"].float(), s["tokens"].long()
    on = tokens >= 0
    m = z.amax(1)
    d = z - m[:, None]
    e = d.exp()
    total = e.sum(1)
    log_total = total.log()
    zt = z.gather(1, tokens.clamp(min=0)[:, None])
    at = torch.arange(c["V"], device=z.device)
    before = (z > zt) | ((z == zt) & (at < tokens[:, None]))
    out = {
        "logprob": torch.where(on, zt[:, 0] - m - log_total, 0.0),
        "entropy": torch.where(on, log_total - (e * d).sum(1) / total, 0.0),
        "rank": torch.where(on, before.sum(1) + 1, 0).to(torch.int32),
        "row_max": torch.where(on, m, -math.inf),
        "row_sumexp": torch.where(on, total, 0.0),
    }
    if c["top"]:
        # one whole number for each value and place: the larger value first, then the lower place
        bits = z.view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) + (c["V"] - 1 - at)
        ids = c["V"] - 1 - (key.topk(c["top"], 1).values & 0xFFFFFFFF)
        out["top_ids"] = torch.where(on[:, None], ids, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(on[:, None], z.gather(1, ids) - m[:, None] - log_total[:, None], -math.inf)
    return out


def _plain_logprobs_grad(s):
    z, tokens = s["logits"].float(), s["tokens"].long()
    on = (tokens >= 0)[:, None]
    log_p = z - s["row_max"][:, None] - s["row_sumexp"].log()[:, None]
    p = log_p.exp()
    d = -p * (s["d_logprob"][:, None] + s["d_entropy"][:, None] * (log_p + s["entropy"][:, None]))
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], s["d_logprob"][:, None])
    return {"d_logits": torch.where(on, d, 0.0).to(s["logits"].dtype)}


def _plain_distill(s):
    c = s["case"]
    tau = c["temperature"]
    z = s["logits"].float() / tau
    z = z - z.amax(1, keepdim=True)
    log_q = z - z.exp().sum(1, keepdim=True).log()
    ids, on = s["teacher_ids"].long().clamp(min=0), s["teacher_ids"] >= 0
    t = torch.where(on, s["teacher_logits"] / tau, -math.inf)
    t = t - t.amax(1, keepdim=True)
    log_p = t - t.exp().sum(1, keepdim=True).log()
    p, log_qk = log_p.exp(), log_q.gather(1, ids)
    q = log_qk.exp()
    kl = torch.where(on, p * (log_p - log_qk), 0.0).sum(1)
    tv = torch.where(on, (p - q).clamp(min=0.0), 0.0).sum(1)
    labels = s["labels"].long()
    named = labels >= 0
    ce = torch.where(named, -log_q.gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    w = s["weights"]
    out = {"loss": w * (c["kl"] * kl + c["tv"] * tv + c["ce"] * ce),
           "accept": torch.where(w != 0, torch.where(on, torch.minimum(p, q), 0.0).sum(1), 0.0)}
    if c["form"] == "gradient":
        short = on & (q < p)
        back = c["kl"] * p * on + c["tv"] * q * short
        name = c["ce"] * named
        d = log_q.exp() * (back.sum(1) + name)[:, None]
        d.scatter_add_(1, ids, -back)
        d.scatter_add_(1, labels.clamp(min=0)[:, None], -name[:, None])
        out["d_logits"] = (d * (w / tau)[:, None]).to(s["logits"].dtype)
    return out


def _plain_embed(s):
    on, ids = (s["ids"] >= 0)[:, None], s["ids"].long().clamp(min=0)
    return {"out": torch.where(on, s["W"][ids].float() * s["case"]["scale"], 0.0).to(s["W"].dtype)}


def _plain_embed_grad(s):
    c = s["case"]
    ids = torch.where(s["ids"] >= 0, s["ids"], c["V"]).long()
    d = torch.zeros(c["V"] + 1, c["D"], device=ids.device)
    d.index_add_(0, ids, s["d_out"].float())
    return {"d_W": (d[:c["V"]] * c["scale"]).to(s["d_out"].dtype)}


# ------------------------------------------------------------------------ one pass

def _own(s):
    import speculative_decoding_03_gb300 as ds
    c = s["case"]
    out, ws = s.get("out"), s.get("ws")
    if ws is None:  # a program keeps its workspace from call to call
        nbytes = ds.embed_grad_workspace_bytes(c["n"], c["V"], c["D"]) if (c["op"], c["form"]) == ("embed", "gradient") else 256
        ws = s["ws"] = ds.Workspace.of_bytes(nbytes)
    if c["op"] == "logprobs" and c["form"] == "forward":
        out = ds.token_logprobs(s["logits"], s["tokens"], c["top"], ws, out)
    elif c["op"] == "logprobs":
        out = ds.token_logprobs_grad(s["logits"], s["tokens"], s["row_max"], s["row_sumexp"], s["entropy"],
                                     s["d_logprob"], s["d_entropy"], ws, out)
    elif c["op"] == "distill":
        call = ds.distill_loss_grad if c["form"] == "gradient" else ds.distill_loss
        out = call(s["logits"], s["teacher_ids"], s["teacher_logits"], ws, s["labels"], s["weights"],
                   temperature=c["temperature"], kl=c["kl"], tv=c["tv"], ce=c["ce"], out=out)
    elif c["form"] == "forward":
        out = ds.embed(s["W"], s["ids"], ws, c["scale"], out)
    else:
        out = ds.embed_grad(s["d_out"], s["ids"], c["V"], ws, c["scale"], out)
    s["out"] = out  # and its output buffers
    if c["op"] == "embed":
        return {"out": out} if c["form"] == "forward" else {"d_W": out}
    return {"d_logits": out} if (c["op"], c["form"]) == ("logprobs", "gradient") else out


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "logprobs":
        return _plain_logprobs(state) if c["form"] == "forward" else _plain_logprobs_grad(state)
    if c["op"] == "distill":
        return _plain_distill(state)
    return _plain_embed(state) if c["form"] == "forward" else _plain_embed_grad(state)


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"] == "embed":
        n, V, D = case["n"], case["V"], case["D"]
        if case["form"] == "forward":
            return {"bytes": 4 * n + 2 * n * D * e, "flops": n * D}
        return {"bytes": 4 * n + (n + V) * D * e, "flops": n * D + V * D}
    rows, kept, V, top = case["rows"], case["kept"], case["V"], case["top"]
    if case["op"] == "logprobs":
        if case["form"] == "forward":
            # a row without a token is not read
            return {"bytes": kept * V * e + rows * (24 + 8 * top), "flops": 6 * kept * V}
        return {"bytes": (kept + rows) * V * e + 24 * rows, "flops": 6 * kept * V}
    small = rows * (16 + 8 * top)
    if case["form"] == "forward":
        return {"bytes": kept * V * e + small, "flops": 4 * kept * V}
    return {"bytes": (kept + rows) * V * e + small, "flops": 7 * kept * V}


# -------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """What ``run`` returns, from the definitions, in 64 bits and unrounded."""
    s = prepare(case, seed)
    if case["op"] == "embed":
        keep = s["ids"] >= 0
        if case["form"] == "forward":
            out = torch.zeros(case["n"], case["D"], dtype=torch.float64, device="cuda")
            out[keep] = case["scale"] * s["W"][s["ids"][keep].long()].double()
            return {"out": out}
        out = torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
        out.index_put_((s["ids"][keep].long(),), case["scale"] * s["d_out"][keep].double(), accumulate=True)
        return {"d_W": out}
    x = s["logits"].double()
    if case["op"] == "logprobs":
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        y = s["tokens"][at].long()
        logp = torch.log_softmax(x[at], 1)
        p = logp.exp()
        lpy = torch.gather(logp, 1, y[:, None])[:, 0]
        if case["form"] == "gradient":
            gl, gh = s["d_logprob"][at].double(), s["d_entropy"][at].double()
            H = -(p * logp).sum(1)
            d = torch.zeros_like(x)
            part = -gl[:, None] * p - gh[:, None] * p * (logp + H[:, None])
            part[torch.arange(len(at), device="cuda"), y] += gl
            d[at] = part
            return {"d_logits": d}
        new = lambda v, fill: torch.full((case["rows"],) + v.shape[1:], fill, dtype=v.dtype, device="cuda").index_copy_(0, at, v)  # noqa: E731
        top = x[at].amax(1)
        out = {"logprob": new(lpy, 0.0), "entropy": new(-(p * logp).sum(1), 0.0), "rank": None,
               "row_max": new(top, -math.inf), "row_sumexp": new((x[at] - top[:, None]).exp().sum(1), 0.0)}
        if case["top"]:
            out["top_ids"] = None
            out["top_logprobs"] = new(logp.topk(case["top"], 1).values, -math.inf)
        return out
    tau = case["temperature"]
    logq = torch.log_softmax(x / tau, 1)
    hole = s["teacher_ids"] < 0
    at = s["teacher_ids"].long().masked_fill(hole, 0)
    t = (s["teacher_logits"].double() / tau).masked_fill(hole, -math.inf)
    p = torch.softmax(t, 1)
    lq = logq.gather(1, at)
    q = lq.exp().masked_fill(hole, 0.0)
    kl = (torch.special.xlogy(p, p) - p * lq).sum(1)
    y = s["labels"].long()
    given = (y >= 0).double()
    ce = -logq.gather(1, y.clamp(min=0)[:, None])[:, 0] * given
    w = s["weights"].double()
    out = {"loss": w * (case["kl"] * kl + case["tv"] * torch.relu(p - q).sum(1) + case["ce"] * ce),
           "accept": torch.minimum(p, q).sum(1) * (w != 0)}
    if case["form"] == "gradient":
        # d/dz of -sum_k a_k log q_k is (sum a) q - a, with a = kl p + tv q [q < p] and the label
        a = case["kl"] * p + case["tv"] * q * (q < p)
        target = torch.zeros_like(x).scatter_add_(1, at, a).scatter_add_(1, y.clamp(min=0)[:, None], (case["ce"] * given)[:, None])
        out["d_logits"] = (logq.exp() * target.sum(1, keepdim=True) - target) * (w / tau)[:, None]
    return out
