"""The operators of the target's side of a step: cases and plain forms.

  append   keys and values of the drafted tokens into a paged cache, with queries and keys
           normalised for each head and rotated by their position on the way (``cache_append``)
  attend   attention of the drafted tokens, a tree or a chain, over the cache
           (``tree_attention``)
  verify   verification of a tree or a chain of drafted tokens against the target's
           probabilities from given random numbers (``tree_verify``)
  keep     the accepted tokens' keys and values moved together in every layer's cache
           (``cache_keep``)

A case names its operator in "op".  Rows of tokens are packed ([rows, ...] with the requests'
starts) or padded ([B, N, ...] with the requests' counts).  ``run`` makes one pass: the plain
form in torch (``own`` false), or the framework's calls (``own`` true).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
#: The most that a pass moves: the largest listed case's bytes.
MOST_BYTES = 1.08e9


# ------------------------------------------------------------------------------- cases

def _append(name, B, N, low, high, Hq, Hkv, D, page, dtype, rotated=128, interleaved=False, norm=False,
            tree=False, packed=False):
    return dict(name=name, op="append", B=B, N=N, low=low, high=high, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype,
                rotated=rotated, interleaved=interleaved, norm=norm, tree=tree, packed=packed)


def _attend(name, B, N, low, high, Hq, Hkv, D, page, dtype, tree=False, packed=False):
    return dict(name=name, op="attend", B=B, N=N, low=low, high=high, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype,
                tree=tree, packed=packed)


def _verify(name, B, N, V, dtype, points=False, tree=False, packed=False):
    return dict(name=name, op="verify", B=B, N=N, V=V, dtype=dtype, points=points, tree=tree, packed=packed)


def _keep(name, B, N, low, high, layers, Hkv, D, page, dtype):
    return dict(name=name, op="keep", B=B, N=N, low=low, high=high, layers=layers, Hkv=Hkv, D=D, page=page, dtype=dtype)


def listed():
    return [
        # one token of one request: what a step costs at least
        _append("append_token", 1, 1, 1000, 1000, 32, 8, 128, 16, "bf16"),
        # trees of up to 16 tokens of 32 requests, queries and keys normalised
        _append("append_trees", 32, 16, 100, 2000, 32, 8, 128, 16, "bf16", norm=True, tree=True, packed=True),
        # four prompts of unequal length, half of each head rotated, neighbours in pairs
        _append("append_prompts", 4, 6001, 0, 500, 28, 4, 128, 64, "f16", rotated=64, interleaved=True, packed=True),
        # one token of one request over a short context
        _attend("attend_token", 1, 1, 1000, 1000, 32, 8, 128, 16, "bf16"),
        # trees of up to 16 tokens of 32 requests
        _attend("attend_trees", 32, 16, 3500, 4500, 32, 8, 128, 16, "bf16", tree=True, packed=True),
        # two requests with long documents, chains of 8
        _attend("attend_long", 2, 8, 130001, 131000, 32, 8, 128, 64, "bf16"),
        # scheduled chains of a large batch: small heads, odd and very unequal lengths
        _attend("attend_chains", 128, 8, 1, 2999, 16, 2, 64, 32, "f16", packed=True),
        # a block of 7 drafted tokens of one request
        _verify("verify_one", 1, 8, 151936, "f32"),
        # blocks of 5 of 256 requests
        _verify("verify_chains", 256, 6, 129280, "f32"),
        # trees of the draft's most probable tokens
        _verify("verify_trees", 64, 16, 151936, "bf16", points=True, tree=True, packed=True),
        # one request, 36 layers
        _keep("keep_one", 1, 16, 1000, 1000, 36, 8, 128, 16, "bf16"),
        # 32 requests
        _keep("keep_batch", 32, 32, 200, 480, 16, 8, 128, 16, "bf16"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(("append", "attend", "attend", "verify", "keep"))
    dtype = rng.choice(("bf16", "f16"))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    tree = rng.random() < 0.5
    packed = rng.random() < 0.5
    if kind == "append":
        D = rng.choice((64, 96, 128, 256))
        B = _log_uniform(rng, 1, 128)
        Hq = Hkv * rng.choice((1, 2, 3, 4, 7, 8))
        most = int(2.0e8 / (B * (Hq + 2 * Hkv) * D * 4))
        N = _log_uniform(rng, 1, max(1, min(64 if tree else 6001, most)))
        case = _append("", B, N, rng.choice((0, 1, 50)), rng.choice((51, 900, 4001)), Hq, Hkv, D, page, dtype,
                       rng.choice((0, 32, 64, D)), rng.random() < 0.4, rng.random() < 0.5, tree, packed)
    elif kind == "attend":
        D = rng.choice((64, 128))
        B = _log_uniform(rng, 1, 128)
        N = rng.choice((1, 2, 4, 6, 8, 11, 16, 17, 32, 64))
        Hq = Hkv * rng.choice((1, 2, 4, 7, 8))
        most = min(MOST_BYTES / 2 / (B * Hkv * D * 4), 50 * MOST_BYTES / (4 * B * N * Hq * D))
        high = _log_uniform(rng, 16, max(17, min(131000, int(most))))
        case = _attend("", B, N, int(high * rng.choice((0.0, 0.3, 0.9))), high, Hq, Hkv, D, page, dtype, tree, packed)
    elif kind == "verify":
        dtype = rng.choice(("f32", "bf16", "f16"))
        V = _log_uniform(rng, 1000, 152000)
        V = V // 8 * 8 if rng.random() < 0.6 else V | 1
        N = rng.choice((1, 2, 6, 8, 16, 17, 32))
        B = _log_uniform(rng, 1, max(1, min(256, int(8e8 / (N * V * SIZES[dtype])))))
        case = _verify("", B, N, V, dtype, rng.random() < 0.5, tree, packed)
    else:
        layers = rng.choice((1, 16, 36))
        D = rng.choice((64, 128))
        B = _log_uniform(rng, 1, max(1, min(128, int(1.0e9 / (layers * 700 * Hkv * D * 4)))))
        case = _keep("", B, rng.choice((2, 8, 16, 33, 64)), rng.choice((0, 100)), rng.choice((101, 480)), layers, Hkv, D, page, dtype)
    return {k: v for k, v in case.items() if k != "name"}


def _spread(low, high, n):
    """n whole numbers from low to high, evenly."""
    return [low + (high - low) * i // max(1, n - 1) if n > 1 else high for i in range(n)]


def _counts(case):
    """How many tokens the requests have; every seed deals them over the requests in another order."""
    return _spread(1, case["N"], case["B"])


# ------------------------------------------------------------------------------ inputs

def _dealt(values, g):
    order = torch.rand(len(values), generator=g, device="cuda").argsort()
    return torch.tensor(values, dtype=torch.int32, device="cuda")[order].contiguous()


def _parents(rows, local, tree, g):
    """Each token's parent by its place in the request, -1 for the first; None for a chain."""
    if not tree:
        return None
    u = torch.rand(rows, generator=g, device="cuda")
    # the nearer the likelier: trees as deep as drafted ones are
    return torch.where(local > 0, (local * u.sqrt()).long().clamp(max=63), -1).to(torch.int32).minimum(local - 1).contiguous()


def _layout(case, g):
    """Counts, and where the rows are: of each row its request (B: of none) and place."""
    B, N = case["B"], case["N"]
    counts = _dealt(_counts(case), g)
    s = {"case": case, "counts": counts, "starts": None}
    if case.get("packed"):
        ends = counts.cumsum(0)
        rows = (sum(_counts(case)) + 7) // 8 * 8  # a batch padded to a multiple of 8 rows
        at = torch.arange(rows, device="cuda")
        s["request"] = torch.searchsorted(ends, at, right=True)
        s["starts"] = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
        s["local"] = (at - s["starts"].long()[s["request"]]).to(torch.int32)
        s["live"] = s["request"] < B
    else:
        rows = B * N
        s["request"] = torch.arange(rows, device="cuda") // N
        s["local"] = (torch.arange(rows, device="cuda") % N).to(torch.int32)
        s["live"] = s["local"] < counts[s["request"]]
    s["rows"] = rows
    return s


def _cache(case, g, layers=0, room=0):
    """Keys and values of one layer (or of several) and the requests' pages, dealt at random; the
    pages hold what earlier requests left."""
    B, page, dtype = case["B"], case["page"], TYPES[case["dtype"]]
    each = -(-(case["high"] + room) // page)
    P = B * each + 3
    shape = ((layers,) if layers else ()) + (P, page, case["Hkv"], case["D"])
    make = lambda: torch.randn(shape, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    pages = torch.rand(P, generator=g, device="cuda").argsort()[:B * each].to(torch.int32).view(B, each).contiguous()
    return make(), make(), pages, _dealt(_spread(case["low"], case["high"], B), g)


def _prepare_verify(case, s, g):
    rows, V, dtype = s["rows"], case["V"], TYPES[case["dtype"]]
    # the draft's logits and the target's, as near as a good draft's are
    z = torch.randn(rows, V, generator=g, device="cuda").mul_(3.0)
    z.add_(torch.rand(rows, V, generator=g, device="cuda").lt_(0.01), alpha=8.0)
    parents = s["parents"] if s["parents"] is not None else s["local"] - 1
    first = torch.arange(rows, device="cuda") - s["local"]
    up = (first + parents).clamp(min=0)  # the parent's row
    if case["points"]:
        # a child is its parent's most probable token that no earlier child is
        place = torch.zeros(rows, dtype=torch.long, device="cuda")
        for back in range(1, case["N"]):
            same = torch.zeros(rows, dtype=torch.bool, device="cuda")
            same[back:] = (first[back:] == first[:-back]) & (parents[back:] == parents[:-back])
            place += same
        tokens = z.topk(case["N"], 1).indices[up, place]
    else:
        # children are drawn from the draft's probabilities
        tokens = torch.empty(rows, dtype=torch.long, device="cuda")
        s["q"] = torch.softmax(z, 1)
        for a in range(0, rows, 256):
            u = torch.rand(s["q"][a:a + 256].shape, generator=g, device="cuda").clamp_(min=1e-12)
            tokens[a:a + 256] = u.log_().neg_().log_().neg_().add_(z[up[a:a + 256]]).argmax(1)
        s["q"] = s["q"].to(dtype)
    s["tokens"] = tokens.to(torch.int32)
    z.add_(torch.randn(rows, V, generator=g, device="cuda"), alpha=0.6)
    s["p"] = torch.softmax(z, 1).to(dtype)
    s["uniforms"] = torch.rand(rows, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    if case["op"] == "keep":
        B, N = case["B"], case["N"]
        s = {"case": case}
        s["k"], s["v"], s["pages"], s["lengths"] = _cache(case, g, case["layers"], N)
        s["accept_len"] = _dealt(_accepted(case), g)
        # a path's nodes rise
        order = torch.rand(B, N - 1, generator=g, device="cuda").argsort(1) + 1
        keep = torch.arange(N - 1, device="cuda") < s["accept_len"][:, None]
        path = torch.where(keep, order, N).sort(1).values
        s["path"] = torch.cat([torch.where(keep, path, -1), torch.full((B, 1), -1, device="cuda")], 1).to(torch.int32).contiguous()
        return s
    s = _layout(case, g)
    s["parents"] = _parents(s["rows"], s["local"], case["tree"], g)
    if case["op"] == "verify":
        _prepare_verify(case, s, g)
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    s["k_cache"], s["v_cache"], s["pages"], s["lengths"] = _cache(case, g, 0, case["N"])
    lead = (s["rows"],) if case["packed"] else (case["B"], case["N"])
    if case["op"] == "attend":
        s["q"] = torch.randn(lead + (Hq, D), generator=g, device="cuda").mul_(1.5).to(dtype)
        s["out"] = torch.zeros(lead + (Hq, D), dtype=dtype, device="cuda")
        return s
    # one projection's output holds queries, keys and values side by side
    qkv = torch.randn(lead + (Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
    s["q"], s["k"], s["v"] = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
    s["q_out"] = torch.zeros(lead + (Hq, D), dtype=dtype, device="cuda")
    R = case["rotated"]
    s["inv_freq"] = (1e6 ** -(torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))).float() if R else None
    if case["norm"]:
        s["q_weight"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["k_weight"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    return s


def _accepted(case):
    return [i * 5 % (min(case["N"], 8)) for i in range(1, case["B"] + 1)]


# ------------------------------------------------------------------------- plain forms

def _depths(s):
    """Each row's distance from its request's first token."""
    if s["parents"] is None:
        return s["local"].long()
    first = torch.arange(s["rows"], device="cuda") - s["local"]
    up, depth = s["parents"].long(), torch.zeros(s["rows"], dtype=torch.long, device="cuda")
    for _ in range(s["case"]["N"] - 1):
        on = up >= 0
        depth += on
        up = torch.where(on, s["parents"].long()[(first + up).clamp(min=0)], -1)
    return depth


def _plain_append(s):
    c = s["case"]
    live = s["live"]
    request = s["request"][live]
    slot = s["lengths"].long()[request] + s["local"].long()[live]
    position = s["lengths"].long()[request] + _depths(s)[live]

    def turned(x, weight):
        x = x.reshape((s["rows"],) + x.shape[-2:])[live].float()
        if c["norm"]:
            x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight
        R = c["rotated"]
        if R:
            angle = position.double()[:, None] * s["inv_freq"].double()
            cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
            a, b = (x[..., 0:R:2], x[..., 1:R:2]) if c["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
            turn = (a * cos - b * sin, b * cos + a * sin)
            turn = torch.stack(turn, -1).flatten(-2) if c["interleaved"] else torch.cat(turn, -1)
            x = torch.cat([turn, x[..., R:]], -1)
        return x.to(TYPES[c["dtype"]])

    at = (s["pages"].long()[request, slot // c["page"]], slot % c["page"])
    s["k_cache"].index_put_(at, turned(s["k"], s.get("k_weight")))
    s["v_cache"].index_put_(at, s["v"].reshape((s["rows"],) + s["v"].shape[-2:])[live])
    s["q_out"].view((s["rows"],) + s["q_out"].shape[-2:])[live] = turned(s["q"], s.get("q_weight"))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _seen(s, L, of):
    """Of the rows `of` [.., N] of requests: which of L slots each attends to."""
    N, B = s["case"]["N"], s["case"]["B"]
    reach = torch.zeros(s["rows"] + 1, N, dtype=torch.bool, device="cuda")
    place = torch.arange(N, device="cuda")
    if s["parents"] is None:
        reach[:-1] = place <= s["local"][:, None]
    else:
        first = torch.arange(s["rows"], device="cuda") - s["local"]
        up = s["local"].long()
        for _ in range(N):
            reach[:-1] |= (place == up[:, None]) & (up >= 0)[:, None]
            up = torch.where(up >= 0, s["parents"].long()[(first + up.clamp(min=0)).clamp(max=s["rows"] - 1)], -1)
    reach = reach[of]  # [B, N, N]
    back = torch.arange(L, device="cuda") - s["lengths"][:, None]  # a slot's place among the request's tokens
    tree = reach.gather(2, back[:, None].clamp(0, N - 1).expand(B, N, L))
    return torch.where(back[:, None] < 0, True, tree & (back[:, None] < N))


def _padded_rows(s):
    """[B, N]: the row of each request's token (s["rows"]: none)."""
    c = s["case"]
    at = torch.full((c["B"], c["N"]), s["rows"], dtype=torch.long, device="cuda")
    live = s["live"]
    at[s["request"][live], s["local"].long()[live]] = torch.arange(s["rows"], device="cuda")[live]
    return at


def _plain_attend(s):
    c = s["case"]
    B, N, Hkv, D = c["B"], c["N"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    of = _padded_rows(s)
    k = s["k_cache"][s["pages"].long()].float().view(B, -1, Hkv, D)
    L = k.shape[1]
    q = torch.cat([s["q"].reshape(s["rows"], Hkv, G, D).float(), torch.zeros(1, Hkv, G, D, device="cuda")])[of]
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D), k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    del k
    x = x.view(B, Hkv, N, G, L).masked_fill_(~_seen(s, L, of)[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = x.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    v = s["v_cache"][s["pages"].long()].float().view(B, L, Hkv, D)
    o = torch.matmul(e.view(B, Hkv, N * G, L), v.transpose(1, 2)).view(B, Hkv, N, G, D) / total
    live = s["live"]
    rows = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hkv * G, D)[s["request"][live], s["local"].long()[live]]
    s["out"].view(s["rows"], Hkv * G, D)[live] = rows.to(TYPES[c["dtype"]])
    return {"out": s["out"]}


def _plain_verify(s):
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    of = _padded_rows(s)
    row = lambda node: of.gather(1, node[:, None])[:, 0].clamp(max=s["rows"] - 1)  # noqa: E731
    every = torch.arange(B, device="cuda")
    at = torch.zeros(B, dtype=torch.long, device="cuda")  # the node where each request stands
    here = row(at)
    r = s["p"][here].float()
    left = torch.ones(B, dtype=torch.float64, device="cuda")
    accept_len = torch.zeros(B, dtype=torch.long, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.long, device="cuda")
    out_tokens = torch.full((B, N), -1, dtype=torch.long, device="cuda")
    for i in range(1, N):
        mine = row(torch.full_like(at, i))
        parent = s["parents"].long()[mine] if s["parents"] is not None else torch.full_like(at, i - 1)
        tried = (of[:, i] < s["rows"]) & (parent == at)
        x = s["tokens"].long()[mine]
        drawn = s["q"][here].float() if not c["points"] else None
        qx = drawn[every, x].double() if drawn is not None else 1.0
        yes = tried & (s["uniforms"][mine].double() * qx * left < r[every, x].double())
        no = tried & ~yes
        if drawn is None:
            left = torch.where(no, left - r[every, x].double(), left)
            r[every, x] = torch.where(no, 0.0, r[every, x])
        else:
            # one rounding to 32 bits of r - left q, and one of its sum
            rest = (r.double() - left[:, None] * drawn.double()).clamp_(min=0.0).float()
            r = torch.where(no[:, None], rest, r)
            left = torch.where(no, rest.double().sum(1).float().double(), left)
        at = torch.where(yes, i, at)
        here = row(at)
        r = torch.where(yes[:, None], s["p"][here].float(), r)
        left = torch.where(yes, 1.0, left)
        path[every, accept_len] = torch.where(yes, i, path[every, accept_len])
        out_tokens[every, accept_len] = torch.where(yes, x, out_tokens[every, accept_len])
        accept_len += yes
    total = r.double().sum(1)
    r = torch.where((total > 0)[:, None], r, s["p"][here].float())  # nothing is left: from the target's own
    up_to = r.double().cumsum(1)
    t = s["uniforms"][row(torch.zeros_like(at))].double() * up_to[:, -1]
    last = torch.where(r > 0, torch.arange(V, device="cuda"), -1).amax(1)
    final = torch.searchsorted(up_to, t[:, None], right=True)[:, 0].minimum(last)
    out_tokens[every, accept_len] = final
    whole = lambda v: v.to(torch.int32)  # noqa: E731
    return {"accept_len": whole(accept_len), "path": whole(path), "out_tokens": whole(out_tokens), "n_out": whole(accept_len + 1)}


def _plain_keep(s):
    c = s["case"]
    on = s["path"] >= 0
    request, j = torch.nonzero(on, as_tuple=True)
    place = lambda slot: (s["pages"].long()[request, slot // c["page"]], slot % c["page"])  # noqa: E731
    base = s["lengths"].long()[request]
    source, target = place(base + s["path"].long()[on]), place(base + 1 + j)
    for x in (s["k"], s["v"]):
        x[:, target[0], target[1]] = x[:, source[0], source[1]]
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------------ one pass

def _own(s):
    import speculative_decoding_03_gb300 as ds
    c, op = s["case"], s["case"]["op"]
    ws = s.get("ws")
    if ws is None:  # a program keeps its workspace and its cache's handle from call to call
        nbytes = ds.tree_attention_workspace_bytes(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]) if op == "attend" else 256
        ws = s["ws"] = ds.Workspace.of_bytes(nbytes)
        if op != "verify":
            s["cache"] = ds.PagedCache(s["k"], s["v"]) if op == "keep" else ds.PagedCache(s["k_cache"], s["v_cache"])
    if op == "keep":
        ds.cache_keep(s["cache"], s["pages"], s["lengths"], s["path"], s["accept_len"], ws)
        return {"k": s["k"], "v": s["v"]}
    rows = dict(starts=s["starts"], nodes=c["N"]) if c["packed"] else dict(counts=s["counts"])
    if op == "append":
        ds.cache_append(s["cache"], s["k"], s["v"], s["pages"], s["lengths"], ws, q=s["q"], q_out=s["q_out"],
                        parents=s["parents"], inv_freq=s["inv_freq"], interleaved=c["interleaved"],
                        q_weight=s.get("q_weight"), k_weight=s.get("k_weight"), eps=1e-6, **rows)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "attend":
        ds.tree_attention(s["q"], s["cache"], s["pages"], s["lengths"], ws, parents=s["parents"], out=s["out"], **rows)
        return {"out": s["out"]}
    lead = (-1,) if c["packed"] else (c["B"], c["N"])
    shaped = lambda t: None if t is None else t.view(lead + t.shape[1:])  # noqa: E731
    s["answer"] = ds.tree_verify(shaped(s["p"]), shaped(s["tokens"]), shaped(s["uniforms"]), ws, q=shaped(s.get("q")),
                                 parents=shaped(s["parents"]), out=s.get("answer"), **rows)
    return s["answer"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "verify": _plain_verify, "keep": _plain_keep}[state["case"]["op"]](state)


def work(case):
    B, e = case["B"], SIZES[case["dtype"]]
    if case["op"] == "keep":
        moved = sum(_accepted(case)) * case["layers"] * case["Hkv"] * case["D"] * 2
        return {"bytes": 2 * moved * e + 4 * B * case["N"], "flops": 0}
    counts = _counts(case)
    if case["op"] == "verify":
        # a row of p, and of q where a token is rejected: the last node of some chains is reached
        rows = B * (1.0 if case["points"] else 1.8)
        return {"bytes": rows * case["V"] * e + 12 * sum(counts), "flops": 3 * rows * case["V"]}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        elements = sum(counts) * (Hq + 2 * Hkv) * D
        return {"bytes": 2 * elements * e, "flops": 8 * elements}
    # any request may have any count: a count's mean stands for each
    lengths, n = _spread(case["low"], case["high"], B), sum(counts) / B
    slots = sum(l + n for l in lengths)
    return {"bytes": slots * 2 * Hkv * D * e + 2 * sum(counts) * Hq * D * e, "flops": 4 * slots * n * Hq * D}


# -------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """What ``run`` returns, from the definitions, in 64 bits and unrounded; None for whole numbers
    and for copies."""
    if case["op"] in ("verify", "keep"):
        return None
    s = prepare(case, seed)
    starts = s["starts"].tolist() if case["packed"] else [b * case["N"] for b in range(case["B"])]
    counts, lengths = s["counts"].tolist(), s["lengths"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else None
    flat = lambda t: t.reshape((s["rows"],) + t.shape[-2:])  # noqa: E731
    up = lambda b, i: i - 1 if parents is None else parents[starts[b] + i]  # noqa: E731
    if case["op"] == "append":
        q_out, keys = s["q_out"].double(), s["k_cache"].double()
        rows, where, slots = [], [], []
        for b in range(case["B"]):
            depth = []
            for i in range(counts[b]):
                depth.append(0 if i == 0 else depth[up(b, i)] + 1)
            rows += range(starts[b], starts[b] + counts[b])
            where += [lengths[b] + d for d in depth]
            slots += [(b, lengths[b] + i) for i in range(counts[b])]
        rows, slots = torch.tensor(rows, device="cuda"), torch.tensor(slots, device="cuda")
        place = torch.tensor(where, device="cuda", dtype=torch.float64)
        page, line = s["pages"].long()[slots[:, 0], slots[:, 1] // case["page"]], slots[:, 1] % case["page"]

        def rotated(x, weight):
            x = flat(x)[rows].double()
            if case["norm"]:
                x = weight.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + 1e-6)
            if case["rotated"]:
                half = case["rotated"] // 2
                z = x[..., :2 * half].unflatten(-1, (half, 2)) if case["interleaved"] else x[..., :2 * half].unflatten(-1, (2, half)).transpose(-1, -2)
                turn = torch.polar(torch.ones_like(place)[:, None], place[:, None] * s["inv_freq"].double())
                z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * turn[:, None])
                x = torch.cat([(z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., 2 * half:]], -1)
            return x

        flat(q_out)[rows] = rotated(s["q"], s.get("q_weight"))
        keys[page, line] = rotated(s["k"], s.get("k_weight"))
        values = s["v_cache"].double()
        values[page, line] = flat(s["v"])[rows].double()
        return {"q": q_out, "k_cache": keys, "v_cache": values}
    Hkv, D = case["Hkv"], case["D"]
    out = s["out"].double()
    for b in range(case["B"]):
        n, l = counts[b], lengths[b]
        if n == 0:
            continue
        slots = torch.arange(l + n, device="cuda")
        page, line = s["pages"].long()[b, slots // case["page"]], slots % case["page"]
        sees = torch.zeros(n, l + n, dtype=torch.bool)
        sees[:, :l] = True
        for i in range(n):
            if i and up(b, i) >= 0:
                sees[i, l:] = sees[up(b, i), l:]
            sees[i, l + i] = True
        sees = sees.cuda()
        rows = slice(starts[b], starts[b] + n)
        for h in range(Hkv):
            k, v = s["k_cache"][page, line, h].double(), s["v_cache"][page, line, h].double()
            q = flat(s["q"])[rows].unflatten(1, (Hkv, -1))[:, h].double()
            score = torch.einsum("ngd,ld->ngl", q, k) / math.sqrt(D)
            p = torch.softmax(score.masked_fill(~sees[:, None], -math.inf), -1)
            flat(out)[rows].unflatten(1, (Hkv, -1))[:, h] = torch.einsum("ngl,ld->ngd", p, v)
    return {"out": out}
