"""A whole step: tokens of the framework's own draft, as many as its schedule says, through the target's side,
against the framework's verification from the same uniform numbers."""
import numpy as np
import pytest

import workloads

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")
import oracle  # noqa: E402

if torch.cuda.is_available():
    from _target import Batch, attention_reference, attention_tolerance, fill_cache, gen, new_cache, verify_reference

BF16 = torch.bfloat16
B, GAMMA, V, HQ, HKV, D = 8, 4, 3000, 6, 2, 64
N = GAMMA + 1


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("seed", [2, 3, 8])       # (every test's u - p / q is 0.01 or more, by the oracle)
@pytest.mark.parametrize("greedy", [False, True])
def test_steps_of_the_draft(greedy, seed, full):
    """Draft, confidence, schedule; then append, attend, verify and keep over two layers.  From the
    numbers that ``verify`` draws for itself ``tree_verify`` accepts the same tokens, and the next step
    attends to them."""
    w = workloads.scaled(workloads.get("qwen3_4b_like"), B=B, gamma=GAMMA, V=V, r=64, H=32)
    inp = workloads.generate(w)
    dev = ds.to_device(inp)
    U, T, W1, W2, anchor = (dev[k] for k in ("U", "T", "W1", "W2", "anchor"))
    n = torch.arange(B * N + 1, device="cuda")
    sps = dev["sps"] if full else 1.0 / (1.0 + 0.1 * (n - 20).clamp(min=0))    # all scheduled, or one or two
    dws = ds.Workspace(B, GAMMA, V, w.r, w.H)

    d = ds.draft_greedy(U, W1, W2, anchor, dws) if greedy else ds.draft(U, W1, W2, anchor, seed, dws)
    _, a = ds.confidence(dev["h"], anchor, d["tokens"], W1, dev["w_c"], float(inp.b_c), dws)
    ell, _, _ = ds.schedule(a, sps.float().contiguous(), dws)
    want = ds.verify_greedy(T, d["tokens"], ell, seed, dws) if greedy else \
        ds.verify(T, U, W1, W2, anchor, d["tokens"], d["q_tok"], d["row_max"], d["row_sumexp"], ell, seed, dws)

    # what the target's side takes of it
    tokens = torch.cat([anchor[:, None], d["tokens"]], 1)
    counts = ell + 1
    q = None
    if not greedy:                                # whole rows of what the tokens were drawn from
        bias = ds.markov_bias(W1, W2, tokens[:, :GAMMA].contiguous(), dws).view(B, GAMMA, V)
        q = torch.zeros(B, N, V, device="cuda")   # (the last token has no children)
        q[:, :GAMMA] = torch.softmax(U + bias, -1)
    p = torch.softmax(T, -1)
    u = torch.tensor([[oracle.u01(oracle.draw(seed, b, i, 0, 1)) for i in range(N)] for b in range(B)],
                     dtype=torch.float32, device="cuda")

    batch = Batch(counts.tolist(), [0, 7, 31, 60, 128, 200, 15, 16], 16, N=N, room=N)
    batch.kw["counts"] = counts
    kc, vc = new_cache(batch, HKV, D, BF16, layers=2)
    for t in (0, 1):
        fill_cache(batch, kc[t], vc[t], seed=100 + t, tokens=False)
    cache = ds.PagedCache(kc, vc)
    ws = ds.Workspace.of_bytes(ds.tree_attention_workspace_bytes(B, N, HQ, HKV, D))
    inv = (1e4 ** -(torch.arange(0, D, 2, device="cuda") / D)).float()
    g = gen(101)
    for _ in range(2):
        for t in (0, 1):
            x = torch.randn(B, N, HQ + 2 * HKV, D, generator=g, device="cuda").to(BF16)
            y = ds.cache_append(cache, x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], batch.pages, batch.lens, ws,
                                q=x[:, :, :HQ], inv_freq=inv, layer=t, **batch.kw)
            out = ds.tree_attention(y, cache, batch.pages, batch.lens, ws, layer=t, **batch.kw)
            ref, _, spread, size = attention_reference(batch, y, kc[t], vc[t], D ** -0.5)
            err = (out.view(B * N, HQ, D)[batch.live_rows()].double() - ref).abs()
            assert (err <= attention_tolerance(batch, ref, spread, size, vc[t], BF16)).all()
        got = ds.tree_verify(p, tokens, u, ws, q=q, **batch.kw)
        before = kc.clone(), vc.clone()
        ds.cache_keep(cache, batch.pages, batch.lens, got["path"], got["accept_len"], ws)
        assert ws.status() == 0 and dws.status() == 0
        # a chain's accepted tokens are where they stay
        assert all(torch.equal(torch.nan_to_num(s), torch.nan_to_num(t)) for s, t in zip(before, (kc, vc)))
        assert torch.equal(got["accept_len"], want["accept_len"]) and torch.equal(got["n_out"], want["n_out"])
        accepted = torch.arange(N, device="cuda") < got["accept_len"][:, None]
        assert torch.equal(got["out_tokens"][accepted], want["out_tokens"][accepted])
        assert torch.equal(got["out_tokens"] >= 0, want["out_tokens"] >= 0)      # (the last token is drawn otherwise)
        for key, value in verify_reference(batch, p, tokens, u, q).items():
            np.testing.assert_array_equal(got[key].cpu().numpy(), value, err_msg=key)
        batch.lens += 1 + got["accept_len"]
        batch.lengths = batch.lens.tolist()
    assert want["accept_len"].max() > 0
