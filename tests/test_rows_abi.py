"""Refusals of the calls on rows of logits and of tables: host-side validation returns before
anything is launched, so these run without a GPU."""
import ctypes

import pytest

import speculative_decoding_03_gb300 as ds

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000000          # an aligned address that is never dereferenced by these calls
F32, BF16, F16 = 0, 1, 2


def logprobs(z=FAKE, dtype=F32, ld=1000, tokens=FAKE, N=4, V=1000, K=5, logprob=FAKE, entropy=FAKE,
             rank=FAKE, row_max=FAKE, row_sumexp=FAKE, ids=FAKE, top=FAKE, ws=FAKE, ws_bytes=256):
    return ds.lib().dspark_token_logprobs(z, dtype, ld, tokens, N, V, K, logprob, entropy, rank, row_max,
                                          row_sumexp, ids, top, ws, ws_bytes, None)


def logprobs_grad(z=FAKE, dtype=F32, ld=1000, tokens=FAKE, N=4, V=1000, row_max=FAKE, row_sumexp=FAKE,
                  entropy=FAKE, d_logprob=FAKE, d_entropy=FAKE, dz=FAKE, ld_d=1000, ws=FAKE, ws_bytes=256):
    return ds.lib().dspark_token_logprobs_grad(z, dtype, ld, tokens, N, V, row_max, row_sumexp, entropy,
                                               d_logprob, d_entropy, dz, ld_d, ws, ws_bytes, None)


def distill(grad=True, z=FAKE, dtype=F32, ld=1000, ids=FAKE, t=FAKE, labels=FAKE, weights=FAKE, d_loss=FAKE,
            N=4, V=1000, K=8, tau=1.0, kl=1.0, tv=0.0, ce=0.0, loss=FAKE, accept=FAKE, dz=FAKE, ld_d=1000,
            ws=FAKE, ws_bytes=256):
    f = [ctypes.c_float(x) for x in (tau, kl, tv, ce)]
    if grad:
        return ds.lib().dspark_distill_loss_grad(z, dtype, ld, ids, t, labels, weights, d_loss, N, V, K, *f,
                                                 loss, accept, dz, ld_d, ws, ws_bytes, None)
    return ds.lib().dspark_distill_loss(z, dtype, ld, ids, t, labels, weights, N, V, K, *f, loss, accept, ws,
                                        ws_bytes, None)


def embed(W=FAKE, dtype=BF16, ld=256, ids=FAKE, N=4, V=1000, D=256, scale=1.0, out=FAKE, out_dtype=BF16,
          ld_out=256, ws=FAKE, ws_bytes=256):
    return ds.lib().dspark_embed(W, dtype, ld, ids, N, V, D, ctypes.c_float(scale), out, out_dtype, ld_out, ws,
                                 ws_bytes, None)


def embed_grad(d_out=FAKE, dtype=BF16, ld=256, ids=FAKE, N=4, V=1000, D=256, scale=1.0, accumulate=0, dW=FAKE,
               w_dtype=BF16, ld_w=256, ws=FAKE, ws_bytes=1 << 30):
    return ds.lib().dspark_embed_grad(d_out, dtype, ld, ids, N, V, D, ctypes.c_float(scale), accumulate, dW,
                                      w_dtype, ld_w, ws, ws_bytes, None)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("bad", [
    dict(z=None), dict(z=FAKE + 2), dict(dtype=3), dict(dtype=-1), dict(ld=999), dict(N=-1), dict(V=0, ld=0),
    dict(K=-1), dict(tokens=FAKE + 2), dict(tokens=None), dict(logprob=None), dict(rank=None), dict(ids=None),
    dict(top=None), dict(K=0), dict(entropy=FAKE + 1), dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=255)])
def test_token_logprobs_refuses(bad):
    assert logprobs(**bad) == INVALID


def test_token_logprobs_limits_and_no_rows():
    assert logprobs(K=129) == UNSUPPORTED
    assert logprobs(N=1 << 21) == UNSUPPORTED
    assert logprobs(V=(1 << 30) + 8, ld=(1 << 30) + 8) == UNSUPPORTED
    assert logprobs(N=0, z=None, tokens=None, logprob=None, rank=None) == OK
    assert logprobs(N=0, ws=None) == INVALID


@pytest.mark.parametrize("bad", [
    dict(z=None), dict(dtype=BF16, z=FAKE + 1), dict(dz=None), dict(ld_d=999), dict(ld=10), dict(tokens=None),
    dict(row_max=None), dict(row_sumexp=None), dict(entropy=None), dict(d_logprob=FAKE + 2), dict(ws=FAKE + 128),
    dict(dz=FAKE, z=FAKE, ld_d=1001)])
def test_token_logprobs_grad_refuses(bad):
    assert logprobs_grad(**bad) == INVALID


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("bad", [
    dict(z=None), dict(dtype=7), dict(ld=1), dict(N=-2), dict(K=-1), dict(ids=None), dict(t=None), dict(K=0),
    dict(loss=None), dict(accept=FAKE + 2), dict(labels=FAKE + 1), dict(weights=FAKE + 3), dict(tau=0.0),
    dict(tau=-1.0), dict(tau=NAN), dict(tau=INF), dict(tau=1e-45), dict(kl=-1.0), dict(tv=NAN), dict(ce=INF),
    dict(ws=None), dict(ws_bytes=0)])
def test_distill_refuses(grad, bad):
    assert distill(grad, **bad) == INVALID


def test_distill_grad_refuses_and_limits():
    assert distill(dz=None) == INVALID
    assert distill(dz=FAKE + 2) == INVALID
    assert distill(ld_d=999) == INVALID
    assert distill(ld_d=1001) == INVALID                 # in place with another stride
    assert distill(d_loss=FAKE + 1) == INVALID
    assert distill(K=129) == UNSUPPORTED
    assert distill(N=1 << 21) == UNSUPPORTED
    assert distill(N=0, z=None, loss=None, accept=None, dz=None) == OK


@pytest.mark.parametrize("bad", [
    dict(W=None), dict(W=FAKE + 1), dict(dtype=5), dict(ld=255), dict(ids=None), dict(V=0), dict(D=0), dict(N=-1),
    dict(scale=NAN), dict(scale=INF), dict(out=None), dict(out_dtype=F16), dict(ld_out=10), dict(ws=None)])
def test_embed_refuses(bad):
    assert embed(**bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(d_out=None), dict(dtype=-3), dict(ld=255), dict(ids=None), dict(ids=FAKE + 2), dict(V=0), dict(D=0),
    dict(N=-1), dict(scale=NAN), dict(dW=None), dict(w_dtype=F16), dict(ld_w=255), dict(ws=FAKE + 4),
    dict(ws_bytes=1024)])
def test_embed_grad_refuses(bad):
    assert embed_grad(**bad) == INVALID


def test_embed_limits_and_no_rows():
    assert embed(N=0, ids=None, out=None) == OK
    assert embed(D=70000, ld=70000, ld_out=70000) == UNSUPPORTED
    assert embed_grad(D=70000, ld=70000, ld_w=70000) == UNSUPPORTED
    assert embed_grad(N=0, ids=None, d_out=None, accumulate=1) == OK      # nothing to add
    L = ds.lib()
    assert L.dspark_embed_grad_workspace_bytes(-1, 10, 10) == 0
    assert L.dspark_embed_grad_workspace_bytes(10, 0, 10) == 0
    assert L.dspark_embed_grad_workspace_bytes(10, 10, 0) == 0
    assert L.dspark_embed_grad_workspace_bytes(1 << 21, 10, 10) == 0
    small, large = (L.dspark_embed_grad_workspace_bytes(n, 1000, 64) for n in (100, 100000))
    assert 256 < small < large and small % 256 == 0
    assert embed_grad(N=100, D=64, ld=64, ld_w=64, ws_bytes=small - 1) == INVALID


def test_a_workspace_holds_the_status_word():
    with pytest.raises(ValueError):
        ds.Workspace.of_bytes(255)
