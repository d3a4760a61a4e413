"""Training the low-rank Markov draft head by distillation, and a step with the trained head.

The target's rows give the teacher's top logits (``token_logprobs``); the student's logits are
the backbone's base logits plus the head's bias (``markov_bias``); ``distill_loss_grad`` gives
the loss, the acceptance expected of a target cut to those top logits (here 32 of 1024, which
hold about 0.6 of its probability) and the gradient in place of the logits; the head's two
matrices get theirs from two plain products and ``embed_grad``.  The loss is the DSpark pages'
(weigao.cc DSpark-vs-MTP page, "loss": total variation 0.9, cross entropy 0.1, weights that
fall over the block's positions).  Synthetic data: the target differs from the base logits by
a hidden head of the same form, so the acceptance of the trained head's drafts rises.

    python examples/train_draft_head.py [steps]
"""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class DraftHead:
    """fp32 master weights of the head, their bf16 copies, and the training step's buffers."""

    def __init__(self, B, gamma, V, r, seed=0, top=32):
        import torch
        import speculative_decoding_03_gb300 as ds
        self.torch, self.ds = torch, ds
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.W1 = torch.randn(V, r, generator=g, device="cuda") * 0.5
        self.W2 = torch.randn(r, V, generator=g, device="cuda") * 0.1
        self.top, self.n = top, B * gamma
        self.ws = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(B * gamma, V, r))
        # position weights exp(-(k - 1) / 4), summing to 1 over the batch
        w = torch.exp(-torch.arange(gamma, device="cuda") / 4.0).repeat(B, 1)
        self.weights = (w / w.sum()).contiguous()
        self.half()

    def half(self):
        self.W1h, self.W2h = (w.to(self.torch.bfloat16) for w in (self.W1, self.W2))

    def teacher(self, T):
        """The target's top log probabilities of every position [B, gamma, V] (no token is
        given, so every row is used)."""
        out = self.ds.token_logprobs(T, None, self.top, self.ws)
        return out["top_ids"], out["top_logprobs"]

    def step(self, U, prev, labels, ids, logprobs, lr):
        """One step of gradient descent on a batch; returns (loss, mean expected acceptance)
        before it, as device scalars."""
        ds, ws = self.ds, self.ws
        B, gamma, V = U.shape
        z = ds.markov_bias(self.W1h, self.W2h, prev.view(-1), ws).view(B, gamma, V)
        z += U
        buf = dict(loss=self.torch.empty_like(self.weights), accept=self.torch.empty_like(self.weights), d_logits=z)
        out = ds.distill_loss_grad(z, ids, logprobs, ws, labels, self.weights, kl=0.0, tv=0.9, ce=0.1, out=buf)
        dz = out["d_logits"].view(-1, V)                       # in place of the logits
        E = ds.embed(self.W1h, prev.view(-1), ws, dtype=self.torch.float32)
        dW2 = E.t() @ dz
        dW1 = ds.embed_grad(dz @ self.W2h.float().t(), prev.view(-1), V, ws)
        self.W1.add_(dW1, alpha=-lr)
        self.W2.add_(dW2, alpha=-lr)
        self.half()
        return out["loss"].sum(), out["accept"].mean()


def batch(B, gamma, V, hidden, seed):
    """Base logits, predecessors and the target's rows (base logits plus the hidden head)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    U = torch.randn(B, gamma, V, generator=g, device="cuda")
    prev = torch.randint(0, V, (B, gamma), generator=g, device="cuda", dtype=torch.int32)
    T = U + hidden[0][prev.long()] @ hidden[1]
    gumbel = -torch.log(-torch.log(torch.rand(T.shape, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    labels = (T + gumbel).argmax(2).to(torch.int32)
    return U, prev, T, labels


def main(steps=200, B=32, gamma=4, V=1024, r=16, lr=300.0, log=print):
    import torch
    import speculative_decoding_03_gb300 as ds
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    hidden = (torch.randn(V, r, generator=g, device="cuda"), torch.randn(r, V, generator=g, device="cuda") * 0.5)
    head = DraftHead(B, gamma, V, r)
    history = []
    for i in range(steps):
        U, prev, T, labels = batch(B, gamma, V, hidden, 100 + i)
        ids, logprobs = head.teacher(T)
        loss, accept = head.step(U, prev, labels, ids, logprobs, lr)
        history.append((loss, accept))
        if i % 50 == 0 or i + 1 == steps:
            log(f"step {i}: loss {loss.item():.4f}, expected acceptance {accept.item():.4f}")
    if head.ws.status() != 0:
        raise RuntimeError("device status word set during training")

    # a speculative step with the trained head, and the log probabilities of its answer
    U, prev, T, _ = batch(B, gamma + 1, V, hidden, 7)
    sps = torch.from_numpy((1.0 / (1.0 + 0.001 * np.arange(B * (gamma + 1) + 1))).astype(np.float32)).cuda()
    H = 16
    dev = dict(U=U[:, :gamma].contiguous(), T=T.contiguous(), W1=head.W1h, W2=head.W2h,
               anchor=prev[:, 0].contiguous(), h=torch.zeros(B, gamma, H, device="cuda"),
               w_c=torch.zeros(H + r, device="cuda"), sps=sps)
    step = ds.Step(dev, 1.0).run(seed=3)
    answer = step.verify_out["out_tokens"]                     # -1 past each request's answer
    lp = ds.token_logprobs(T, answer, 5, head.ws)
    given = answer >= 0
    log(f"a step answers {given.sum().item()} tokens, mean log probability "
        f"{lp['logprob'][given].mean().item():.3f}, mean entropy {lp['entropy'][given].mean().item():.3f}")
    return [(a.item(), b.item()) for a, b in history], answer, lp


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
