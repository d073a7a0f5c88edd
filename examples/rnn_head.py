"""Train the RNN head by distillation and serve what was learned.

    python examples/rnn_head.py [steps]

A target (an RNN head of fixed random weights over the same base logits) writes blocks; a student
head starts from noise and is fitted to the target's top logits:

    rnn_scan -> logits -> distill (loss and gradient) -> rnn_scan_grad -> Adam

Then the student drafts new blocks (rnn_draft) and the target verifies them (verify_probs), as it
did before the training: the accepted length is what the training is for.  Synthetic data."""

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from rank_markov_draft_gb300 import binding  # noqa: E402

B, K, V, R, D, TOP = 64, 8, 1024, 64, 128, 32


class Head:
    """W1 [V, R], W2 [R, V], Wa and Wg [D, R]: fp32 values, used as bf16."""

    def __init__(self, gen, std):
        def normal(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.w = dict(W1=std * normal(V, R), W2=std * normal(R, V), Wa=normal(D, R) / D ** 0.5,
                      Wg=normal(D, R) / D ** 0.5)
        self.m = {n: torch.zeros_like(w) for n, w in self.w.items()}
        self.v = {n: torch.zeros_like(w) for n, w in self.w.items()}
        self.steps = 0

    def bf16(self):
        return {n: w.bfloat16() for n, w in self.w.items()}

    def adam(self, grads, lr=0.02, b1=0.9, b2=0.99):
        self.steps += 1
        for n, g in grads.items():
            self.m[n].lerp_(g, 1 - b1)
            self.v[n].lerp_(g * g, 1 - b2)
            m, v = self.m[n] / (1 - b1 ** self.steps), self.v[n] / (1 - b2 ** self.steps)
            self.w[n] -= lr * m / (v.sqrt() + 1e-8)


def backbone(gen):
    """Base logits, hidden states and anchors of B blocks (a position more, for the bonus token)."""
    U = torch.randn(B, K + 1, V, generator=gen, device="cuda")
    h = torch.randn(B, K + 1, D, generator=gen, device="cuda").bfloat16()
    return U, h, torch.randint(0, V, (B,), generator=gen, device="cuda", dtype=torch.int32)


def draft(ctx, head, U, h, anchors, seed):
    w = head.bf16()
    return binding.rnn_draft(ctx, U, w["W1"], w["W2"], anchors, h, w["Wa"], Wg=w["Wg"], seed=seed)["tokens"]


def logits_of(ctx, head, U, h, prev):
    w = head.bf16()
    return binding.rnn_logits(ctx, U, w["W1"], w["W2"], prev, h, w["Wa"], Wg=w["Wg"])


def train_step(ctx, head, target, gen, seed):
    """One step on B blocks that the target writes; the mean loss."""
    U, h, anchors = backbone(gen)
    U, h = U[:, :K].contiguous(), h[:, :K].contiguous()
    tokens = draft(ctx, target, U, h, anchors, seed)
    prev = torch.cat([anchors[:, None], tokens[:, :-1]], 1)
    known = logits_of(ctx, target, U, h, prev)
    top = torch.topk(known["logits"], TOP, dim=2)
    rest = 1 - (top.values - known["lse"][..., None]).exp().sum(2)
    weight = torch.exp(-torch.arange(K, device="cuda") / 4.0).expand(B, K) / (B * K)

    w = head.bf16()
    e, za, zg = w["W1"][prev.long()], h @ w["Wa"], h @ w["Wg"]
    s = binding.rnn_scan(ctx, za, zg, e)["s"]
    logits = U + s.float() @ w["W2"].float()
    out = binding.distill(ctx, logits, top.indices.int(), top.values, teacher_rest=rest,
                          row_weight=weight.contiguous(), grad=logits)  # in place of the logits
    ds = (logits @ w["W2"].float().T).bfloat16()
    g = binding.rnn_scan_grad(ctx, za, zg, e, s, ds)
    rows = h.reshape(-1, D).float()
    head.adam(dict(W1=torch.zeros_like(head.w["W1"]).index_add_(0, prev.flatten().long(), g["de"].reshape(-1, R).float()),
                   W2=s.reshape(-1, R).float().T @ logits.view(-1, V),
                   Wa=rows.T @ g["dza"].reshape(-1, R).float(), Wg=rows.T @ g["dzg"].reshape(-1, R).float()))
    return float(out["loss"].sum())


def accepted(ctx, head, target, gen, seed):
    """Mean accepted length of B drafted blocks of K tokens."""
    U, h, anchors = backbone(gen)
    tokens = draft(ctx, head, U[:, :K].contiguous(), h[:, :K].contiguous(), anchors, seed)
    prev = torch.cat([anchors[:, None], tokens], 1)
    P = torch.softmax(logits_of(ctx, target, U, h, prev)["logits"], 2)
    Q = torch.softmax(logits_of(ctx, head, U[:, :K].contiguous(), h[:, :K].contiguous(), prev[:, :K].contiguous())["logits"], 2)
    out = binding.verify_probs(ctx, P, tokens, torch.rand(B, K, generator=gen, device="cuda"),
                               torch.rand(B, generator=gen, device="cuda"), Q=Q)
    return float(out["n_acc"].float().mean())


def run(steps=300):
    gen = torch.Generator("cuda").manual_seed(1)
    with binding.Context(0, B_max=B, V_max=V, K_max=K + 1) as ctx:
        target, head = Head(gen, std=0.8), Head(gen, std=0.1)
        before = accepted(ctx, head, target, gen, seed=0)
        losses = [train_step(ctx, head, target, gen, seed=1 + i) for i in range(steps)]
        after = accepted(ctx, head, target, gen, seed=1 + steps)
        torch.cuda.synchronize()
        if ctx.status() != 0:
            raise RuntimeError(f"device status {ctx.status()}")
    return dict(losses=losses, before=before, after=after)


if __name__ == "__main__":
    out = run(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
    for i in range(0, len(out["losses"]), max(1, len(out["losses"]) // 10)):
        print(f"step {i:4d}  loss {out['losses'][i]:.4f}")
    print(f"accepted tokens of {K}: {out['before']:.2f} before, {out['after']:.2f} after")
