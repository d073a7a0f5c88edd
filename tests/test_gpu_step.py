"""One training step of the RNN head through the library alone: embedding, gates, recurrence, logits,
distillation and back, then clipping; against autograd in 64 bits, eager and as a captured graph."""

import pytest
import torch

from rank_markov_draft_gb300 import binding
from tests.test_gpu_embed import normal, tokens

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
B, K, V, R, D, TOP = 6, 8, 1000, 64, 96, 12


def inputs(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    prev = tokens(seed, B * K, V, padding=0.0).view(B, K)
    U = normal(seed + 1, B, K, V)
    h = normal(seed + 2, B, K, D).to(BF16)
    t = torch.topk(U + normal(seed + 3, B, K, V), TOP, dim=2)
    rest = 0.1 * torch.rand(B, K, generator=g, device="cuda")
    return dict(prev=prev, U=U, h=h, ids=t.indices.int(), t=t.values.contiguous(), rest=rest)


def weights():
    return dict(W1=0.5 * normal(11, V, R), W2=(0.5 * normal(12, R, V)).to(BF16), Wz=(normal(13, D, 2 * R) / D ** 0.5).to(BF16),
                bz=normal(14, 2 * R))


def train_step(ctx, a, w, limit):
    """Gradients of W1, W2, Wz and bz, clipped in place; the losses and the norm."""
    e = binding.embed(ctx, w["W1"], a["prev"], dtype=BF16)
    z = binding.linear(ctx, a["h"], w["Wz"], bias=w["bz"])["y"]
    s = binding.rnn_scan(ctx, z[..., :R], z[..., R:], e)["s"]
    logits = binding.linear(ctx, s, w["W2"], residual=a["U"])["y"]
    d = binding.distill(ctx, logits, a["ids"], a["t"], teacher_rest=a["rest"], alpha_kl=1.0, alpha_tv=0.0, grad=logits)
    gl = binding.linear_grad(ctx, s, w["W2"], logits)
    gs = binding.rnn_scan_grad(ctx, z[..., :R], z[..., R:], e, s, gl["dx"])
    dz = gs["dza"].as_strided((B, K, 2 * R), (K * 2 * R, 2 * R, 1))  # both halves, one tensor
    gz = binding.linear_grad(ctx, a["h"], w["Wz"], dz, dx=False, dbias=True)
    g = dict(W1=binding.embed_grad(ctx, a["prev"], gs["de"], V), W2=gl["dW"], Wz=gz["dW"], bz=gz["dbias"])
    norm = binding.clip_grads(ctx, list(g.values()), limit)
    return g, d["loss"], norm


def reference(a, w, limit):
    p = {n: t.double().requires_grad_() for n, t in w.items()}
    e = p["W1"][a["prev"].long()]
    z = a["h"].double() @ p["Wz"] + p["bz"]
    s, out = torch.zeros(B, R, dtype=torch.float64, device="cuda"), []
    for k in range(K):
        s = torch.sigmoid(z[:, k, :R]) * s + torch.sigmoid(z[:, k, R:]) * e[:, k]
        out.append(s)
    q = torch.softmax(a["U"].double() + torch.stack(out, 1) @ p["W2"], 2)
    qi = q.gather(2, a["ids"].long())
    rho = a["rest"].double()
    pi = (1 - rho)[..., None] * torch.softmax(a["t"].double(), 2)
    loss = (pi * (pi.log() - qi.log())).sum(2) + rho * (rho.log() - (1 - qi.sum(2)).log())
    loss.sum().backward()
    g = {n: t.grad for n, t in p.items()}
    norm = torch.sqrt(sum((v * v).sum() for v in g.values()))
    return {n: v * min(1.0, limit / float(norm)) for n, v in g.items()}, loss.detach(), norm


def compare(got, want):
    """What the path holds in bf16 (e, z, s, logits, their gradient, ds, dza, dzg, de: ten roundings of
    2^-9 of each value at most, whose errors partly cancel) moves a gradient by less than ten of
    their sum."""
    (g, loss, norm), (wg, wl, wn) = got, want
    for n in wg:
        assert (g[n].double() - wg[n]).norm() <= 10 * 2.0 ** -8 * wg[n].norm(), n
    assert abs(float(norm) - float(wn)) <= 10 * 2.0 ** -8 * float(wn)
    # a logit's own rounding: 2^-9 of up to 6 for each of the row's events, and its inputs'
    assert (loss.double() - wl).abs().max() <= 10 * 2.0 ** -8 * 6


@pytest.mark.parametrize("limit", [0.05, 1e9])
def test_step_against_autograd(dsp, limit):
    a, w = inputs(20), weights()
    got = train_step(dsp, a, w, limit)
    torch.cuda.synchronize()
    assert dsp.status() == 0
    compare(got, reference(a, w, limit))


def test_captured_step(dsp):
    a, w = inputs(20), weights()
    for _ in range(2):
        train_step(dsp, a, w, 0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, loss, norm = train_step(dsp, a, w, 0.5)
    for seed in (30, 40):
        for n, t in inputs(seed).items():
            a[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert dsp.status() == 0
        eg, el, en = train_step(dsp, a, w, 0.5)
        assert torch.equal(loss, el) and torch.equal(norm, en) and all(torch.equal(g[n], eg[n]) for n in g)
        compare((g, loss, norm), reference(a, w, 0.5))
