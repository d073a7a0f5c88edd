"""Cases of the training and verification operators and their plain forms.

Three operators, each called as a program that trains or runs a drafter calls it:

* ``verify_probs``: accept-or-correct of a drafted block against the target's probabilities,
  from random numbers the caller gives, the draft's probabilities dense or on candidates;
* ``distill``: the loss against a teacher's top logits (KL and total variation over the
  teacher's tokens and the rest of the vocabulary) and its gradient;
* ``rnn_scan`` / ``rnn_scan_grad``: the RNN head's gated recurrence
  s_t = sigmoid(za_t) s_{t-1} + sigmoid(zg_t) e_t over given sequences, and its gradients.

``run`` computes a case in elementary torch operations (``own`` false) or through the library
(``own`` true).  ``exact`` restates each definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
ALPHA_KL, ALPHA_TV = 0.1, 0.9  # the DSpark recipe's weights of the two terms


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one user's request on a small vocabulary: the call's latency
        dict(name="verify one request", op="verify", B=1, K=4, V=4096, m=0),
        # the serving batch with a full-vocabulary drafter
        dict(name="verify serving batch", op="verify", B=128, K=16, V=151936, m=0),
        # the selector's drafts: 16 candidates a position
        dict(name="verify candidates", op="verify", B=256, K=16, V=151936, m=16),
        # a short ragged batch, odd vocabulary (rows that start at no 16-byte boundary)
        dict(name="distill few odd rows", op="distill", N=5, V=32003, k=20, dtype="bf16", T=2.0, grad=True),
        # one training batch of the serving shape (128 blocks of 16), fp32 logits
        dict(name="distill batch fp32", op="distill", N=2048, V=151936, k=32, dtype="fp32", T=1.0, grad=True),
        # the same from a mixed-precision trainer
        dict(name="distill batch bf16", op="distill", N=2048, V=151936, k=64, dtype="bf16", T=1.0, grad=True),
        # the validation loss: no gradient asked for
        dict(name="distill loss only", op="distill", N=1024, V=151936, k=64, dtype="bf16", T=1.0, grad=False),
        # serving, one token a request: state in, state out
        dict(name="scan one token", op="scan", N=128, L=1, D=256, dtype="bf16", reset=False),
        # teacher-forced draft blocks of a training batch
        dict(name="scan blocks", op="scan", N=8192, L=16, D=256, dtype="bf16", reset=False),
        # one long packed sequence, few channels
        dict(name="scan long", op="scan", N=1, L=65536, D=256, dtype="fp32", reset=True),
        # the two above backward
        dict(name="scan grad blocks", op="scan_grad", N=8192, L=16, D=256, dtype="bf16", reset=False),
        dict(name="scan grad long", op="scan_grad", N=4, L=16384, D=256, dtype="bf16", reset=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "distill", "distill", "scan", "scan_grad"])
    if op == "verify":
        V = _log(rng, 1000, 151936)
        K = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        B = _log(rng, 1, max(1, min(256, 256 * 17 * 151936 // ((K + 1) * V))))
        return dict(op=op, B=B, K=K, V=V, m=rng.choice([0, 0, 1, rng.randint(2, 32)]))
    if op == "distill":
        V = _log(rng, 1000, 151936)
        if rng.random() < 0.5:
            V = V // 8 * 8
        N = _log(rng, 1, max(1, min(8192, 2048 * 151936 // V)))
        return dict(op=op, N=N, V=V, k=_log(rng, 1, 128), dtype=rng.choice(["fp32", "bf16"]),
                    T=rng.choice([1.0, 1.0, 0.7, 2.0]), grad=rng.random() < 0.75)
    D = rng.choice([64, 128, 192, 256, 256, 512, rng.randint(1, 300), 1024])
    L = _log(rng, 1, 65536)
    N = _log(rng, 1, max(1, min(8192, 8192 * 16 * 256 // (L * D))))
    return dict(op=op, N=N, L=L, D=D, dtype=rng.choice(["fp32", "bf16"]), reset=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _spread_ids(g, rows, k, V):
    """k distinct token ids a row: a random start and equal strides around the vocabulary."""
    start = torch.randint(0, V, (rows, 1), generator=g, device="cuda")
    return (start + torch.arange(k, device="cuda") * (V // k)) % V


def prepare(case, seed):
    g = _rng(seed)
    op = case["op"]
    if op == "verify":
        return _prepare_verify(case, g)
    if op == "distill":
        return _prepare_distill(case, g)
    return _prepare_scan(case, g)


def _prepare_verify(c, g):
    """The draft's logits 3 N(0, 1) with 8 tokens raised by U(8, 12), the target's those plus
    N(0, 1); tokens drawn from the draft's distribution; windows of mixed length."""
    B, K, V, m = c["B"], c["K"], c["V"], c["m"]
    U = 3.0 * _normal(g, B, K, V)
    ids = _spread_ids(g, B * K, min(8, V), V).view(B, K, -1)
    U.scatter_add_(2, ids, 8.0 + 4.0 * torch.rand(ids.shape, generator=g, device="cuda"))
    P = torch.empty(B, K + 1, V, device="cuda")
    torch.add(U, _normal(g, B, K, V), out=P[:, :K])
    P[:, K] = 3.0 * _normal(g, B, V)
    st = dict(case=c, P=torch.softmax(P, 2), Q=None, cand=None, cand_q=None)
    del P
    if m:
        top = torch.topk(U, min(m, V), dim=2)
        st["cand"] = top.indices.to(torch.int32).contiguous()
        st["cand_q"] = torch.softmax(top.values, 2).contiguous()
        race = st["cand_q"] / torch.empty_like(st["cand_q"]).exponential_(generator=g)
        slot = race.argmax(2, keepdim=True)
        st["tokens"] = torch.gather(st["cand"], 2, slot)[:, :, 0].contiguous()
    else:
        st["Q"] = torch.softmax(U, 2)
        race = st["Q"] / U.exponential_(generator=g)
        st["tokens"] = race.argmax(2).to(torch.int32)
    st["u_accept"] = torch.rand(B, K, generator=g, device="cuda")
    st["u_draw"] = torch.rand(B, generator=g, device="cuda")
    st["ell"] = torch.randint(max(0, K - 4), K + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return st


def _prepare_distill(c, g):
    """Student logits 3 N(0, 1) with the teacher's first 8 tokens raised by U(8, 12); the
    teacher's logits those plus N(0, 1), its rest up to a tenth; position weights
    exp(-k / 4) over blocks of 16, one row in ten padding (weight 0); some short lists."""
    N, V = c["N"], c["V"]
    k = min(c["k"], V)
    x = 3.0 * _normal(g, N, V)
    ids = _spread_ids(g, N, k, V)
    x.scatter_add_(1, ids[:, :8], 8.0 + 4.0 * torch.rand(N, min(k, 8), generator=g, device="cuda"))
    logits = x.to(DTYPES[c["dtype"]])
    t = torch.gather(logits, 1, ids).float() + _normal(g, N, k)
    t, order = torch.sort(t, dim=1, descending=True)
    ids = torch.gather(ids, 1, order).to(torch.int32)
    short = torch.rand(N, 1, generator=g, device="cuda") < 0.2
    slot = torch.arange(k, device="cuda")
    ids = torch.where(short & (slot >= (k + 1) // 2), torch.full_like(ids, -1), ids)
    pos = (torch.arange(N, device="cuda") % 16).float()
    w = torch.exp(-pos / 4.0) / N
    if N > 1:
        w = torch.where(torch.rand(N, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
    rest = 0.1 * torch.rand(N, generator=g, device="cuda")
    return dict(case=c, logits=logits, ids=ids.contiguous(), t=t.contiguous(), rest=rest, w=w)


def _prepare_scan(c, g):
    """Decay gates near 0.9 and input gates near 0.5 as two halves of one projection's output,
    rows of the embedding table as the input term; resets every 512 steps on average."""
    N, L, D = c["N"], c["L"], c["D"]
    dt = DTYPES[c["dtype"]]
    z = _normal(g, N, L, 2 * D)
    z[..., :D].mul_(1.5).add_(2.0)
    z = z.to(dt)
    st = dict(case=c, za=z[..., :D], zg=z[..., D:], e=_normal(g, N, L, D).to(dt), s0=_normal(g, N, D), reset=None)
    if c["reset"]:
        st["reset"] = (torch.rand(N, L, generator=g, device="cuda") < 1.0 / 512).to(torch.uint8)
    if c["op"] == "scan_grad":
        st["s"] = _scan_plain(st)[0]
        st["ds"] = _normal(g, N, L, D).to(dt)
        st["ds_last"] = _normal(g, N, D)
    return st


# ------------------------------------------------------------------------------ one pass
_ctx = None


def _context():
    """The library's context, made once by a program and kept."""
    global _ctx
    if _ctx is None:
        from rank_markov_draft_gb300 import binding
        _ctx = binding.Context(0, B_max=1, V_max=4096, K_max=1)
    return _ctx


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from rank_markov_draft_gb300 import binding
    c, ctx = st["case"], _context()
    if c["op"] == "verify":
        out = binding.verify_probs(ctx, st["P"], st["tokens"], st["u_accept"], st["u_draw"], Q=st["Q"],
                                   cand=st["cand"], cand_q=st["cand_q"], ell=st["ell"])
        return [out["n_acc"], out["next_token"], out["accept_prob"]]
    if c["op"] == "distill":
        out = binding.distill(ctx, st["logits"], st["ids"], st["t"], teacher_rest=st["rest"], row_weight=st["w"],
                              temperature=c["T"], alpha_kl=ALPHA_KL, alpha_tv=ALPHA_TV, grad=c["grad"])
        return [out["loss"], out["tv"]] + ([out["grad"]] if c["grad"] else [])
    if c["op"] == "scan":
        out = binding.rnn_scan(ctx, st["za"], st["zg"], st["e"], s0=st["s0"], reset=st["reset"])
        return [out["s"], out["s_last"]]
    out = binding.rnn_scan_grad(ctx, st["za"], st["zg"], st["e"], st["s"], st["ds"], s0=st["s0"],
                                ds_last=st["ds_last"], reset=st["reset"])
    return [out["dza"], out["dzg"], out["de"], out["ds0"]]


def _run_plain(st):
    op = st["case"]["op"]
    if op == "verify":
        return _verify_plain(st)
    if op == "distill":
        return _distill_plain(st)
    if op == "scan":
        return list(_scan_plain(st))
    return _scan_grad_plain(st)


def _verify_plain(st):
    """Comparisons and cumulative sums in 64 bits: a token is the index where a sum of up to
    151936 probabilities passes a given number."""
    c = st["case"]
    B, K, V, m = c["B"], c["K"], c["V"], c["m"]
    P, x = st["P"], st["tokens"].long()
    px = torch.gather(P[:, :K], 2, x[..., None])[..., 0].double()
    if m:
        qx = (st["cand_q"] * (st["cand"] == st["tokens"][..., None])).sum(2).double()
    else:
        qx = torch.gather(st["Q"], 2, x[..., None])[..., 0].double()
    window = torch.arange(K, device=P.device) < st["ell"][:, None]
    ok = (st["u_accept"].double() * qx < px) & window
    n_acc = torch.cumprod(ok.int(), 1).sum(1)
    row = torch.arange(B, device=P.device)
    p = P[row, n_acc].double()
    r = p
    pos = torch.clamp(n_acc, max=K - 1)
    rejected = (n_acc < st["ell"])[:, None]
    if m:
        cid = st["cand"][row, pos].long()
        cq = torch.where(rejected, st["cand_q"][row, pos].double(), 0.0)
        r = torch.scatter(p, 1, cid, torch.clamp(torch.gather(p, 1, cid) - cq, min=0.0))
    else:
        r = torch.where(rejected, torch.clamp(p - st["Q"][row, pos], min=0.0), p)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    cdf = torch.cumsum(r, 1)
    nxt = (cdf <= st["u_draw"].double()[:, None] * cdf[:, -1:]).sum(1)
    nxt = torch.where(cdf[:, -1] > 0, nxt, -1)
    prob = torch.clamp(px / qx, max=1.0)
    prob = torch.where(qx > 0, prob, (px > 0).double())
    prob = torch.where(window, prob, -1.0).float()
    return [n_acc.int(), nxt.int(), prob]


def _distill_plain(st):
    """The vocabulary in 32 bits; the teacher's few tokens in 64, where the sign of p - q
    decides a gradient."""
    c = st["case"]
    T, w = c["T"], st["w"]
    z = st["logits"].float() / T
    slot = st["ids"] >= 0
    ids = torch.where(slot, st["ids"], st["ids"][:, :1]).long()
    zi = torch.where(slot, torch.gather(st["logits"], 1, ids).double() / T, -math.inf)
    z.scatter_(1, ids, -math.inf)
    m = z.amax(1, keepdim=True)
    ez = torch.exp(z - m)
    del z
    sum_out = ez.sum(1, keepdim=True)
    top = torch.maximum(m.double(), zi.amax(1, keepdim=True))
    ei = torch.exp(zi - top)
    out = sum_out.double() * torch.exp(m.double() - top)
    total = out + ei.sum(1, keepdim=True)
    q, q_rest = ei / total, (out / total)[:, 0]
    rho = st["rest"].double()
    ti = torch.where(slot, st["t"].double() / T, -math.inf)
    pe = torch.exp(ti - ti.amax(1, keepdim=True))
    p = (1.0 - rho)[:, None] * pe / pe.sum(1, keepdim=True)
    zero = torch.zeros_like(p)
    kl = torch.where(p > 0, p * (torch.log(p) - torch.log(q)), zero).sum(1)
    kl = kl + torch.where(rho > 0, rho * (torch.log(rho) - torch.log(q_rest)), zero[:, 0])
    tv = 0.5 * ((p - q).abs().sum(1) + (rho - q_rest).abs())
    wd = w.double()
    loss = torch.where(w > 0, wd * (ALPHA_KL * kl + ALPHA_TV * tv), 0.0).float()
    tv = torch.where(w > 0, tv, 0.0).float()
    if not c["grad"]:
        return [loss, tv]
    sgn, sgn_r = torch.sign(q - p), torch.sign(q_rest - rho)
    S = (sgn * q).sum(1) + sgn_r * q_rest
    gi = ALPHA_KL * (q - p) + 0.5 * ALPHA_TV * (sgn - S[:, None]) * q
    go = ALPHA_KL * (q_rest - rho) + 0.5 * ALPHA_TV * (sgn_r - S) * q_rest
    grad = ez.mul_(((wd / T * go).float()[:, None]) / sum_out)
    # a short list's empty slots name its first token again and add nothing to it
    grad.scatter_add_(1, ids, torch.where(slot, (wd / T)[:, None] * gi, zero).float())
    grad = torch.where(w[:, None] > 0, grad, 0.0)
    return [loss, tv, grad.to(st["logits"].dtype)]


def _gates(st):
    a = 1.0 / (1.0 + torch.exp(-st["za"].float()))
    g = 1.0 / (1.0 + torch.exp(-st["zg"].float()))
    if st["reset"] is not None:
        a = a * (st["reset"] == 0)[..., None]
    return a, g


def _linear_scan(a, b):
    """y_t = a_t y_{t-1} + b_t along dimension 1 (y_{-1} = 0): spans double, log2(L) times (a
    recurrence has no form without a loop that does not overflow over long sequences)."""
    span = 1
    while span < a.shape[1]:
        b = torch.cat([b[:, :span], b[:, span:] + a[:, span:] * b[:, :-span]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return b


def _scan_plain(st):
    a, g = _gates(st)
    b = g * st["e"].float()
    b[:, 0] += a[:, 0] * st["s0"]
    s = _linear_scan(a, b)
    return s.to(st["e"].dtype), s[:, -1].clone()


def _scan_grad_plain(st):
    a, g = _gates(st)
    e, dt = st["e"].float(), st["e"].dtype
    d = st["ds"].float()
    d[:, -1] += st["ds_last"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    delta = _linear_scan(later.flip(1), d.flip(1)).flip(1)
    before = torch.cat([st["s0"][:, None], st["s"][:, :-1].float()], 1)
    dza = delta * before * a * (1.0 - a)
    dzg = delta * e * g * (1.0 - g)
    return [dza.to(dt), dzg.to(dt), (delta * g).to(dt), a[:, 0] * delta[:, 0]]


# ------------------------------------------------------------------------------ what a pass needs
def work(case):
    c = case
    if c["op"] == "verify":
        rows = 1 if c["m"] else 2  # the draw row of the target, and of the draft where it is dense
        small = c["B"] * (c["K"] * (4 * 4 + 8 * c["m"]) + 16)
        return {"bytes": c["B"] * c["V"] * 4 * rows + small, "flops": 2 * rows * c["B"] * c["V"]}
    if c["op"] == "distill":
        size = 4 if c["dtype"] == "fp32" else 2
        n = c["N"] * c["V"]
        return {"bytes": n * size * (2 if c["grad"] else 1) + c["N"] * (8 * c["k"] + 16),
                "flops": n * (8 if c["grad"] else 4)}
    size = 4 if c["dtype"] == "fp32" else 2
    n, state = c["N"] * c["L"] * c["D"], c["N"] * c["D"] * 4
    flags = c["N"] * c["L"] if c["reset"] else 0
    if c["op"] == "scan":
        return {"bytes": 4 * n * size + 2 * state + flags, "flops": 10 * n}
    return {"bytes": 8 * n * size + 3 * state + flags, "flops": 20 * n}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return _verify_exact(st)
    if op == "distill":
        return _distill_exact(st)
    return _scan_exact(st) if op == "scan" else _scan_grad_exact(st)


def _verify_exact(st):
    """min(1, p / q) of each drafted token in its window, -1 beyond it."""
    c = st["case"]
    b = torch.arange(c["B"], device="cuda").repeat_interleave(c["K"])
    k = torch.arange(c["K"], device="cuda").repeat(c["B"])
    x = st["tokens"].reshape(-1).long()
    p = st["P"][b, k, x].cpu().numpy().astype(np.float64)
    if c["m"]:
        hit = (st["cand"].reshape(-1, st["cand"].shape[2]) == x[:, None].int())
        q = st["cand_q"].reshape(hit.shape)[hit].cpu().numpy().astype(np.float64)
    else:
        q = st["Q"][b, k, x].cpu().numpy().astype(np.float64)
    prob = np.where(q <= p, np.where(p > 0, 1.0, 0.0), p / np.maximum(q, 1e-300))
    inside = k.cpu().numpy() < st["ell"].cpu().numpy()[b.cpu().numpy()]
    return [None, None, np.where(inside, prob, -1.0).reshape(c["B"], c["K"])]


def _distill_exact(st):
    """Row blocks of the whole distribution in 64 bits: softmax over all tokens, the events'
    derivative by the chain rule through it."""
    c = st["case"]
    T, N, V = c["T"], c["N"], c["V"]
    step = max(1, min(N, (1 << 26) // V))
    loss, tv, grad = [], [], []
    for r0 in range(0, N, step):
        x = st["logits"][r0:r0 + step].double() / T
        ids, t = st["ids"][r0:r0 + step].long(), st["t"][r0:r0 + step].double() / T
        rho, w = st["rest"][r0:r0 + step].double(), st["w"][r0:r0 + step].double()
        real = ids >= 0
        q = torch.softmax(x, 1)
        lq = torch.log_softmax(x, 1)
        p = (1 - rho)[:, None] * torch.softmax(t.masked_fill(~real, -math.inf), 1)
        # slots of -1 are sent to a column of their own behind the vocabulary
        at = torch.where(real, ids, V)
        p_full = torch.zeros(x.shape[0], V + 1, dtype=torch.float64, device="cuda").scatter_(1, at, p)[:, :V]
        listed_ = torch.zeros(x.shape[0], V + 1, dtype=torch.bool, device="cuda").scatter_(1, at, True)[:, :V]
        o = q.masked_fill(listed_, 0.0)
        q_rest = o.sum(1)
        kl = torch.xlogy(p_full, p_full).sum(1) - (p_full * lq).sum(1)
        kl = kl + torch.xlogy(rho, rho / q_rest)
        tv_ = 0.5 * ((p_full - q).abs().masked_fill(~listed_, 0.0).sum(1) + (rho - q_rest).abs())
        live = w != 0
        loss.append(torch.where(live, w * (ALPHA_KL * kl + ALPHA_TV * tv_), 0.0))
        tv.append(torch.where(live, tv_, 0.0))
        if c["grad"]:
            # dL/dq of each token's event, then (diag(q) - q q^T) of it
            dq = torch.where(listed_, -ALPHA_KL * p_full / q + 0.5 * ALPHA_TV * torch.sign(q - p_full),
                             (-ALPHA_KL * rho / q_rest + 0.5 * ALPHA_TV * torch.sign(q_rest - rho))[:, None])
            gq = q * dq
            gx = (gq - q * gq.sum(1, keepdim=True)) * (w / T)[:, None]
            grad.append(torch.where(live[:, None], gx, 0.0))
    return [torch.cat(loss), torch.cat(tv)] + ([torch.cat(grad)] if c["grad"] else [])


def _scan_exact(st):
    """The recurrence step by step."""
    z, zg, e = st["za"].double(), st["zg"].double(), st["e"].double()
    a, b = torch.sigmoid(z), torch.sigmoid(zg) * e
    keep = torch.ones_like(a[:, :, :1]) if st["reset"] is None else (st["reset"] == 0).double()[..., None]
    a = a * keep
    s, cur = torch.empty_like(a), st["s0"].double()
    for t in range(a.shape[1]):
        cur = torch.addcmul(b[:, t], a[:, t], cur)
        s[:, t] = cur
    return [s, cur.clone()]


def _scan_grad_exact(st):
    a, g, e = torch.sigmoid(st["za"].double()), torch.sigmoid(st["zg"].double()), st["e"].double()
    if st["reset"] is not None:
        a = a.masked_fill((st["reset"] != 0)[..., None], 0.0)
    L = a.shape[1]
    delta, cur = st["ds"].double(), st["ds_last"].double()
    for t in range(L - 1, -1, -1):
        cur = delta[:, t] + cur
        delta[:, t] = cur
        cur = a[:, t] * cur
    prev = torch.empty_like(a)
    prev[:, 0] = st["s0"].double()
    prev[:, 1:] = st["s"][:, :-1].double()
    return [delta * prev * a * (1 - a), delta * e * g * (1 - g), delta * g, cur.clone()]
