"""Cases of the training step's operators around the heads, and their plain forms.

What a step that trains a drafting head does beside the recurrence and the distillation:

* ``embed`` / ``embed_grad``: rows of the Markov table W1 by token, scaled and converted, and the
  table's gradient, the rows' gradients summed token by token;
* ``clip_grads``: the norm of all gradients together and their scaling down to a limit;
* ``linear`` / ``linear_grad``: act(x W + bias) + residual in one product (the gates h Wa, h Wg,
  and the logits U + s W2), and the gradients of x, W and the bias.

``run`` computes a case in elementary torch operations (``own`` false) or through the library
(``own`` true).  ``exact`` restates each definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # serving: the last token of each request, from the served table
        dict(name="embed one token", op="embed", N=128, V=151936, D=256, table="bf16", out="bf16", scale=1.0),
        # the predecessors of a training batch (8192 blocks of 16), from the fp32 master table
        dict(name="embed blocks", op="embed", N=131072, V=151936, D=256, table="fp32", out="bf16", scale=1.0),
        # a short batch, odd sizes: the call's latency
        dict(name="embed grad few odd rows", op="embed_grad", N=77, V=32003, D=100, de="fp32", grad="fp32", scale=10.0),
        # the training batch backward
        dict(name="embed grad blocks", op="embed_grad", N=131072, V=151936, D=256, de="bf16", grad="fp32", scale=1.0),
        # rows as wide as a backbone's hidden state
        dict(name="embed grad wide", op="embed_grad", N=16384, V=16000, D=2048, de="bf16", grad="bf16", scale=45.25),
        # a model of many small tensors of both types
        dict(name="clip many tensors", op="clip", count=48, total=12000000, types="mixed", limit=1.0),
        # the RNN head of the serving vocabulary: W1, W2, Wa, Wg
        dict(name="clip head", op="clip", count=4, total=2 * 256 * (151936 + 4096), types="fp32", limit=1.0),
        # the gate of one position of the serving batch
        dict(name="linear gate of a position", op="linear", M=128, K=4096, N=256, act="sigmoid", bias=True,
             residual=None, out="bf16"),
        # both gates of the RNN head over a training batch (128 blocks of 16)
        dict(name="linear rnn gates", op="linear", M=2048, K=4096, N=512, act=None, bias=True, residual=None, out="bf16"),
        # the calibrated logits U + s W2 of that batch, for a mixed-precision loss
        dict(name="linear logits", op="linear", M=2048, K=256, N=151936, act=None, bias=False, residual="fp32", out="bf16"),
        # a gate backward on odd sizes
        dict(name="linear grad odd gate", op="linear_grad", M=333, K=1000, N=250, act="sigmoid", bias=True, dy="bf16"),
        # the logits backward: gradients of the states and of W2
        dict(name="linear grad logits", op="linear_grad", M=2048, K=256, N=151936, act=None, bias=False, dy="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "clip", "linear", "linear", "linear_grad", "linear_grad"])
    if op in ("embed", "embed_grad"):
        D = rng.choice([64, 128, 256, 256, 512, 1024, 2048, rng.randint(1, 300)])
        V = _log(rng, 1000, max(1001, min(151936, 151936 * 256 // D)))
        N = _log(rng, 1, max(1, min(131072, 131072 * 256 // D)))
        types = [rng.choice(["fp32", "bf16"]) for _ in range(2)]
        names = ("table", "out") if op == "embed" else ("de", "grad")
        return dict(op=op, N=N, V=V, D=D, scale=rng.choice([1.0, 1.0, D ** 0.5]), **dict(zip(names, types)))
    if op == "clip":
        total = _log(rng, 1000, 2 * 256 * (151936 + 4096))
        return dict(op=op, count=_log(rng, 1, 60), total=total, types=rng.choice(["fp32", "bf16", "mixed"]),
                    limit=rng.choice([0.5, 1.0, 1e6]))
    # a table of logits (few inputs, many outputs) or a projection
    if rng.random() < 0.5:
        K, N = rng.choice([64, 128, 256, 256, rng.randint(1, 256)]), _log(rng, 1000, 151936)
        N = N // 8 * 8 if rng.random() < 0.7 else N
    else:
        K, N = _log(rng, 1, 4096), _log(rng, 1, 4096)
        K, N = (K, N) if rng.random() < 0.5 else (max(64, K // 64 * 64), max(64, N // 64 * 64))
    act = rng.choice([None, None, "sigmoid", "silu", "gelu", "tanh", "relu"])
    case = dict(op=op, M=0, K=K, N=N, act=act, bias=rng.random() < 0.5)
    if op == "linear":
        case.update(residual=rng.choice([None, "fp32", "bf16"]), out=rng.choice(["fp32", "bf16"]))
    else:
        case.update(dy=rng.choice(["bf16", "bf16", "fp32"]))
    # rows up to half of the large cases' products and of their outputs (all of the plainest gradient's)
    share = 2 if op == "linear" or act or case["dy"] == "fp32" else 1
    case["M"] = _log(rng, 1, max(1, min(8192, 2048 * 151936 // (share * N), 2048 * 256 * 151936 // (share * K * N))))
    return case


# ------------------------------------------------------------------------------ inputs
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, N, V):
    """Token ids as text has them: the id's probability falls as 1 / (id + 1); one position in
    fifty is padding (-1)."""
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    return torch.where(torch.rand(N, generator=g, device="cuda") < 0.02, -1, ids).to(torch.int32)


def _sizes(count, total):
    """Element counts of a model's tensors: a few large ones, most of them small, odd ones too."""
    if count == 4 and total % 512 == 0 and total // 512 > 4096:  # W1, W2, Wa, Wg
        V = total // 512 - 4096
        return [256 * V, 256 * V, 256 * 4096, 256 * 4096]
    weight = [1.0 / (1 + (i * 7919) % count) for i in range(count)]
    s = sum(weight)
    return [max(1, int(total * w / s)) for w in weight]


def prepare(case, seed):
    c, g = case, _rng(seed)
    if c["op"] == "embed":
        return dict(case=c, table=(0.02 * _normal(g, c["V"], c["D"])).to(DTYPES[c["table"]]), ids=_tokens(g, c["N"], c["V"]))
    if c["op"] == "embed_grad":
        return dict(case=c, ids=_tokens(g, c["N"], c["V"]), de=(_normal(g, c["N"], c["D"]) / c["N"]).to(DTYPES[c["de"]]))
    if c["op"] == "clip":
        types = {"fp32": ["fp32"], "bf16": ["bf16"], "mixed": ["fp32", "bf16"]}[c["types"]]
        grads = [(0.01 * _normal(g, n)).to(DTYPES[types[i % len(types)]]) for i, n in enumerate(_sizes(c["count"], c["total"]))]
        # the raw gradients are kept (for the statistics that a trainer logs): the clipped ones go beside them
        return dict(case=c, grads=grads, out=[torch.empty_like(t) for t in grads])
    M, K, N = c["M"], c["K"], c["N"]
    st = dict(case=c, x=_normal(g, M, K).bfloat16(), W=(_normal(g, K, N) / K ** 0.5).bfloat16(), bias=None, residual=None, pre=None)
    if c["bias"]:
        st["bias"] = 0.5 * _normal(g, N)
    if c["op"] == "linear":
        if c["residual"]:
            st["residual"] = (3.0 * _normal(g, M, N)).to(DTYPES[c["residual"]])
        return st
    # gradients of logits: a softmax less a few tokens' shares, averaged over the rows
    dy = torch.softmax(3.0 * _normal(g, M, N), 1)
    hit = torch.randint(0, N, (M, 4), generator=g, device="cuda")
    st["dy"] = (dy.scatter_add_(1, hit, torch.full((M, 4), -0.25, device="cuda")) / M).to(DTYPES[c["dy"]])
    if c["act"]:
        st["pre"] = _normal(g, M, N).to(torch.bfloat16)
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
    if c["op"] == "embed":
        return binding.embed(ctx, st["table"], st["ids"], scale=c["scale"], dtype=DTYPES[c["out"]])
    if c["op"] == "embed_grad":
        return binding.embed_grad(ctx, st["ids"], st["de"], c["V"], scale=c["scale"], dtype=DTYPES[c["grad"]])
    if c["op"] == "clip":
        return [binding.clip_grads(ctx, st["grads"], c["limit"], out=st["out"])] + st["out"]
    if c["op"] == "linear":
        return binding.linear(ctx, st["x"], st["W"], bias=st["bias"], act=c["act"], residual=st["residual"],
                              dtype=DTYPES[c["out"]])["y"]
    out = binding.linear_grad(ctx, st["x"], st["W"], st["dy"], act=c["act"], pre=st["pre"], dbias=c["bias"])
    return [out["dx"], out["dW"]] + ([out["dbias"]] if c["bias"] else [])


def _run_plain(st):
    c = st["case"]
    if c["op"] == "embed":
        rows = st["table"][st["ids"].clamp(min=0).long()].float() * c["scale"]
        return torch.where(st["ids"][:, None] >= 0, rows, 0.0).to(DTYPES[c["out"]])
    if c["op"] == "embed_grad":
        grad = torch.zeros(c["V"] + 1, c["D"], device="cuda")
        # padding goes to a row of its own behind the table
        grad.index_add_(0, torch.where(st["ids"] >= 0, st["ids"], c["V"]), st["de"].float())
        return (grad[:c["V"]] * c["scale"]).to(DTYPES[c["grad"]])
    if c["op"] == "clip":
        norm = torch.sqrt(sum((t.float() * t.float()).sum(dtype=torch.float64) for t in st["grads"])).float()
        coef = torch.clamp(c["limit"] / (norm + 1e-6), max=1.0)
        return [norm] + [(t.float() * coef).to(t.dtype) for t in st["grads"]]
    return _linear_plain(st) if c["op"] == "linear" else _linear_grad_plain(st)


def _linear_plain(st):
    c = st["case"]
    z = st["x"].float() @ st["W"].float()
    if c["bias"]:
        z = z + st["bias"]
    if c["act"] == "sigmoid":
        z = 1.0 / (1.0 + torch.exp(-z))
    elif c["act"] == "tanh":
        z = torch.tanh(z)
    elif c["act"] == "relu":
        z = torch.clamp(z, min=0.0)
    elif c["act"] == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif c["act"] == "gelu":
        z = 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if c["residual"]:
        z = z + st["residual"].float()
    return z.to(DTYPES[c["out"]])


def _linear_grad_plain(st):
    c = st["case"]
    dz = st["dy"].float()
    if c["act"]:
        z = st["pre"].float()
        if c["act"] == "sigmoid":
            s = 1.0 / (1.0 + torch.exp(-z))
            dz = dz * (s * (1.0 - s))
        elif c["act"] == "tanh":
            t = torch.tanh(z)
            dz = dz * (1.0 - t * t)
        elif c["act"] == "relu":
            dz = dz * (z > 0)
        elif c["act"] == "silu":
            s = 1.0 / (1.0 + torch.exp(-z))
            dz = dz * (s * (1.0 + z * (1.0 - s)))
        else:
            dz = dz * (0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / (2.0 * math.pi)) ** 0.5)
    dx = (dz @ st["W"].float().T).bfloat16()
    dW = st["x"].float().T @ dz
    return [dx, dW] + ([dz.sum(0)] if c["bias"] else [])


# ------------------------------------------------------------------------------ what a pass needs
def work(case):
    c = case
    size = {"fp32": 4, "bf16": 2}
    if c["op"] == "embed":
        rows = min(c["N"], c["V"])  # a row that several tokens name is read once
        return {"bytes": c["D"] * (rows * size[c["table"]] + c["N"] * size[c["out"]]) + 4 * c["N"], "flops": c["N"] * c["D"]}
    if c["op"] == "embed_grad":
        return {"bytes": c["D"] * (c["N"] * size[c["de"]] + c["V"] * size[c["grad"]]) + 4 * c["N"], "flops": c["N"] * c["D"]}
    if c["op"] == "clip":
        each = {"fp32": 4, "bf16": 2, "mixed": 3}[c["types"]]
        return {"bytes": 2 * each * c["total"], "flops": 3 * c["total"]}
    M, K, N = c["M"], c["K"], c["N"]
    if c["op"] == "linear":
        each = size[c["out"]] + (size[c["residual"]] if c["residual"] else 0)
        return {"bytes": 2 * K * (M + N) + M * N * each + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    each = size[c["dy"]] + (2 if c["act"] else 0)
    return {"bytes": 2 * K * (M + N) + M * N * each + 2 * M * K + 4 * K * N + (4 * N if c["bias"] else 0),
            "flops": 4 * M * N * K}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "embed":
        padded = torch.cat([st["table"].double(), torch.zeros(1, c["D"], dtype=torch.float64, device="cuda")])
        return padded.index_select(0, st["ids"].long() % (c["V"] + 1)) * c["scale"]  # -1: the row behind the table
    if c["op"] == "embed_grad":
        return _embed_grad_exact(st)
    if c["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(t.double(), t.double())) for t in st["grads"]))
        factor = min(1.0, c["limit"] / (norm + 1e-6))
        return [np.float64(norm)] + [t.double() * factor for t in st["grads"]]
    return _linear_exact(st) if c["op"] == "linear" else _linear_grad_exact(st)


def _embed_grad_exact(st):
    """Rows in the order of their tokens, differences of their running sum at the tokens' ends;
    blocks of channels, so that the running sums fit."""
    c = st["case"]
    order = torch.argsort(st["ids"])
    ends = torch.searchsorted(st["ids"][order].long().contiguous(), torch.arange(-1, c["V"], device="cuda"), right=True)
    out = []
    for d0 in range(0, c["D"], 256):
        total = torch.cumsum(st["de"][order, d0:d0 + 256].double(), 0)
        total = torch.cat([torch.zeros_like(total[:1]), total])
        out.append(c["scale"] * torch.diff(total[ends], dim=0))
    return torch.cat(out, 1)


def _act(name, z):
    """Value and derivative of an activation in 64 bits."""
    if name is None:
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.relu(z), (z > 0).double()
    if name == "tanh":
        return torch.tanh(z), 1 / torch.cosh(z) ** 2
    s = torch.sigmoid(z)
    if name == "sigmoid":
        return s, s * torch.sigmoid(-z)
    if name == "silu":
        return z * s, s + z * s * torch.sigmoid(-z)
    cdf = torch.special.ndtr(z)
    return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def _linear_exact(st):
    c = st["case"]
    z = torch.mm(st["x"].double(), st["W"].double())
    if c["bias"]:
        z += st["bias"].double()
    if c["act"]:
        z = _act(c["act"], z)[0]
    return z if st["residual"] is None else z.add_(st["residual"])


def _linear_grad_exact(st):
    c = st["case"]
    dz = st["dy"].double()
    if c["act"]:
        dz = dz * _act(c["act"], st["pre"].double())[1]
    out = [torch.mm(dz, st["W"].double().t()), torch.mm(st["x"].double().t(), dz)]
    return out + ([dz.sum(0)] if c["bias"] else [])
