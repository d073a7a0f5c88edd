"""Plain 64-bit torch statements of the training step's operators around the heads.

Straight from the formulas, on whatever device the inputs are; used by the tests only.  The error
bounds returned beside the values are first-order bounds of the operators' arithmetic (32-bit sums,
matrix products in steps of 16); the tests add the rounding of the output type to them.
"""

from __future__ import annotations

import math

import torch

EPS32 = 2.0 ** -24  # half a step of float32, relative
ACTS = (None, "sigmoid", "tanh", "relu", "silu", "gelu")


def embed(table, ids, scale=1.0):
    """scale * table[ids] [..., D] (negative ids: zeros) and its bound (one rounded product)."""
    rows = torch.where((ids >= 0)[..., None], table.double()[ids.clamp(min=0).long()], 0.0) * scale
    return rows, rows.abs() * EPS32


def embed_grad(ids, de, V, scale=1.0, before=None):
    """Gradient of the table (added to `before`); a sum of n terms in any order is off by at most
    n - 1 roundings of the sum of their sizes, then come the scale and the addition."""
    flat, d = ids.flatten().long(), de.double().flatten(0, -2)
    keep = (flat >= 0) & (flat < V)
    flat, d = flat[keep], d[keep]
    s = torch.zeros(V, d.shape[1], dtype=torch.float64, device=d.device).index_add_(0, flat, d)
    size = torch.zeros_like(s).index_add_(0, flat, d.abs())
    n = torch.bincount(flat, minlength=V)[:, None].double()
    out, bound = scale * s, abs(scale) * size * (n + 1) * EPS32
    if before is not None:
        out = out + before.double()
        bound = bound + out.abs() * EPS32
    return out, bound


def clip(grads, max_norm):
    """The common norm and the scaled tensors."""
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    factor = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g.double() * factor for g in grads]


def act(name, z):
    if name is None:
        return z
    return {"sigmoid": lambda: 1 / (1 + torch.exp(-z)), "tanh": lambda: torch.tanh(z), "relu": lambda: torch.clamp(z, min=0),
            "silu": lambda: z / (1 + torch.exp(-z)), "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2))}[name]()


def slope(name, z):
    """d act / d z (0 at relu's kink), without a difference from 1 that a far argument leaves nothing of."""
    if name is None:
        return torch.ones_like(z)
    e = torch.exp(-z.abs())
    s = torch.where(z < 0, e, 1.0) / (1 + e)
    return {"sigmoid": lambda: e / (1 + e) ** 2, "tanh": lambda: 4 * e ** 2 / (1 + e ** 2) ** 2, "relu": lambda: (z > 0).double(),
            "silu": lambda: s * (1 + z * torch.where(z < 0, 1.0, e) / (1 + e)),
            "gelu": lambda: 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[name]()


def product(a, b, parts=1):
    """a b and its bound: the terms (of `parts` exact numbers an element) are exact, their sum is taken 16 at a
    time, each step rounded (or cut: a whole step of float32) relative to what has been added up so far,
    for 512 terms at most; up to 64 sums of these, and these, are added up in float32."""
    K = parts * a.shape[-1]
    cuts, adds = min(K / 16, 32) + 16, min(K / 64, 64) + K / 512
    return a @ b, (2 * cuts + adds) * EPS32 * (a.abs() @ b.abs())


def linear(x, W, bias=None, name=None, residual=None):
    """y, pre and their bounds.  No activation here is steeper than 1.13; the functions' own values
    are taken to be right to 8 roundings."""
    z, dz = product(x.double(), W.double())
    if bias is not None:
        z = z + bias.double()
        dz = dz + z.abs() * EPS32
    y = act(name, z)
    dy = 1.13 * dz + (0 if name is None else 8 * EPS32 * (y.abs() + (z.abs() * y.abs()).clamp(max=1) + EPS32))
    if residual is not None:
        y = y + residual.double()
        dy = dy + y.abs() * EPS32
    return y, z, dy, dz


def linear_grad(x, W, dy, name=None, pre=None):
    """dx, dW, dbias and their bounds.  dz is right to the activation's roundings; where it is no
    bf16 number it enters the products as three, 2^-25 of itself at most away."""
    d = dy.double()
    err = torch.zeros_like(d)
    if name is not None:
        k = slope(name, pre.double())
        # the functions' own roundings and a few products'; SiLU's and GELU's slopes are sums of two terms
        # of up to 1.13 that may cancel
        err = d.abs() * (24 if name in ("silu", "gelu") else 12 * k) * EPS32
        d = d * k
    rest, parts = err.clone(), 1
    if name is not None or dy.dtype != torch.bfloat16:
        rest, parts = rest + d.abs() * 2.0 ** -25, 3
    Wd, xd = W.double(), x.double()
    dx, ex = product(d, Wd.T, parts)
    dW, ew = product(xd.T, d, parts)
    db, eb = d.sum(0), d.abs().sum(0) * d.shape[0] * EPS32 + err.sum(0)
    return dict(dx=(dx, ex + rest @ Wd.abs().T), dW=(dW, ew + xd.abs().T @ rest), dbias=(db, eb))
