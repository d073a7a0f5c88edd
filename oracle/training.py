"""Plain 64-bit numpy statements of the training and probability-verification operators.

Straight from the formulas, with loops where the formulas have them; used by the tests only.
The error bounds returned beside the values are first-order bounds of 32-bit evaluation: the
tests add the rounding of the output type to them.
"""

from __future__ import annotations

import numpy as np

EPS32 = 2.0 ** -24  # half a step of float32, relative


def verify_probs(P, tokens, u_accept, u_draw, *, Q=None, cand=None, cand_q=None, ell=None):
    """n_acc [B], next_token [B], accept_prob [B, K] (min(1, p/q), -1 outside the window)."""
    top = float(np.finfo(np.float32).max)
    P = np.asarray(P, np.float64)
    P = np.where((P > 0) & (P <= top), P, 0.0)  # negative or not finite: nothing
    B, K = tokens.shape
    V = P.shape[2]
    n_acc, nxt = np.zeros(B, np.int64), np.zeros(B, np.int64)
    prob = np.full((B, K), -1.0)

    def draft_row(b, k):
        row = plain_row(b, k)
        return np.where(row < 0, 0.0, row)

    def plain_row(b, k):
        if cand is None:
            return np.asarray(Q[b, k], np.float64)
        row = np.zeros(V)
        for v, q in list(zip(cand[b, k], cand_q[b, k]))[::-1]:  # the first of equal ids counts
            if 0 <= v < V:
                row[v] = q
        return row

    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(B):
            n = K if ell is None else int(np.clip(ell[b], 0, K))
            j = n
            for k in range(n):
                x = tokens[b, k]
                p, q = P[b, k, x], draft_row(b, k)[x]
                prob[b, k] = min(1.0, p / q) if q > 0 else float(p > 0 and q == 0)
                if j == n and not float(u_accept[b, k]) * q < p:
                    j = k
            r = P[b, j]
            if j < n:
                r = r - draft_row(b, j)
            w = np.where(r > 0, r, 0.0)
            if not w.sum() > 0:
                w = P[b, j]
            n_acc[b] = j
            cum = np.cumsum(w)
            nxt[b] = int(np.argmax(cum > float(u_draw[b]) * cum[-1])) if cum[-1] > 0 else -1
    return n_acc, nxt, prob


def distill_row(x, ids, t, rho, w, T, a_kl, a_tv):
    """Loss, tv, gradient and gradient error bound of one row (1-D arrays)."""
    x = np.asarray(x, np.float64)
    V = x.size
    zero = (0.0, 0.0, np.zeros(V), np.zeros(V), 0.0)
    seen, slots = set(), []
    for i, v in enumerate(ids):
        if 0 <= v < V and v not in seen:
            seen.add(int(v))
            slots.append(i)
    t = np.array([float(t[i]) for i in slots])
    at = np.array([int(ids[i]) for i in slots], np.int64)
    if w == 0 or not slots or t.max() == -np.inf or x.max() == -np.inf:
        return zero
    with np.errstate(divide="ignore", invalid="ignore"):
        rho = min(max(float(rho), 0.0), 1.0)
        z = x / T
        ez = np.exp(z - z.max())
        q = ez / ez.sum()
        out = np.ones(V, bool)
        out[at] = False
        q_rest = q[out].sum()
        eo = np.exp(z[out] - (z[out].max() if out.any() and z[out].max() > -np.inf else 0.0))
        o = eo / eo.sum() if eo.sum() > 0 else eo
        pt = np.exp((t - t.max()) / T)
        p = (1 - rho) * pt / pt.sum()
        qi = q[at]
        kl = sum(pi * (np.log(pi) - np.log(v)) for pi, v in zip(p, qi) if pi > 0)
        if rho > 0:
            kl += rho * (np.log(rho) - np.log(q_rest))
        tv = 0.5 * (np.abs(p - qi).sum() + abs(rho - q_rest))
        loss = w * ((a_kl * kl if a_kl else 0.0) + a_tv * tv)
        sgn, sgn_r = np.sign(qi - p), np.sign(q_rest - rho)
        S = (sgn * qi).sum() + sgn_r * q_rest
        g = np.zeros(V)
        g[at] = w / T * (a_kl * (qi - p) + 0.5 * a_tv * (sgn - S) * qi)
        g[out] = w / T * o * (a_kl * (q_rest - rho) + 0.5 * a_tv * (sgn_r - S) * q_rest)
    # relative error of a softmax entry in 32 bits: the exponent's three roundings (difference,
    # scale, product) times its size, the exponential, and the sum's tree (2 + log2 V deep)
    live = z[z > -np.inf]
    span = min(max(live.max() - live.min(), (t.max() - t[t > -np.inf].min()) / T), 104.0)
    E = EPS32 * (2 * (3 * span + 4) + 2 * (2 + np.log2(max(V, 2))) + 8)
    size = np.zeros(V)
    size[at] = abs(a_kl) * (qi + p) + abs(a_tv) * 2 * qi
    size[out] = o * (abs(a_kl) * (q_rest + rho) + abs(a_tv) * 2 * q_rest)
    bound = abs(w) / T * np.abs(size) * E
    return loss, tv, g, bound, E


def sigmoid(z):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def _gate_error(z):
    """Relative error of 1 / (1 + 2^(-z log2 e)) in 32 bits: the exponent's rounding times its
    size, the exponential, the sum and the division."""
    return EPS32 * (2 * np.minimum(np.abs(np.asarray(z, np.float64)), 104.0) + 12)


def rnn_scan(za, zg, e, s0=None, reset=None):
    """States s [N, L, D] in 64 bits and a bound of their 32-bit error."""
    a, e = sigmoid(za), np.asarray(e, np.float64)
    g = np.ones_like(a) if zg is None else sigmoid(zg)
    rel = _gate_error(za) + (0 if zg is None else _gate_error(zg)) + 4 * EPS32
    if reset is not None:
        a = np.where(np.asarray(reset, bool)[..., None], 0.0, a)
    N, L, D = a.shape
    s, err = np.empty((N, L, D)), np.empty((N, L, D))
    cur = np.zeros((N, D)) if s0 is None else np.asarray(s0, np.float64)
    size, bad = np.abs(cur), np.zeros((N, D))
    for t in range(L):
        b = g[:, t] * e[:, t]
        drop = a[:, t] == 0
        with np.errstate(invalid="ignore"):
            cur = np.where(drop, b, a[:, t] * cur + b)
            size = np.where(drop, np.abs(b), a[:, t] * size + np.abs(b))
            bad = np.where(drop, 0.0, a[:, t] * bad) + rel[:, t] * size
        s[:, t], err[:, t] = cur, bad
    return s, err


def rnn_scan_grad(za, zg, e, s, ds, s0=None, ds_last=None, reset=None):
    """dza, dzg, de, ds0 in 64 bits, each with a bound of its 32-bit error."""
    a, e = sigmoid(za), np.asarray(e, np.float64)
    g = np.ones_like(a) if zg is None else sigmoid(zg)
    ga = _gate_error(za)
    gg = np.zeros_like(a) if zg is None else _gate_error(zg)
    na = sigmoid(-np.asarray(za, np.float64))
    ng = np.zeros_like(a) if zg is None else sigmoid(-np.asarray(zg, np.float64))
    if reset is not None:
        a = np.where(np.asarray(reset, bool)[..., None], 0.0, a)
    s, ds = np.asarray(s, np.float64), np.asarray(ds, np.float64)
    N, L, D = a.shape
    out = [np.zeros((N, L, D)) for _ in range(3)]
    bound = [np.zeros((N, L, D)) for _ in range(3)]
    delta = np.zeros((N, D)) if ds_last is None else np.asarray(ds_last, np.float64)
    size, bad = np.abs(delta), np.zeros((N, D))
    for t in range(L - 1, -1, -1):
        delta = delta + ds[:, t]
        size = size + np.abs(ds[:, t])
        bad = bad + 4 * EPS32 * size
        prev = s[:, t - 1] if t > 0 else (np.zeros((N, D)) if s0 is None else np.asarray(s0, np.float64))
        drop = a[:, t] == 0
        with np.errstate(invalid="ignore"):
            for i, f, rel in ((0, np.where(drop, 0.0, prev * a[:, t] * na[:, t]), 2 * ga[:, t]),
                              (1, e[:, t] * g[:, t] * ng[:, t], 2 * gg[:, t]), (2, g[:, t], gg[:, t])):
                out[i][:, t] = delta * f
                bound[i][:, t] = np.abs(f) * (bad + size * (rel + 6 * EPS32))
            delta = np.where(drop, 0.0, a[:, t] * delta)
            size = np.where(drop, 0.0, a[:, t] * size)
            bad = np.where(drop, 0.0, a[:, t] * bad) + (ga[:, t] + 2 * EPS32) * size
    return (*out, delta), (*bound, bad)
