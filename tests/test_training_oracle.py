"""The 64-bit statements of the training and verification operators against hand values,
differences and sampling (CPU), and the host-side refusals of the calls."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import training as tr
from rank_markov_draft_gb300 import binding, build

KW = dict(T=0.8, a_kl=0.3, a_tv=0.9)


def _row(seed, V=23, k=5):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(V)[:k]
    return rng.normal(0, 2, V), ids, rng.normal(0, 2, k), rng.uniform(0, 0.4)


@pytest.mark.parametrize("seed", range(4))
def test_distill_gradient_equals_differences(seed):
    x, ids, t, rho = _row(seed)
    _, _, g, _, _ = tr.distill_row(x, ids, t, rho, 1.7, **KW)
    h = 1e-6
    for v in range(x.size):
        up, dn = x.copy(), x.copy()
        up[v] += h
        dn[v] -= h
        d = (tr.distill_row(up, ids, t, rho, 1.7, **KW)[0] - tr.distill_row(dn, ids, t, rho, 1.7, **KW)[0]) / (2 * h)
        assert abs(d - g[v]) < 1e-8  # central differences: h^2 times a third derivative of order one


def test_distill_of_equal_distributions_is_zero():
    rng = np.random.default_rng(3)
    x = rng.normal(0, 2, 11)
    q = np.exp(x) / np.exp(x).sum()
    ids = np.array([4, 0, 7])
    loss, tv, g, _, _ = tr.distill_row(x, ids, x[ids], 1 - q[ids].sum(), 1.0, 1.0, 1.0, 0.0)
    assert abs(loss) < 1e-14 and tv < 1e-14 and np.abs(g).max() < 1e-15


def test_distill_tv_is_at_most_the_vocabularys():
    """One event for the rest hides what moves inside it: 1 - tv is at least the acceptance
    probability sum min(p, q), and equals it where the teacher's list is the vocabulary."""
    rng = np.random.default_rng(4)
    for k in (1, 3, 11):
        x, t = rng.normal(0, 2, 11), rng.normal(0, 2, 11)
        q, p = np.exp(x) / np.exp(x).sum(), np.exp(t) / np.exp(t).sum()
        ids = np.argsort(-t)[:k]
        accept = np.minimum(p, q).sum()
        tv = tr.distill_row(x, ids, t[ids], 1 - p[ids].sum(), 1.0, 1.0, 1.0, 1.0)[1]
        assert 1 - tv >= accept - 1e-15 and (k == 11) == (abs(1 - tv - accept) < 1e-12)


def test_distill_rows_without_anything_are_zero():
    x, ids, t, rho = _row(5)
    for case in (dict(w=0.0), dict(ids=np.full_like(ids, -1)), dict(t=np.full_like(t, -np.inf)),
                 dict(x=np.full_like(x, -np.inf))):
        a = dict(x=x, ids=ids, t=t, rho=rho, w=1.0) | case
        loss, tv, g, _, _ = tr.distill_row(**a, **KW)
        assert loss == 0 and tv == 0 and not g.any()


def test_scan_gradient_equals_differences():
    rng = np.random.default_rng(7)
    N, L, D = 2, 5, 3
    za, zg, e = (rng.normal(0, 1, (N, L, D)) for _ in range(3))
    s0, wl = rng.normal(0, 1, (N, D)), rng.normal(0, 1, (N, D))
    ds = rng.normal(0, 1, (N, L, D))
    reset = np.zeros((N, L), np.uint8)
    reset[0, 3] = 1

    def f(za, zg, e, s0):
        s, _ = tr.rnn_scan(za, zg, e, s0, reset)
        return (s * ds).sum() + (s[:, -1] * wl).sum()

    s, _ = tr.rnn_scan(za, zg, e, s0, reset)
    grads, _ = tr.rnn_scan_grad(za, zg, e, s, ds, s0, wl, reset)
    args = [za, zg, e, s0]
    for i, g in enumerate(grads):
        for at in np.ndindex(*args[i].shape):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += 1e-6
            dn[i][at] -= 1e-6
            assert abs((f(*up) - f(*dn)) / 2e-6 - g[at]) < 1e-8


def test_scan_reset_drops_whatever_came_before():
    za = np.zeros((1, 3, 1))
    e = np.array([[[np.inf], [2.0], [4.0]]])
    s, _ = tr.rnn_scan(za, None, e, np.array([[np.nan]]), np.array([[1, 1, 0]], np.uint8))
    assert s[0, :, 0].tolist() == [np.inf, 2.0, 5.0]


def test_verification_keeps_the_target_distribution():
    """Committed first tokens of many blocks follow the target whatever the draft."""
    rng = np.random.default_rng(11)
    n, V = 40000, 5
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    P = np.broadcast_to(p, (n, 2, V))
    tok = rng.choice(V, size=(n, 1), p=q).astype(np.int32)
    acc, nxt, _ = tr.verify_probs(P, tok, rng.random((n, 1)), rng.random(n), Q=np.broadcast_to(q, (n, 1, V)))
    first = np.where(acc > 0, tok[:, 0], nxt)
    chi2 = ((np.bincount(first, minlength=V) - n * p) ** 2 / (n * p)).sum()
    assert chi2 < 23.5  # 0.9999 quantile at 4 degrees of freedom


def test_verification_edge_rows():
    P = np.array([[[0.25, 0.75, 0.0], [0.0, 0.0, 0.0]]])
    u = np.array([[0.5]])
    same = P[:, :1]
    # equal rows: accepted, and the row after the window has no mass
    assert [x.tolist() for x in tr.verify_probs(P, np.array([[1]]), u, np.array([0.9]), Q=same)[:2]] == [[1], [-1]]
    # a token the target gives nothing is rejected; nothing is left over, so the target's row
    acc, nxt, prob = tr.verify_probs(P, np.array([[2]]), u, np.array([0.9]), Q=same)
    assert (acc[0], nxt[0], prob[0, 0]) == (0, 1, 0.0)
    # candidates: the first of equal ids counts
    acc, nxt, prob = tr.verify_probs(P, np.array([[0]]), u, np.array([0.0]), cand=np.array([[[0, 0, -1]]]),
                                     cand_q=np.array([[[0.5, 0.1, 9.0]]]))
    assert (acc[0], nxt[0], prob[0, 0]) == (0, 1, 0.5)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, -0.5])
def test_verification_of_entries_that_are_no_probabilities(bad):
    """A drafted token whose p is no probability is rejected (0); one whose q is negative counts
    as undrafted, and one whose q is infinite or NaN is rejected and not drawn either."""
    p = np.array([[[0.5, 0.5], [0.5, 0.5]]])
    q = np.array([[[0.5, 0.5]]])
    token, u, u_draw = np.array([[0]]), np.array([[0.25]]), np.array([0.0])
    broken = p.copy()
    broken[0, 0, 0] = bad
    with_q = lambda x: np.array([[[x, 0.5]]])  # noqa: E731
    acc, nxt, prob = tr.verify_probs(broken, token, u, u_draw, Q=q)
    assert (acc[0], nxt[0], prob[0, 0]) == (0, 1, 0.0)
    acc, nxt, prob = tr.verify_probs(p, token, u, u_draw, Q=with_q(bad))
    assert (acc[0], prob[0, 0]) == ((1, 1.0) if bad < 0 else (0, 0.0))
    # both: rejected, and the target's other token is drawn, its own mass being left
    acc, nxt, prob = tr.verify_probs(broken, token, u, u_draw, Q=with_q(bad))
    assert (acc[0], nxt[0], prob[0, 0]) == (0, 1, 0.0)
    # a negative q adds nothing to what is left over
    acc, nxt, _ = tr.verify_probs(np.array([[[0.0, 0.5, 0.5], [1.0, 0.0, 0.0]]]), token, u, np.array([0.6]),
                                  Q=np.array([[[0.5, -8.0, 0.0]]]))
    assert (acc[0], nxt[0]) == (0, 2)


# ------------------------------------------------------------------ host-side refusals
P = ctypes.c_void_p
GOOD, ODD = P(0x1000), P(0x1002)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_verify_probs_argument_checks(lib):
    E = binding
    v = lambda p=GOOD, Q=GOOD, cand=None, cq=None, m=0, B=4, K=16, V=4097, tok=GOOD, nxt=GOOD: (  # noqa: E731
        lib.dspark_verify_probs(None, p, Q, cand, cq, m, tok, GOOD, GOOD, None, B, K, V, GOOD, nxt, None, None))
    assert v() == E.INVALID_ARG  # valid, no context
    assert v(K=65) == E.UNSUPPORTED
    assert v(V=(1 << 18) + 1) == E.UNSUPPORTED
    assert v(Q=None, cand=GOOD, cq=GOOD, m=257) == E.UNSUPPORTED
    for bad in (dict(p=None), dict(Q=None), dict(cand=GOOD), dict(m=4), dict(m=-1), dict(Q=None, cand=GOOD, m=4),
                dict(B=0), dict(K=0), dict(V=0), dict(tok=None), dict(nxt=None), dict(p=ODD)):
        assert v(**({"V": 1 << 19} | bad)) == E.INVALID_ARG, bad  # found before the size


def test_distill_argument_checks(lib):
    E = binding
    d = lambda x=GOOD, dt=0, ld=4097, k=8, N=4, V=4097, T=1.0, a=0.1, b=0.9, loss=GOOD, g=None, ldg=4097: (  # noqa: E731
        lib.dspark_distill(None, x, dt, ld, GOOD, GOOD, k, None, None, N, V, T, a, b, loss, None, g, ldg, None))
    assert d() == E.INVALID_ARG  # valid, no context
    assert d(V=(1 << 18) + 1, ld=1 << 19) == E.UNSUPPORTED
    assert d(k=257) == E.UNSUPPORTED
    assert d(N=1 << 31) == E.UNSUPPORTED
    big = dict(k=257)  # a size that only a call past the other checks reports
    for bad in (dict(x=None), dict(dt=2), dict(ld=4096), dict(N=0), dict(V=0), dict(loss=None), dict(g=GOOD, ldg=4096),
                dict(g=GOOD, ld=5000), dict(k=0), dict(T=0.0), dict(T=-1.0), dict(T=float("nan")),
                dict(T=float("inf")), dict(a=float("inf")), dict(b=float("nan")), dict(x=ODD),
                dict(x=P(0x1001), dt=1)):
        assert d(**(big | bad)) == E.INVALID_ARG, bad


def test_scan_argument_checks(lib):
    E = binding
    f = lambda za=GOOD, zg=GOOD, e=GOOD, dt=0, la=64, lg=64, le=64, N=2, L=3, D=64, s=GOOD: (  # noqa: E731
        lib.dspark_rnn_scan(None, za, zg, e, dt, la, lg, le, None, None, N, L, D, s, None, None))
    assert f() == E.INVALID_ARG  # valid, no context
    assert f(N=1 << 20, L=1 << 11) == E.UNSUPPORTED
    assert f(N=1 << 25, L=1) == E.UNSUPPORTED
    assert f(la=1 << 31) == E.UNSUPPORTED
    big = dict(N=1 << 25, L=1)
    for bad in (dict(za=None), dict(e=None), dict(dt=7), dict(N=0), dict(L=0), dict(D=0), dict(la=63), dict(lg=63),
                dict(le=63), dict(za=ODD), dict(zg=ODD), dict(e=P(0x1001), dt=1)):
        assert f(**(big | bad)) == E.INVALID_ARG, bad
    g = lambda zg=GOOD, s=GOOD, ds=GOOD, da=GOOD, dg=GOOD, de=GOOD, lda=64, ldg=64, N=2: (  # noqa: E731
        lib.dspark_rnn_scan_grad(None, GOOD, zg, GOOD, s, ds, 1, 64, 64, 64, None, None, None, N, 3, 64, da, dg, lda,
                                 ldg, de, None, None))
    assert g() == E.INVALID_ARG
    assert g(N=1 << 25) == E.UNSUPPORTED
    assert g(lda=1 << 31) == E.UNSUPPORTED
    for bad in (dict(s=None), dict(ds=None), dict(da=None), dict(de=None), dict(dg=None), dict(zg=None), dict(lda=63),
                dict(ldg=63)):
        assert g(**({"lda": 1 << 31} | bad)) == E.INVALID_ARG, bad


def test_binding_refuses_shapes_types_and_layouts():
    z = torch.zeros
    with pytest.raises(ValueError, match="P: shape"):
        binding.verify_probs(None, z(2, 3, 8), z(2, 3, dtype=torch.int32), z(2, 3), z(2), Q=z(2, 3, 8))
    with pytest.raises(ValueError, match="u_draw"):
        binding.verify_probs(None, z(2, 4, 8), z(2, 3, dtype=torch.int32), z(2, 3), z(3), Q=z(2, 3, 8))
    with pytest.raises(ValueError, match="teacher_logits"):
        binding.distill(None, z(4, 8), z(4, 2, dtype=torch.int32), z(4, 3))
    with pytest.raises(ValueError, match="zg: shape"):
        binding.rnn_scan(None, z(2, 3, 8), z(2, 3, 4), z(2, 3, 8))
    with pytest.raises(TypeError, match="float16"):
        binding._dtype(z(2, dtype=torch.float16), "e")
    with pytest.raises(TypeError):
        binding._rows(z(4, 8), torch.bfloat16, "za")
    with pytest.raises(ValueError, match="CUDA"):
        binding._rows(z(4, 8), torch.float32, "za")
