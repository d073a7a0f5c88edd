"""The 64-bit statements of the training step's operators against differences and torch's autograd,
and the operators' refusals, all on the CPU."""

import ctypes

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding, build


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("name", step.ACTS)
def test_slopes_are_differences(name):
    z = normal(1, 400) * 3
    z = z[z.abs() > 1e-3]  # (relu's kink)
    h = 1e-5
    diff = (step.act(name, z + h) - step.act(name, z - h)) / (2 * h)
    assert (diff - step.slope(name, z)).abs().max() < 1e-9


@pytest.mark.parametrize("name", step.ACTS)
def test_linear_grad_is_differences(name):
    x, W, b, dy = normal(2, 5, 7), normal(3, 7, 6), normal(4, 6), normal(5, 5, 6)
    z = step.linear(x, W, b, name)[1]
    g = step.linear_grad(x, W, dy, name, z)
    f = lambda x, W, b: (step.linear(x, W, b, name)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for i, key in ((0, "dx"), (1, "dW"), (2, "dbias")):
        step_of = normal(6 + i, *(x, W, b)[i].shape)
        up, down = [x, W, b], [x, W, b]
        up[i], down[i] = up[i] + h * step_of, down[i] - h * step_of
        assert abs((f(*up) - f(*down)) / (2 * h) - (g[key][0] * step_of).sum()) < 1e-6


def test_embed_grad_is_embeds_transpose():
    ids = torch.tensor([3, 0, -1, 3, 9, 3])
    table, de = normal(1, 10, 4), normal(2, 6, 4)
    out = step.embed(table, ids, 2.5)[0]
    grad = step.embed_grad(ids, de, 10, 2.5)[0]
    assert abs((out * de).sum() - (table * grad).sum()) < 1e-12
    assert (out[2] == 0).all() and (grad[1] == 0).all()


def test_clip_has_the_limit_as_its_norm():
    grads = [normal(1, 100), normal(2, 3, 5)]
    norm, out = step.clip(grads, 0.5)
    assert abs(torch.cat([g.flatten() for g in out]).norm() - 0.5) < 1e-6
    assert step.clip(grads, 2 * norm)[1][0].equal(grads[0])


# ------------------------------------------------------------------------------ refusals
P = ctypes.c_void_p
GOOD, ODD = P(0x1000), P(0x1001)  # never dereferenced by the host checks
E = binding
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_embed_argument_checks(lib):
    def f(table=GOOD, tt=0, ldt=8, ids=GOOD, N=4, V=100, D=8, out=P(0x2000), ot=1, ldo=8):
        return lib.dspark_embed(None, table, tt, ldt, ids, N, V, D, 1.0, out, ot, ldo, None)

    assert f() == E.INVALID_ARG  # valid arguments, no context
    for bad in (dict(table=None), dict(tt=2), dict(ot=-1), dict(ids=None), dict(out=None), dict(N=-1), dict(V=0), dict(D=0),
                dict(ldt=7), dict(ldo=7), dict(table=ODD), dict(ids=P(0x1002)), dict(out=ODD), dict(out=P(0x1000))):
        assert f(**bad) == E.INVALID_ARG, bad
    for bad in (dict(V=(1 << 18) + 1), dict(N=BIG), dict(ldt=BIG), dict(ldo=BIG)):
        assert f(**bad) == E.UNSUPPORTED, bad
    assert f(N=0, ids=None, out=None) == E.INVALID_ARG  # nothing to do: only the context is missing


def test_embed_grad_argument_checks(lib):
    def f(ids=GOOD, de=GOOD, dt=1, ld=8, N=4, V=100, D=8, grad=P(0x2000), gt=0, ldg=8):
        return lib.dspark_embed_grad(None, ids, de, dt, ld, N, V, D, 1.0, 0, grad, gt, ldg, None)

    assert f() == E.INVALID_ARG
    for bad in (dict(ids=None), dict(de=None), dict(dt=2), dict(ld=7), dict(N=-1), dict(V=0), dict(D=0), dict(grad=None),
                dict(gt=2), dict(ldg=7), dict(de=ODD), dict(grad=P(0x1002)), dict(grad=P(0x1000))):
        assert f(**bad) == E.INVALID_ARG, bad
    for bad in (dict(N=(1 << 20) + 1), dict(V=(1 << 18) + 1), dict(D=(1 << 16) + 1, ld=1 << 17, ldg=1 << 17), dict(ld=BIG),
                dict(ldg=BIG)):
        assert f(**bad) == E.UNSUPPORTED, bad


def test_clip_argument_checks(lib):
    def f(ptr=0x1000, n=5, dtype=0, count=1, limit=1.0, out=0x2000, norm=GOOD, lists=True):
        g = (P * 1)(ptr) if lists else None
        o = None if out is None else (P * 1)(out)
        return lib.dspark_clip_grads(None, g, (ctypes.c_int64 * 1)(n), (ctypes.c_int32 * 1)(dtype), count, limit, o, norm, None)

    assert f() == E.INVALID_ARG
    for bad in (dict(ptr=None), dict(ptr=0x1002), dict(n=-1), dict(dtype=2), dict(count=-1), dict(limit=-1.0),
                dict(limit=float("nan")), dict(out=0x2001), dict(out=0), dict(norm=None), dict(norm=P(0x1002)), dict(lists=False)):
        assert f(**bad) == E.INVALID_ARG, bad
    assert f(n=(1 << 40) + 1) == E.UNSUPPORTED


def test_linear_argument_checks(lib):
    def f(x=GOOD, ldx=8, W=P(0x5000), ldw=16, bias=None, act=0, res=None, rt=0, ldr=16, M=4, K=8, N=16, y=P(0x2000), yt=0, ldy=16,
          pre=None, ldp=16, ws=None, size=0, sized=True):
        n = ctypes.c_int64(size)
        return lib.dspark_linear(None, x, ldx, W, ldw, bias, act, res, rt, ldr, M, K, N, y, yt, ldy, pre, ldp, ws,
                                 ctypes.byref(n) if sized else None, None)

    assert f() == E.INVALID_ARG
    for bad in (dict(x=None), dict(W=None), dict(y=None), dict(ldx=7), dict(ldw=15), dict(ldy=15), dict(act=6), dict(act=-1),
                dict(res=GOOD, rt=2), dict(res=GOOD, ldr=15), dict(res=P(0x1002)), dict(M=-1), dict(K=0), dict(N=0), dict(yt=2),
                dict(pre=P(0x3000), ldp=15), dict(pre=P(0x2000)), dict(pre=GOOD), dict(pre=P(0x4000), res=P(0x4000)), dict(y=GOOD),
                dict(y=P(0x5000)), dict(x=ODD), dict(W=ODD), dict(bias=P(0x1002)), dict(y=P(0x1002)),
                dict(ws=P(0x1010), size=64), dict(size=-1), dict(sized=False), dict(res=P(0x2000), rt=1),
                dict(res=P(0x2000), ldr=17)):
        assert f(**bad) == E.INVALID_ARG, bad
    for bad in (dict(M=BIG), dict(ldx=BIG), dict(ldw=BIG), dict(ldy=BIG), dict(K=(1 << 22) + 1, ldx=1 << 23),
                dict(N=(1 << 22) + 1, ldw=1 << 23, ldy=1 << 23)):
        assert f(**bad) == E.UNSUPPORTED, bad


def test_linear_grad_argument_checks(lib):
    def f(x=GOOD, ldx=8, W=P(0x2000), ldw=16, dy=P(0x3000), dt=1, ldy=16, act=0, pre=None, pt=1, ldp=16, M=4, K=8, N=16,
          dx=P(0x4000), xt=1, lddx=8, dW=P(0x5000), wt=0, lddw=16, db=P(0x6000), size=0):
        n = ctypes.c_int64(size)
        return lib.dspark_linear_grad(None, x, ldx, W, ldw, dy, dt, ldy, act, pre, pt, ldp, M, K, N, dx, xt, lddx, dW, wt, lddw,
                                      db, None, ctypes.byref(n), None)

    assert f() == E.INVALID_ARG
    for bad in (dict(x=None), dict(W=None), dict(dy=None), dict(dt=2), dict(ldy=15), dict(act=6), dict(act=1), dict(act=1, pre=ODD),
                dict(act=1, pre=GOOD, ldp=15), dict(act=1, pre=GOOD, pt=2), dict(M=-1), dict(K=0), dict(N=0), dict(xt=2),
                dict(lddx=7), dict(wt=2), dict(lddw=15), dict(ldx=7), dict(ldw=15), dict(db=P(0x1002)), dict(dx=ODD), dict(size=-1),
                dict(dx=None, dW=None, db=None), dict(dx=P(0x3000)), dict(dx=GOOD), dict(dW=P(0x2000)), dict(dW=P(0x4000))):
        assert f(**bad) == E.INVALID_ARG, bad
    for bad in (dict(M=BIG), dict(ldy=BIG), dict(lddx=BIG)):
        assert f(**bad) == E.UNSUPPORTED, bad


def test_wrappers_check_shapes():
    t = torch.zeros
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bias"):
        binding.linear(None, t(2, 4, **bf), t(4, 6, **bf), bias=t(5))
    with pytest.raises(ValueError, match="residual"):
        binding.linear(None, t(2, 4, **bf), t(4, 6, **bf), residual=t(1, 6))
    with pytest.raises(ValueError, match="dy"):
        binding.linear_grad(None, t(2, 4, **bf), t(4, 6, **bf), t(2, 5, **bf))
    with pytest.raises(ValueError, match="de"):
        binding.embed_grad(None, t(3, dtype=torch.int32), t(4, 6), 10)
    with pytest.raises(ValueError, match="accumulate"):
        binding.embed_grad(None, t(4, dtype=torch.int32), t(4, 6), 10, accumulate=True)
    with pytest.raises(ValueError, match="act"):
        binding._act("swish")
