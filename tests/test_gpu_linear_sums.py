"""Accuracy of the linear layers' sums, against 64 bits with bounds much finer than an output of bf16.

Terms are positive, of 1 to 1.57 each, so that a sum's size is the sum and what the accumulators cut adds
up instead of cancelling.  An accumulator takes 512 terms, 16 at a time: 32 cuts, each of less than a step
of fp32 (2^-23) of what it then holds, k / 32 of its end on average, and 1.25 times that where the first
terms are the largest: 21 of its ends together.  What the accumulators held is added up in fp32, a rounding
(2^-24) each of what has been added up so far: K / 1024 of the sum together, and a few (terms shared out among
blocks make fewer cuts and at most 64 parts).
So no sum is further off than (42 + K / 1024 + 4) 2^-24 of itself.  A cut is half a step on average, and
a rounding none: the mean of many sums is off by 16.5 half steps, 1e-6, whatever K is."""

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding
from tests.test_gpu_embed import done, wide

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
MEAN = 1.1e-6


def worst(terms):
    return (46 + terms / 1024) * step.EPS32


def half_step(want, dtype):
    """Half a step of `dtype` at each value: the most that one rounding is off."""
    bits = {F32: 24, BF16: 8}[dtype]
    return torch.ldexp(torch.ones_like(want), torch.frexp(want)[1] - bits - 1)


def positive(seed, *shape):
    """bf16 numbers of [1, 1.25]."""
    g = torch.Generator("cuda").manual_seed(seed)
    return (1 + 0.25 * torch.rand(*shape, generator=g, device="cuda")).to(BF16)


def product(ctx, kind, A, B, dtype):
    """A [I, C] times B [C, J] as y, dx or dW of a layer."""
    (I, C), J = A.shape, B.shape[1]
    if kind == "y":
        out = binding.linear(ctx, A, B, dtype=dtype)["y"]
    elif kind == "dx":
        out = binding.linear_grad(ctx, torch.empty(I, J, dtype=BF16, device="cuda"), B.T.contiguous(), A, dW=False,
                                  dx=torch.empty(I, J, dtype=dtype, device="cuda"))["dx"]
    else:
        out = binding.linear_grad(ctx, A.T.contiguous(), torch.empty(I, J, dtype=BF16, device="cuda"), B, dx=False,
                                  dW=torch.empty(I, J, dtype=dtype, device="cuda"))["dW"]
    done(ctx)
    return out


def check(got, want, terms):
    err = (got.double() - want).abs()
    allowed = worst(terms) * want + (0 if got.dtype == F32 else half_step(want, got.dtype))
    bad = err > allowed
    assert not bad.any(), (int(bad.sum()), float((err / want).max()))
    if got.dtype == F32:
        assert float((err / want).mean()) <= MEAN


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["y", "dx", "dW"])
@pytest.mark.parametrize("terms", [512, 2048, 4096, 17000, 50000])
def test_sums_of_few_tiles(dsp, terms, kind, dtype):
    """(whose terms are shared out among blocks)"""
    A, B = positive(terms, 130, terms), positive(terms + 1, terms, 72)
    check(product(dsp, kind, A, B, dtype), A.double() @ B.double(), terms)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["y", "dx", "dW"])
@pytest.mark.parametrize("terms", [4096, 50000])
def test_sums_of_many_tiles(dsp, terms, kind, dtype):
    """(of which a block takes all terms): rows and columns of a small product, again and again."""
    A, B = positive(terms, 64, terms), positive(terms + 1, terms, 128)
    want = A.double() @ B.double()
    got = product(dsp, kind, A.repeat(64, 1), B.repeat(1, 38), dtype)
    first = got[:64, :128]
    check(first, want, terms)
    assert torch.equal(got, first.repeat(64, 38))


@pytest.mark.parametrize("dw_dtype", [F32, BF16])
def test_sums_of_both_gradients_at_once(dsp, dw_dtype):
    M, K, N = 2048, 192, 30000
    x, W, dy = positive(1, M, K), positive(2, K, N), positive(3, M, N)
    g = binding.linear_grad(dsp, x, W, dy, dW=torch.empty(K, N, dtype=dw_dtype, device="cuda"))
    done(dsp)
    check(g["dx"], dy.double() @ W.double().T, N)
    check(g["dW"], x.double().T @ dy.double(), M)


# dz in 32 bits: sums of one term, three numbers of bf16 that together leave 2^-25 of it, and three cuts.
ONE = (2 * 3 + 1) * step.EPS32


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dy_of_32_bits_enters_the_products_whole(dsp, dtype):
    dy = 1 + torch.rand(3000, 1, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    W = positive(2, 40, 1)
    dx = binding.linear_grad(dsp, torch.empty(3000, 40, dtype=BF16, device="cuda"), W, dy, dW=False,
                             dx=torch.empty(3000, 40, dtype=dtype, device="cuda"))["dx"]
    row = dy.T.contiguous()
    x = positive(3, 1, 40)
    dW = binding.linear_grad(dsp, x, torch.empty(40, 3000, dtype=BF16, device="cuda"), row, dx=False,
                             dW=torch.empty(40, 3000, dtype=dtype, device="cuda"))["dW"]
    done(dsp)
    for got, want in ((dx, dy.double() @ W.double().T), (dW, x.double().T @ row.double())):
        err = (got.double() - want).abs()
        bad = err > ONE * want + (0 if dtype == F32 else half_step(want, dtype))
        assert not bad.any(), (int(bad.sum()), float((err / want).max()))


@pytest.mark.parametrize("M,K,N,act,dtype", [(700, 256, 50000, None, BF16), (2048, 100, 20000, None, F32), (1500, 136, 24000, "silu", BF16)])
def test_large_gradients_wherever_they_lie_give_equal_bits(dsp, M, K, N, act, dtype):
    """Both products of a large dz share the blocks out by sizes, not by where dW lies."""
    x, W, dy = positive(1, M, K), positive(2, K, N), positive(3, M, N).to(dtype)
    pre = positive(4, M, N) if act else None
    for dw_dtype in (F32, BF16):
        want = binding.linear_grad(dsp, x, W, dy, act=act, pre=pre, dW=torch.empty(K, N, dtype=dw_dtype, device="cuda"))
        for extra, at in ((3, 1), (8, 0), (16, 4)):
            dW = wide(torch.zeros(K, N, dtype=dw_dtype, device="cuda"), extra, at)[1]
            dx = wide(torch.zeros(M, K, dtype=BF16, device="cuda"), extra, at)[1]
            binding.linear_grad(dsp, x, W, dy, act=act, pre=pre, dx=dx, dW=dW)
            done(dsp)
            assert torch.equal(dx, want["dx"]) and torch.equal(dW, want["dW"]), (extra, at)
