"""The linear layers' activations and slopes of 32 bits, one argument at a time against 64 bits, relative to
themselves: layers of one input, whose products are the argument.

The functions called are right to: expf one unit in the last place (two roundings, 2^-24 each), the quick
division two units, erfcf four, tanhf two; then come a sum of 1 and a product or two."""

import math

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding
from tests.test_gpu_embed import done

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TINY = 2.0 ** -125  # results below count as zero


def arguments():
    """bf16 numbers of either sign: all between 2^-12 and 100 in steps of seven, and zero."""
    z = torch.arange(0x3980, 0x42C8, 7, dtype=torch.int16).view(BF16)
    return torch.cat([-z, torch.zeros(1, dtype=BF16), z]).cuda()


def value(name, z):
    """Without cancellation."""
    if name in ("sigmoid", "silu"):
        s = torch.where(z >= 0, 1 / (1 + torch.exp(-z.abs())), torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())))
        return s if name == "sigmoid" else z * s
    return step.act(name, z)


def slope(name, z):
    e = torch.exp(-z.abs())
    if name == "sigmoid":
        return e / (1 + e) ** 2
    if name == "tanh":
        return 4 * e ** 2 / (1 + e ** 2) ** 2
    return step.slope(name, z)


def roundings(name, z):
    """Of a value, of itself.  GELU's argument is off by its scale's and a rounding of its own (1.5 together), and
    erfc(x) moves by 2 x^2 + 2 of what x does (x^2 = z^2 / 2)."""
    return {"sigmoid": 2 + 1 + 4, "silu": 2 + 1 + 4 + 1, "tanh": 4, "relu": 0, "gelu": 8 + 2 + 1.5 * (z * z + 2)}[name]


@pytest.mark.parametrize("name", step.ACTS[1:])
@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("K", [1, 4096])
def test_values_of_32_bits(dsp, name, rows, K):
    """K > 1: the same argument beside zeros, in a product of several parts."""
    z = arguments()
    W = torch.zeros(K, z.numel(), dtype=BF16, device="cuda")
    W[K // 2] = z
    y = binding.linear(dsp, torch.ones(rows, K, dtype=BF16, device="cuda"), W, act=name, dtype=F32)["y"]
    done(dsp)
    want = value(name, z.double())
    err = (y[-1].double() - want).abs()
    bad = err > roundings(name, z.double()) * step.EPS32 * want.abs() + TINY
    assert not bad.any(), (z[bad][:3], y[-1][bad][:3], want[bad][:3])
    assert torch.equal(y, y[:1].expand_as(y))


@pytest.mark.parametrize("name", ["sigmoid", "tanh", "silu", "gelu"])
def test_slopes_of_32_bits(dsp, name):
    """dW of one row is x times dz, and dbias is dz; three bf16 numbers of dz leave 2^-25 of it, their sum cuts three
    times.  (SiLU's and GELU's slopes are sums of two terms of either sign: relative to those.)"""
    z = arguments()
    dy = torch.full((1, z.numel()), 1.5, dtype=BF16, device="cuda")
    g = binding.linear_grad(dsp, torch.ones(1, 1, dtype=BF16, device="cuda"), torch.ones(1, z.numel(), dtype=BF16, device="cuda"),
                            dy, act=name, pre=z[None], dx=False, dbias=True)
    done(dsp)
    d = z.double()
    want = slope(name, d)
    if name == "sigmoid":
        allowed = (2 + 2 + 4 + 1) * want
    elif name == "tanh":
        allowed = (2 + 2 + 4 + 2) * want
    elif name == "silu":
        s = value("sigmoid", d)
        allowed = 9 * s + (9 + 9 + 2) * s * d.abs() * value("sigmoid", -d) + want.abs()
    else:
        # the exponential's argument z^2 / 2 is rounded twice
        allowed = roundings("gelu", d) * 0.5 * torch.erfc(-d / math.sqrt(2)) + (2 + d * d + 4) * d.abs() * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi) + want.abs()
    for got, more in ((g["dW"][0], 7), (g["dbias"], 1)):
        err = (got.double() - 1.5 * want).abs()
        bad = err > 1.5 * (allowed + more * want.abs()) * step.EPS32 + TINY
        assert not bad.any(), (z[bad][:3], got[bad][:3], 1.5 * want[bad][:3])
