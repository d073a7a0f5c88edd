"""Layers whose x, W and dz are of very different shapes and all need copies (rows off 16-byte boundaries)."""

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding
from tests.test_gpu_embed import done, near, normal

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("M,K,N,act,dtype", [(9000, 3, 5001, "sigmoid", BF16), (7000, 100, 1025, None, F32), (3, 5001, 257, "tanh", F32),
                                             (20000, 1, 1, "silu", BF16), (1, 9, 40003, "gelu", BF16), (2500, 4099, 3, None, F32)])
def test_tall_beside_wide(dsp, M, K, N, act, dtype):
    x, W = normal(M, M, K).to(BF16), (normal(M + 1, K, N) / K ** 0.5).to(BF16)
    out = binding.linear(dsp, x, W, act=act, pre=True, dtype=F32)
    dy = normal(M + 2, M, N).to(dtype)
    g = binding.linear_grad(dsp, x, W, dy, act=act, pre=out["pre"] if act else None, dbias=True)
    done(dsp)
    y, z, ey, ez = step.linear(x, W, None, act)
    near(out["y"], y, ey, "y")
    near(out["pre"], z, ez, "pre")
    for name, (want, bound) in step.linear_grad(x, W, dy, act, out["pre"]).items():
        near(g[name], want, bound, name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [F32, BF16])
@pytest.mark.parametrize("N", [640, 641])
def test_residuals_beside_long_sums(dsp, N, residual, dtype):
    """Accumulators that start again while residuals arrive, over more tiles than blocks."""
    M, K = 20050, 1100
    x, W = normal(1, M, K).to(BF16), (normal(2, K, N) / K ** 0.5).to(BF16)
    res, bias = (3 * normal(3, M, N)).to(residual), normal(4, N)
    out = binding.linear(dsp, x, W, bias=bias, act="silu", residual=res, dtype=dtype)["y"]
    done(dsp)
    want, _, bound, _ = step.linear(x, W, bias, "silu", res)
    near(out, want, bound)
    if residual == dtype:
        binding.linear(dsp, x, W, bias=bias, act="silu", residual=res, out=res)
        done(dsp)
        assert torch.equal(res, out)
