"""Embedding rows of any width: rows shared out among blocks, up to the widest that an index takes, and the refusal
of more blocks than a launch has."""

import ctypes

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding, build
from tests.test_gpu_embed import TYPES, done, near, normal, wide

BF16 = torch.bfloat16


def test_more_blocks_than_a_launch_has_are_refused():
    build.build()
    lib, P = binding.load(), ctypes.c_void_p

    def f(N, D):
        return lib.dspark_embed(None, P(0x1000), 1, (1 << 31) - 1, P(0x1000), N, 100, D, 1.0, P(0x2000), 1, (1 << 31) - 1, None)

    most = (1 << 31) - 1
    for N, D in ((most, 1025), (1 << 30, 2048), (1025, most), (1 << 21, 1 << 20)):
        assert f(N, D) == binding.UNSUPPORTED, (N, D)
    for N, D in ((most, 1024), (1, most), (1023, most), ((1 << 21) - 1, 1 << 20)):
        assert f(N, D) == binding.INVALID_ARG, (N, D)  # (there is no context)


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [1023, 1024, 1025, 2049, 8184, 8192, 8200, 16392, 100003, 1 << 20])
def test_wide_rows(dsp, D, types):
    table, ids = normal(D, 5, D).to(types[0]), torch.tensor([[4, 0], [-1, 4], [2, 3]], dtype=torch.int32, device="cuda")
    full, out = wide(torch.zeros(6, D, dtype=types[1], device="cuda"), 8)
    before = full.clone()
    binding.embed(dsp, table, ids, scale=1.3, out=out.unflatten(0, (3, 2)))
    done(dsp)
    near(out, *(t.flatten(0, 1) for t in step.embed(table, ids, 1.3)))
    before[:, :D] = out
    assert torch.equal(full.nan_to_num(7.0), before.nan_to_num(7.0))


@pytest.mark.gpu
def test_the_widest_rows(dsp):
    D = (1 << 31) - 1
    table = torch.arange(1 << 16, device="cuda").to(BF16).repeat(1 << 15)[None, :D]
    for ids in ([0], [-1]):
        out = binding.embed(dsp, table, torch.tensor(ids, dtype=torch.int32, device="cuda"))
        done(dsp)
        assert torch.equal(out, table) if ids == [0] else not out.any()
