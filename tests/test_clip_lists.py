"""Lists of gradients that name one tensor twice: both places would scale it at one time."""

import pytest
import torch

from rank_markov_draft_gb300 import binding


def test_addresses_are_listed_once():
    binding._each_once([], [], "out")
    binding._each_once([16, 32, 48], [5, 5, 5], "out")
    binding._each_once([0, 16, 0], [0, 5, 0], "out")  # tensors of no elements lie nowhere
    binding._each_once([16, 16], [0, 5], "out")
    for pointers, numel in (([16, 16], [5, 5]), ([16, 32, 0, 0, 16], [5, 1, 0, 0, 2])):
        with pytest.raises(ValueError, match="out: the same tensor twice"):
            binding._each_once(pointers, numel, "out")


@pytest.mark.gpu
def test_calls_refuse_them_and_leave_the_tensors(dsp):
    a, b = torch.full((100,), 2.0, device="cuda"), torch.full((50,), 3.0, device="cuda")
    for grads, out in (([a, b, a], None), ([a, b], [torch.empty_like(a)[:50]] * 2)):
        with pytest.raises(ValueError):
            binding.clip_grads(dsp, grads, 1.0, out=out)
    same = torch.empty_like(b)
    with pytest.raises(ValueError, match="twice"):
        binding.clip_grads(dsp, [b, b.clone()], 1.0, out=[same, same])
    torch.cuda.synchronize()
    assert (a == 2.0).all() and (b == 3.0).all() and dsp.status() == 0
    # a norm counts it twice, as the formula does
    assert abs(float(binding.grad_norm(dsp, [a, a])) - 800 ** 0.5) < 1e-4
    none = [torch.empty(0, device="cuda") for _ in range(3)]
    assert float(binding.clip_grads(dsp, none + [b], 1e9)) == pytest.approx(450 ** 0.5, rel=1e-6)
