"""GPU parity of the gradients' common norm and clipping (dspark_clip_grads) against the 64-bit
statement.  A thread adds at most 32 squares to one 32-bit sum before 64-bit sums take over, so the
sum of squares is right to 40 roundings, the norm to half of that and its own."""

import math

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NORM = 21 * step.EPS32


def make(seed, sizes, types, std=0.01):
    g = torch.Generator("cuda").manual_seed(seed)
    return [(std * torch.randn(n, generator=g, device="cuda")).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def check(ctx, grads, limit, norm, out):
    torch.cuda.synchronize()
    assert ctx.status() == 0
    want, scaled = step.clip(grads, limit)
    assert abs(float(norm) - want) <= NORM * want
    for o, s in zip(out, scaled):
        half = torch.finfo(o.dtype).eps / 2
        # the factor: the norm's error, its own rounding; then the product's
        assert ((o.double() - s).abs() <= s.abs() * (half * (1 + 1e-6) + NORM + 3 * step.EPS32) + 2.0 ** -133).all()


LISTS = [[1], [5], [16384], [16385, 7], [0, 3, 0], [100000], [3] * 31, [1000 + i for i in range(32)], [33] * 33,
         [1 + 37 * i for i in range(511)], [9] * 512, [9] * 513, [20000] * 600, [5] * 1300, [3000001, 2, 64]]


@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_lists(dsp, sizes, types):
    grads = make(len(sizes), sizes, types)
    norm = binding.grad_norm(dsp, grads)
    torch.cuda.synchronize()
    want = step.clip(grads, 1.0)[0]
    assert abs(float(norm) - want) <= NORM * want
    for limit in (0.3 * want, 3 * want):
        out = [torch.full_like(g, 9.0) for g in grads]
        check(dsp, grads, limit, binding.clip_grads(dsp, grads, limit, out=out), out)
        mine = [g.clone() for g in grads]
        same = binding.clip_grads(dsp, mine, limit)
        assert all(torch.equal(a, b) for a, b in zip(mine, out)) and float(same) == float(norm)
        if limit > want:
            assert all(torch.equal(a, b) for a, b in zip(mine, grads))


@pytest.mark.parametrize("offset", [1, 3, 4, 5])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_misaligned_tensors(dsp, offset, dtype):
    base = make(7, [50000], (dtype,))[0]
    grads = [base[offset:20003], base[20004:40001], base[40001:]]
    store = torch.zeros(60000, dtype=dtype, device="cuda")
    out = [store[:20003 - offset], store[20007:20007 + 19997], store[50001:50001 + 9999]]
    check(dsp, grads, 0.5, binding.clip_grads(dsp, grads, 0.5, out=out), out)
    used = torch.zeros(60000, dtype=torch.bool, device="cuda")
    for a, o in zip((0, 20007, 50001), out):
        used[a:a + o.numel()] = True
    assert (store[~used] == 0).all()
    mine = base.clone()
    parts = [mine[offset:20003], mine[20004:40001], mine[40001:]]
    binding.clip_grads(dsp, parts, 0.5)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(parts, out))
    assert torch.equal(mine[:offset], base[:offset]) and mine[20003] == base[20003]


def test_shapes_and_views(dsp):
    grads = [make(1, [60], (F32,))[0].view(3, 4, 5), make(2, [1], (BF16,))[0][0]]
    out = [torch.empty_like(g) for g in grads]
    check(dsp, grads, 0.01, binding.clip_grads(dsp, grads, 0.01, out=out), out)


def test_any_iterable(dsp):
    grads = make(1, [50, 60], (F32,))
    want = float(binding.grad_norm(dsp, grads))
    assert float(binding.grad_norm(dsp, (g for g in grads))) == want
    mine = [g.clone() for g in grads]
    assert float(binding.clip_grads(dsp, (g for g in mine), 0.01)) == want
    check(dsp, grads, 0.01, binding.clip_grads(dsp, tuple(grads), 0.01, out=tuple(torch.empty_like(g) for g in grads)), mine)


def test_no_tensors(dsp):
    assert float(binding.grad_norm(dsp, [])) == 0.0 and float(binding.clip_grads(dsp, [], 1.0)) == 0.0
    grads = [torch.zeros(100, device="cuda")]
    assert float(binding.clip_grads(dsp, grads, 0.0)) == 0.0 and (grads[0] == 0).all()
    assert dsp.status() == 0


@pytest.mark.parametrize("value,norm,rest", [(math.inf, math.inf, 0.0), (-math.inf, math.inf, 0.0), (math.nan, math.nan, math.nan)])
def test_nonfinite_gradients_follow_the_formula(dsp, value, norm, rest):
    grads = make(3, [40000, 7], (F32, BF16))
    grads[0][12345] = value
    got = float(binding.clip_grads(dsp, grads, 1.0))
    assert got == norm or (math.isnan(got) and math.isnan(norm))
    assert math.isnan(float(grads[0][12345]))  # inf * 0
    assert all(float(v) == rest or math.isnan(rest) and math.isnan(float(v)) for v in (grads[0][0], grads[1][6]))


def test_limits(dsp):
    grads = make(4, [1000], (F32,))
    for limit in (0.0, math.inf):
        out = [torch.empty_like(grads[0])]
        binding.clip_grads(dsp, grads, limit, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out[0], grads[0] if limit else torch.zeros_like(grads[0]))


def test_many_elements_of_one_sign(dsp):
    """300 million ones: 32-bit sums would stop growing at 2^24."""
    grads = [torch.ones(300_000_000, dtype=BF16, device="cuda")]
    norm = float(binding.grad_norm(dsp, grads))
    assert abs(norm - math.sqrt(3e8)) <= NORM * norm


def test_refusals(dsp):
    g = make(5, [10, 20], (F32,))
    with pytest.raises(binding.DSparkError):
        binding.clip_grads(dsp, g, -1.0)
    with pytest.raises(ValueError):
        binding.clip_grads(dsp, g, 1.0, out=g[:1])
    with pytest.raises(ValueError):
        binding.clip_grads(dsp, g, 1.0, out=[g[0], g[1].bfloat16()])
    with pytest.raises(TypeError):
        binding.grad_norm(dsp, [g[0].double()])
    with pytest.raises(ValueError):
        binding.grad_norm(dsp, [g[0][::2]])
    with pytest.raises(ValueError):
        binding.grad_norm(dsp, [g[0].cpu()])
    for other in (None, 1.0, "g"):
        with pytest.raises(TypeError):
            binding.grad_norm(dsp, [g[0], other])


def test_side_stream_graph_and_equal_bits(dsp):
    grads = make(6, [70000, 3, 16384, 501], (F32, BF16))
    out = [torch.empty_like(g) for g in grads]
    want = binding.clip_grads(dsp, grads, 0.1, out=out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [torch.empty_like(g) for g in grads]
    norm = binding.clip_grads(dsp, grads, 0.1, out=again, stream=side)
    side.synchronize()
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(again, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = binding.clip_grads(dsp, grads, 0.1, out=again)
    for seed in (7, 8):
        for g, new in zip(grads, make(seed, [70000, 3, 16384, 501], (F32, BF16))):
            g.copy_(new)
        graph.replay()
        check(dsp, grads, 0.1, norm, again)
