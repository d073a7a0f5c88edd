"""GPU parity of embedding rows and their gradient (dspark_embed, dspark_embed_grad) against the
64-bit statements, whose bounds (one rounded product; n - 1 roundings of a sum of n terms) plus half
a step of the output type are the tolerances."""

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]


def near(got, want, bound, what=""):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - want).abs()
    bad = ~(err <= bound + half * want.abs() * (1 + 1e-6) + 2.0 ** -126)
    assert not bad.any(), (what, bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), want[bad][:3].tolist())


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def tokens(seed, N, V, padding=0.1, skew=True):
    g = torch.Generator("cuda").manual_seed(seed)
    u = torch.rand(N, generator=g, device="cuda")
    ids = ((V + 1.0) ** u - 1 if skew else u * V).long().clamp(0, V - 1)
    return torch.where(torch.rand(N, generator=g, device="cuda") < padding, -1 - ids, ids).to(torch.int32)


def wide(t, extra, at=0):
    """The same values as columns [at, at + D) of a wider tensor."""
    w = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    w[:, at:at + t.shape[1]] = t
    return w, w[:, at:at + t.shape[1]]


def done(ctx):
    torch.cuda.synchronize()
    assert ctx.status() == 0


SHAPES = [(1, 1, 1), (1, 5, 8), (128, 1000, 256), (33, 7, 100), (2, 300, 2048), (1000, 50, 1), (5, 3, 9000), (4097, 700, 24),
          (257, 1 << 18, 40)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("N,V,D", SHAPES)
def test_embed(dsp, N, V, D, types):
    table, ids = normal(N + D, V, D).to(types[0]), tokens(N, N, V)
    out = binding.embed(dsp, table, ids, scale=1.7, dtype=types[1])
    done(dsp)
    near(out, *step.embed(table, ids, 1.7))
    if types[0] == types[1]:  # unscaled rows are copies
        out = binding.embed(dsp, table, ids)
        assert torch.equal(out, torch.where(ids[:, None] >= 0, table[ids.clamp(min=0).long()], 0))


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("extra,at", [(8, 0), (8, 8), (3, 0), (16, 1)])
def test_embed_strides(dsp, types, extra, at):
    table, ids = normal(3, 90, 64).to(types[0]), tokens(4, 70, 90).view(7, 10)
    full, out = wide(torch.zeros(70, 64, dtype=types[1], device="cuda"), extra, at)
    before = full.clone()
    binding.embed(dsp, wide(table, extra, at)[1], ids, scale=0.5, out=out.unflatten(0, (7, 10)))
    done(dsp)
    near(out, *(t.flatten(0, 1) for t in step.embed(table, ids, 0.5)))
    before[:, at:at + 64] = out
    assert torch.equal(full.nan_to_num(7.0), before.nan_to_num(7.0))  # nothing beside the rows is written


def test_embed_special_values_pass_through(dsp):
    table = torch.tensor([[float("inf")] * 8, [float("-inf")] * 8, [float("nan")] * 8, [0.0] * 8], device="cuda")
    out = binding.embed(dsp, table, torch.tensor([0, 1, 2, 3, -5], dtype=torch.int32, device="cuda"), scale=2.0)
    done(dsp)
    assert torch.equal(out.nan_to_num(5.0, 3.0, 2.0)[:, 0].cpu(), torch.tensor([3.0, 2.0, 5.0, 0.0, 0.0]))


def test_embed_no_rows(dsp):
    out = binding.embed(dsp, normal(1, 5, 8), torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    done(dsp)
    assert out.shape == (0, 3, 8) and dsp.last_launches == 0


def test_offsets_past_32_bits(dsp):
    V, D = 1 << 18, 8200
    table = torch.zeros(V, D, dtype=BF16, device="cuda")
    table[V - 1], table[V // 2] = 3.0, 2.0
    ids = torch.tensor([V - 1, V // 2, 0], dtype=torch.int32, device="cuda")
    out = binding.embed(dsp, table, ids)
    done(dsp)
    assert (out.float().mean(1).cpu() == torch.tensor([3.0, 2.0, 0.0])).all()
    grad = binding.embed_grad(dsp, ids, out, V, dtype=BF16, grad=table)
    done(dsp)
    assert (grad[V - 1] == 3).all() and (grad[V // 2] == 2).all() and (grad[0] == 0).all()
    assert int((grad[:, 17] != 0).sum()) == 2


@pytest.mark.parametrize("bad", [[100], [100, 3, 2 ** 31 - 1]])
def test_ids_out_of_range_are_reported_and_skipped(bad):
    ids = torch.tensor([1] + bad + [99], dtype=torch.int32, device="cuda")
    with binding.Context(0, B_max=1, V_max=4096, K_max=1) as ctx:
        table = normal(1, 100, 16)
        out = binding.embed(ctx, table, ids)
        torch.cuda.synchronize()
        assert ctx.status() == binding.DEVICE_OOB
        inside = ids < 100
        assert torch.equal(out[inside], table[ids[inside].long()]) and (out[~inside] == 0).all()
        with pytest.raises(binding.DSparkError):
            binding.embed(ctx, table, ids)
        ctx.reset()
        grad = binding.embed_grad(ctx, ids, out, 100)
        torch.cuda.synchronize()
        assert ctx.status() == binding.DEVICE_OOB
        near(grad, *step.embed_grad(ids, out, 100))


GRAD_SHAPES = [(1, 1, 1), (1, 300, 8), (77, 1000, 100), (2, 7, 256), (1000, 50, 1), (300, 3, 700), (4096, 700, 64),
               (4097, 5000, 24), (33000, 20000, 32), (70000, 151936, 8), (20000, 1, 16), (5000, 1 << 18, 16), (600, 40, 2056)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("N,V,D", GRAD_SHAPES)
def test_embed_grad(dsp, N, V, D, types):
    ids, de = tokens(N + V, N, V), normal(N, N, D).to(types[0])
    grad = binding.embed_grad(dsp, ids, de, V, scale=0.7, dtype=types[1])
    done(dsp)
    near(grad, *step.embed_grad(ids, de, V, 0.7))
    again = binding.embed_grad(dsp, ids, de, V, scale=0.7, dtype=types[1])
    assert torch.equal(grad, again)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("N,V,D", [(1, 9, 8), (500, 2000, 100), (9000, 30, 64), (40000, 151936, 16)])
def test_embed_grad_accumulates(dsp, N, V, D, types):
    ids, de, before = tokens(N, N, V), normal(1, N, D).to(types[0]), normal(2, V, D).to(types[1])
    grad = binding.embed_grad(dsp, ids, de, grad=before.clone(), scale=0.7, accumulate=True)
    done(dsp)
    near(grad, *step.embed_grad(ids, de, V, 0.7, before))
    named = torch.zeros(V, dtype=torch.bool, device="cuda")
    named[ids[ids >= 0].long()] = True
    assert torch.equal(grad[~named], before[~named])


@pytest.mark.parametrize("N", [31, 32, 33, 1023, 1024, 1025, 4095, 16384, 16385, 65537, 131072, 131073, 262145])
@pytest.mark.parametrize("V", [2, 513, 151936])
def test_embed_grad_around_tiles(dsp, N, V):
    ids, de = tokens(N, N, V, padding=0.01), normal(N, N, 8)
    grad = binding.embed_grad(dsp, ids, de, V)
    done(dsp)
    near(grad, *step.embed_grad(ids, de, V))


def test_embed_grad_most_rows(dsp):
    N, V = 1 << 20, 151936
    ids, de = tokens(5, N, V), normal(6, N, 8).to(BF16)
    grad = binding.embed_grad(dsp, ids, de, V)
    done(dsp)
    near(grad, *step.embed_grad(ids, de, V))


@pytest.mark.parametrize("kind", ["one token", "all padding", "each once", "last alone", "two in turn"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_token_patterns(dsp, kind, accumulate):
    N, V = 5000, 6000
    n = torch.arange(N, device="cuda")
    ids = {"one token": torch.full_like(n, 4242), "all padding": torch.full_like(n, -1), "each once": (n * 7) % V,
           "last alone": torch.where(n == N - 1, V - 1, -1), "two in turn": torch.where(n % 2 == 0, 0, V - 1)}[kind].to(torch.int32)
    de, before = normal(3, N, 40), normal(4, V, 40)
    grad = binding.embed_grad(dsp, ids, de, scale=2.0, grad=before.clone(), accumulate=accumulate)
    done(dsp)
    near(grad, *step.embed_grad(ids, de, V, 2.0, before if accumulate else None), what=kind)


@pytest.mark.parametrize("extra,at", [(8, 0), (8, 8), (3, 0), (16, 1)])
@pytest.mark.parametrize("types", TYPES)
def test_embed_grad_strides(dsp, types, extra, at):
    ids, de = tokens(4, 700, 90), normal(3, 700, 64).to(types[0])
    full, grad = wide(torch.zeros(90, 64, dtype=types[1], device="cuda"), extra, at)
    before = full.clone()
    binding.embed_grad(dsp, ids, wide(de, extra, at)[1], grad=grad)
    done(dsp)
    near(grad, *step.embed_grad(ids, de, 90))
    before[:, at:at + 64] = grad
    assert torch.equal(full.nan_to_num(7.0), before.nan_to_num(7.0))


def test_embed_grad_no_rows(dsp):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    before = normal(1, 50, 24)
    assert (binding.embed_grad(dsp, none, torch.empty(0, 24, device="cuda"), 50) == 0).all()
    grad = binding.embed_grad(dsp, none, torch.empty(0, 24, device="cuda"), grad=before.clone(), accumulate=True)
    done(dsp)
    assert torch.equal(grad, before)


def test_embed_grad_nonfinite_rows_stay_with_their_tokens(dsp):
    ids = torch.tensor([5, 6, 5, 7, -1, 8], dtype=torch.int32, device="cuda")
    de = torch.ones(6, 8, device="cuda")
    de[2], de[3], de[4] = float("inf"), float("nan"), float("nan")
    grad = binding.embed_grad(dsp, ids, de, 10)[:, 0]
    done(dsp)
    assert grad.nan_to_num(99.0, 88.0).tolist() == [0, 0, 0, 0, 0, 88, 1, 99, 1, 0]


def test_embed_and_gradient_are_transposes(dsp):
    ids, table, de = tokens(1, 3000, 800), normal(2, 800, 48), normal(3, 3000, 48)
    out = binding.embed(dsp, table, ids, scale=3.0)
    grad = binding.embed_grad(dsp, ids, de, 800, scale=3.0)
    done(dsp)
    a, b = (out.double() * de.double()).sum(), (table.double() * grad.double()).sum()
    size = (out.double() * de.double()).abs().sum()
    assert (a - b).abs() <= 800 * step.EPS32 * size  # the commonest token has some hundred rows


def test_side_stream_and_graph(dsp):
    V, N, D = 3000, 5000, 64
    ids, de, table = tokens(1, N, V), normal(2, N, D), normal(3, V, D)
    want_out, want = binding.embed(dsp, table, ids), binding.embed_grad(dsp, ids, de, V)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, grad = torch.empty_like(want_out), torch.empty_like(want)
    binding.embed(dsp, table, ids, out=out, stream=side)
    binding.embed_grad(dsp, ids, de, grad=grad, stream=side)
    side.synchronize()
    assert torch.equal(out, want_out) and torch.equal(grad, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.embed(dsp, table, ids, out=out)
        binding.embed_grad(dsp, ids, de, grad=grad)
    for seed in (4, 5):
        ids.copy_(tokens(seed, N, V))
        de.copy_(normal(seed, N, D))
        graph.replay()
        done(dsp)
        near(out, *step.embed(table, ids))
        near(grad, *step.embed_grad(ids, de, V))
