"""GPU parity of the RNN head's recurrence over given sequences (dspark_rnn_scan and its
gradients) against the 64-bit statement, whose error bound (accumulated along the sequence from
the gates' and products' 32-bit roundings) plus half a step of the output type is the tolerance."""

import numpy as np
import pytest
import torch

from oracle import training as tr
from rank_markov_draft_gb300 import binding
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

HALF = {torch.float32: torch.finfo(torch.float32).eps / 2, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
DTYPES = [torch.float32, torch.bfloat16]


def make(seed, N, L, D, dtype, gated=True, reset=0.0, decay=2.0):
    rng = np.random.default_rng(seed)
    t = lambda m, s, *shape: torch.from_numpy(rng.normal(m, s, shape).astype(np.float32)).to(dtype)  # noqa: E731
    a = dict(za=t(decay, 1.5, N, L, D), zg=t(0, 1, N, L, D) if gated else None, e=t(0, 1, N, L, D),
             s0=rng.normal(0, 1, (N, D)).astype(np.float32), reset=None, ds=t(0, 1, N, L, D),
             ds_last=rng.normal(0, 1, (N, D)).astype(np.float32))
    if reset:
        a["reset"] = (rng.random((N, L)) < reset).astype(np.uint8)
    return a


def f64(x):
    return None if x is None else x.double().cpu().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)


def cuda(x):
    return None if x is None else x.cuda() if isinstance(x, torch.Tensor) else dev(x)


def near(got, want, bound, half, what):
    bad = ~(np.abs(f64(got) - want) <= bound + half * np.abs(want) * (1 + 1e-6) + 2.0 ** -126)
    at = np.argwhere(bad)[:3]
    assert not bad.any(), (what, at.tolist(), [(f64(got)[tuple(i)], want[tuple(i)], bound[tuple(i)]) for i in at])


def forward(ctx, a, **kw):
    out = binding.rnn_scan(ctx, cuda(a["za"]), cuda(a["zg"]), cuda(a["e"]), s0=cuda(a["s0"]), reset=cuda(a["reset"]), **kw)
    torch.cuda.synchronize()
    assert ctx.status() == 0
    return out


def check_forward(ctx, a):
    out = forward(ctx, a)
    s, err = tr.rnn_scan(f64(a["za"]), f64(a["zg"]), f64(a["e"]), a["s0"], a["reset"])
    near(out["s"], s, err, HALF[a["e"].dtype], "s")
    near(out["s_last"], s[:, -1], err[:, -1], HALF[torch.float32], "s_last")
    return out


def check_backward(ctx, a, s):
    out = binding.rnn_scan_grad(ctx, cuda(a["za"]), cuda(a["zg"]), cuda(a["e"]), s, cuda(a["ds"]), s0=cuda(a["s0"]),
                                ds_last=cuda(a["ds_last"]), reset=cuda(a["reset"]))
    torch.cuda.synchronize()
    assert ctx.status() == 0
    want, bound = tr.rnn_scan_grad(f64(a["za"]), f64(a["zg"]), f64(a["e"]), f64(s), f64(a["ds"]), a["s0"], a["ds_last"], a["reset"])
    half = HALF[a["e"].dtype]
    for i, name in enumerate(("dza", "dzg", "de")):
        if name in out:
            near(out[name], want[i], bound[i], half, name)
    near(out["ds0"], want[3], bound[3], HALF[torch.float32], "ds0")
    assert ("dzg" in out) == (a["zg"] is not None)
    return out


SHAPES = [(1, 1, 1), (128, 1, 256), (3, 1, 7), (1, 2, 3), (2, 5, 33), (7, 16, 64), (2000, 16, 8), (300, 15, 256), (5, 17, 100),
          (1, 4097, 1), (1, 1000, 65), (2, 777, 256), (1, 12289, 64), (3, 2048, 40), (40, 513, 512), (4, 300, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(dsp, shape, dtype):
    a = make(sum(shape), *shape, dtype)
    check_backward(dsp, a, check_forward(dsp, a)["s"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 1, 8), (2, 300, 24), (1, 9001, 16), (4, 130, 257)])
@pytest.mark.parametrize("gated,reset", [(False, 0.0), (True, 0.05), (False, 1.0)])
def test_gates_and_resets(dsp, shape, gated, reset, dtype):
    a = make(sum(shape) + 1, *shape, dtype, gated, reset)
    check_backward(dsp, a, check_forward(dsp, a)["s"])
    a["s0"] = a["ds_last"] = None
    check_backward(dsp, a, check_forward(dsp, a)["s"])


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_memory(dsp, dtype):
    """Decays of 1 - 3e-4: a state carries thousands of steps across every split of the sequence."""
    a = make(5, 1, 30000, 32, dtype, decay=9.0)
    check_backward(dsp, a, check_forward(dsp, a)["s"])


def test_state_handed_on_in_one_buffer(dsp):
    """A long sequence whose last state lands on its first, and the gradients likewise."""
    a = make(13, 2, 20000, 48, torch.float32)
    want = forward(dsp, a)
    state, s = dev(a["s0"]), torch.empty_like(want["s"])
    binding.dspark_rnn_scan(dsp, cuda(a["za"]), cuda(a["zg"]), cuda(a["e"]), state, None, 2, 20000, 48, s, state)
    assert torch.equal(s, want["s"]) and torch.equal(state, want["s_last"])
    args = [cuda(a[n]) for n in ("za", "zg", "e")] + [s, cuda(a["ds"])]
    g = binding.rnn_scan_grad(dsp, *args, s0=dev(a["s0"]), ds_last=dev(a["ds_last"]))
    dza, dzg, de, d = torch.empty_like(s), torch.empty_like(s), torch.empty_like(s), dev(a["ds_last"])
    binding.dspark_rnn_scan_grad(dsp, *args, dev(a["s0"]), None, d, 2, 20000, 48, dza, dzg, de, d)
    assert torch.equal(dza, g["dza"]) and torch.equal(dzg, g["dzg"]) and torch.equal(de, g["de"]) and torch.equal(d, g["ds0"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 511, 32), (1, 512, 32), (1, 513, 64), (1, 1024, 2), (9, 1040, 512), (19, 515, 256),
                                   (1, 40000, 3), (150, 600, 64)])
def test_around_the_cut_into_segments(dsp, shape, dtype):
    a = make(sum(shape), *shape, dtype, reset=0.002)
    check_backward(dsp, a, check_forward(dsp, a)["s"])
    a["s0"] = a["ds_last"] = a["reset"] = None
    check_backward(dsp, a, check_forward(dsp, a)["s"])


def test_saturated_gates(dsp):
    """Gates of exactly 0 and 1, and beyond: infinities, the type's lowest and largest values."""
    a = make(6, 2, 700, 24, torch.float32)
    big = torch.finfo(torch.float32).max
    for i, v in enumerate((torch.inf, -torch.inf, big, -big, 200.0, -200.0, 88.0, -88.0, 40.0, -40.0)):
        a["za"][:, i::37, i] = v
        a["zg"][:, i::41, i + 10] = v
    check_backward(dsp, a, check_forward(dsp, a)["s"])


@pytest.mark.parametrize("L", [5, 5000])
def test_a_reset_drops_infinities_and_nan(dsp, L):
    a = make(7, 2, L, 48, torch.float32)
    clean = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    r = L // 2
    a["reset"] = np.zeros((2, L), np.uint8)
    a["reset"][:, r] = 3
    clean["reset"] = a["reset"]
    a["e"][0, r - 1] = torch.inf
    a["e"][1, 0] = torch.nan
    a["s0"] = a["s0"].copy()
    a["s0"][0] = np.nan
    out, ref = forward(dsp, a), forward(dsp, clean)
    assert torch.equal(out["s"][:, r:], ref["s"][:, r:]) and torch.equal(out["s_last"], ref["s_last"])
    assert torch.isnan(out["s"][:, r - 1]).all() or torch.isinf(out["s"][0, r - 1]).all()
    # and a gradient after the reset does not pass it
    a["ds"][:, r + 1] = torch.nan
    g = binding.rnn_scan_grad(dsp, a["za"].cuda(), a["zg"].cuda(), clean["e"].cuda(), ref["s"], a["ds"].cuda(),
                              s0=dev(clean["s0"]), reset=dev(a["reset"]))
    w = binding.rnn_scan_grad(dsp, a["za"].cuda(), a["zg"].cuda(), clean["e"].cuda(), ref["s"], clean["ds"].cuda(),
                              s0=dev(clean["s0"]), reset=dev(a["reset"]))
    for name in ("dza", "dzg", "de"):
        assert torch.equal(g[name][:, :r], w[name][:, :r]), name
        assert torch.isfinite(g[name][:, :r]).all()
    assert torch.equal(g["ds0"], w["ds0"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [3, 8, 40, 256])
def test_strided_rows(dsp, D, dtype):
    """Halves of a projection, rows of a padded table, at any alignment, and gradients written
    into such halves."""
    a = make(8 + D, 3, 70, D, dtype)
    want = forward(dsp, a)
    z = torch.empty(3, 70, 2 * D + 1, dtype=dtype, device="cuda")
    z[..., :D], z[..., D + 1:] = a["za"].cuda(), a["zg"].cuda()
    e = torch.empty(3, 70, D + 5, dtype=dtype, device="cuda")
    e[..., 5:] = a["e"].cuda()
    got = binding.rnn_scan(dsp, z[..., :D], z[..., D + 1:], e[..., 5:], s0=dev(a["s0"]))
    assert torch.equal(got["s"], want["s"]) and torch.equal(got["s_last"], want["s_last"])
    g = binding.rnn_scan_grad(dsp, a["za"].cuda(), a["zg"].cuda(), a["e"].cuda(), want["s"], a["ds"].cuda(), s0=dev(a["s0"]))
    dz = torch.full((3, 70, 2 * D + 3), 5.0, dtype=dtype, device="cuda")
    de, ds0 = torch.empty_like(want["s"]), torch.empty(3, D, device="cuda")
    binding.dspark_rnn_scan_grad(dsp, z[..., :D], z[..., D + 1:], e[..., 5:], want["s"], a["ds"].cuda(), dev(a["s0"]), None,
                                 None, 3, 70, D, dz[..., :D], dz[..., D + 2:2 * D + 2], de, ds0)
    assert torch.equal(dz[..., :D], g["dza"]) and torch.equal(dz[..., D + 2:2 * D + 2], g["dzg"])
    assert torch.equal(de, g["de"]) and torch.equal(ds0, g["ds0"])
    assert torch.all(dz[..., D:D + 2] == 5.0) and torch.all(dz[..., 2 * D + 2:] == 5.0)


def test_one_token_steps_equal_the_sequence(dsp):
    """Serving: the state handed from call to call in one buffer gives the sequence's states."""
    a = make(9, 33, 12, 96, torch.bfloat16)
    want = forward(dsp, a)
    state = dev(a["s0"])
    for t in range(12):
        s = torch.empty(33, 1, 96, dtype=torch.bfloat16, device="cuda")
        za, zg, e = (a[n][:, t:t + 1].cuda() for n in ("za", "zg", "e"))
        binding.dspark_rnn_scan(dsp, za, zg, e, state, None, 33, 1, 96, s, state)
        assert torch.equal(s[:, 0], want["s"][:, t])
    assert torch.equal(state, want["s_last"])


def test_offsets_past_32_bits(dsp):
    """Rows 2^28 elements apart: the last ones lie beyond the 32-bit range."""
    N, L, D, ld = 3, 4, 64, 1 << 28
    a = make(10, N, L, D, torch.bfloat16)
    buf = torch.empty((N * L - 1) * ld + D, dtype=torch.bfloat16, device="cuda").as_strided((N, L, D), (L * ld, ld, 1))
    want = forward(dsp, a)
    for name in ("za", "zg", "e"):
        buf.copy_(a[name].cuda())
        args = [buf if n == name else a[n].cuda() for n in ("za", "zg", "e")]
        got = binding.rnn_scan(dsp, *args, s0=dev(a["s0"]))
        assert torch.equal(got["s"], want["s"]), name


@pytest.mark.parametrize("shape", [(6, 16, 64), (1, 6000, 32)])
def test_side_stream_graph_and_repeat(dsp, shape):
    a = make(11, *shape, torch.bfloat16)
    want = forward(dsp, a)
    za, zg, e, s0 = a["za"].cuda(), a["zg"].cuda(), a["e"].cuda(), dev(a["s0"])
    ds = a["ds"].cuda()
    wantg = binding.rnn_scan_grad(dsp, za, zg, e, want["s"], ds, s0=s0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = binding.rnn_scan(dsp, za, zg, e, s0=s0)
        g = binding.rnn_scan_grad(dsp, za, zg, e, out["s"], ds, s0=s0)
    side.synchronize()
    assert torch.equal(out["s"], want["s"])
    assert all(torch.equal(g[n], wantg[n]) for n in wantg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.rnn_scan(dsp, za, zg, e, s0=s0)
        g = binding.rnn_scan_grad(dsp, za, zg, e, out["s"], ds, s0=s0)
    for k in (2.0, 1.0):
        e.copy_(a["e"].cuda() * k)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["s"], want["s"])
    assert all(torch.equal(g[n], wantg[n]) for n in wantg)


def test_refusals(dsp):
    a = make(12, 2, 3, 16, torch.float32)
    z = a["za"].cuda()
    with pytest.raises(TypeError):
        binding.rnn_scan(dsp, z.bfloat16(), None, a["e"].cuda())
    with pytest.raises(TypeError, match="float16"):
        binding.rnn_scan(dsp, z.half(), None, a["e"].cuda().half())
    with pytest.raises(ValueError, match="evenly"):
        binding.rnn_scan(dsp, torch.empty(2, 5, 16, device="cuda")[:, :3], None, a["e"].cuda())
    with pytest.raises(ValueError, match="last dimension"):
        binding.rnn_scan(dsp, torch.empty(2, 3, 32, device="cuda")[..., ::2], None, a["e"].cuda())
    with pytest.raises(binding.DSparkError) as err:  # broadcast rows overlap
        binding.rnn_scan(dsp, torch.zeros(1, 1, 16, device="cuda").expand(2, 3, 16), None, a["e"].cuda())
    assert err.value.code == binding.INVALID_ARG
