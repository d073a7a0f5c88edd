"""GPU parity of the distillation loss and its gradient (dspark_distill) against the 64-bit
statement.

Tolerances: a gradient element is off by the 32-bit evaluation's bound (oracle.training, built
from the exponents' sizes and the sum's depth) and half a step of its type; a loss by the same
relative error of every p, q and logarithm."""

import numpy as np
import pytest
import torch

from oracle import training as tr
from rank_markov_draft_gb300 import binding
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

HALF = {torch.float32: torch.finfo(torch.float32).eps / 2, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
DTYPES = [torch.float32, torch.bfloat16]
KW = dict(temperature=1.3, alpha_kl=0.4, alpha_tv=0.9)


def make(seed, N, V, k, dtype, spread=2.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(0, spread, (N, V)).astype(np.float32)).to(dtype)
    ids = np.stack([rng.permutation(V)[:k] if k <= V else np.arange(k) - (k - V) for _ in range(N)]).astype(np.int32)
    return dict(x=x, ids=ids, t=rng.normal(0, spread, (N, k)).astype(np.float32),
                rho=rng.uniform(0, 0.3, N).astype(np.float32), w=rng.uniform(0.1, 2, N).astype(np.float32))


def call(ctx, a, logits=None, grad=True, **kw):
    o = {n: None if a[n] is None else dev(a[n]) for n in ("ids", "t", "rho", "w")}
    return binding.distill(ctx, a["x"].cuda() if logits is None else logits, o["ids"], o["t"], teacher_rest=o["rho"],
                           row_weight=o["w"], grad=grad, **(KW | kw))


def compare(a, out, rows=None, **kw):
    kw = KW | kw
    x = a["x"].double().numpy()
    loss, tv = host(out["loss"]), host(out["tv"])
    grad = None if "grad" not in out else out["grad"].double().cpu().numpy()
    half = HALF[a["x"].dtype]
    for n in range(x.shape[0]) if rows is None else rows:
        w = 1.0 if a["w"] is None else float(a["w"][n])
        L, d, g, b, E = tr.distill_row(x[n], a["ids"][n], a["t"][n], 0.0 if a["rho"] is None else a["rho"][n], w,
                                       kw["temperature"], kw["alpha_kl"], kw["alpha_tv"])
        # KL: each of p, q and ln(p / q) is off by E relative (the logarithm's argument) once
        span = abs(L / w) / max(abs(kw["alpha_kl"]), 1e-9) if w and np.isfinite(L) else 0.0
        tol = abs(w) * (abs(kw["alpha_kl"]) * (2 + 2 * span) + 2 * abs(kw["alpha_tv"])) * E
        if np.isfinite(L):
            assert abs(loss[n] - L) <= tol + 1e-45, (n, loss[n], L, tol)
        else:
            assert loss[n] == L, (n, loss[n], L)
        assert abs(tv[n] - d) <= 2 * E, (n, tv[n], d)
        if grad is not None:
            # (2^-126: below it float32 itself is coarser)
            bad = ~(np.abs(grad[n] - g) <= b + half * np.abs(g) * (1 + 1e-6) + 2.0 ** -126)
            assert not bad.any(), (n, np.flatnonzero(bad)[:5], grad[n][bad][:5], g[bad][:5], b[bad][:5])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 255, 256, 257, 2047, 2048, 4099, 32003])
def test_vocabularies(dsp, V, dtype):
    a = make(V, 6, V, min(V, 9), dtype)
    out = call(dsp, a)
    torch.cuda.synchronize()
    assert dsp.status() == 0
    compare(a, out)
    alone = call(dsp, a, grad=False)
    assert "grad" not in alone and torch.equal(alone["loss"], out["loss"]) and torch.equal(alone["tv"], out["tv"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [65536, 100001, 151936, 1 << 18])
def test_large_vocabularies(dsp, V, dtype):
    a = make(V, 3, V, 64, dtype, spread=3.0)
    compare(a, call(dsp, a))


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64, 128, 129, 255, 256])
def test_teacher_lists(dsp, k):
    a = make(k, 8, 1500, k, torch.float32)
    a["ids"][1, k // 2:] = -1
    a["ids"][2] = -1                   # no teacher: nothing
    a["ids"][3, :] = a["ids"][3, 0]    # one token, repeated
    a["t"][4, : k // 2] = -np.inf
    a["t"][5] = -np.inf                # no mass: nothing
    out = call(dsp, a)
    compare(a, out)
    assert host(out["loss"])[2] == 0 and host(out["loss"])[5] == 0 and not out["grad"][[2, 5]].any()


@pytest.mark.parametrize("V,k", [(4, 4), (5, 8), (3, 256)])
def test_every_token_is_the_teachers(dsp, V, k):
    a = make(V + k, 5, V, k, torch.float32)
    a["rho"] = None
    compare(a, call(dsp, a))
    a["rho"] = np.full(5, 0.2, np.float32)  # mass where the student cannot have any
    out = call(dsp, a)
    assert np.all(np.isposinf(host(out["loss"]))) and torch.isfinite(out["grad"]).all()
    out = call(dsp, a, alpha_kl=0.0)
    compare(a, out, alpha_kl=0.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_student_logits(dsp, dtype):
    a = make(31, 8, 3001, 12, dtype)
    lowest = torch.finfo(dtype).min
    a["x"][0, ::2] = -torch.inf
    a["x"][1, 5:] = -torch.inf
    a["x"][2] = -torch.inf                 # nothing at all: zero
    a["x"][3] = lowest                     # uniform at the lowest value
    a["x"][4, ::3] = lowest
    a["x"][5] = -torch.inf
    a["x"][5, int(a["ids"][5, 3])] = 1.0   # only a teacher's token is left
    a["x"][6, torch.from_numpy(a["ids"][6].astype(np.int64))] = -torch.inf
    a["x"][7, 17] = torch.finfo(dtype).max
    out = call(dsp, a)
    assert not out["grad"][2].any() and float(out["loss"][2]) == 0 and float(out["tv"][2]) == 0
    assert torch.isfinite(out["grad"]).all()
    compare(a, out, rows=[0, 1, 2, 3, 4, 5, 6])
    # row 7: the whole mass on one token
    g = out["grad"][7].double().cpu().numpy()
    want = tr.distill_row(a["x"][7].double().numpy(), a["ids"][7], a["t"][7], a["rho"][7], a["w"][7], 1.3, 0.4, 0.9)
    assert np.abs(g - want[2]).max() <= 8 * HALF[dtype] * np.abs(want[2]).max()


def test_nan_stays_in_its_row(dsp):
    a = make(32, 5, 901, 6, torch.float32)
    a["x"][1, 700] = torch.nan
    a["x"][3] = torch.nan
    out = call(dsp, a)
    assert torch.isnan(out["loss"]).tolist() == [False, True, False, True, False]
    assert torch.isnan(out["grad"]).any(1).tolist() == [False, True, False, True, False]
    compare(a, out, rows=[0, 2, 4])


@pytest.mark.parametrize("V", [901, 39001])
def test_teachers_rest_that_is_no_probability(dsp, V):
    """NaN goes through to its row's loss and gradient; the rest is clamped to [0, 1]."""
    a = make(45, 5, V, 6, torch.float32)
    a["rho"][:] = (0.1, np.nan, -0.5, 1.5, -np.inf)
    out = call(dsp, a)
    assert torch.isnan(out["loss"]).tolist() == torch.isnan(out["tv"]).tolist() == [False, True, False, False, False]
    assert torch.isnan(out["grad"]).all(1).tolist() == [False, True, False, False, False]
    compare(a, out, rows=[0, 2, 3, 4])
    assert torch.isnan(call(dsp, a, grad=False)["loss"]).tolist() == [False, True, False, False, False]


def test_rows_of_no_weight_are_not_read(dsp):
    a = make(33, 6, 777, 5, torch.bfloat16)
    a["w"][[0, 4]] = 0.0
    a["x"][0] = torch.nan
    a["t"][4] = np.nan
    a["ids"][4] = 10 ** 6
    out = call(dsp, a)
    torch.cuda.synchronize()
    assert dsp.status() == 0
    compare(a, out)
    assert not out["grad"][[0, 4]].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_padded_rows_and_the_gradient_in_place(dsp, dtype, pad):
    """Rows of a wider buffer: the padding is neither read into the loss nor written."""
    a = make(34 + pad, 7, 1003, 9, dtype)
    buf = torch.full((7, 1003 + pad), torch.nan, dtype=dtype, device="cuda")
    buf[:, :1003] = a["x"].cuda()
    gbuf = torch.full((7, 1003 + 2 * pad + 1), 7.0, dtype=dtype, device="cuda")
    got = call(dsp, a, logits=buf[:, :1003], grad=gbuf[:, :1003])
    compare(a, got)
    assert torch.all(gbuf[:, 1003:] == 7.0)
    same = call(dsp, a, logits=buf[:, :1003], grad=buf[:, :1003])
    assert torch.equal(buf[:, :1003], got["grad"]) and torch.equal(same["loss"], got["loss"])
    assert torch.isnan(buf[:, 1003:]).all()


def test_block_shapes_and_defaults(dsp):
    a = make(35, 12, 640, 4, torch.float32)
    flat = call(dsp, a | dict(rho=None, w=None))
    compare(a | dict(rho=None, w=None), flat)
    out = binding.distill(dsp, a["x"].cuda().view(3, 4, 640), dev(a["ids"]).view(3, 4, 4), dev(a["t"]).view(3, 4, 4), **KW)
    assert out["loss"].shape == (3, 4) and out["grad"].shape == (3, 4, 640)
    assert torch.equal(out["loss"].flatten(), flat["loss"]) and torch.equal(out["grad"].view(12, 640), flat["grad"])


@pytest.mark.parametrize("T", [0.05, 1.0, 20.0])
@pytest.mark.parametrize("kl,tv", [(1.0, 0.0), (0.0, 1.0), (0.1, 0.9), (-0.5, 0.25)])
def test_temperatures_and_weights(dsp, T, kl, tv):
    a = make(36, 5, 1200, 10, torch.float32)
    a["rho"][:3] = (0.0, 1.0, 1e-6)
    kw = dict(temperature=T, alpha_kl=kl, alpha_tv=tv)
    compare(a, call(dsp, a, **kw), **kw)


def test_equal_student_and_teacher(dsp):
    """p = q: the loss is zero up to rounding, and so is KL's gradient."""
    a = make(37, 4, 500, 20, torch.float32)
    x = a["x"].double().numpy()
    q = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    a["t"] = np.take_along_axis(x, a["ids"].astype(np.int64), 1).astype(np.float32)
    a["rho"] = (1 - np.take_along_axis(q, a["ids"].astype(np.int64), 1).sum(1)).astype(np.float32)
    out = call(dsp, a, temperature=1.0, alpha_kl=1.0, alpha_tv=0.0)
    E = tr.distill_row(x[0], a["ids"][0], a["t"][0], a["rho"][0], 1.0, 1.0, 1.0, 0.0)[4]
    assert out["loss"].abs().max() <= 2 * 2 * E
    assert out["grad"].abs().max() <= 2 * 2 * E


# 39001 logits are a long row.
@pytest.mark.parametrize("V", [500, 39001])
def test_signs_next_to_tvs_kinks(dsp, V):
    """p and q of every event nearly equal: slots 4e-6 apart, the rest 2e-5.  What decides are sums
    of 32 bits.  A slots' sum: exponentials off by 2^-22, of exponents up to 2 log2 e with three
    roundings, and at most 13 additions, so 2^-22 + (3 * 2 + 13) 2^-24 = 1.4e-6, two of them
    2.8e-6.  The outside's: exponents up to 14 (3 * 14 * ln 2 * 2^-24 = 1.7e-6), at most 90 additions
    a lane and ten on the way together, 7.9e-6 in all, of which a slot's q feels the outside's
    share of the whole, below a tenth."""
    N, k = 40, 64
    a = make(43, N, V, k, torch.float32, spread=1.0)
    rng = np.random.default_rng(44)
    at = a["ids"].astype(np.int64)
    a["x"].scatter_(1, torch.from_numpy(at), torch.from_numpy(rng.uniform(9, 11, (N, k)).astype(np.float32)))
    x = a["x"].double().numpy()
    q = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    side = rng.choice([-1.0, 1.0], (N, k))
    side[:, ::2] = -side[:, 1::2]  # as many above as below, of all weights
    s = np.take_along_axis(x, at, 1)
    a["t"] = (s + 8e-6 * side).astype(np.float32)
    qs = np.take_along_axis(q, at, 1)
    a["rho"] = ((1 - qs.sum(1)) * (1 + 2.5e-5 * rng.choice([-1.0, 1.0], N))).astype(np.float32)
    t = a["t"].astype(np.float64)
    p = np.exp(t) / np.exp(t).sum(1, keepdims=True) * (1 - a["rho"].astype(np.float64))[:, None]
    # (the rest's step moves every slot by a part of its own)
    far = np.abs(p / qs - 1) >= 4e-6
    rows = np.flatnonzero(far.all(1))
    assert rows.size >= N // 4 and (1 - qs.sum(1)).max() < 0.1 and (np.abs(a["rho"] / (1 - qs.sum(1)) - 1) >= 2e-5).all()
    assert (p < qs)[rows].any() and (p > qs)[rows].any()
    out = call(dsp, a, temperature=1.0)
    compare(a, out, rows=rows, temperature=1.0)


def test_gradient_equals_differences(dsp):
    """The call's own loss, differenced by its own logits (32 bits: steps of 2^-6)."""
    a = make(38, 1, 12, 4, torch.float32)
    g = host(call(dsp, a)["grad"])[0]
    h = 2.0 ** -6
    for v in range(12):
        L = []
        for s in (h, -h):
            b = dict(a, x=a["x"].clone())
            b["x"][0, v] += s
            L.append(float(call(dsp, b, grad=False)["loss"][0]))
        # second-order remainder h^2 / 6 of a third derivative below w (|a_kl| + a_tv), and the
        # losses' own rounding over 2 h
        assert abs((L[0] - L[1]) / (2 * h) - g[v]) <= float(a["w"][0]) * 1.3 * (h * h + 2e-6 / h)


def test_offsets_past_32_bits(dsp):
    N, V, ld = 10, 1003, 1 << 28
    a = make(39, N, V, 6, torch.bfloat16)
    buf = torch.empty(N * ld - (ld - V), dtype=torch.bfloat16, device="cuda").as_strided((N, V), (ld, 1))
    buf.copy_(a["x"].cuda())
    out = call(dsp, a, logits=buf, grad=buf)
    compare(a, dict(out, grad=buf.contiguous()))


def test_teacher_token_out_of_range_is_reported():
    a = make(40, 3, 50, 4, torch.float32)
    b = {k: v.copy() if k == "ids" else v for k, v in a.items()}
    b["ids"][1, 2] = 50
    with binding.Context(0, B_max=1, V_max=8, K_max=1) as ctx:
        out = call(ctx, b)
        torch.cuda.synchronize()
        assert ctx.status() == binding.DEVICE_OOB
        b["ids"][1, 2] = -1  # skipped like an empty slot
        compare(b, out)


def test_side_stream_graph_and_repeat(dsp):
    a = make(41, 9, 5000, 8, torch.bfloat16)
    want = call(dsp, a)
    x = a["x"].cuda()
    ids, t, rho, w = (dev(a[n]) for n in ("ids", "t", "rho", "w"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = binding.distill(dsp, x, ids, t, teacher_rest=rho, row_weight=w, **KW)
    side.synchronize()
    assert torch.equal(out["grad"], want["grad"]) and torch.equal(out["loss"], want["loss"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.distill(dsp, x, ids, t, teacher_rest=rho, row_weight=w, **KW)
    for s in (0.5, 1.0):
        x.copy_(a["x"].cuda() * s)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["grad"], want["grad"]) and torch.equal(out["loss"], want["loss"])


# 16-byte pieces of a row at which the number that a thread holds, or the threads, change.
STEPS = sorted({p + d for p in [96, 192, 288, 384, 480, 512, 576, 640, 768, 864, 1024, 1152, 1344, 1536, 1728, 1792, 2016, 2304, 2592,
                                 2688, 3136, 3456, 3584, 4096, 4608, 5120, 7168, 9216, 9728]
                for d in (0, 1)} | {1760, 1791})


@pytest.mark.parametrize("dtype,per", [(torch.float32, 4), (torch.bfloat16, 8)])
@pytest.mark.parametrize("pieces", STEPS)
def test_every_way_a_short_row_is_dealt_out(dsp, dtype, per, pieces):
    for V in (pieces * per, pieces * per + 3):
        a = make(V, 3, V, 12, dtype)
        a["ids"][0, :3] = (V - 1, 0, V - 2)
        compare(a, call(dsp, a))


# Rows past 155,648 bytes (608 * 16 pieces of 16) take the other kernel: 38,912 fp32 logits, 77,824
# bf16.  (The smaller sizes are those where three CTAs, then two, no longer fit an SM.)
@pytest.mark.parametrize("dtype,V", [(dt, base + d) for dt, base in ((torch.float32, 10368), (torch.bfloat16, 20736),
                                                         (torch.float32, 18432), (torch.bfloat16, 36864),
                                                         (torch.float32, 38912), (torch.bfloat16, 77824))
                                     for d in (-9, -1, 0, 1, 7, 33, 130)])
def test_around_the_longest_short_row(dsp, dtype, V):
    a = make(V, 5, V, 33, dtype)
    a["ids"][0, :3] = (V - 1, 0, V - 2)
    a["ids"][1, :4] = (V // 2, -1, V // 2, V // 2 + 1)
    compare(a, call(dsp, a))


@pytest.mark.parametrize("dtype,V", [(torch.float32, 40003), (torch.bfloat16, 40003), (torch.bfloat16, 80007)])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_long_rows_padded_and_in_place(dsp, dtype, V, pad):
    """As above for rows in segments: logits and gradient at different offsets modulo 16 bytes."""
    N = 7
    a = make(50 + pad, N, V, 21, dtype)
    buf = torch.full((N, V + pad), torch.nan, dtype=dtype, device="cuda")
    buf[:, :V] = a["x"].cuda()
    gbuf = torch.full((N, V + 2 * pad + 1), 7.0, dtype=dtype, device="cuda")
    got = call(dsp, a, logits=buf[:, :V], grad=gbuf[:, :V])
    compare(a, got)
    assert torch.all(gbuf[:, V:] == 7.0)
    same = call(dsp, a, logits=buf[:, :V], grad=buf[:, :V])
    assert torch.equal(buf[:, :V], got["grad"]) and torch.equal(same["loss"], got["loss"])
    assert torch.isnan(buf[:, V:]).all()


@pytest.mark.parametrize("dtype,V", [(torch.float32, 50021), (torch.bfloat16, 50021), (torch.bfloat16, 90021)])
def test_long_rows_masked_and_without_weight(dsp, dtype, V):
    a = make(60, 10, V, 12, dtype)
    lowest = torch.finfo(dtype).min
    a["x"][0, ::2] = -torch.inf
    a["x"][1, 5:] = -torch.inf             # whole segments of nothing
    a["x"][2] = -torch.inf                 # nothing at all: zero
    a["x"][3] = lowest                     # uniform at the lowest value
    a["x"][4] = -torch.inf
    a["x"][4, int(a["ids"][4, 3])] = 1.0   # only a teacher's token is left
    a["x"][5, torch.from_numpy(a["ids"][5].astype(np.int64))] = -torch.inf
    a["w"][[6, 8]] = 0.0
    a["x"][6] = torch.nan                  # not looked at
    a["ids"][8] = 10 ** 6
    a["x"][7, 40000] = torch.nan
    out = call(dsp, a)
    torch.cuda.synchronize()
    assert dsp.status() == 0
    assert not out["grad"][[2, 6, 8]].any() and float(out["loss"][2]) == 0
    assert torch.isnan(out["loss"]).tolist() == [n == 7 for n in range(10)]
    assert torch.isnan(out["grad"]).any(1).tolist() == [n == 7 for n in range(10)]
    compare(a, out, rows=[0, 1, 2, 3, 4, 5, 6, 8, 9])


@pytest.mark.parametrize("dtype,V", [(torch.float32, 12007), (torch.bfloat16, 24001), (torch.float32, 39001),
                                     (torch.bfloat16, 78001)])
@pytest.mark.parametrize("grad", [True, False])
def test_many_long_rows(dsp, dtype, V, grad):
    """More rows than one launch takes (2048), over many rounds, a run of them without weight."""
    N, k = 2300, 7
    rng = np.random.default_rng(V)
    base = make(V, 8, V, k, dtype)
    pick = rng.integers(0, 8, N)
    a = {n: base[n][pick] for n in ("x", "ids", "t", "rho")} | dict(w=rng.uniform(0.1, 2, N).astype(np.float32))
    a["w"][300:900] = 0.0
    a["w"][2047:2050] = 0.0
    out = call(dsp, a, grad=grad)
    torch.cuda.synchronize()
    assert dsp.status() == 0
    rows = [0, 1, 299, 300, 901, 1500, 2046, 2048, 2050, 2051, N - 1]
    compare(a, out, rows=rows)
    # every other row against the one of the same logits: the loss is linear in its weight, with
    # two roundings, and TV does not depend on it
    alone = call(dsp, base | dict(w=np.ones(8, np.float32)), grad=False)
    want = host(alone["loss"])[pick] * a["w"]
    live = a["w"] != 0
    assert np.abs(host(out["loss"]) - want).max() <= 1e-5 * np.abs(want).max()
    assert (host(out["loss"])[~live] == 0).all()
    assert np.abs(host(out["tv"])[live] - host(alone["tv"])[pick][live]).max() <= 1e-5


@pytest.mark.parametrize("dtype,V,N", [(torch.float32, 131075, 500), (torch.float32, 131072, 77), (torch.bfloat16, 151936, 600),
                                       (torch.bfloat16, 78001, 2100)])
@pytest.mark.parametrize("T", [1.3, 0.25])
def test_every_gradient_of_many_long_rows(dsp, dtype, V, N, T):
    """Many rounds of segments, up to 64 of a row: every element of every row, which has the
    logits of one of eight and a weight of its own, against the 64-bit gradient times the weight;
    weights of 1e6 bring coefficients above one, rows of none are zeros."""
    rng = np.random.default_rng(V + N)
    base = make(V, 8, V, 40, dtype)
    pick = rng.integers(0, 8, N)
    w = rng.uniform(0.1, 2, N).astype(np.float32)
    w[::7] *= 1e6
    w[rng.random(N) < 0.2] = 0.0
    w[N // 3:N // 2] = 0.0
    at = torch.from_numpy(pick).cuda()
    x = base["x"].cuda()[at]
    ids, t, rho = (dev(base[n][pick]) for n in ("ids", "t", "rho"))
    out = binding.distill(dsp, x, ids, t, teacher_rest=rho, row_weight=dev(w), **KW | dict(temperature=T))
    torch.cuda.synchronize()
    assert dsp.status() == 0
    del x
    row = [tr.distill_row(base["x"][n].double().numpy(), base["ids"][n], base["t"][n], base["rho"][n], 1.0, T,
                          KW["alpha_kl"], KW["alpha_tv"]) for n in range(8)]
    want, bound = (torch.from_numpy(np.stack([r[i] for r in row])).cuda() for i in (2, 3))
    for n in range(N):
        if w[n] == 0:
            assert not out["grad"][n].any() and float(out["loss"][n]) == 0, n
            continue
        g = want[pick[n]] * float(w[n])
        bad = ~((out["grad"][n].double() - g).abs() <= bound[pick[n]] * float(w[n]) + HALF[dtype] * g.abs() * (1 + 1e-6) + 2.0 ** -126)
        assert not bad.any(), (n, w[n], bad.nonzero()[:3].flatten().tolist())
    loss, E = np.array([r[0] for r in row])[pick] * w, max(r[4] for r in row)
    tol = w * (KW["alpha_kl"] * (2 + 2 * np.abs(loss / np.maximum(w, 1e-30)) / KW["alpha_kl"]) + 2 * KW["alpha_tv"]) * E
    assert (np.abs(host(out["loss"]) - loss) <= tol).all()


@pytest.mark.parametrize("V", [60000, 120000])
def test_long_rows_on_a_side_stream_in_a_graph_and_repeated(dsp, V):
    a = make(61, 9, V, 8, torch.bfloat16)
    want = call(dsp, a)
    x = a["x"].cuda()
    ids, t, rho, w = (dev(a[n]) for n in ("ids", "t", "rho", "w"))
    for _ in range(3):  # the context's scratch is used again
        out = binding.distill(dsp, x, ids, t, teacher_rest=rho, row_weight=w, **KW)
        assert torch.equal(out["grad"], want["grad"]) and torch.equal(out["loss"], want["loss"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = binding.distill(dsp, x, ids, t, teacher_rest=rho, row_weight=w, **KW)
    side.synchronize()
    assert torch.equal(out["grad"], want["grad"]) and torch.equal(out["loss"], want["loss"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.distill(dsp, x, ids, t, teacher_rest=rho, row_weight=w, **KW)
    for s in (0.5, 1.0):
        x.copy_(a["x"].cuda() * s)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["grad"], want["grad"]) and torch.equal(out["loss"], want["loss"])


def test_refusals(dsp):
    a = make(42, 3, 64, 4, torch.float32)
    with pytest.raises(binding.DSparkError) as err:
        call(dsp, a, temperature=0.0)
    assert err.value.code == binding.INVALID_ARG
    with pytest.raises(TypeError, match="float16"):
        call(dsp, a, logits=a["x"].cuda().half())
    with pytest.raises(ValueError, match="last dimension"):
        call(dsp, a, logits=a["x"].cuda().t().contiguous().t())
    with pytest.raises(TypeError):
        call(dsp, a, grad=torch.empty(3, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="grad: shape"):
        call(dsp, a, grad=torch.empty(3, 65, device="cuda"))
