"""GPU parity of the linear layers (dspark_linear, dspark_linear_grad) against the 64-bit statements,
whose bounds (matrix products added up 16 terms at a time; dz as one or two bf16 numbers) plus half a
step of the output type are the tolerances."""

import pytest
import torch

from oracle import step
from rank_markov_draft_gb300 import binding
from tests.test_gpu_embed import done, near, normal, wide

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(seed, M, K, N):
    return normal(seed, M, K).to(BF16), (normal(seed + 1, K, N) / K ** 0.5).to(BF16)


def check(ctx, x, W, dtype=BF16, **kw):
    out = binding.linear(ctx, x, W, dtype=dtype, pre=True, **kw)
    done(ctx)
    lead = x.shape[:-1].numel()
    res = kw.get("residual")
    y, z, dy, dz = step.linear(x.reshape(lead, -1), W, kw.get("bias"), kw.get("act"), None if res is None else res.reshape(lead, -1))
    near(out["y"].reshape(lead, -1), y, dy, "y")
    near(out["pre"].reshape(lead, -1), z, dz, "pre")
    plain = binding.linear(ctx, x, W, dtype=dtype, **kw)
    assert "pre" not in plain and torch.equal(plain["y"], out["y"])
    return out


def check_grad(ctx, x, W, dy, act=None, pre=None, dx_dtype=BF16, dw_dtype=F32, **kw):
    dx, dW = torch.full_like(x, 9.0, dtype=dx_dtype), torch.full_like(W, 9.0, dtype=dw_dtype)
    out = binding.linear_grad(ctx, x, W, dy, act=act, pre=pre, dx=dx, dW=dW, dbias=True, **kw)
    done(ctx)
    for name, (want, bound) in step.linear_grad(x, W, dy, act, pre).items():
        near(out[name], want, bound, name)
    for name in ("dx", "dW", "dbias"):  # each by itself
        only = binding.linear_grad(ctx, x, W, dy, act=act, pre=pre, dx=name == "dx", dW=name == "dW", dbias=name == "dbias")
        assert list(only) == [name]
        if only[name].dtype == out[name].dtype:
            assert torch.equal(only[name], out[name]), name
    return out


SHAPES = [(1, 1, 1), (1, 64, 64), (128, 4096, 256), (2, 7, 9), (127, 63, 65), (129, 65, 127), (256, 128, 256), (300, 1000, 250),
          (5, 256, 4003), (64, 8, 1000), (1000, 8, 8), (33, 2048, 64), (1, 5000, 3), (2048, 256, 640), (700, 72, 520), (3, 16, 20000)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear(dsp, M, K, N, dtype):
    check(dsp, *make(M + K, M, K, N), dtype=dtype)


@pytest.mark.parametrize("act", step.ACTS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [None, F32, BF16])
@pytest.mark.parametrize("M,K,N", [(150, 96, 200), (40, 33, 77), (16, 2048, 64)])
def test_epilogues(dsp, M, K, N, act, bias, residual):
    x, W = make(3, M, K, N)
    for dtype in (F32, BF16):
        check(dsp, x, W, dtype=dtype, act=act, bias=normal(5, N) if bias else None,
              residual=None if residual is None else (3 * normal(6, M, N)).to(residual))


@pytest.mark.parametrize("act", step.ACTS)
def test_activations_far_out(dsp, act):
    """Arguments of up to +-3e4 and next to zero: no overflow, no NaN."""
    W = torch.tensor([[-30000.0, -100.0, -20.0, -1e-3, 0.0, 1e-3, 20.0, 100.0, 30000.0]], device="cuda").to(BF16)
    x = torch.ones(3, 1, dtype=BF16, device="cuda")
    out = check(dsp, x, W, dtype=F32, act=act)
    dy = torch.ones(3, 9, dtype=BF16, device="cuda")
    check_grad(dsp, x, W, dy, act=act, pre=out["pre"] if act else None)


@pytest.mark.parametrize("extra,at", [(8, 0), (8, 8), (3, 0), (16, 1), (4, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dsp, extra, at, dtype):
    M, K, N = 140, 72, 136
    x, W = make(1, M, K, N)
    res = normal(2, M, N).to(dtype)
    want = binding.linear(dsp, x, W, residual=res, dtype=dtype, act="silu", pre=True)
    xs, ws, rs = wide(x, extra, at)[1], wide(W, extra, at)[1], wide(res, extra, at)[1]
    full, out = wide(torch.zeros_like(res), extra, at)
    before = full.clone()
    pre_full, pre = wide(torch.zeros_like(res), extra, at)
    binding.linear(dsp, xs, ws, residual=rs, out=out, act="silu", pre=pre)
    done(dsp)
    assert torch.equal(out, want["y"]) and torch.equal(pre, want["pre"])
    before[:, at:at + N] = out
    assert torch.equal(full.nan_to_num(7.0), before.nan_to_num(7.0))
    dy = normal(3, M, N).to(dtype)
    dx, dW = wide(torch.zeros_like(x), extra, at), wide(torch.zeros_like(W), extra, at)
    for a in (None, "silu"):
        want_g = binding.linear_grad(dsp, x, W, dy, act=a, pre=want["pre"] if a else None, dW=torch.empty_like(W))
        binding.linear_grad(dsp, xs, ws, wide(dy, extra, at)[1], act=a, pre=pre if a else None, dx=dx[1], dW=dW[1])
        done(dsp)
        assert torch.equal(dx[1], want_g["dx"]) and torch.equal(dW[1], want_g["dW"])
    for full, mine in (dx, dW):
        mine.zero_()
        assert int(full.isnan().sum()) == full.shape[0] * extra


def test_residual_in_place_and_leading_dimensions(dsp):
    x, W = make(1, 60, 32, 96)
    res = normal(2, 3, 20, 96)
    want = check(dsp, x.view(3, 20, 32), W, dtype=F32, residual=res)["y"]
    mine = res.clone()
    out = binding.linear(dsp, x.view(3, 20, 32), W, residual=mine, out=mine)
    done(dsp)
    assert out["y"] is mine and torch.equal(mine, want)


def test_no_rows(dsp):
    x, W = make(1, 0, 32, 96)
    assert binding.linear(dsp, x, W)["y"].shape == (0, 96) and dsp.last_launches == 0
    g = binding.linear_grad(dsp, x, W, torch.empty(0, 96, dtype=BF16, device="cuda"), dbias=True)
    done(dsp)
    assert g["dx"].shape == (0, 32) and (g["dW"] == 0).all() and (g["dbias"] == 0).all()


def test_nonfinite_inputs_stay_in_their_rows(dsp):
    x, W = make(1, 200, 70, 90)
    clean = binding.linear(dsp, x, W)["y"]
    x[3, 5], x[150, 69] = float("nan"), float("inf")
    y = binding.linear(dsp, x, W)["y"]
    done(dsp)
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[3] = keep[150] = False
    assert torch.equal(y[keep], clean[keep]) and y[3].isnan().all() and not y[150].isfinite().any()


GRAD_SHAPES = [(1, 1, 1), (333, 1000, 250), (128, 64, 64), (129, 65, 127), (2, 300, 7), (700, 8, 72), (64, 256, 5003),
               (2048, 256, 640), (1, 128, 4096), (5000, 16, 24), (200, 2000, 8)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K,N", GRAD_SHAPES)
def test_linear_grad(dsp, M, K, N, dtype):
    x, W = make(M + K, M, K, N)
    check_grad(dsp, x, W, (normal(9, M, N) / M).to(dtype))


@pytest.mark.parametrize("act", step.ACTS[1:])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("M,K,N", [(150, 96, 200), (40, 33, 77), (600, 16, 64)])
def test_linear_grad_activations(dsp, M, K, N, act, types):
    x, W = make(3, M, K, N)
    check_grad(dsp, x, W, normal(5, M, N).to(types[0]), act, (2 * normal(6, M, N)).to(types[1]))


@pytest.mark.parametrize("dx_dtype", [F32, BF16])
@pytest.mark.parametrize("dw_dtype", [F32, BF16])
def test_gradient_types(dsp, dx_dtype, dw_dtype):
    x, W = make(3, 260, 136, 200)
    check_grad(dsp, x, W, normal(5, 260, 200).to(BF16), dx_dtype=dx_dtype, dw_dtype=dw_dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(384, 256, 50000), (384, 200, 50001), (40100, 64, 64), (40100, 64, 61), (20050, 96, 128), (20050, 33, 101),
                                   (20050, 300, 130)])
def test_residuals_of_many_tiles(dsp, M, K, N, residual, dtype):
    """More tiles than blocks: each residual arrives while another tile is worked on; and in place."""
    x, W = make(1, M, K, N)
    res = (3 * normal(2, M, N)).to(residual)
    y = binding.linear(dsp, x, W, residual=res, dtype=dtype)["y"]
    done(dsp)
    want, _, bound, _ = step.linear(x, W, residual=res)
    near(y, want, bound)
    if residual == dtype:
        assert binding.linear(dsp, x, W, residual=res, out=res)["y"] is res
        done(dsp)
        assert torch.equal(res, y)


def gap(M, N, ld, dtype):
    """A matrix with elements beside its rows and after them, and all of them."""
    store = torch.full((M * ld + 5,), 777.0, dtype=dtype, device="cuda")
    return store[:M * ld].view(M, ld)[:, :N], store


def beside(store, M, N, ld):
    kept = store.clone()
    kept[:M * ld].view(M, ld)[:, :N] = 777
    return bool((kept == 777).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K,N,ld", [(65, 67, 67, 72), (65, 40, 65, 68), (40, 72, 1, 8), (300, 97, 300, 304), (300, 66, 1001, 1008),
                                      (2048, 256, 20001, 20008)])
def test_nothing_beside_an_output(dsp, M, K, N, ld, residual, dtype):
    """Rows on boundaries for vectors and TMA that end within one."""
    x, W = make(1, M, K, N)
    y, all_y = gap(M, N, ld, dtype)
    pre, all_pre = gap(M, N, ld, dtype)
    res = normal(3, M, N).to(dtype) if residual else None
    want = binding.linear(dsp, x, W, residual=res, dtype=dtype, act="silu", pre=True)
    binding.linear(dsp, x, W, residual=res, out=y, act="silu", pre=pre)
    done(dsp)
    assert torch.equal(y, want["y"]) and torch.equal(pre, want["pre"])
    assert beside(all_y, M, N, ld) and beside(all_pre, M, N, ld)
    if residual:
        return
    dy, ldk = normal(4, M, N).to(BF16), (K + 8) // 8 * 8
    dx, all_dx = gap(M, K, ldk, dtype)
    dW, all_dW = gap(K, N, ld, dtype)
    for act, z in ((None, None), ("silu", want["pre"])):
        binding.linear_grad(dsp, x, W, dy, act=act, pre=z, dx=dx, dW=dW)
        done(dsp)
        bounds = step.linear_grad(x, W, dy, act, z)
        near(dx, *bounds["dx"], "dx")
        near(dW, *bounds["dW"], "dW")
        assert beside(all_dx, M, K, ldk) and beside(all_dW, K, N, ld)


@pytest.mark.parametrize("act", [None, "sigmoid", "gelu"])
@pytest.mark.parametrize("residual", [F32, BF16])
@pytest.mark.parametrize("first", [0, 1, 2, 3, 7])
@pytest.mark.parametrize("M,N,ld", [(1, 1, 1), (2, 1, 3), (33, 31, 31), (130, 33, 34), (65, 67, 68), (129, 97, 101), (3, 1000, 1001), (300, 64, 65)])
def test_residuals_at_any_address(dsp, M, N, ld, first, residual, act):
    """Rows that begin within a word, with values beside them that must not count (the largest there are)."""
    x, W = make(M + N, M, 40, N)
    store = torch.full((first + M * ld + 5,), torch.finfo(residual).max, dtype=residual, device="cuda")
    res = store[first:first + M * ld].view(M, ld)[:, :N]
    res.copy_(3 * normal(3, M, N))
    check(dsp, x, W, residual=res, act=act)
    kept = store.clone()
    y = binding.linear(dsp, x, W, residual=res, dtype=residual, act=act)["y"]
    assert binding.linear(dsp, x, W, residual=res, out=res, act=act)["y"] is res
    done(dsp)
    assert torch.equal(res, y)
    res.copy_(kept[first:first + M * ld].view(M, ld)[:, :N])
    assert torch.equal(store, kept)


def test_logits_of_a_large_vocabulary(dsp):
    """A ragged vocabulary, more tiles than blocks; the gradients' long contraction."""
    M, K, V = 384, 256, 50003
    x, W = make(1, M, K, V)
    U = 3 * normal(2, M, V)
    check(dsp, x, W, residual=U)
    x, W = make(1, M, K, 50000)
    check(dsp, x, W, residual=U[:, :50000])
    check_grad(dsp, x, W, (torch.softmax(U[:, :50000], 1) / M).to(BF16))


def test_offsets_past_32_bits(dsp):
    M, K, N = 70000, 16, 65536
    x, W = make(1, M, K, N)
    y = binding.linear(dsp, x, W)["y"]
    done(dsp)
    for rows in (slice(0, 50), slice(34990, 35010), slice(M - 50, M)):
        want, _, bound, _ = step.linear(x[rows], W)
        near(y[rows], want, bound)
    g = binding.linear_grad(dsp, x, W, y, dW=False)
    done(dsp)
    for rows in (slice(0, 50), slice(M - 50, M)):
        near(g["dx"][rows], *step.linear_grad(x[rows], W, y[rows])["dx"])


def test_workspace_of_the_caller(dsp):
    """Rows that do not start on 16-byte boundaries need a workspace: too small a one is refused with
    the size, the size suffices, and nothing beyond it is written."""
    import ctypes
    x, W = make(1, 100, 33, 77)
    dy, pre = normal(2, 100, 77), normal(3, 100, 77)
    y = torch.empty(100, 77, device="cuda")
    out = dict(dx=torch.empty_like(x), dW=torch.empty(33, 77, device="cuda"), db=torch.empty(77, device="cuda"))
    p = lambda t: t.data_ptr()  # noqa: E731

    def forward(ws, n):
        return dsp.lib.dspark_linear(dsp.handle, p(x), 33, p(W), 77, None, 0, None, 0, 0, 100, 33, 77, p(y), 0, 77, None, 0, ws, n,
                                     torch.cuda.current_stream().cuda_stream)

    def backward(ws, n):
        return dsp.lib.dspark_linear_grad(dsp.handle, p(x), 33, p(W), 77, p(dy), 0, 77, 4, p(pre), 0, 77, 100, 33, 77, p(out["dx"]),
                                          1, 33, p(out["dW"]), 0, 77, p(out["db"]), ws, n, torch.cuda.current_stream().cuda_stream)

    for call in (forward, backward):
        n = ctypes.c_int64(0)
        assert call(None, ctypes.byref(n)) == binding.CAPACITY and n.value > 0
        need = n.value
        n = ctypes.c_int64(need - 1)
        ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
        assert call(ws.data_ptr(), ctypes.byref(n)) == binding.CAPACITY and n.value == need
        assert call(ws.data_ptr(), ctypes.byref(n)) == 0
        done(dsp)
        assert (ws[need:] == 77).all()
    want, _, bound, _ = step.linear(x, W)
    near(y, want, bound)
    for name, (want, bound) in zip(("dx", "dW", "db"), step.linear_grad(x, W, dy, "silu", pre).values()):
        near(out[name], want, bound)
    x, W = make(1, 100, 64, 80)
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    binding.linear(dsp, x, W, workspace=ws)
    binding.linear_grad(dsp, x, W, normal(2, 100, 80).to(BF16), workspace=ws)
    done(dsp)


@pytest.mark.parametrize("N", [640, 77])
def test_side_stream_and_graph(dsp, N):
    M, K = 300, 128
    x, W = make(1, M, K, N)
    dy = normal(2, M, N)
    want, want_g = binding.linear(dsp, x, W, act="gelu", pre=True), None
    want_g = binding.linear_grad(dsp, x, W, dy, act="gelu", pre=want["pre"], dbias=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.linear(dsp, x, W, act="gelu", pre=True, stream=side)
    got_g = binding.linear_grad(dsp, x, W, dy, act="gelu", pre=got["pre"], dbias=True, stream=side)
    side.synchronize()
    assert torch.equal(got["y"], want["y"]) and all(torch.equal(got_g[n], want_g[n]) for n in want_g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.linear(dsp, x, W, act="gelu", pre=True)
        out_g = binding.linear_grad(dsp, x, W, dy, act="gelu", pre=out["pre"], dbias=True)
    for seed in (4, 6):
        x.copy_(make(seed, M, K, N)[0])
        dy.copy_(normal(seed, M, N))
        graph.replay()
        done(dsp)
        y, z, ey, ez = step.linear(x, W, None, "gelu")
        near(out["y"], y, ey)
        for name, (w, b) in step.linear_grad(x, W, dy, "gelu", out["pre"]).items():
            near(out_g[name], w, b, name)


BOTH = [(700, 256, 50000, None, BF16), (3000, 136, 12000, None, BF16), (300, 200, 40008, "silu", BF16), (257, 64, 50008, None, F32),
        (140, 520, 100000, "sigmoid", F32)]


@pytest.mark.parametrize("dw_dtype", [F32, BF16])
@pytest.mark.parametrize("M,K,N,act,dtype", BOTH)
def test_both_products_of_a_large_gradient(dsp, M, K, N, act, dtype, dw_dtype):
    """dz beyond what L2 keeps: both products in one launch, of one to three parts."""
    x, W = make(M, M, K, N)
    dy, pre = (normal(1, M, N) / M).to(dtype), normal(2, M, N).to(BF16) if act else None
    dW = torch.full_like(W, 9.0, dtype=dw_dtype)
    out = binding.linear_grad(dsp, x, W, dy, act=act, pre=pre, dW=dW)
    done(dsp)
    want = step.linear_grad(x, W, dy, act, pre)
    near(out["dx"], *want["dx"], "dx")
    near(dW, *want["dW"], "dW")
    again = binding.linear_grad(dsp, x, W, dy, act=act, pre=pre, dW=torch.empty_like(dW))
    assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["dW"], dW)


@pytest.mark.parametrize("M,K,N,act", [(1100, 64, 31080, None), (1100, 130, 31240, None), (700, 65, 48008, None), (2048, 60, 17000, None),
                                       (2048, 1024, 8360, "sigmoid"), (3000, 256, 5001, "tanh"), (5000, 64, 120, "relu")])
def test_gradients_of_tiles_that_reach_beyond(dsp, M, K, N, act):
    """Tiles of which whole boxes lie outside, in one launch or two, and the column sums of many parts."""
    x, W = make(M, M, K, N)
    dy, pre = (normal(1, M, N) / M).to(BF16), normal(2, M, N).to(BF16) if act else None
    out = binding.linear_grad(dsp, x, W, dy, act=act, pre=pre, dbias=True)
    done(dsp)
    for name, (want, bound) in step.linear_grad(x, W, dy, act, pre).items():
        near(out[name], want, bound, name)
    again = binding.linear_grad(dsp, x, W, dy, act=act, pre=pre, dbias=True)
    assert all(torch.equal(again[name], out[name]) for name in out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(1000, 2000, 1000), (3000, 1500, 1400), (2000, 1024, 4096), (257, 9000, 264)])
def test_products_that_bound_the_time(dsp, M, K, N, dtype):
    """Many stages a tile: pairs of blocks, splits, accumulators that start again."""
    x, W = make(M + K, M, K, N)
    check(dsp, x, W, dtype=dtype, bias=normal(5, N), act="sigmoid")
    check_grad(dsp, x, W, normal(9, M, N).to(BF16), dx_dtype=dtype)


def test_rows_wherever_they_lie_give_equal_bits(dsp):
    for M, K, N in ((1000, 2000, 1000), (520, 256, 3000)):
        x, W = make(1, M, K, N)
        want = binding.linear(dsp, x, W, dtype=F32)["y"]
        out = wide(torch.zeros(M, N, device="cuda"), 1)[1]
        binding.linear(dsp, wide(x, 3, 1)[1], wide(W, 5, 2)[1], out=out)
        done(dsp)
        assert torch.equal(out, want)


@pytest.mark.parametrize("backward,N,cta", [(False, 512, 0), (False, 512, 1), (True, 512, 0), (True, 512, 1), (True, 50000, 0),
                                            (True, 50000, 1), (True, 50000, 100)])
def test_waits_that_run_out(backward, N, cta):
    """A block that loads nothing: its waits end, the status says so, and the context works again."""
    x, W = make(1, 700, 128, N)
    with binding.Context(0, B_max=1, V_max=4096, K_max=1) as ctx:
        ctx.debug_set(cta=cta, timeout_ms=20)
        if backward:
            binding.linear_grad(ctx, x, W, normal(2, 700, N).to(BF16))
        else:
            binding.linear(ctx, x, W)
        torch.cuda.synchronize()
        assert ctx.status() == binding.TIMEOUT
        with pytest.raises(binding.DSparkError):
            binding.linear(ctx, x, W)
        ctx.reset()
        check(ctx, x, W)
        dy = normal(2, 700, N).to(BF16)
        out, want = binding.linear_grad(ctx, x, W, dy), step.linear_grad(x, W, dy)
        done(ctx)
        near(out["dx"], *want["dx"])
        near(out["dW"], *want["dW"])
