"""Calls with stream=: their outputs and workspaces are memory of that stream, which work still queued on the
caller's does not use, although neither stream waits for the other."""

import pytest
import torch

from rank_markov_draft_gb300 import binding
from tests.test_gpu_embed import done, normal, tokens

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def owner(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for v in (out.values() if isinstance(out, dict) else out) for t in tensors(v)]


def calls(ctx):
    x, W, dy = normal(1, 70, 33).to(BF16), normal(2, 33, 50).to(BF16), normal(3, 70, 50)
    ids, table = tokens(4, 70, 300), normal(5, 300, 40)
    e, reset = normal(6, 3, 20, 16).to(BF16), None
    s = binding.rnn_scan(ctx, e, e, e)["s"]
    logits, top = normal(7, 6, 500), torch.topk(normal(8, 6, 500), 5)
    teacher = top.indices.int(), top.values.contiguous()
    P, drafted = torch.softmax(normal(9, 2, 4, 100), 2), tokens(10, 6, 100, padding=0.0).view(2, 3)
    u, cand = torch.rand(2, 3, device="cuda"), torch.rand(2, 3, 100, device="cuda")
    U, W1, W2 = normal(11, 2, 4, 512), normal(12, 512, 32).to(BF16), normal(13, 32, 512).to(BF16)
    anchors = torch.tensor([3, 500], dtype=torch.int32, device="cuda")
    return dict(
        embed=lambda **k: binding.embed(ctx, table, ids, **k),
        embed_grad=lambda **k: binding.embed_grad(ctx, ids, dy, 300, **k),
        grad_norm=lambda **k: binding.grad_norm(ctx, [dy, x], **k),
        clip_grads=lambda **k: binding.clip_grads(ctx, [dy, x], 1e9, **k),
        linear=lambda **k: binding.linear(ctx, x, W, act="silu", pre=True, **k),
        linear_grad=lambda **k: binding.linear_grad(ctx, x, W, dy, act="tanh", pre=dy, dbias=True, **k),
        rnn_scan=lambda **k: binding.rnn_scan(ctx, e, e, e, **k),
        rnn_scan_grad=lambda **k: binding.rnn_scan_grad(ctx, e, e, e, s, e, **k),
        distill=lambda **k: binding.distill(ctx, logits, *teacher, **k),
        verify_probs=lambda **k: binding.verify_probs(ctx, P, drafted, u, u[:, 0].contiguous(), Q=cand, **k),
        markov_draft=lambda **k: binding.markov_draft(ctx, U, W1, W2, anchors, **k),
        markov_logits=lambda **k: binding.markov_logits(ctx, U, W1, W2, drafted.repeat(1, 2)[:, :4].contiguous(), **k),
    )


NAMES = ["embed", "embed_grad", "grad_norm", "clip_grads", "linear", "linear_grad", "rnn_scan", "rnn_scan_grad", "distill",
         "verify_probs", "markov_draft", "markov_logits"]


@pytest.mark.parametrize("by_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_lie_in_the_calls_stream(dsp, name, by_handle):
    call = calls(dsp)[name]
    want = [t.clone() for t in tensors(call())]
    done(dsp)
    side = torch.cuda.Stream()
    got = tensors(call(stream=side.cuda_stream if by_handle else side))
    done(dsp)
    assert all(owner(t) == side.cuda_stream for t in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want)


@pytest.mark.parametrize("backward", [False, True])
def test_workspace_lies_in_the_calls_stream(dsp, backward):
    """Nothing but a workspace of 16 MB is left to allocate."""
    M, K, N = 4096, 1000, 63
    x, W, dy = normal(1, M, K + 1)[:, :K].to(BF16), normal(2, K, N).to(BF16), normal(3, M, N)
    x = torch.zeros(M, K + 1, dtype=BF16, device="cuda")[:, 1:].copy_(x)
    y, dx, dW = torch.empty(M, N, dtype=BF16, device="cuda"), torch.empty(M, K, dtype=BF16, device="cuda"), torch.empty(K, N, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    size = lambda: {s: sum(g["total_size"] for g in torch.cuda.memory_snapshot() if g["stream"] == s)  # noqa: E731
                    for s in (torch.cuda.current_stream().cuda_stream, side.cuda_stream)}
    side = torch.cuda.Stream()
    before = size()
    if backward:
        binding.linear_grad(dsp, x, W, dy, dx=dx, dW=dW, stream=side)
    else:
        binding.linear(dsp, x, W, out=y, stream=side)
    done(dsp)
    after = size()
    mine, sides = torch.cuda.current_stream().cuda_stream, side.cuda_stream
    assert after[mine] == before[mine] and after[sides] - before[sides] >= 2 * M * K


def test_work_queued_on_the_callers_stream_keeps_its_memory(dsp):
    """A tensor freed while its last reading is queued; a call on a side stream that runs at once, of outputs and a
    workspace of the same size; and the other way round, an output dropped while the side stream still writes it."""
    M, N, K = 4096, 4096, 40
    x, W = normal(1, M, K).to(BF16), normal(2, K, N + 1).to(BF16)[:, 1:]
    big, ones = normal(3, 4096, 4096), torch.ones(N, N, dtype=BF16, device="cuda")
    want = binding.linear(dsp, x, W, dtype=F32)["y"]
    done(dsp)
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()

    def busy():
        y = big
        for _ in range(40):  # some milliseconds
            y = (big @ y).mul_(1e-2)

    with torch.cuda.stream(side):
        busy()
    busy()
    torch.cuda.synchronize()
    freed = [torch.full((M, N), 3.0, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    busy()
    sums = [t.double().sum() for t in freed]
    del freed
    got = [binding.linear(dsp, x, W, dtype=F32, stream=side)["y"] for _ in range(6)]
    torch.cuda.synchronize()
    assert all(float(s) == 3.0 * M * N for s in sums) and all(torch.equal(g, want) for g in got)
    del got
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    for _ in range(6):
        binding.linear(dsp, x, W, dtype=F32, stream=side)  # dropped at once
    fills = [torch.full((M, N), 5.0, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    assert all((t == 5.0).all() for t in fills) and ones.sum() > 0
    assert dsp.status() == 0


def test_captured_on_a_forked_stream(dsp):
    x, W = normal(1, 300, 33).to(BF16), normal(2, 33, 77).to(BF16)
    want = binding.linear(dsp, x, W, act="tanh")["y"]
    done(dsp)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = binding.linear(dsp, x, W, act="tanh", stream=side)["y"]
        binding.linear(dsp, x, W, act="tanh", stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for scale in (1.0, 2.0):
        x.mul_(scale)
        want = binding.linear(dsp, x, W, act="tanh")["y"]
        got.zero_()
        graph.replay()
        done(dsp)
        assert torch.equal(got, want)
