"""GPU parity of verification from given probabilities and random numbers
(dspark_verify_probs) against the 64-bit statement.

Tokens and counts are decided by comparisons of exact products and of sums kept to 2^-48, so
they are equal; an acceptance probability is one division in 32 bits, off by half a step."""

import numpy as np
import pytest
import torch

from oracle import training as tr
from rank_markov_draft_gb300 import binding
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

HALF = torch.finfo(torch.float32).eps / 2


def make(seed, B, K, V, m=0, spread=2.0, noise=1.0):
    rng = np.random.default_rng(seed)
    U = rng.normal(0, spread, (B, K, V))
    T = np.concatenate([U + rng.normal(0, noise, (B, K, V)), rng.normal(0, spread, (B, 1, V))], 1)
    soft = lambda x: (np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
    a = dict(P=soft(T), Q=None, cand=None, cand_q=None)
    if m:
        a["cand"] = np.argsort(-U, 2)[:, :, :m].astype(np.int32)
        a["cand_q"] = soft(np.take_along_axis(U, a["cand"].astype(np.int64), 2))
        slot = (a["cand_q"].cumsum(2) < rng.random((B, K, 1))).sum(2).clip(0, m - 1)
        a["tokens"] = np.take_along_axis(a["cand"], slot[..., None], 2)[..., 0].astype(np.int32)
    else:
        a["Q"] = soft(U)
        a["tokens"] = (a["Q"].cumsum(2) < rng.random((B, K, 1))).sum(2).clip(0, V - 1).astype(np.int32)
    a["u_accept"] = rng.random((B, K)).astype(np.float32)
    a["u_draw"] = rng.random(B).astype(np.float32)
    a["ell"] = None
    return a


def call(ctx, a, **kw):
    up = {k: None if v is None else dev(v) for k, v in a.items()}
    return binding.verify_probs(ctx, up["P"], up["tokens"], up["u_accept"], up["u_draw"], Q=up["Q"], cand=up["cand"],
                                cand_q=up["cand_q"], ell=up["ell"], **kw)


def check(ctx, a):
    out = call(ctx, a)
    torch.cuda.synchronize()
    assert ctx.status() == 0
    n, t, p = tr.verify_probs(a["P"], a["tokens"], a["u_accept"], a["u_draw"], Q=a["Q"], cand=a["cand"],
                              cand_q=a["cand_q"], ell=a["ell"])
    assert np.array_equal(host(out["n_acc"]), n)
    assert np.array_equal(host(out["next_token"]), t)
    assert np.all(np.abs(host(out["accept_prob"]) - p) <= HALF * np.abs(p))
    return n, t


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 32, 127, 128, 129, 1000, 4099, 32003, 50000])
@pytest.mark.parametrize("m", [0, 3])
def test_vocabularies(dsp, V, m):
    B, K = (9, 4) if V < 5000 else (5, 3)
    check(dsp, make(V + m, B, K, V, min(m, V)))


@pytest.mark.parametrize("V", [15359, 15360, 15361, 15364, 30720, 30721])
@pytest.mark.parametrize("m", [0, 20])
def test_around_the_tokens_of_one_cta(dsp, V, m):
    """Up to 15,360 tokens one CTA makes a request's tests and its draw."""
    a = make(V + m, 6, 3, V, m, noise=0.5)
    a["ell"] = np.array([0, 1, 2, 3, 3, 3], np.int32)
    check(dsp, a)


@pytest.mark.parametrize("B,V", [(1101, 40), (1030, 15364)])
def test_more_requests_than_a_launch_takes(dsp, B, V):
    check(dsp, make(B, B, 1, V, noise=0.3))


@pytest.mark.parametrize("B,K", [(1, 1), (1, 64), (3, 33), (200, 2)])
def test_batches_and_blocks(dsp, B, K):
    n, _ = check(dsp, make(B + K, B, K, 517, noise=0.3))
    if B == 200:
        assert set(n) == {0, 1, 2}


def test_full_vocabulary(dsp):
    check(dsp, make(3, 2, 2, 151936))
    check(dsp, make(4, 1, 1, 1 << 18))
    check(dsp, make(5, 2, 2, 151935, 16))


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 256])
def test_candidates(dsp, m):
    a = make(m, 40, 5, 1201, m, noise=0.5)
    check(dsp, a)
    a["cand"][::2, :, m // 2:] = -1  # empty slots, and a repeated id whose first slot counts
    a["cand"][:, :, m - 1] = a["cand"][:, :, 0]
    check(dsp, a)


def test_windows(dsp):
    a = make(8, 12, 6, 301, noise=0.2)
    a["ell"] = np.array([0, 1, 2, 3, 4, 5, 6, 7, -3, 100, 0, 6], np.int32)
    check(dsp, a)


def test_random_numbers_at_their_ends(dsp):
    for u in (0.0, 1.0 - 2.0 ** -24):
        a = make(9, 30, 3, 777)
        a["u_draw"][:] = u
        check(dsp, a)
        a["u_accept"][:] = u
        check(dsp, a)


def test_rows_without_mass(dsp):
    """Nothing left over (p = q), a target row that is all zero, tokens of no probability, and
    entries that are negative, infinite or NaN (which have no mass)."""
    a = make(10, 16, 3, 263)
    a["P"][0, :3] = a["Q"][0]
    a["P"][1] = 0.0
    a["tokens"][2:5] = 7
    a["P"][2, :, 7] = 0.0
    a["P"][3, :, 7] = np.nan
    a["P"][4, :, 7] = -1.0
    a["Q"][5] = 0.0
    a["Q"][6] = np.nan
    a["Q"][7, :, ::2] = np.inf
    a["P"][8, :, ::3] = np.inf
    a["P"][9, :, ::3] = np.nan
    a["P"][10, :, ::2] = -0.5
    a["P"][11] = 0.0
    a["P"][11, :, 262] = 1e-38
    # the compared acceptance probabilities are those of finite pairs
    out = call(dsp, a)
    torch.cuda.synchronize()
    assert dsp.status() == 0
    n, t, p = tr.verify_probs(a["P"], a["tokens"], a["u_accept"], a["u_draw"], Q=a["Q"])
    assert np.array_equal(host(out["n_acc"]), n) and np.array_equal(host(out["next_token"]), t)
    fine = [0, 1, 2, 5, 11, 12, 13, 14, 15]
    assert np.all(np.abs(host(out["accept_prob"])[fine] - p[fine]) <= HALF * np.abs(p[fine]))
    assert t[1] == -1


@pytest.mark.parametrize("V", [263, 20004])  # one CTA; several, in 16-byte pieces
@pytest.mark.parametrize("m", [0, 5])
def test_entries_that_are_no_probabilities(dsp, V, m):
    """A p that is negative or not finite is nothing, a negative q likewise; a token whose q is
    infinite or NaN is rejected and left out: the acceptance probability, the test and the
    draw agree on each, one such entry among good ones and whole rows of them."""
    a = make(V + m, 64, 3, V, m, noise=0.5)
    rng = np.random.default_rng(V)
    q = a["cand_q"] if m else a["Q"]
    values = [np.nan, np.inf, -np.inf, -0.25]
    for b in range(64):
        p_bad, q_bad = values[b % 4], values[b // 4 % 4]
        x = a["tokens"][b]
        if b & 16:  # the drafted token's p
            a["P"][b, np.arange(3), x] = p_bad
        if b & 32:  # and its q
            if m:
                q[b][a["cand"][b] == x[:, None]] = q_bad
            else:
                q[b, np.arange(3), x] = q_bad
        if b & 48 == 0:  # many entries of both
            a["P"][b][rng.random((4, V)) < 0.3] = p_bad
            q[b][rng.random(q[b].shape) < 0.3] = q_bad
    check(dsp, a)
    a["u_accept"][:] = 0.0
    check(dsp, a)


def test_acceptance_probability_of_every_row_without_mass(dsp):
    """The rows of test_rows_without_mass, all compared."""
    a = make(10, 16, 3, 263)
    a["tokens"][2:5] = 7
    a["P"][2, :, 7], a["P"][3, :, 7], a["P"][4, :, 7] = 0.0, np.nan, -1.0
    a["Q"][5], a["Q"][6] = 0.0, np.nan
    a["Q"][7, :, ::2] = np.inf
    a["P"][8, :, ::3], a["P"][9, :, ::3], a["P"][10, :, ::2] = np.inf, np.nan, -0.5
    a["tokens"][7:11] = 6
    check(dsp, a)


def test_tiny_mass_decides(dsp):
    """A row of one large and many rare tokens: the draw lands among the rare ones, whose
    probabilities a 32-bit running sum would lose beside the large one."""
    V = 40000
    a = make(12, 64, 1, V)
    a["P"][:, :, 0] = 1.0
    a["P"][:, :, 1:] = 2.0 ** -40
    a["Q"][:] = 0.0
    a["Q"][:, :, 5] = 1.0
    a["tokens"][:] = 5
    a["u_accept"][:] = 0.5
    a["u_draw"] = (1.0 - 2.0 ** -24 * np.arange(1, 65)).astype(np.float32)
    check(dsp, a)
    a["P"][:, :, 0] = 2.0 ** -22  # rare tokens' whole mass about 2^-25 of it
    check(dsp, a)


def test_token_out_of_range_is_reported():
    a = make(13, 2, 2, 100)
    a["tokens"][1, 0] = 100
    with binding.Context(0, B_max=1, V_max=8, K_max=1) as ctx:
        call(ctx, a)
        torch.cuda.synchronize()
        assert ctx.status() == binding.DEVICE_OOB


def test_offsets_past_32_bits(dsp):
    """P of 2^32 + entries; the last request's rows lie beyond the 32-bit range."""
    B, K, V = 1030, 15, 1 << 18
    P = torch.zeros(B, K + 1, V, device="cuda")
    P[B - 1, :, V - 3] = 1.0
    cand = torch.full((B, K, 1), V - 3, dtype=torch.int32, device="cuda")
    q = torch.ones(B, K, 1, device="cuda")
    u = torch.full((B, K), 0.25, device="cuda")
    out = binding.verify_probs(dsp, P, cand[:, :, 0].contiguous(), u, u[:, 0].contiguous(), cand=cand, cand_q=q)
    assert host(out["n_acc"]).tolist() == [0] * (B - 1) + [K]
    assert host(out["next_token"]).tolist() == [-1] * (B - 1) + [V - 3]


def test_misaligned_rows_side_stream_and_graph(dsp):
    """Tensors that start 4 bytes after a 16-byte boundary, on another stream, then replayed
    from a graph on new random numbers."""
    a = make(14, 6, 3, 1000)
    up = {k: dev(a[k]) for k in ("tokens", "u_accept", "u_draw")}
    shift = lambda x: torch.cat([torch.zeros(1, device="cuda"), dev(x).flatten()])[1:].view(x.shape)  # noqa: E731
    P, Q = shift(a["P"]), shift(a["Q"])
    assert P.data_ptr() % 16 == 4
    want = tr.verify_probs(a["P"], a["tokens"], a["u_accept"], a["u_draw"], Q=a["Q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = binding.verify_probs(dsp, P, up["tokens"], up["u_accept"], up["u_draw"], Q=Q)
    side.synchronize()
    assert np.array_equal(host(out["next_token"]), want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.verify_probs(dsp, P, up["tokens"], up["u_accept"], up["u_draw"], Q=Q)
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        a["u_accept"], a["u_draw"] = rng.random((6, 3)).astype(np.float32), rng.random(6).astype(np.float32)
        up["u_accept"].copy_(dev(a["u_accept"]))
        up["u_draw"].copy_(dev(a["u_draw"]))
        graph.replay()
        torch.cuda.synchronize()
        want = tr.verify_probs(a["P"], a["tokens"], a["u_accept"], a["u_draw"], Q=a["Q"])
        assert np.array_equal(host(out["n_acc"]), want[0]) and np.array_equal(host(out["next_token"]), want[1])


def test_selector_drafts_are_verified(dsp):
    """The walk's drafts: candidates and their probabilities under the walk, verified against a
    target, agree with the statement on the same numbers."""
    rng = np.random.default_rng(21)
    B, K, V, r = 8, 4, 2048, 64
    U = dev(rng.normal(0, 3, (B, K, V)).astype(np.float32))
    A, Bt = (torch.randn(V, r, device="cuda").mul_(0.3).to(torch.bfloat16) for _ in range(2))
    anchors = dev(rng.integers(0, V, B).astype(np.int32))
    sc = binding.selector_scores(dsp, U, A, Bt, anchors, topk=16)
    walk = binding.selector_walk(dsp, sc["cand"], sc["scores"], anchors, V=V, temperature=1.0, seed=3)
    tok, cand = host(walk["tokens"]), host(sc["cand"])
    slot = (cand == tok[..., None]).argmax(2)
    came = np.concatenate([np.zeros((B, 1), np.int64), slot[:, :-1]], 1)
    s = np.take_along_axis(host(sc["scores"]), came[:, :, None, None], 2)[:, :, 0].astype(np.float64)
    q = (np.exp(s - s.max(2, keepdims=True)) / np.exp(s - s.max(2, keepdims=True)).sum(2, keepdims=True)).astype(np.float32)
    assert np.abs(np.log(np.take_along_axis(q, slot[..., None], 2)[..., 0]) - host(walk["logprobs"])).max() < 1e-4
    P = torch.softmax(torch.cat([U + torch.randn_like(U), U[:, :1]], 1), 2)
    a = dict(P=host(P), Q=None, cand=cand, cand_q=q, tokens=tok, ell=None,
             u_accept=rng.random((B, K)).astype(np.float32), u_draw=rng.random(B).astype(np.float32))
    check(dsp, a)


def test_refusals(dsp):
    a = make(15, 2, 2, 64)
    up = {k: None if v is None else dev(v) for k, v in a.items()}
    with pytest.raises(binding.DSparkError) as err:  # no draft probabilities
        binding.verify_probs(dsp, up["P"], up["tokens"], up["u_accept"], up["u_draw"])
    assert err.value.code == binding.INVALID_ARG
    with pytest.raises(ValueError, match="contiguous"):
        binding.verify_probs(dsp, up["P"].transpose(0, 1).contiguous().transpose(0, 1), up["tokens"], up["u_accept"],
                             up["u_draw"], Q=up["Q"])
    with pytest.raises(TypeError, match="dtype"):
        binding.verify_probs(dsp, up["P"].double(), up["tokens"], up["u_accept"], up["u_draw"], Q=up["Q"])
