"""Routing by scores (moe_select, moe_route_scored) against its definition in
float64, and its refusals.

The chosen experts are compared for equality: the choice is made on scores in 64
bits, whose rounding (about 2^-52) moves no order of the drawn values, and
where values are equal by construction the lower id has to come first. Weights
are formed in 64 bits and rounded once (2^-24), except for the softmax over all
experts, whose float32 terms may each be off by 2^-22 (exponential and its
argument) and whose sum by 2^-24 for each of at most 22 additions in a row: 30 x 2^-24 with
the last rounding.
"""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import expert_token_routing_amd as M
from expert_token_routing_amd import _binding as B
from tests.gpu_helpers import device, say

F32 = torch.float32
FAKE = ctypes.c_void_p(0x10000)
gpu = pytest.mark.gpu


def oracle(logits, bias, k, score="softmax", n_group=1, topk_group=1, group_score="max", renormalize=True, scale=1.0):
    """(ids, weights) in float64, token by token."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    nan = np.isnan(l)
    l = np.where(nan, -np.inf, l)
    ids, ws = np.zeros((T, k), np.int64), np.zeros((T, k))
    n = E // n_group
    with np.errstate(all="ignore"):
        for t in range(T):
            m = l[t].max()
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-l[t]))
            else:
                s = np.where(l[t] == m, 1.0, np.exp(l[t] - m))
                s = s / math.fsum(s)
            c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
            c = np.where(nan[t] | np.isnan(c), -np.inf, c)
            value = []
            for g in range(n_group):
                part = sorted(c[g * n:(g + 1) * n], reverse=True)
                v = part[0] + part[1] if group_score == "top2" and n > 1 else part[0]
                value.append(-np.inf if np.isnan(v) else v)
            kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            among = sorted(e for g in kept for e in range(g * n, (g + 1) * n))
            ids[t] = sorted(among, key=lambda e: (-c[e], e))[:k]
            w = s[ids[t]]
            ws[t] = np.nan if m == -np.inf else scale * (w / w.sum() if renormalize else w)
    return ids, ws


def check(logits, bias, k, **kw):
    dev = device()
    say(f"select T={logits.shape[0]} E={logits.shape[1]} k={k} bias={bias is not None} {kw}")
    idx, w = M.moe_select(logits.to(dev), k, None if bias is None else bias.to(dev), **kw)
    want_i, want_w = oracle(logits.numpy(), None if bias is None else bias.numpy(), k, **kw)
    assert idx.dtype == torch.int32 and w.dtype == F32
    np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
    steps = 30 if kw.get("score", "softmax") == "softmax" and not kw.get("renormalize", True) else 2
    got = w.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want_w))
    assert np.all((np.abs(got - want_w) <= steps * 2.0 ** -24 * np.abs(want_w) + 2.0 ** -149) | np.isnan(want_w))
    return idx, w


def draw(T, E, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, E, generator=g) * spread, torch.randn(E, generator=g) * 0.1


# --------------------------------------------------------------------------- #
# Refusals (CPU)                                                               #
# --------------------------------------------------------------------------- #
SELECT = dict(logits=FAKE, bias=FAKE, T=4, E=64, k=4, score=1, G=8, top=2, rule=1, renorm=1, scale=1.0, idx=FAKE, w=FAKE)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), M.MOE_ERR_INVALID_ARG), (dict(E=0), M.MOE_ERR_INVALID_ARG), (dict(k=0), M.MOE_ERR_INVALID_ARG),
    (dict(k=65), M.MOE_ERR_INVALID_ARG), (dict(k=17), M.MOE_ERR_INVALID_ARG),        # two groups hold 16
    (dict(score=2), M.MOE_ERR_INVALID_ARG), (dict(score=-1), M.MOE_ERR_INVALID_ARG),
    (dict(rule=2), M.MOE_ERR_INVALID_ARG), (dict(rule=-1), M.MOE_ERR_INVALID_ARG),
    (dict(G=0), M.MOE_ERR_INVALID_ARG), (dict(G=7), M.MOE_ERR_INVALID_ARG), (dict(top=0), M.MOE_ERR_INVALID_ARG),
    (dict(top=9), M.MOE_ERR_INVALID_ARG), (dict(scale=math.nan), M.MOE_ERR_INVALID_ARG),
    (dict(scale=math.inf), M.MOE_ERR_INVALID_ARG), (dict(logits=None), M.MOE_ERR_INVALID_ARG),
    (dict(idx=None), M.MOE_ERR_INVALID_ARG), (dict(w=None), M.MOE_ERR_INVALID_ARG),
    (dict(E=1032), M.MOE_ERR_UNSUPPORTED), (dict(E=128, G=128, top=64), M.MOE_ERR_UNSUPPORTED),
    (dict(E=64, k=33, G=1, top=1), M.MOE_ERR_UNSUPPORTED), (dict(T=2 ** 30), M.MOE_ERR_UNSUPPORTED),
    (dict(T=0, logits=None, idx=None, w=None), M.MOE_OK),
])
def test_select_rejects(kw, want):
    a = {**SELECT, **kw}
    assert M.lib().moe_select(a["logits"], a["bias"], a["T"], a["E"], a["k"], a["score"], a["G"], a["top"], a["rule"],
                              a["renorm"], a["scale"], a["idx"], a["w"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(H=12), M.MOE_ERR_INVALID_ARG), (dict(k=17), M.MOE_ERR_INVALID_ARG), (dict(score=5), M.MOE_ERR_INVALID_ARG),
    (dict(x=None), M.MOE_ERR_INVALID_ARG), (dict(x=ctypes.c_void_p(0x10004)), M.MOE_ERR_INVALID_ARG),
    (dict(logits=None), M.MOE_ERR_INVALID_ARG), (dict(ws=None), M.MOE_ERR_WORKSPACE), (dict(nws=16), M.MOE_ERR_WORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10010)), M.MOE_ERR_WORKSPACE), (dict(T=0, x=None), M.MOE_OK),
])
def test_route_scored_rejects(kw, want):
    a = {**SELECT, "x": FAKE, "wr": FAKE, "H": 64, "ws": FAKE, "nws": 1 << 30, **kw}
    assert M.lib().moe_route_scored(a["x"], a["wr"], None, a["bias"], a["T"], a["H"], a["E"], a["k"], a["score"], a["G"],
                                    a["top"], a["rule"], a["renorm"], a["scale"], a["logits"], a["idx"], a["w"], a["ws"],
                                    a["nws"], None) == want


def test_select_rejects_mismatched_tensors():
    l = torch.zeros(4, 64)
    for kw, exc, match in ((dict(logits=l.double()), TypeError, "logits must be"), (dict(logits=l[0]), ValueError, "logits has"),
                           (dict(bias=torch.zeros(63)), ValueError, "bias has shape"), (dict(k=0), ValueError, "k must be"),
                           (dict(k=2.0), ValueError, "k must be"), (dict(k=65), ValueError, "k must be"),
                           (dict(score="tanh"), ValueError, "score must be one of"), (dict(score=1), ValueError, "score must be"),
                           (dict(group_score="sum"), ValueError, "group_score must be"),
                           (dict(n_group=7), ValueError, "do not divide"), (dict(n_group=0), ValueError, "n_group must be"),
                           (dict(n_group=8, topk_group=9), ValueError, "exceeds n_group"),
                           (dict(n_group=8, topk_group=1, k=9), ValueError, "exceeds the 8 experts"),
                           (dict(topk_idx=torch.zeros(4, 5, dtype=torch.int32)), ValueError, "topk_idx has shape"),
                           (dict(topk_w=torch.zeros(4, 4, dtype=torch.float64)), TypeError, "topk_w must be"),
                           (dict(), ValueError, "must live on a GPU")):
        a = dict(logits=l, k=4)
        a.update(kw)
        with pytest.raises(exc, match=match):
            M.moe_select(a.pop("logits"), a.pop("k"), **a)
    x, wr = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64)
    for kw, exc, match in ((dict(choice_bias=torch.zeros(15)), ValueError, "choice_bias has shape"),
                           (dict(n_group=3), ValueError, "do not divide"), (dict(score=""), ValueError, "score must be"),
                           (dict(logits=torch.zeros(4, 15)), ValueError, "logits has shape"),
                           (dict(), ValueError, "must live on a GPU")):
        a = dict(bias=None, choice_bias=None, k=4)
        a.update(kw)
        with pytest.raises(exc, match=match):
            M.moe_route_scored(x, wr, **a)


# --------------------------------------------------------------------------- #
# Against the definition                                                       #
# --------------------------------------------------------------------------- #
SHAPES = [  # T, E, k, groups, of which stay
    (1, 256, 8, 8, 4), (5, 256, 8, 8, 4), (130, 256, 8, 8, 4), (67, 256, 16, 4, 1), (33, 256, 8, 1, 1), (21, 256, 3, 32, 5),
    (9, 256, 20, 8, 4), (40, 128, 6, 4, 2), (19, 128, 1, 16, 16), (50, 64, 6, 8, 3), (17, 64, 4, 64, 7), (70, 32, 4, 1, 1),
    (31, 32, 2, 8, 2), (3, 1, 1, 1, 1), (13, 7, 7, 7, 7), (11, 33, 5, 3, 2), (29, 100, 9, 10, 3), (23, 160, 6, 8, 3),
    (12, 160, 6, 16, 2), (6, 257, 8, 1, 1), (8, 384, 8, 1, 1), (7, 512, 10, 8, 4), (5, 1000, 32, 8, 4), (4, 1024, 32, 64, 5),
    (2051, 256, 8, 8, 4), (2049, 64, 8, 1, 1),
]


@gpu
@pytest.mark.parametrize("T,E,k,G,top", SHAPES)
def test_matches_the_definition(T, E, k, G, top):
    kinds = list(itertools.product(("sigmoid", "softmax"), ("max", "top2"), (False, True), (False, True)))
    for i, (score, rule, with_bias, renorm) in enumerate(kinds if T < 1000 else kinds[::5]):
        logits, bias = draw(T, E, seed=100 * i + E)
        check(logits, bias if with_bias else None, k, score=score, n_group=G, topk_group=top, group_score=rule,
              renormalize=renorm, scale=1.0 if i % 2 else 2.5)


@gpu
@pytest.mark.parametrize("E,G,top,k", [(256, 8, 4, 8), (64, 1, 1, 8), (160, 8, 3, 6), (1000, 10, 4, 12)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_id(E, G, top, k, score):
    g = torch.Generator().manual_seed(E)
    for values in (1, 2, 5):  # few values: nearly everything is tied, groups too
        logits = torch.randint(0, values, (37, E), generator=g).float()
        bias = 0.25 * torch.randint(0, 2, (E,), generator=g).float()
        for rule in ("max", "top2"):
            check(logits, None, k, score=score, n_group=G, topk_group=top, group_score=rule)
            check(logits, torch.zeros(E), k, score=score, n_group=G, topk_group=top, group_score=rule)
        if score == "sigmoid":  # (softmax scores plus a bias: equal sums only where equally rounded)
            check(logits, bias, k, score=score, n_group=G, topk_group=top, group_score="max")


@gpu
@pytest.mark.parametrize("E", [32, 64, 128, 256, 200])
def test_scores_that_float32_cannot_tell_apart(E):
    """Sigmoids near 1 and biases next to each other: sums that differ by 1e-9 and less."""
    g = torch.Generator().manual_seed(3)
    logits = 14 + 1e-3 * torch.randn(64, E, generator=g)
    check(logits, None, 8, score="sigmoid")
    check(logits, torch.full((E,), 0.5), 8, score="sigmoid", n_group=4, topk_group=2, group_score="top2")
    bias = 0.5 + 2.0 ** -24 * torch.randint(0, 3, (E,), generator=g)
    check(logits, bias, 8, score="sigmoid", n_group=4, topk_group=2, group_score="top2")
    near = 1e-6 * torch.randn(64, E, generator=g)
    check(near, bias, 8, score="softmax", n_group=4, topk_group=3, group_score="top2", renormalize=False)


@gpu
@pytest.mark.parametrize("E,G,top", [(64, 1, 1), (256, 1, 1), (256, 8, 4), (160, 8, 3), (1000, 10, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_logits_next_to_zero(E, G, top, score):
    """Logits whose scores are equal in 64 bits, the smallest steps of float32 among them, and
    logits 2^-30 apart, whose scores are not (but are in float32)."""
    g = torch.Generator().manual_seed(E)
    steps = torch.randint(-300, 300, (9, E), generator=g).double()
    for unit in (2.0 ** -149, 2.0 ** -100, 2.0 ** -70, 2.0 ** -30):
        l = (steps * unit).float()
        for renorm in (True, False):
            check(l, None, 6, score=score, n_group=G, topk_group=top, renormalize=renorm)
        check(l, None, 6, score=score, n_group=G, topk_group=top, group_score="top2")


@gpu
@pytest.mark.parametrize("E,G,top", [(64, 8, 4), (256, 8, 4), (100, 4, 2)])
def test_far_logits(E, G, top):
    logits, bias = draw(40, E, seed=9, spread=40.0)
    for score in ("sigmoid", "softmax"):
        check(logits, bias, 6, score=score, n_group=G, topk_group=top, group_score="top2")
        check(logits - 600, None, 6, score=score, renormalize=score == "softmax")


@gpu
@pytest.mark.parametrize("E,G,top,k", [(64, 8, 4, 8), (256, 8, 4, 8), (100, 5, 3, 20)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_infinities_and_nan(E, G, top, k, score, renorm):
    logits, bias = draw(12, E, seed=5)
    inf = float("inf")
    logits[0, ::2] = float("nan")
    logits[1] = float("nan")
    logits[2] = -inf
    logits[3, : E // G * 2] = -inf
    logits[4, 3:] = -inf                 # fewer finite logits than selections
    logits[5, 7] = float("nan")
    logits[5, 9] = inf
    logits[6, 11:13] = inf
    logits[7, E // 2:] = float("nan")
    logits[8, 1:] = float("nan")
    dev = device()
    kw = dict(score=score, n_group=G, topk_group=top, group_score="top2", renormalize=renorm)
    check(logits, None, k, **kw)
    bias[3], bias[5], bias[10] = -inf, inf, float("nan")
    # the ids are the definition's, and valid, also where a bias is infinite or NaN
    idx, _ = M.moe_select(logits.to(dev), k, bias.to(dev), **kw)
    want, _ = oracle(logits.numpy(), bias.numpy(), k, **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    for row in idx.tolist():
        assert len(set(row)) == k and min(row) >= 0 and max(row) < E


@gpu
def test_no_tokens_views_and_given_outputs():
    dev = device()
    idx, w = M.moe_select(torch.zeros(0, 64, device=dev), 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    # logits and bias that start at an odd address
    flat, bias = draw(1, 21 * 64 + 1, seed=2)[0][0].to(dev), draw(1, 65, seed=3)[1].to(dev)
    l, b = flat[1:].view(21, 64), bias[1:]
    io, wo = torch.full((21, 4), -7, dtype=torch.int32, device=dev), torch.full((21, 4), -7.0, device=dev)
    r = M.moe_select(l, 4, b, score="sigmoid", n_group=8, topk_group=3, topk_idx=io, topk_w=wo)
    assert r[0] is io or r[0].data_ptr() == io.data_ptr()
    want, _ = oracle(l.cpu().numpy(), b.cpu().numpy(), 4, score="sigmoid", n_group=8, topk_group=3)
    np.testing.assert_array_equal(io.cpu().numpy(), want)
    assert torch.equal(l, flat[1:].view(21, 64))


@gpu
@pytest.mark.parametrize("T,E", [(3, 256), (3000, 256), (3000, 100)])
def test_stream_and_graph(T, E):
    dev = device()
    logits, bias = (v.to(dev) for v in draw(T, E, seed=T))
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2")
    want = M.moe_select(logits, 8, bias, **kw)
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    got = M.moe_select(logits, 8, bias, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.moe_select(logits, 8, bias, **kw)
    for rep in range(3):
        logits.copy_(draw(T, E, seed=T + rep + 1)[0])
        want = M.moe_select(logits, 8, bias, **kw)
        for o in out:
            o.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), rep


@gpu
def test_rows_past_32_bit_offsets():
    dev = device()
    T, E = (1 << 32) // 1024 + 40, 1024  # the last rows start past 2^32 values
    logits = torch.zeros(T, E, device=dev)
    tail, bias = draw(30, E, seed=1)
    logits[-30:] = tail.to(dev)
    idx, w = M.moe_select(logits, 8, bias.to(dev), score="sigmoid", n_group=8, topk_group=4)
    want, ws = oracle(tail.numpy(), bias.numpy(), 8, score="sigmoid", n_group=8, topk_group=4)
    np.testing.assert_array_equal(idx[-30:].cpu().numpy(), want)
    assert np.allclose(w[-30:].cpu().numpy(), ws, rtol=2 * 2.0 ** -24, atol=0)


@gpu
@pytest.mark.parametrize("T,H,E", [(1, 7168, 256), (40, 128, 32), (300, 200, 60), (2100, 256, 64)])
def test_route_scored_is_its_two_calls(T, H, E):
    """Its logits are moe_route's bits, its choice moe_select's of them."""
    dev = device()
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, H, generator=g) * H ** -0.5).to(torch.bfloat16).to(dev)
    wr, lb, cb = (torch.randn(*s, generator=g).to(dev) for s in ((E, H), (E,), (E,)))
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2", scale=2.5)
    say(f"route_scored T={T} H={H} E={E}")
    for bias in (None, lb):
        logits, idx, w = M.moe_route_scored(x, wr, bias, 0.1 * cb, 5, **kw)
        assert torch.equal(logits, M.moe_route(x, wr, bias, 5)[0])
        i2, w2 = M.moe_select(logits, 5, 0.1 * cb, **kw)
        assert torch.equal(idx, i2) and torch.equal(w, w2)
        check(logits.cpu(), 0.1 * cb.cpu(), 5, **kw)
    assert B.MAX_GROUPS == 64
