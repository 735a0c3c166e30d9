"""moe_select where its float32 candidates and groups are nearly tied: inputs that
lie next to the bounds by which it trusts a float32 value, made on the CPU, and the
choice compared with the definition in 64 bits (tests/test_select.py's oracle)."""
import numpy as np
import pytest
import torch

import expert_token_routing_amd as M
from tests.gpu_helpers import device, say
from tests.test_select import check, oracle

f32 = np.float32
gpu = pytest.mark.gpu


def sigmoid32(l):
    """A sigmoid as float32 instructions form it: each step rounded to nearest (the GPU's
    exponential and reciprocal may be a step off that)."""
    e = np.exp2(((-l).astype(f32) * f32(1.44269504)).astype(np.float64)).astype(f32)
    return (1 / (f32(1) + e).astype(np.float64)).astype(f32)


def sigmoid64(l):
    return 1 / (1 + np.exp(-l.astype(np.float64)))


def low_pairs(level, rows, seed):
    """Logits [rows, 4] about `level` whose first two and last two have nearly the same sum of
    scores, in the wrong order where float32 forms it, by more than 5 steps of 2^-24 of the
    largest score for each of the four (what four sigmoids near 1 may be off)."""
    rng = np.random.default_rng(seed)
    got = []
    while sum(map(len, got)) < rows:
        l = (level + 0.1 * rng.standard_normal((400000, 4))).astype(f32)
        s = sigmoid64(l)
        last = s[:, 0] + s[:, 1] - s[:, 2]
        l = l[last > 0]
        last = last[last > 0]
        l[:, 3] = np.log(last / (1 - last)).astype(f32)
        s, q = sigmoid64(l), sigmoid32(l)
        right = (s[:, 0] + s[:, 1]) - (s[:, 2] + s[:, 3])
        seen = (q[:, 0] + q[:, 1]).astype(np.float64) - (q[:, 2] + q[:, 3])
        margin = 4 * s.max(1) * 5 * 2.0 ** -24 + q.max(1) * 2.0 ** -22
        got.append(l[(right * seen < 0) & (np.abs(seen) > 1.1 * margin)])
    return np.concatenate(got)[:rows]


@gpu
@pytest.mark.parametrize("level", [-13.0, -25.0, -31.0, -60.0])
@pytest.mark.parametrize("E,G,top,at", [(4, 2, 1, (0, 1)), (32, 8, 4, (2, 6)), (60, 5, 2, (4, 1)), (256, 8, 4, (5, 3))])
def test_groups_of_low_sigmoids(level, E, G, top, at):
    """A sigmoid far below 0 is off by |logit| steps in float32: two groups whose sums differ by
    less than that, at the border of those that stay."""
    pairs = torch.from_numpy(low_pairs(level, 200, 7 + E))
    per = E // G
    rng = torch.Generator().manual_seed(E)
    logits = level - 3 - torch.rand(len(pairs), E, generator=rng)
    above = [g for g in range(G) if g not in at][: top - 1]
    for g in above:  # groups that stay whatever the two are
        logits[:, g * per:g * per + 2] = pairs.max(1, keepdim=True).values + 0.03
    for g, p in zip(at, (pairs[:, :2], pairs[:, 2:])):
        logits[:, g * per:g * per + 2] = p
    for bias in (None, torch.zeros(E)):
        check(logits, bias, 2 * top, score="sigmoid", n_group=G, topk_group=top, group_score="top2")


@gpu
@pytest.mark.parametrize("level", [-13.0, -25.0, -60.0])
@pytest.mark.parametrize("E,k", [(256, 8), (64, 4), (100, 6)])
def test_low_sigmoids_beside_a_bias_that_cancels_them(level, E, k):
    """Choice values of 1e-4 of the scores, whose order float32's error of a score hides."""
    g = torch.Generator().manual_seed(E)
    logits = level + 1e-4 * torch.randn(300, E, generator=g)
    bias = torch.full((E,), -float(sigmoid64(np.array([level], f32))[0]))
    check(logits, bias, k, score="sigmoid")
    check(logits, bias, k, score="sigmoid", n_group=4, topk_group=2, group_score="max")


def seconds(call, times=30):
    """Median time of one of `times` calls on an otherwise idle GPU."""
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(times + 1)]
    for _ in range(3):
        call()
    marks[0].record()
    for m in marks[1:]:
        call()
        m.record()
    torch.cuda.synchronize()
    return float(np.median([a.elapsed_time(b) for a, b in zip(marks, marks[1:])]))


@gpu
@pytest.mark.parametrize("G,top", [(10, 4), (5, 2), (3, 1)])
def test_groups_that_leave_lanes_empty_are_chosen_in_float32(G, top):
    """Only rows at the border go the 64-bit way, also where the groups are no power of two and
    leave lanes without any: the time is not a multiple of that of a power of two (all rows in 64
    bits: 2.6 to 3.6 times as long)."""
    dev = device()
    g = torch.Generator(device=dev).manual_seed(G)
    T, per = 65536, 16
    logits, bias = torch.randn(T, per * 16, generator=g, device=dev), 0.1 * torch.randn(per * 16, generator=g, device=dev)

    def call(n_group, topk_group):
        l, b = logits.view(-1)[:T * per * n_group].view(T, per * n_group), bias[:per * n_group]
        return lambda: M.moe_select(l, 4, b, score="sigmoid", n_group=n_group, topk_group=topk_group, group_score="top2")
    full = 4 if G < 8 else 16
    say(f"times of {G} and {full} groups")
    mine, other = seconds(call(G, top)), seconds(call(full, top))
    print(f"{G} groups {1e3 * mine:.1f} us, {full} groups {1e3 * other:.1f} us")
    assert mine <= 2 * other


@gpu
@pytest.mark.parametrize("E,G,top", [(64, 1, 1), (256, 8, 4), (160, 8, 3), (1000, 10, 4)])
@pytest.mark.parametrize("largest", [17.0, 500.0])
def test_logits_that_their_distance_to_the_largest_makes_equal(E, G, top, largest):
    """exp(l - m) of logits next to 0: l - m rounds to 2^-49 at 17 and to 2^-44 at 500, so logits
    less than that apart have the same score in 64 bits and go by id."""
    g = torch.Generator().manual_seed(E)
    steps = torch.randint(-3, 4, (60, E), generator=g).double()
    for unit in (2.0 ** -51, 2.0 ** -49, 2.0 ** -46, 2.0 ** -44, 2.0 ** -42):
        l = (steps * unit).float()
        l[:, 5] = largest
        for renorm in (True, False):
            check(l, None, 6, n_group=G, topk_group=top, renormalize=renorm)


@gpu
@pytest.mark.parametrize("E,G,top,k", [(64, 1, 1, 4), (256, 8, 4, 8), (160, 8, 3, 6), (99, 3, 2, 12),
                                       (512, 1, 1, 16), (1000, 10, 4, 12)])
@pytest.mark.parametrize("spread", [0.01, 1.0, 8.0])
def test_weights_of_a_softmax_over_all_experts(E, G, top, k, spread):
    """Without renormalisation the denominator counts. Its terms' exponentials may be a step
    (2 x 2^-24) off and round once more, the weight rounds once: 4 x 2^-24, whatever kernel and
    way the sizes take."""
    g = torch.Generator().manual_seed(E)
    logits = spread * torch.randn(300, E, generator=g)
    logits[0, 1::2] = -float("inf")
    logits[1, ::3] = float("nan")
    logits[2] = 0.25
    logits[3] += 1000.0
    for bias in (None, 0.01 * torch.randn(E, generator=g)):
        for rule in ("max", "top2"):
            kw = dict(n_group=G, topk_group=top, group_score=rule, renormalize=False, scale=1.0)
            _, w = check(logits, bias, k, **kw)
            _, want = oracle(logits.numpy(), None if bias is None else bias.numpy(), k, **kw)
            assert np.all(np.abs(w.cpu().numpy() - want) <= 4.1 * 2.0 ** -24 * want + 2.0 ** -126)


@gpu
@pytest.mark.parametrize("E,G,top", [(64, 1, 1), (256, 8, 4), (100, 5, 3), (1000, 10, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_bias_does_not_bring_a_nan_logit_back(E, G, top, score):
    """A logit of -infinity has score 0 and its bias; one that is NaN has no choice value at all."""
    g = torch.Generator().manual_seed(E)
    logits, bias = torch.randn(20, E, generator=g), 0.1 * torch.randn(E, generator=g)
    per = E // G
    logits[:, 3], logits[:, per // 2] = float("nan"), float("nan")
    logits[:, 4] = -float("inf")
    bias[3], bias[4], bias[per // 2] = 9.0, 8.0, 7.0
    for rule in ("max", "top2"):
        idx, _ = check(logits, bias, 4, score=score, n_group=G, topk_group=top, group_score=rule)
        assert bool((idx[:, 0] == 4).all()) and not bool(((idx == 3) | (idx == per // 2)).any())


@gpu
@pytest.mark.parametrize("E,k,G,top", [(64, 1, 1, 1), (64, 2, 8, 8), (256, 4, 1, 1), (69, 2, 3, 1), (160, 6, 8, 3), (32, 8, 8, 6),
                                       (100, 1, 5, 2)])
@pytest.mark.parametrize("score,level", [("softmax", -4.0), ("softmax", -52.0), ("softmax", 3.0), ("sigmoid", -4.0)])
def test_negative_values_in_the_last_bits_of_a_key(E, k, G, top, score, level):
    """The largest two values of a row next to each other in the bits that a key drops, the larger
    one at the higher id, every other value far from the next: the first candidates come the wrong
    way round, and values below 0 have to be put right as those above are."""
    g = torch.Generator().manual_seed(E)
    logits = level - 0.5 - 0.05 * torch.rand(200, E, generator=g).argsort(1).float()
    step = abs(level) * 2.0 ** -22
    ends = torch.rand(200, E, generator=g).argsort(1)[:, :2].sort(1).values
    for t, (a, b) in enumerate(ends.tolist()):
        logits[t, a], logits[t, b] = level, level + step * (1 + t % 8)
    check(logits, None, k, score=score, n_group=G, topk_group=top)
    # choice values below 0 beside a bias
    check(logits, torch.full((E,), -2.0), k, score="sigmoid", n_group=G, topk_group=top)
    bias = -2.0 - 0.01 * torch.rand(E, generator=g).argsort().float()
    a, b = sorted(torch.rand(E, generator=g).argsort()[:2].tolist())
    bias[a], bias[b] = -1.5, -1.5 + 2.0 ** -21
    check(torch.zeros(8, E), bias, k, score=score, n_group=G, topk_group=top)


@gpu
@pytest.mark.parametrize("E,G,top", [(160, 10, 4), (100, 5, 2), (96, 3, 2), (140, 7, 5)])
def test_negative_groups_beside_lanes_without_one(E, G, top):
    """Groups of negative value where lanes hold none: the definition's, and as quick as positive
    ones (those lanes do not count as groups above)."""
    g = torch.Generator().manual_seed(E)
    logits, bias = torch.randn(300, E, generator=g), -1.0 - torch.rand(E, generator=g)
    for score in ("sigmoid", "softmax"):
        check(logits - 5, None, 4, score=score, n_group=G, topk_group=top, group_score="max")
        check(logits, bias, 4, score=score, n_group=G, topk_group=top, group_score="top2")
    dev = device()
    l, b = torch.randn(65536, E, device=dev), bias.to(dev)
    kw = dict(score="sigmoid", n_group=G, topk_group=top, group_score="top2")
    below, above = seconds(lambda: M.moe_select(l, 4, b, **kw)), seconds(lambda: M.moe_select(l, 4, -b, **kw))
    print(f"{G} groups below 0 {1e3 * below:.1f} us, above {1e3 * above:.1f} us")
    assert below <= 1.5 * above


@gpu
@pytest.mark.parametrize("E,k,G,top", [(64, 1, 1, 1), (64, 3, 8, 2), (256, 8, 8, 4), (100, 4, 5, 2), (1000, 4, 10, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_renormalised_weights_of_scores_that_are_all_zero(E, k, G, top, score):
    """A bias selects experts whose logits are -infinity, or NaN: 0 / 0 is NaN, as by the formula; with one
    finite logit among them that one has the whole weight."""
    g = torch.Generator().manual_seed(E)
    per = E // G
    logits, bias = torch.randn(12, E, generator=g), torch.zeros(E)
    chosen = [per * (j % top) + j // top for j in range(k)]
    for j, e in enumerate(chosen):
        bias[e] = 50.0 - j
        logits[:, e] = -float("inf")
    logits[6:, chosen[-1]] = -700.0 if score == "sigmoid" else -30.0
    _, w = check(logits, bias, k, score=score, n_group=G, topk_group=top)
    assert bool(torch.isnan(w[:6]).all()) and bool((w[6:, -1] == 1).all())


@gpu
@pytest.mark.parametrize("E,G,top,k", [(4, 1, 1, 3), (16, 1, 1, 6), (64, 8, 1, 6), (256, 8, 2, 8), (100, 5, 3, 12), (1000, 10, 1, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_minus_infinity_comes_before_nan(E, G, top, k, score):
    """Fewer finite logits than selections: the experts at -infinity (score 0) before the NaN ones (no
    choice value), also where these have the lower ids."""
    g = torch.Generator().manual_seed(E)
    logits = torch.full((20, E), float("nan"))
    for t in range(20):
        order = torch.rand(E, generator=g).argsort()
        logits[t, order[: E // 2]] = -float("inf")
        logits[t, order[: max(1, min(k - 1, t % k))]] = torch.randn(max(1, min(k - 1, t % k)), generator=g)
    for renorm in (True, False):
        for rule in ("max", "top2"):
            check(logits, None, k, score=score, n_group=G, topk_group=top, group_score=rule, renormalize=renorm)
