"""Infinities and NaN in token vectors, router weights and activations: what
they make of their own token, and that no other token's output moves.

A router logit that is NaN counts as -infinity, so the selected ids stay
distinct and inside [0, E): dispatch and the expert MLPs index memory with
them. Rows are independent in every kernel, so the other tokens' outputs are
compared bit for bit with those of a call on finite inputs of the same shape.
"""
import math

import pytest
import torch

import expert_token_routing_amd as M

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = math.nan, math.inf
gpu = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@gpu
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,H,E,k", [
    (9, 40, 8, 3), (9, 128, 100, 7), (5, 72, 1000, 32),                      # one wave per token, any E
    (9, 64, 64, 4), (9, 256, 128, 8), (9, 72, 256, 8), (300, 64, 512, 2), (9, 64, 1024, 32),  # vector loads
    (2100, 64, 32, 4), (2051, 64, 64, 16), (2048, 72, 128, 5), (2099, 64, 256, 8),  # a row of 16 lanes per token
])
def test_route_ids_are_valid_with_nan(T, H, E, k, renormalize):
    g = _gen(1)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    w = torch.randn((E, H), generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda")
    print(f"[gpu] route with NaN T={T} H={H} E={E} k={k}", flush=True)
    clean = [t.clone() for t in M.moe_route(x, w, bias, k, renormalize)]
    bad = x.clone()
    rows = sorted({0, 3, T - 1})
    bad[rows[0], 5] = NAN
    bad[rows[1], :] = NAN
    bad[rows[2], 1] = INF
    logits, idx, tw = M.moe_route(bad, w, bias, k, renormalize)
    torch.cuda.synchronize()
    assert int(idx.min()) >= 0 and int(idx.max()) < E
    assert bool(idx.sort(1)[0].diff(dim=1).gt(0).all()), "an expert was picked twice"
    assert torch.isnan(logits[rows[0]]).all() and torch.isnan(logits[rows[1]]).all()
    assert idx[rows[0]].tolist() == idx[rows[1]].tolist() == list(range(k))
    assert torch.isnan(tw[rows[:2]]).all()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[rows] = False
    for a, b in zip((logits, idx, tw), clean):
        assert _same_bits(a[others], b[others])
    # one expert without a score: never taken while others have one
    wn = w.clone()
    wn[E // 2, 0] = NAN
    logits, idx, tw = M.moe_route(x, wn, bias, min(k, E - 1), renormalize)
    torch.cuda.synchronize()
    assert torch.isnan(logits[:, E // 2]).all()
    assert int(idx.min()) >= 0 and int(idx.max()) < E and not idx.eq(E // 2).any()
    assert bool(idx.sort(1)[0].diff(dim=1).gt(0).all()) and torch.isfinite(tw).all()


def _bf16_weights(g, E, H, I):
    return ((torch.randn((E, H, 2 * I), generator=g, device="cuda") / H ** 0.5).to(BF),
            (torch.randn((E, I, H), generator=g, device="cuda") / I ** 0.5).to(BF))


def _share(name, x, wr, gu, dn, k, e0):
    if name == "moe_forward_i8":
        return M.moe_forward_i8(x, wr, None, *M.moe_quantize_weights(gu), *M.moe_quantize_weights(dn), k, e0)[0]
    return getattr(M, name)(x, wr, None, gu, dn, k, e0)[0]


@gpu
@pytest.mark.parametrize("name,T,H,I,E,k,e0,El", [
    ("moe_forward", 40, 128, 96, 8, 2, 0, 8), ("moe_forward", 2200, 256, 64, 64, 4, 0, 16),
    ("moe_forward_f32", 40, 72, 40, 12, 3, 0, 6), ("moe_forward_fused", 700, 128, 96, 8, 2, 0, 4),
    ("moe_forward_i8", 1, 128, 96, 8, 2, 0, 8), ("moe_forward_i8", 40, 272, 48, 12, 3, 0, 5),
    ("moe_forward_i8", 2200, 256, 64, 64, 4, 0, 16), ("moe_forward_i8", 900, 256, 400, 16, 4, 0, 6)])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_share_keeps_nonfinite_tokens_to_themselves(name, T, H, I, E, k, e0, El, value):
    g = _gen(2)
    x = (torch.randn((T, H), generator=g, device="cuda") / H ** 0.5).to(BF)
    wr = torch.randn((E, H), generator=g, device="cuda")
    gu, dn = _bf16_weights(g, El, H, I)
    print(f"[gpu] {name} with {value} T={T} H={H} I={I} E={E}", flush=True)
    clean = _share(name, x, wr, gu, dn, k, e0).clone()
    rows = sorted({0, T // 2, T - 1})
    for t in rows:
        x[t, (5 * t + 1) % H] = value
    y = _share(name, x, wr, gu, dn, k, e0)
    torch.cuda.synchronize()
    # (an infinity can leave one expert +inf and so send the token to another rank: zeros here)
    idx = M.moe_route(x, wr, None, k)[1][rows]
    local = idx.ge(e0).logical_and(idx.lt(e0 + El)).any(1)
    assert torch.isnan(y[rows][local]).all() and y[rows][~local].eq(0).all()
    assert local.all() or not math.isnan(value)
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert torch.isfinite(y[others]).all() and _same_bits(y[others], clean[others])


@gpu
@pytest.mark.parametrize("T", [5, 24])
@pytest.mark.parametrize("rdtype", [BF, F32])
def test_block_keeps_nonfinite_tokens_to_themselves(T, rdtype):
    """Both of the block's layers (the one for a few tokens adds its sums in
    another order where other experts are in use: compared to a step of bf16
    of the largest value)."""
    H, I, E, k = 256, 96, 8, 2
    g = _gen(3)
    r = torch.randn((T, H), generator=g, device="cuda").to(rdtype)
    wr, wn = torch.randn((E, H), generator=g, device="cuda"), torch.rand(H, generator=g, device="cuda") + 0.5
    gu, dn = _bf16_weights(g, E, H, I)
    print(f"[gpu] block with NaN T={T}", flush=True)
    clean = [t.clone() for t in M.moe_block_forward(r, wn, wr, None, gu, dn, k, wn, w_next=wn)[:2]]
    r[1, 7], r[T - 1, 0] = NAN, INF
    got = M.moe_block_forward(r, wn, wr, None, gu, dn, k, wn, w_next=wn)[:2]
    torch.cuda.synchronize()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[[1, T - 1]] = False
    for a, b in zip(got, clean):
        assert torch.isnan(a[1]).all() and torch.isnan(a[T - 1]).all()
        a, b = a[others].float(), b[others].float()
        assert torch.isfinite(a).all() and float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())


@gpu
@pytest.mark.parametrize("fn", ["moe_forward_few", "moe_forward_few_f32", "moe_forward"])
@pytest.mark.parametrize("T,H,I,k", [(3, 72, 40, 2), (24, 256, 136, 4)])
def test_few_infinite_h(fn, T, H, I, k):
    """silu(g) u past the largest float32: every h of two tokens is an infinity,
    and so is their y (all selections weighted by the bias alone, all products
    of one sign: no 0 inf and no inf - inf). The experts in use stay the same,
    and with them the order of the other tokens' sums."""
    E = 4
    g = _gen(4)
    x = torch.rand((T, H), generator=g, device="cuda").to(BF)
    wr, bias = torch.zeros((E, H), device="cuda"), torch.randn(E, generator=g, device="cuda")
    gu, dn = (w.abs() for w in _bf16_weights(g, E, H, I))
    print(f"[gpu] {fn} with infinite h T={T}", flush=True)
    clean = [getattr(M, fn)(x, wr, bias, gu, d, k, 0)[0].clone() for d in (dn, -dn)]
    x[1] *= 2.0 ** 70
    x[2] *= 2.0 ** 100
    up = getattr(M, fn)(x, wr, bias, gu, dn, k, 0)[0]
    down = getattr(M, fn)(x, wr, bias, gu, -dn, k, 0)[0]
    torch.cuda.synchronize()
    assert torch.isposinf(up[1:3]).all() and torch.isneginf(down[1:3]).all()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[1:3] = False
    assert _same_bits(up[others], clean[0][others]) and _same_bits(down[others], clean[1][others])


@gpu
@pytest.mark.parametrize("segs,H,I,behind", [([3, 0, 5], 272, 48, 2), ([9], 2880, 768, 0), ([100, 0, 240], 144, 208, 5),
                                             ([600, 300, 0, 33], 256, 400, 0)])
def test_expert_ffn_i8_keeps_nonfinite_rows_to_themselves(segs, H, I, behind):
    """A row that holds an infinity or NaN gets an infinite or NaN scale and
    quantised zeros: its output is NaN, also where only its h is not finite."""
    g = _gen(5)
    n, E = sum(segs), len(segs)
    x = torch.randn((n + behind, H), generator=g, device="cuda").to(BF)
    w = [t for p in _bf16_weights(g, E, H, I) for t in M.moe_quantize_weights(p)]
    off = torch.tensor([0, *segs], device="cuda").cumsum(0).to(torch.int32)
    print(f"[gpu] expert_ffn_i8 with NaN segs={segs} H={H} I={I}", flush=True)
    clean = M.moe_expert_ffn_i8(x, off, *w)[0][:n].clone()
    rows = [0, n // 2, n - 2, n - 1]
    x[rows[0], 3], x[rows[1], H - 1], x[rows[2], 0] = NAN, INF, -INF
    x[rows[3]] *= 2.0 ** 70  # finite, but its h is past float32
    x[n:] = NAN
    out = M.moe_expert_ffn_i8(x, off, *w)[0][:n]
    torch.cuda.synchronize()
    assert torch.isnan(out[rows]).all()
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert torch.isfinite(clean).all() and _same_bits(out[others], clean[others])


@gpu
@pytest.mark.parametrize("fn", ["moe_forward_few", "moe_forward_few_f32"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 72, 40, 8, 2), (4, 128, 64, 100, 7), (9, 72, 136, 40, 3), (24, 256, 136, 8, 2),
                                       (32, 64, 40, 300, 5)])
def test_few_keeps_nonfinite_tokens_to_themselves(fn, T, H, I, E, k):
    """Every selection kernel; the other tokens' sums are added in another order
    where other experts are in use: compared to a step of bf16 of the largest."""
    g = _gen(6)
    x = (torch.randn((T, H), generator=g, device="cuda") / H ** 0.5).to(BF)
    wr = torch.randn((E, H), generator=g, device="cuda")
    gu, dn = _bf16_weights(g, E, H, I)
    print(f"[gpu] {fn} with NaN T={T} H={H} I={I} E={E}", flush=True)
    clean = getattr(M, fn)(x, wr, None, gu, dn, k, 0)[0].float()
    rows = sorted({0, T // 2, T - 1})
    for t, v in zip(rows, (NAN, INF, -INF)):
        x[t, (3 * t + 1) % H] = v
    y = getattr(M, fn)(x, wr, None, gu, dn, k, 0)[0].float()
    torch.cuda.synchronize()
    assert torch.isnan(y[rows]).all()
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[rows] = False
    if T > 3:
        a, b = y[others], clean[others]
        assert torch.isfinite(a).all() and float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())
