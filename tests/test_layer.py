"""moe_layer_forward: the share with scored routing plus the shared expert,
against its steps and against the oracle, and its refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import expert_token_routing_amd as M
import oracle.moe_oracle as O
from tests.gpu_helpers import OUT_TOL, bf16_bits, device, rel_max_err, say
from tests.test_select import oracle as choose

BF, F32 = torch.bfloat16, torch.float32
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
gpu = pytest.mark.gpu


@pytest.mark.parametrize("kw,want", [
    (dict(H=12), M.MOE_ERR_INVALID_ARG), (dict(I=4), M.MOE_ERR_INVALID_ARG), (dict(Is=4), M.MOE_ERR_INVALID_ARG),
    (dict(Is=-8), M.MOE_ERR_INVALID_ARG), (dict(Is=0), M.MOE_ERR_INVALID_ARG),   # weights without a size
    (dict(sg=None), M.MOE_ERR_INVALID_ARG), (dict(sd=None), M.MOE_ERR_INVALID_ARG), (dict(sg=ODD), M.MOE_ERR_INVALID_ARG),
    (dict(yt=2), M.MOE_ERR_INVALID_ARG), (dict(y=None), M.MOE_ERR_INVALID_ARG), (dict(y=ODD), M.MOE_ERR_INVALID_ARG),
    (dict(e0=60), M.MOE_ERR_INVALID_ARG), (dict(k=17), M.MOE_ERR_INVALID_ARG), (dict(score=2), M.MOE_ERR_INVALID_ARG),
    (dict(scale=math.nan), M.MOE_ERR_INVALID_ARG), (dict(x=None), M.MOE_ERR_INVALID_ARG),
    (dict(H=1 << 14, I=1 << 15), M.MOE_ERR_UNSUPPORTED), (dict(H=1 << 14, Is=1 << 15), M.MOE_ERR_UNSUPPORTED),
    (dict(ws=None), M.MOE_ERR_WORKSPACE), (dict(ws=ODD), M.MOE_ERR_WORKSPACE), (dict(nws=100), M.MOE_ERR_WORKSPACE),
    (dict(T=0, x=None, y=None), M.MOE_OK),
])
def test_layer_rejects(kw, want):
    p = dict(x=FAKE, wr=FAKE, gu=FAKE, dn=FAKE, sg=FAKE, sd=FAKE, T=4, H=64, I=32, Is=32, E=64, k=4, e0=0, El=8, score=1, G=8,
             top=2, rule=1, renorm=1, scale=1.0, y=FAKE, yt=0, ws=FAKE, nws=1 << 40)
    p.update(kw)
    assert M.lib().moe_layer_forward(p["x"], p["wr"], None, None, p["gu"], p["dn"], p["sg"], p["sd"], p["T"], p["H"], p["I"],
                                     p["Is"], p["E"], p["k"], p["e0"], p["El"], p["score"], p["G"], p["top"], p["rule"],
                                     p["renorm"], p["scale"], p["y"], p["yt"], p["ws"], p["nws"], None) == want


def test_layer_rejects_mismatched_tensors():
    x, wr = torch.zeros(4, 64, dtype=BF), torch.zeros(16, 64)
    gu, dn = torch.zeros(16, 64, 64, dtype=BF), torch.zeros(16, 32, 64, dtype=BF)
    sg, sd = torch.zeros(64, 48, dtype=BF), torch.zeros(24, 64, dtype=BF)
    for kw, exc, match in ((dict(shared_down=None), ValueError, "given together"),
                           (dict(shared_gate_up=torch.zeros(64, 47, dtype=BF)), ValueError, "must be even"),
                           (dict(shared_gate_up=torch.zeros(72, 48, dtype=BF)), ValueError, "shared_gate_up has shape"),
                           (dict(shared_down=torch.zeros(32, 64, dtype=BF)), ValueError, "shared_down has shape"),
                           (dict(shared_gate_up=torch.zeros(64, 0, dtype=BF)), ValueError, "no columns"),
                           (dict(choice_bias=torch.zeros(15)), ValueError, "choice_bias has shape"),
                           (dict(n_group=5), ValueError, "do not divide"), (dict(out_dtype=torch.float64), TypeError, "out_dtype"),
                           (dict(y=torch.zeros(4, 72, dtype=BF)), ValueError, "y has shape"), (dict(e0=1), ValueError, "local experts"),
                           (dict(), ValueError, "must live on a GPU")):
        p = dict(bias=None, choice_bias=None, w_gate_up=gu, w_down=dn, k=2, e0=0, shared_gate_up=sg, shared_down=sd)
        p.update(kw)
        with pytest.raises(exc, match=match):
            M.moe_layer_forward(x, wr, **p)


def weights(T, H, I, Is, E, El, seed):
    dev = device()
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*s, scale=1.0):
        return torch.randn(s, generator=g, device=dev) * scale
    return dict(x=randn(T, H, scale=H ** -0.5).to(BF), w_router=randn(E, H), bias=randn(E, scale=0.1),
                choice_bias=randn(E, scale=0.1), w_gate_up=randn(El, H, 2 * I, scale=H ** -0.5).to(BF),
                w_down=randn(El, I, H, scale=I ** -0.5).to(BF),
                shared_gate_up=randn(H, 2 * Is, scale=H ** -0.5).to(BF) if Is else None,
                shared_down=randn(Is, H, scale=Is ** -0.5).to(BF) if Is else None)


def steps(d, k, e0, out_dtype, kw):
    """The layer from its separate calls (the share's as in moe_forward)."""
    E, El = d["w_router"].shape[0], d["w_gate_up"].shape[0]
    _, idx, w = M.moe_route_scored(d["x"], d["w_router"], d["bias"], d["choice_bias"], k, **kw)
    _, off, _, inv, xp = M.moe_dispatch(d["x"], idx, E, e0, El)
    out = M.moe_expert_ffn(xp, off, d["w_gate_up"], d["w_down"])[1]
    if d["shared_gate_up"] is None:
        return (M.moe_combine if out_dtype is BF else M.moe_combine_f32)(out, inv, w)
    share = M.moe_combine_f32(out, inv, w)
    h = M.moe_gemm(d["x"], d["shared_gate_up"][None], activation="swiglu")
    return M.moe_gemm(h, d["shared_down"][None], residual=share, out_dtype=out_dtype)


CASES = [  # T, H, I, Is, E, El, e0, k, G, top
    (200, 128, 96, 64, 16, 4, 8, 4, 4, 2), (33, 256, 128, 128, 64, 64, 0, 8, 8, 4), (1000, 512, 264, 520, 32, 8, 24, 6, 8, 3),
    (17, 136, 40, 8, 8, 3, 5, 3, 1, 1), (64, 128, 64, 0, 16, 16, 0, 2, 4, 4),
]


@gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_layer_is_its_steps(case, out_dtype):
    T, H, I, Is, E, El, e0, k, G, top = case
    d = weights(T, H, I, Is, E, El, T)
    kw = dict(score="sigmoid", n_group=G, topk_group=top, group_score="top2", scale=2.5)
    say(f"layer {case} {out_dtype}")
    y, ws = M.moe_layer_forward(d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], k, e0,
                                d["shared_gate_up"], d["shared_down"], out_dtype=out_dtype, **kw)
    want = steps(d, k, e0, out_dtype, kw)
    # the separate expert MLPs may take the other GEMM kernel, whose bits are the same
    assert torch.equal(y, want)
    assert ws.numel() >= M.layer_workspace_size(T, H, I, Is, E, k, El)


@gpu
@pytest.mark.parametrize("T", [1, 3, 16, 17, 40])
@pytest.mark.parametrize("score,renorm,Is", [("sigmoid", True, 72), ("softmax", False, 72), ("sigmoid", False, 0),
                                             ("sigmoid", True, 136), ("softmax", True, 408)])
def test_layer_against_the_oracle(T, score, renorm, Is):
    H, I, E, El, e0, k = 192, 136, 32, 12, 8, 5
    d = weights(T, H, I, Is, E, El, 10 * T + Is)
    kw = dict(score=score, n_group=8, topk_group=3, group_score="top2", renormalize=renorm, scale=1.5)
    say(f"layer oracle T={T} {score} {renorm} {Is}")
    y, _ = M.moe_layer_forward(d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], k, e0,
                               d["shared_gate_up"], d["shared_down"], **kw)
    # float64 logits; a margin of 1e-6 between the chosen ones is not asked of
    # these few tokens: their choice is the GPU logits', checked beside
    logits, idx, _ = M.moe_route_scored(d["x"], d["w_router"], d["bias"], d["choice_bias"], k, **kw)
    ids, w = choose(logits.cpu().numpy(), d["choice_bias"].cpu().numpy(), k, **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ids)
    x = d["x"].double()
    ref = torch.zeros(T, H, dtype=torch.float64, device=x.device)

    def mlp(v, gu, dn):
        n = dn.shape[0]
        z = v @ gu.double()
        return (torch.nn.functional.silu(z[..., :n]) * z[..., n:]) @ dn.double()
    for t in range(T):
        for e, p in zip(ids[t], w[t]):
            if e0 <= e < e0 + El:
                ref[t] += p * mlp(x[t], d["w_gate_up"][e - e0], d["w_down"][e - e0])
    if Is:
        ref += mlp(x, d["shared_gate_up"], d["shared_down"])
    assert rel_max_err(y.double().cpu().numpy(), ref.cpu().numpy()) <= OUT_TOL
    assert O is not None and bf16_bits(y).shape == (T, H)


@gpu
@pytest.mark.parametrize("T,Is", [(48, 64), (7, 64), (7, 128), (16, 384)])
def test_shares_add_up_to_the_layer(T, Is):
    """The shared expert on one of four ranks; float32 shares added."""
    H, I, E, k = 256, 128, 32, 6
    d = weights(T, H, I, Is, E, E, 3)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_score="top2", out_dtype=F32)
    a = (d["x"], d["w_router"], d["bias"], d["choice_bias"])
    whole, _ = M.moe_layer_forward(*a, d["w_gate_up"], d["w_down"], k, 0, d["shared_gate_up"], d["shared_down"], **kw)
    total = torch.zeros_like(whole)
    for e0 in range(0, E, 8):
        shared = (d["shared_gate_up"], d["shared_down"]) if e0 == 16 else (None, None)
        total += M.moe_layer_forward(*a, d["w_gate_up"][e0:e0 + 8], d["w_down"][e0:e0 + 8], k, e0, *shared, **kw)[0]
    # k + 4 float32 additions of terms below the largest output
    assert float((total - whole).abs().max()) <= 2 * (k + 4) * 2.0 ** -24 * k * float(whole.abs().max())


@gpu
@pytest.mark.parametrize("T,Is", [(1, 136), (16, 136), (300, 136), (1, 128), (13, 256)])
def test_layer_in_a_graph_and_on_a_stream(T, Is):
    H, I, E, k = 256, 128, 64, 8
    d = weights(T, H, I, Is, E, E, T)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_score="top2")

    def call(**more):
        return M.moe_layer_forward(d["x"], d["w_router"], None, d["choice_bias"], d["w_gate_up"], d["w_down"], k, 0,
                                   d["shared_gate_up"], d["shared_down"], **kw, **more)
    want = call()[0]
    side = torch.cuda.Stream(device=d["x"].device)
    side.wait_stream(torch.cuda.current_stream(d["x"].device))
    got = call(stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((M.layer_workspace_size(T, H, I, Is, E, k, E),), 0xFF, dtype=torch.uint8, device=d["x"].device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(workspace=ws)[0]
    for rep in range(3):
        d["x"].copy_(torch.randn(T, H, device=d["x"].device) * H ** -0.5)
        want = call()[0]
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


@gpu
def test_a_decode_chain():
    """Two blocks as a model strings them: norm, layer, norm with the residual."""
    T, H, I, Is, E, k = 5, 256, 64, 64, 32, 4
    dev = device()
    r = torch.randn(T, H, device=dev).to(BF)
    ref = r.double()
    one = torch.ones(H, device=dev)
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2", scale=2.5)

    def norm64(v):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    for layer in range(2):
        d = weights(T, H, I, Is, E, E, 50 + layer)
        x = M.moe_norm_pre(r, one)
        y, _ = M.moe_layer_forward(x, d["w_router"], None, d["choice_bias"], d["w_gate_up"], d["w_down"], k, 0,
                                   d["shared_gate_up"], d["shared_down"], out_dtype=F32, **kw)
        _, idx, w = M.moe_route_scored(x, d["w_router"], None, d["choice_bias"], k, **kw)
        r, _ = M.moe_norm_post(y, r, one)
        xr = norm64(ref)

        def mlp(v, gu, dn):
            z = v @ gu.double()
            return (torch.nn.functional.silu(z[..., :dn.shape[0]]) * z[..., dn.shape[0]:]) @ dn.double()
        yr = mlp(xr, d["shared_gate_up"], d["shared_down"])
        for t in range(T):
            for e, p in zip(idx[t].tolist(), w[t].double()):
                yr[t] += p * mlp(xr[t], d["w_gate_up"][e], d["w_down"][e])
        ref = ref + norm64(yr)
    # each block rounds x, h, y's terms and r to bf16
    assert rel_max_err(r.double().cpu().numpy(), ref.cpu().numpy()) <= OUT_TOL
