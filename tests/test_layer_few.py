"""moe_layer_forward for a few tokens, where the share for a few tokens takes the
experts that were chosen before and the shared expert beside them."""
import ctypes

import pytest
import torch

import expert_token_routing_amd as M
from tests.test_layer import weights

F32 = torch.float32
FAKE = ctypes.c_void_p(0x100000)
KW = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2", scale=2.5)
gpu = pytest.mark.gpu


def internal():
    """moe_layer_forward with its number of workgroups and of polls before a waiting one turns
    to other work as arguments (an entry point for tests)."""
    f = M.lib().moe_internal_layer_forward
    args = M.SIGNATURES["moe_layer_forward"][1]
    f.restype, f.argtypes = ctypes.c_int, args[:-1] + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return f


def layer_with(workgroups, polls, d, k, e0, y, ws):
    names = ("x", "w_router", "bias", "choice_bias", "w_gate_up", "w_down", "shared_gate_up", "shared_down")
    El, I, H = d["w_down"].shape
    st = internal()(*(None if d[n] is None else d[n].data_ptr() for n in names), d["x"].shape[0], H, I,
                    0 if d["shared_down"] is None else d["shared_down"].shape[0], d["w_router"].shape[0], k, e0, El, 1, 4, 2,
                    1, 1, 2.5, y.data_ptr(), 1, ws.data_ptr(), ws.numel(), workgroups, polls,
                    torch.cuda.current_stream().cuda_stream)
    M.check(st, "moe_internal_layer_forward")


@pytest.mark.parametrize("workgroups,polls", [(0, 0), (0, -1), (-1, 1)])
def test_internal_rejects(workgroups, polls):
    assert internal()(FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, 8, 8, 8, 8, 4, 2, 0, 4, 1, 1, 1, 0, 1, 1.0, FAKE, 1,
                      FAKE, 1 << 30, workgroups, polls, None) == M.MOE_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("T,H,I,Is,E,El,e0,k", [(1, 7168, 256, 256, 256, 256, 0, 8), (16, 2048, 1024, 1024, 64, 32, 16, 8),
                                                (5, 136, 40, 120, 32, 8, 8, 6), (13, 520, 264, 0, 16, 16, 0, 3),
                                                (3, 264, 128, 256, 8, 1, 7, 2), (32, 1024, 264, 520, 8, 8, 0, 2),
                                                (17, 136, 64, 72, 32, 12, 8, 6), (25, 2048, 512, 0, 16, 4, 4, 3)])
@pytest.mark.parametrize("workgroups,polls", [(8, 1), (11, 2), (40, 1), (0, 1)])
def test_items_put_aside(T, H, I, Is, E, El, e0, k, workgroups, polls):
    """Workgroups that put waiting items aside for others', as in moe_forward_few's test of it: the
    same bits, from a workspace of any contents, one call after another and two side by side."""
    d = weights(T, H, I, Is, E, El, T + Is)
    ref, ws = M.moe_layer_forward(d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], k, e0,
                                  d["shared_gate_up"], d["shared_down"], out_dtype=F32, **KW)
    ws2 = torch.empty_like(ws)
    ys = [torch.empty_like(ref) for _ in range(3)]
    side = torch.cuda.Stream()
    for i in range(2):
        print(f"[gpu] layer put aside {i} workgroups={workgroups} polls={polls} T={T} H={H} I={I} Is={Is} E={E}", flush=True)
        ws.fill_(85 * i)
        ws2.fill_(255 - 85 * i)
        for y in ys:
            y.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        layer_with(workgroups, polls, d, k, e0, ys[0], ws)
        layer_with(workgroups, polls, d, k, e0, ys[1], ws)
        with torch.cuda.stream(side):
            layer_with(workgroups, polls, d, k, e0, ys[2], ws2)
        torch.cuda.synchronize()
        for y in ys:
            assert torch.equal(y.view(torch.int32), ref.view(torch.int32))


def shared_alone(x, gate_up, down):
    """swiglu(x G) D in float64, and tests/test_few.py's bound of its error in float32 sums: the
    worst of it, and its root mean square."""
    F64, u = torch.float64, 2.0 ** -24
    I, H = down.shape
    nA, nB = H / 4 + 64, I / 4 + 64
    xe, we, d = x.to(F64), gate_up.to(F64), down.to(F64)
    p, q = xe @ we, xe.abs() @ we.abs()
    g, up, G, U = p[:, :I], p[:, I:], q[:, :I], q[:, I:]
    h = g * torch.sigmoid(g) * up
    spread, direct = (1.1 * G * up.abs() + g.abs() * U) @ d.abs(), h.abs() @ d.abs()
    return (h @ d, u * (nA * spread + (nB + 16) * direct),
            u * (nA ** 0.5 * spread + (nB ** 0.5 + 16) * direct))


WIDTHS = [(1, 3176, 136, 96), (2, 328, 2760, 264), (11, 2680, 736, 1128), (16, 1024, 256, 264), (3, 200, 32, 1624),
          (16, 264, 40, 8), (7, 520, 128, 129 * 8), (5, 136, 520, 1000), (4, 72, 8, 64), (13, 1032, 1024, 1016),
          (16, 136, 32, 60 * 128), (1, 264, 136, 60 * 256 - 8),
          (17, 1024, 256, 256), (24, 264, 40, 8), (27, 5336, 208, 1936), (32, 520, 128, 28 * 128), (19, 976, 448, 40),
          (32, 64, 128, 72)]


@gpu
@pytest.mark.parametrize("T,H,I,Is", WIDTHS)
def test_a_shared_expert_of_any_width_keeps_float32(T, H, I, Is):
    """With a scale of 0 only the shared expert is left: its hidden values are not rounded to bf16
    (whose 2^-8 would be far outside), whatever its width beside the local ones'."""
    d = weights(T, H, I, Is, 16, 8, T + Is)
    print(f"[gpu] shared alone T={T} H={H} I={I} Is={Is}", flush=True)
    a = (d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], 4, 4)
    kw = dict(KW, out_dtype=F32)
    y = M.moe_layer_forward(*a, d["shared_gate_up"], d["shared_down"], **dict(kw, scale=0.0))[0].double()
    ref, worst, rms = shared_alone(d["x"], d["shared_gate_up"], d["shared_down"])
    err = (y - ref).abs()
    assert bool((err <= 2.0 ** -24 * ref.abs() + worst).all())
    assert float(err.norm()) <= float((2.0 ** -24 * ref).norm() + rms.norm())
    # beside the local ones: sums of k + n products, in order, each rounded
    whole = M.moe_layer_forward(*a, d["shared_gate_up"], d["shared_down"], **kw)[0].double()
    local = M.moe_layer_forward(*a, None, None, **kw)[0].double()
    terms = 4 - (-Is // I)
    size = torch.maximum(local.abs(), y.abs()).max() * terms
    assert float((whole - local - y).abs().max()) <= 2 * terms * 2.0 ** -24 * float(size)


@gpu
@pytest.mark.parametrize("T,H,I,Is", [(16, 520, 264, 712), (3, 136, 40, 8), (1, 2048, 256, 520), (29, 520, 264, 712)])
def test_a_shared_expert_of_any_width_by_few_workgroups(T, H, I, Is):
    """Its empty blocks and k ranges are items as the others are; nothing of it is read past its
    matrices' ends (NaN behind them)."""
    d = weights(T, H, I, Is, 16, 8, T + Is)
    for name, n in (("shared_gate_up", H * 2 * Is), ("shared_down", Is * H)):
        flat = torch.full((n + 4096,), float("nan"), dtype=torch.bfloat16, device="cuda")
        flat[:n] = d[name].flatten()
        d[name] = flat[:n].view(d[name].shape)
    ref, ws = M.moe_layer_forward(d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], 4, 4,
                                  d["shared_gate_up"], d["shared_down"], out_dtype=F32, **KW)
    assert bool(torch.isfinite(ref).all())
    y = torch.empty_like(ref)
    for i, (workgroups, polls) in enumerate(((8, 1), (11, 2), (40, 1))):
        print(f"[gpu] shared of any width, workgroups={workgroups} T={T} H={H} I={I} Is={Is}", flush=True)
        ws.fill_(85 * i)
        layer_with(workgroups, polls, d, 4, 4, y, ws)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int32), ref.view(torch.int32))


@gpu
@pytest.mark.parametrize("T", [17, 24, 32])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, F32])
def test_up_to_32_tokens_every_expert_keeps_float32(T, out_dtype):
    """Local experts and shared one against the layer in float64, chosen by the GPU's logits. What
    is off beside the sums' roundings: the weights, by those of logits of up to 8 (2^-24 for
    each of at most H / 4 + 64 additions, in root mean square), at most 1e-4 of y, where bf16 hidden
    values are 1e-3 off."""
    H, I, Is, E, El, e0, k = 1024, 256, 264, 16, 8, 4, 4
    d = weights(T, H, I, Is, E, El, T)
    print(f"[gpu] layer in float32 T={T} {out_dtype}", flush=True)
    y = M.moe_layer_forward(d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], k, e0,
                            d["shared_gate_up"], d["shared_down"], out_dtype=out_dtype, **KW)[0].double()
    logits, idx, _ = M.moe_route_scored(d["x"], d["w_router"], d["bias"], d["choice_bias"], k, **KW)
    s = torch.sigmoid(d["x"].double() @ d["w_router"].double().T + d["bias"].double()).gather(1, idx.long())
    w = 2.5 * s / s.sum(1, keepdim=True)
    ref = shared_alone(d["x"], d["shared_gate_up"], d["shared_down"])[0]
    for e in range(El):
        t, j = (idx == e + e0).nonzero(as_tuple=True)
        if len(t):
            ref.index_add_(0, t, w[t, j][:, None] * shared_alone(d["x"][t], d["w_gate_up"][e], d["w_down"][e])[0])
    half = 2.0 ** -8 * ref.abs() if out_dtype is torch.bfloat16 else torch.zeros_like(ref)
    over = ((y - ref).abs() - half).clamp(min=0)  # beyond y's own rounding
    assert float(over.norm()) <= 1e-4 * float(ref.norm())


@gpu
@pytest.mark.parametrize("T,H,I,Is,k", [(32, 128, 128, 20 * 128, 16), (4, 136, 64, 63 * 128, 4), (32, 264, 40, 1024, 32)])
def test_a_shared_expert_too_wide_for_the_tables(T, H, I, Is, k):
    """More parts than the kernel of a few tokens holds: two products onto the float32 share, whose
    hidden values are rounded to bf16 (2^-9 each, at most; the sums' terms are of either sign)."""
    E = 32
    d = weights(T, H, I, Is, E, E, Is)
    print(f"[gpu] shared too wide T={T} H={H} I={I} Is={Is} k={k}", flush=True)
    a = (d["x"], d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], k, 0)
    kw = dict(score="sigmoid", out_dtype=F32)
    y = M.moe_layer_forward(*a, d["shared_gate_up"], d["shared_down"], scale=0.0, **kw)[0].double()
    ref = shared_alone(d["x"], d["shared_gate_up"], d["shared_down"])[0]
    h = d["x"].double() @ d["shared_gate_up"].double()
    h = torch.nn.functional.silu(h[:, :Is]) * h[:, Is:]
    bound = 2.0 ** -8 * (h.abs() @ d["shared_down"].double().abs())
    assert bool(((y - ref).abs() <= bound).all())
    whole = M.moe_layer_forward(*a, d["shared_gate_up"], d["shared_down"], **kw)[0].double()
    local = M.moe_layer_forward(*a, None, None, **kw)[0].double()
    assert float((whole - local - y).abs().max()) <= 4 * 2.0 ** -24 * float(torch.maximum(local.abs(), y.abs()).max())


@gpu
@pytest.mark.parametrize("T,Is", [(17, 136), (24, 128), (32, 264), (32, 0), (5, 72)])
def test_a_few_tokens_in_a_graph_and_on_a_stream(T, Is):
    H, I, E, k = 256, 128, 64, 8
    d = weights(T, H, I, Is, E, E, T)
    print(f"[gpu] few tokens in a graph T={T} Is={Is}", flush=True)

    def call(**more):
        return M.moe_layer_forward(d["x"], d["w_router"], None, d["choice_bias"], d["w_gate_up"], d["w_down"], k, 0,
                                   d["shared_gate_up"], d["shared_down"], **KW, **more)
    want = call()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((M.layer_workspace_size(T, H, I, Is, E, k, E),), 0xFF, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(workspace=ws)[0]
    for rep in range(3):
        d["x"].copy_(torch.randn(T, H, device="cuda") * H ** -0.5)
        want = call()[0]
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


@gpu
def test_tokens_alone_or_among_others():
    """A token's y by itself and among 16 and 32: the sums' order goes by the experts in use, so they
    agree to float32 accuracy of its logits and sums (1e-5 of the largest), not to bf16's."""
    H, I, Is, E, k = 512, 128, 200, 32, 4
    d = weights(32, H, I, Is, E, E, 1)
    a = (d["w_router"], d["bias"], d["choice_bias"], d["w_gate_up"], d["w_down"], k, 0, d["shared_gate_up"], d["shared_down"])
    print("[gpu] tokens alone or among others", flush=True)
    whole = M.moe_layer_forward(d["x"], *a, out_dtype=F32, **KW)[0]
    for lo, n in ((0, 1), (7, 16), (31, 1), (3, 17)):
        y = M.moe_layer_forward(d["x"][lo:lo + n], *a, out_dtype=F32, **KW)[0]
        assert float((y - whole[lo:lo + n]).abs().max()) <= 1e-5 * float(whole.abs().max())
