"""moe_layer_forward up to 16 tokens, where the share for a few tokens takes the
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
                                                (3, 264, 128, 256, 8, 1, 7, 2)])
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
