"""The operators in the order a block uses them: moe_block_forward against its
three steps bit for bit, a chain of blocks whose norms pass on what the next
one takes, and the 8-bit layer between the same norms."""
import ctypes

import pytest
import torch

import expert_token_routing_amd as M

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)
gpu = pytest.mark.gpu
INV, UNS, WSP = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INV), (dict(H=12), INV), (dict(I=12), INV), (dict(k=5), INV), (dict(E=2000), UNS), (dict(H=40000), UNS),
    (dict(H=16384, I=32768), UNS), (dict(rt=2), INV), (dict(kind=1), INV), (dict(gate=FAKE), INV), (dict(kind=5), INV),
    (dict(normed=None), INV), (dict(wn=None), INV), (dict(eps=-1.0), INV), (dict(r=None), INV), (dict(wpre=None), INV),
    (dict(out=None), INV), (dict(dn=None), INV), (dict(wpre=ODD), INV), (dict(wp=ODD), INV), (dict(gu=ODD), INV),
    (dict(normed=ODD), INV), (dict(gate=ODD, kind=1), INV), (dict(ws=None), WSP), (dict(wsb=100), WSP),
    (dict(ws=ctypes.c_void_p(0x100010)), WSP), (dict(T=0, r=None, out=None), M.MOE_OK),
])
def test_block_forward_rejects(kw, want):
    d = dict(r=FAKE, rt=0, wpre=FAKE, wr=FAKE, gu=FAKE, dn=FAKE, wp=FAKE, gate=None, kind=0, wn=FAKE, eps=1e-6, T=8, H=64,
             I=32, E=4, k=2, out=FAKE, normed=FAKE, ws=ctypes.c_void_p(0x100000), wsb=1 << 30)
    d.update(kw)
    got = M.lib().moe_block_forward(d["r"], d["rt"], d["wpre"], d["wr"], None, d["gu"], d["dn"], d["wp"], d["gate"],
                                    d["kind"], 1.0, d["wn"], d["eps"], d["T"], d["H"], d["I"], d["E"], d["k"], 1, d["out"],
                                    d["normed"], d["ws"], d["wsb"], None)
    assert got == want


def test_block_forward_rejects_mismatched_tensors():
    r, w, wr = torch.zeros(4, 64, dtype=BF), torch.zeros(64), torch.zeros(8, 64)
    gu, dn = torch.zeros(8, 64, 64, dtype=BF), torch.zeros(8, 32, 64, dtype=BF)
    for args, kw, exc, match in (((r, w[:8], wr, None, gu, dn, 2), {}, ValueError, "w_pre has shape"),
                                 ((r, w, wr, None, gu[:4], dn, 2), {}, ValueError, "w_gate_up has shape"),
                                 ((r, w, wr, None, gu, dn[:, :8], 2), {}, ValueError, "w_down has shape"),
                                 ((r, w, wr, None, gu, dn, 9), {}, ValueError, "k must be"),
                                 ((r, w, wr, None, gu, dn, 2), dict(gate=torch.zeros(5, 1)), ValueError, "gate has shape"),
                                 ((r, w, wr, None, gu, dn, 2), dict(normed=r), ValueError, "normed is given"),
                                 ((r, w, wr, None, gu, dn, 2), dict(out=torch.zeros(4, 64)), TypeError, "out must be"),
                                 ((r, w, wr, None, gu, dn, 2), {}, ValueError, "must live on a GPU")):
        with pytest.raises(exc, match=match):
            M.moe_block_forward(*args, **kw)


def _layer(seed, H, I, E):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s, k=1.0):
        return torch.randn(s, generator=g, device="cuda") * k

    return dict(w_pre=1 + rn(H, k=0.1), w_router=rn(E, H, k=H ** -0.5), bias=rn(E, k=0.1),
                w_gate_up=rn(E, H, 2 * I, k=H ** -0.5).to(BF), w_down=rn(E, I, H, k=I ** -0.5).to(BF),
                w_post=1 + rn(H, k=0.1), gate=rn(H, k=0.5))


@gpu
@pytest.mark.parametrize("T", [0, 1, 16, 17, 200])
@pytest.mark.parametrize("rt", [BF, F32])
def test_block_equals_its_steps(T, rt):
    H, I, E, k = 264, 136, 6, 2
    p = _layer(0, H, I, E)
    r = torch.randn((T, H), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(rt)
    wn = p["w_post"].flip(0).contiguous()
    print(f"[gpu] block T={T} {rt}", flush=True)
    out, normed, ws = M.moe_block_forward(r, p["w_pre"], p["w_router"], p["bias"], p["w_gate_up"], p["w_down"], k,
                                          p["w_post"], gate=p["gate"], residual_scale=0.5, w_next=wn)
    x = M.moe_norm_pre(r, p["w_pre"])
    f = M.moe_forward_few_f32 if T <= 16 else M.moe_forward_f32
    y, _ = f(x, p["w_router"], p["bias"], p["w_gate_up"], p["w_down"], k, 0)
    o2, n2 = M.moe_norm_post(y, r, p["w_post"], gate=p["gate"], residual_scale=0.5, w_next=wn)
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(normed, n2)
    # in place, replayed
    if T:
        r2 = r.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.moe_block_forward(r2, p["w_pre"], p["w_router"], p["bias"], p["w_gate_up"], p["w_down"], k, p["w_post"],
                                gate=p["gate"], residual_scale=0.5, w_next=wn, out=r2, normed=n2, workspace=ws)
        for _ in range(3):
            r2.copy_(r)
            n2.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(r2, out) and torch.equal(n2, normed)


def _reference_layer(x, p, k):
    """The MoE layer of x (float64) with p's weights in float64."""
    lg = x @ p["w_router"].to(F64).T + p["bias"].to(F64)
    idx = torch.sort(lg, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.softmax(lg.gather(1, idx), 1)
    y = torch.zeros_like(x)
    I = p["w_down"].shape[1]
    for e in range(p["w_down"].shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        gu = x[t] @ p["w_gate_up"][e].to(F64)
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y.index_add_(0, t, w[t, j][:, None] * (h @ p["w_down"][e].to(F64)))
    return y


def _rms(v, w):
    return v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.to(F64)


@gpu
@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("layer", ["bf16", "i8"])
def test_two_blocks_in_a_row(T, layer):
    """Two blocks, the first one's last norm giving the second one's x, against
    the same chain in float64. Each block's x is taken from the GPU's chain (its
    rounding to bf16 could move a selection), so a block's output differs by the
    roundings of one block. Relative to the output's size: the residual's own
    rounding 2^-8; the layer's y (h and, above 16 tokens, the expert outputs
    rounded to bf16: 2 x 2^-8 at worst, of a gated part not above the whole);
    with 8-bit weights and activations, four quantised factors off by at most
    half a step of 1 / 127 of their row's largest value, which is at most 6
    times its size in these normal draws: 4 x 6 / 254 at worst, and at random
    1 / sqrt(3) of that and less: 0.06 of the gated part in norm."""
    H, I, E, k = 512, 256, 8, 2
    ps = [_layer(s, H, I, E) for s in (3, 4)]
    g = torch.Generator(device="cuda").manual_seed(5)
    r = torch.randn((T, H), generator=g, device="cuda").to(BF)
    x = M.moe_norm_pre(r, ps[0]["w_pre"])
    for i, p in enumerate(ps):
        wn = ps[(i + 1) % 2]["w_pre"]
        print(f"[gpu] chain T={T} {layer} block {i}", flush=True)
        if layer == "bf16":
            f = M.moe_forward_few_f32 if T <= M.FEW_TOKENS else M.moe_forward_f32
            y, _ = f(x, p["w_router"], p["bias"], p["w_gate_up"], p["w_down"], k, 0)
        else:
            q = (*M.moe_quantize_weights(p["w_gate_up"]), *M.moe_quantize_weights(p["w_down"]))
            y, _ = M.moe_forward_i8(x, p["w_router"], p["bias"], *q, k, 0)
        ref = r.to(F64) + p["gate"].to(F64) * _rms(_reference_layer(x.to(F64), p, k), p["w_post"])
        r, x = M.moe_norm_post(y, r, p["w_post"], gate=p["gate"], w_next=wn)
        torch.cuda.synchronize()
        assert r.dtype == BF and x.dtype == BF
        err = float((r.to(F64) - ref).norm() / ref.norm())
        assert err <= (3 * 2.0 ** -8 if layer == "bf16" else 3 * 2.0 ** -8 + 0.06), err
        want = _rms(ref, wn)
        assert float((x.to(F64) - want).norm() / want.norm()) <= err + 2 * 2.0 ** -8
