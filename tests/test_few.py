"""The whole share for a few tokens (moe_forward_few, moe_forward_few_f32)
against the layer's definition in float64, and its refusals.

Tolerance. A dot product over K is added in float32 by four waves, at most
K / 4 additions each (K products of exact bf16 values), then over the waves and
ranges (at most 64): every rounding is at most 2^-24 of the sum of the
products' magnitudes, S. So |error| <= (K / 4 + 64) 2^-24 S, and, the roundings
being independent, their root mean square over the outputs is at most
sqrt(K / 4 + 64) 2^-24 of S's. The errors of g and u reach h = silu(g) u through
|d silu / d g| <= 1.1 and |silu(g)| <= |g|, those of h reach y through w |Wd|.
The exponentials, divisions and products between add at most 16 steps of 2^-24.
h's three bf16 parts hold its 24 bits. Rounding y adds half a step.
"""
import ctypes

import pytest
import torch

import expert_token_routing_amd as M

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
gpu = pytest.mark.gpu
INV, UNS, WSP = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_ERR_WORKSPACE


# --------------------------------------------------------------------------- #
# Refusals (CPU)                                                               #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("kw,want", [
    (dict(T=33), UNS), (dict(T=-1), INV), (dict(H=12), INV), (dict(I=12), INV), (dict(I=0), INV), (dict(k=0), INV),
    (dict(k=5), INV), (dict(E=2000), UNS), (dict(E=64, k=33), UNS), (dict(e0=1), INV), (dict(El=0), INV),
    (dict(H=16384, I=32768), UNS), (dict(I=1 << 25, T=16), UNS),
    (dict(H=1 << 25, T=32), UNS), (dict(x=None), INV), (dict(w=None), INV), (dict(gu=None), INV), (dict(d=None), INV),
    (dict(y=None), INV), (dict(x=ODD), INV), (dict(gu=ODD), INV), (dict(d=ODD), INV), (dict(y=ODD), INV),
    (dict(ws=None), WSP), (dict(ws=ctypes.c_void_p(0x100010)), WSP), (dict(wsb=512), WSP),
    (dict(T=0, x=None, y=None, ws=None), M.MOE_OK),
])
@pytest.mark.parametrize("name", ["moe_forward_few", "moe_forward_few_f32"])
def test_few_rejects(name, kw, want):
    a = dict(x=FAKE, w=FAKE, gu=FAKE, d=FAKE, T=8, H=8, I=8, E=4, k=2, e0=0, El=4, y=FAKE, ws=ctypes.c_void_p(0x100000),
             wsb=1 << 30)
    a.update(kw)
    assert getattr(M.lib(), name)(a["x"], a["w"], None, a["gu"], a["d"], a["T"], a["H"], a["I"], a["E"], a["k"], a["e0"],
                                  a["El"], 1, a["y"], a["ws"], a["wsb"], None) == want


def test_few_workspace_size():
    """The partial sums: with n experts in use there are at most min(T k, n T)
    rows, each in at most ceil(1024 / (n panels)) ranges of at least 512."""
    assert M.FEW_TOKENS == 32
    assert M.few_workspace_size(33, 64, 64, 8, 2, 8) == 0
    for T, H, I, E, k, El in ((1, 7168, 256, 256, 8, 256), (16, 7168, 2048, 256, 8, 32), (32, 1024, 2816, 8, 2, 8),
                              (32, 1024, 640, 1024, 32, 512), (1, 8, 8, 1, 1, 1), (5, 72, 4104, 6, 3, 2)):
        cap, pa, pb = T * min(k, El), 2 * -(-I // 128), -(-H // 128)
        need = 0
        for n in range(1, min(El, cap) + 1):
            rows = min(cap, n * T)

            def ranges(K, items):
                u, want = -(-K // 512), -(-1024 // items)
                units = max(1, -(-u // want))
                return -(-u // units)
            need = max(need, rows * ranges(H, n * pa) * pa * 128 * 4 + rows * ranges(I, n * pb) * H * 4)
        assert M.few_workspace_size(T, H, I, E, k, El) >= need + T * E * 4 + cap * I * 4, (T, H, I, E, k, El)


@pytest.mark.parametrize("fn", ["moe_forward_few", "moe_forward_few_f32"])
def test_few_rejects_mismatched_tensors(fn):
    x, wr = torch.zeros(16, 64, dtype=BF), torch.zeros(8, 64)
    gu, dn = torch.zeros(4, 64, 64, dtype=BF), torch.zeros(4, 32, 64, dtype=BF)
    f = getattr(M, fn)
    for args, kw, exc, match in (((x, torch.zeros(8, 72), None, gu, dn, 2, 0), {}, ValueError, "w_router has shape"),
                                 ((x, wr, torch.zeros(7), gu, dn, 2, 0), {}, ValueError, "bias has shape"),
                                 ((x, wr, None, gu, dn[:, :24], 2, 0), {}, ValueError, "w_down has shape"),
                                 ((x, wr, None, gu, dn, 9, 0), {}, ValueError, "k must be"),
                                 ((x, wr, None, gu, dn, 2, 5), {}, ValueError, "local experts"),
                                 ((x, wr, None, gu.float(), dn, 2, 0), {}, TypeError, "w_gate_up must be"),
                                 ((x, wr, None, gu, dn, 2, 0), dict(y=torch.zeros(15, 64, dtype=BF if "32" not in fn else F32)),
                                  ValueError, "y has shape"),
                                 ((x, wr, None, gu, dn, 2, 0), {}, ValueError, "must live on a GPU")):
        with pytest.raises(exc, match=match):
            f(*args, **kw)


# --------------------------------------------------------------------------- #
# The kernels (GPU)                                                            #
# --------------------------------------------------------------------------- #
def _inputs(T, H, I, E, El, bias=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s, k=1.0):
        return torch.randn(s, generator=g, device="cuda") * k

    return ((rn(T, H) * H ** -0.5).to(BF), rn(E, H), rn(E, k=0.5) if bias else None,
            torch.randn((El, H, 2 * I), generator=g, device="cuda", dtype=BF) * H ** -0.5,
            torch.randn((El, I, H), generator=g, device="cuda", dtype=BF) * I ** -0.5)


def _reference(x, wr, bias, gu, dn, k, e0, renormalize):
    """y in float64, and the bounds' worst and root-mean-square sums."""
    T, H = x.shape
    El, I, _ = dn.shape
    lg = x.to(F64) @ wr.to(F64).T
    if bias is not None:
        lg = lg + bias.to(F64)
    idx = torch.sort(lg, dim=1, descending=True, stable=True)[1][:, :k]
    val = lg.gather(1, idx)
    w = torch.softmax(val, 1) if renormalize else torch.softmax(lg, 1).gather(1, idx)
    y, wa, wr_ = (torch.zeros((T, H), dtype=F64, device=x.device) for _ in range(3))
    nA, nB, u = H / 4 + 64, I / 4 + 64, 2.0 ** -24
    for e in range(El):
        t, j = (idx == e + e0).nonzero(as_tuple=True)
        if not len(t):
            continue
        xe, we = x[t].to(F64), gu[e].to(F64)
        p, q = xe @ we, xe.abs() @ we.abs()
        g, up, G, U = p[:, :I], p[:, I:], q[:, :I], q[:, I:]
        h = g * torch.sigmoid(g) * up
        d = dn[e].to(F64)
        scale = w[t, j][:, None]
        spread = (1.1 * G * up.abs() + g.abs() * U) @ d.abs()
        direct = h.abs() @ d.abs()
        y.index_add_(0, t, scale * (h @ d))
        wa.index_add_(0, t, scale * u * (nA * spread + (nB + 16) * direct))
        wr_.index_add_(0, t, scale * u * (nA ** 0.5 * spread + (nB ** 0.5 + 16) * direct))
    return y, wa, wr_


def _compare(y, ref, worst, rms, what):
    half = 2.0 ** -8 if y.dtype == BF else 2.0 ** -24
    err = (y.to(F64) - ref).abs()
    assert bool((err <= half * ref.abs() + worst + 1e-37).all()), what
    lim = float((half * ref).norm() + rms.norm())
    assert float(err.norm()) <= lim, f"{what}: norm {float(err.norm()):.3e}, bound {lim:.3e}"
    untouched = worst.sum(1) == 0  # no local selection: exact zeros
    assert bool(y[untouched].eq(0).all()), what


CASES = [
    (1, 8, 8, 1, 1, 0, 1),
    (1, 128, 64, 4, 1, 0, 4),
    (3, 72, 40, 8, 2, 2, 4),          # ragged panels and k ranges
    (5, 64, 32, 16, 3, 12, 2),        # tokens without a local expert
    (7, 2880, 768, 32, 4, 16, 16),
    (16, 520, 136, 64, 8, 0, 16),
    (17, 256, 96, 8, 2, 0, 8),
    (32, 264, 520, 2, 2, 0, 2),       # every expert has all 32 tokens
    (31, 136, 1032, 3, 1, 1, 1),      # one local expert, up to 31 rows
    (32, 1024, 640, 1024, 32, 100, 512),
    (32, 1024, 2816, 8, 2, 0, 8),
    (2, 4104, 24, 300, 5, 0, 300),
]


@gpu
@pytest.mark.parametrize("T,H,I,E,k,e0,El", CASES)
@pytest.mark.parametrize("bias,renormalize", [(False, True), (True, False)])
def test_few_against_definition(T, H, I, E, k, e0, El, bias, renormalize):
    a = _inputs(T, H, I, E, El, bias)
    ref, worst, rms = _reference(*a, k, e0, renormalize)
    print(f"[gpu] few T={T} H={H} I={I} E={E} k={k} e0={e0} El={El} bias={bias}", flush=True)
    y, ws = M.moe_forward_few(*a, k, e0, renormalize)
    torch.cuda.synchronize()
    _compare(y, ref, worst, rms, "bf16")
    ws.fill_(0xA5)
    y32 = torch.full((T, H), float("nan"), device="cuda")
    out, _ = M.moe_forward_few_f32(*a, k, e0, renormalize, y=y32, workspace=ws)
    torch.cuda.synchronize()
    assert out is y32
    _compare(y32, ref, worst, rms, "float32")
    assert torch.equal(y32.to(BF).view(torch.int16), y.view(torch.int16))
    again, _ = M.moe_forward_few(*a, k, e0, renormalize, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


@gpu
@pytest.mark.parametrize("T,I,E,El,e0", [(1, 256, 256, 256, 0), (16, 2048, 256, 32, 64), (32, 2048, 256, 32, 0)],
                         ids=["tp8_t1", "ep8_t16", "ep8_t32"])
def test_few_dsr1_shapes(T, I, E, El, e0):
    a = _inputs(T, 7168, I, E, El)
    ref, worst, rms = _reference(*a, 8, e0, True)
    print(f"[gpu] few DeepSeek-R1 shapes T={T} I={I} El={El}", flush=True)
    y, _ = M.moe_forward_few(*a, 8, e0)
    torch.cuda.synchronize()
    _compare(y, ref, worst, rms, "y")
    general, _ = M.moe_forward(*a, 8, e0)
    top = float(general.float().abs().max())
    assert float((general.float() - y.float()).abs().max()) <= 2e-2 * top


@gpu
def test_few_ties_and_lowest_values():
    """Equal router rows tie exactly: the lower expert wins; experts at -inf are
    taken last, in order; no local expert leaves zeros."""
    T, H, I, E = 4, 64, 32, 12
    x, wr, _, gu, dn = _inputs(T, H, I, E, E)
    wr = wr[:1].repeat(E, 1).contiguous()
    for bias in (None, torch.tensor([float("-inf")] * 10 + [0.0] * 2, device="cuda"),
                 torch.tensor([torch.finfo(F32).min] * 11 + [0.0], device="cuda")):
        for k, e0, El in ((3, 0, E), (3, 0, 2), (3, 4, 4)):
            a = (x, wr, bias, gu[:El].contiguous(), dn[:El].contiguous())
            ref, worst, rms = _reference(*a, k, e0, True)
            y, _ = M.moe_forward_few(*a, k, e0)
            torch.cuda.synchronize()
            _compare(y, ref, worst, rms, f"k={k} e0={e0} El={El}")


@gpu
def test_few_no_tokens():
    a = _inputs(1, 64, 32, 8, 8)
    y, _ = M.moe_forward_few(a[0][:0], *a[1:], 2, 0)
    assert y.shape == (0, 64)


@gpu
@pytest.mark.parametrize("T,H,I,E,k,e0,El", [(1, 7168, 256, 64, 8, 0, 64), (9, 520, 136, 64, 8, 0, 16), (32, 264, 520, 2, 2, 0, 2)])
def test_few_replayed(T, H, I, E, k, e0, El):
    a = _inputs(T, H, I, E, El)
    ref, ws = M.moe_forward_few(*a, k, e0)
    y = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        M.moe_forward_few(*a, k, e0, y=y, workspace=ws)
    for i in range(4):
        print(f"[gpu] few replay {i} T={T} H={H}", flush=True)
        y.fill_(float("nan"))
        ws.fill_(i * 85)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
        other, _ = M.moe_forward_few(*a, k, e0)
        torch.cuda.synchronize()
        assert torch.equal(other.view(torch.int16), ref.view(torch.int16))


@gpu
def test_few_two_calls_at_once():
    """Two streams, each with its own workspace, their kernels side by side."""
    a = _inputs(16, 2048, 1024, 32, 32, seed=1)
    b = _inputs(32, 1024, 2816, 8, 8, seed=2)
    ra, _ = M.moe_forward_few(*a, 4, 0)
    rb, _ = M.moe_forward_few(*b, 2, 0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ys = []
    print("[gpu] few on two streams", flush=True)
    for _ in range(8):
        ys.append((M.moe_forward_few(*a, 4, 0, stream=s1)[0], ra))
        ys.append((M.moe_forward_few(*b, 2, 0, stream=s2)[0], rb))
    torch.cuda.synchronize()
    for y, r in ys:
        assert torch.equal(y.view(torch.int16), r.view(torch.int16))


def _internal():
    """moe_forward_few_f32 with its number of workgroups and of polls before a
    waiting one turns to other work as arguments (an entry point for tests)."""
    f = M.lib().moe_internal_forward_few
    f.restype = ctypes.c_int
    f.argtypes = M.SIGNATURES["moe_forward_few_f32"][1][:16] + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return f


def _few_with(workgroups, polls, a, k, e0, y, ws):
    x, wr, _, _, dn = a
    st = _internal()(*(t.data_ptr() if t is not None else None for t in a), x.shape[0], x.shape[1], dn.shape[1],
                     wr.shape[0], k, e0, dn.shape[0], 1, y.data_ptr(), ws.data_ptr(), ws.numel(), workgroups, polls,
                     torch.cuda.current_stream().cuda_stream)
    M.check(st, "moe_internal_forward_few")


@pytest.mark.parametrize("workgroups,polls", [(0, 0), (0, -1), (-1, 1)])
def test_few_internal_rejects(workgroups, polls):
    assert _internal()(FAKE, FAKE, None, FAKE, FAKE, 8, 8, 8, 4, 2, 0, 4, 1, FAKE, ctypes.c_void_p(0x100000), 1 << 30,
                       workgroups, polls, None) == INV


@gpu
@pytest.mark.parametrize("T,H,I,E,k,e0,El", CASES + [(1, 7168, 256, 256, 8, 0, 256), (16, 2048, 1024, 64, 8, 16, 32)])
@pytest.mark.parametrize("workgroups,polls", [(8, 1), (11, 2), (40, 1), (0, 1)])
def test_few_items_put_aside(T, H, I, E, k, e0, El, workgroups, polls):
    """Workgroups that find their own queues empty while others still hold items
    put theirs aside and take those: with 11 workgroups on eight queues, up to
    700 items of a call. The same bits, from a workspace of any contents, one call
    after another and two side by side."""
    a = _inputs(T, H, I, E, El, bias=True)
    ref, ws = M.moe_forward_few_f32(*a, k, e0)
    ws2 = torch.empty_like(ws)
    ys = [torch.empty_like(ref) for _ in range(3)]
    side = torch.cuda.Stream()
    for i in range(2):
        print(f"[gpu] few put aside {i} workgroups={workgroups} polls={polls} T={T} H={H} I={I} E={E}", flush=True)
        ws.fill_(85 * i)
        ws2.fill_(255 - 85 * i)
        for y in ys:
            y.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        _few_with(workgroups, polls, a, k, e0, ys[0], ws)
        _few_with(workgroups, polls, a, k, e0, ys[1], ws)
        with torch.cuda.stream(side):
            _few_with(workgroups, polls, a, k, e0, ys[2], ws2)
        torch.cuda.synchronize()
        for y in ys:
            assert torch.equal(y.view(torch.int32), ref.view(torch.int32))
