"""The norms before and after a block (moe_norm_pre, moe_norm_post) against
their formulas in float64, and their refusals.

Tolerance of a value v computed from terms of magnitude m: half a step of its
type (bf16 2^-8, float32 2^-24, relative to v) plus the float32 arithmetic
before it. A row's sum of squares is formed by at most 32 additions per lane,
6 across the wave and 16 across the waves, a relative error of at most
54 x 2^-24 with the mean's product, halved by the square root; the reciprocal
root, the three products and the final addition add at most 6 steps more. So
40 x 2^-24 of m bounds it; n' inherits the error of r' and adds its own.
"""
import ctypes
import math
import sys

import pytest
import torch

import expert_token_routing_amd as M

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 40 * 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)

gpu = pytest.mark.gpu


# --------------------------------------------------------------------------- #
# Refusals (CPU)                                                               #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), M.MOE_ERR_INVALID_ARG), (dict(H=0), M.MOE_ERR_INVALID_ARG), (dict(H=12), M.MOE_ERR_INVALID_ARG),
    (dict(H=32776), M.MOE_ERR_UNSUPPORTED), (dict(eps=-1.0), M.MOE_ERR_INVALID_ARG),
    (dict(eps=math.nan), M.MOE_ERR_INVALID_ARG), (dict(eps=math.inf), M.MOE_ERR_INVALID_ARG),
    (dict(rt=2), M.MOE_ERR_INVALID_ARG), (dict(rt=-1), M.MOE_ERR_INVALID_ARG),
    (dict(r=None), M.MOE_ERR_INVALID_ARG), (dict(w=None), M.MOE_ERR_INVALID_ARG), (dict(out=None), M.MOE_ERR_INVALID_ARG),
    (dict(r=ODD), M.MOE_ERR_INVALID_ARG), (dict(w=ODD), M.MOE_ERR_INVALID_ARG), (dict(out=ODD), M.MOE_ERR_INVALID_ARG),
    (dict(T=0, r=None, out=None), M.MOE_OK),
])
def test_norm_pre_rejects(kw, want):
    a = dict(r=FAKE, rt=0, w=FAKE, eps=EPS, T=4, H=64, out=FAKE)
    a.update(kw)
    assert M.lib().moe_norm_pre(a["r"], a["rt"], a["w"], a["eps"], a["T"], a["H"], a["out"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(yt=2), M.MOE_ERR_INVALID_ARG), (dict(rt=7), M.MOE_ERR_INVALID_ARG), (dict(H=4), M.MOE_ERR_INVALID_ARG),
    (dict(H=40000), M.MOE_ERR_UNSUPPORTED), (dict(eps=math.nan), M.MOE_ERR_INVALID_ARG),
    (dict(kind=4), M.MOE_ERR_INVALID_ARG), (dict(kind=-1), M.MOE_ERR_INVALID_ARG),
    (dict(kind=1), M.MOE_ERR_INVALID_ARG),                 # a kind without a gate
    (dict(gate=FAKE), M.MOE_ERR_INVALID_ARG),              # a gate without a kind
    (dict(wn=None), M.MOE_ERR_INVALID_ARG), (dict(normed=None), M.MOE_ERR_INVALID_ARG),
    (dict(y=None), M.MOE_ERR_INVALID_ARG), (dict(r=None), M.MOE_ERR_INVALID_ARG), (dict(out=None), M.MOE_ERR_INVALID_ARG),
    (dict(y=ODD), M.MOE_ERR_INVALID_ARG), (dict(wp=ODD), M.MOE_ERR_INVALID_ARG), (dict(wn=ODD), M.MOE_ERR_INVALID_ARG),
    (dict(gate=ODD, kind=1), M.MOE_ERR_INVALID_ARG), (dict(gate=ODD, kind=3), M.MOE_ERR_INVALID_ARG),
    (dict(T=0, y=None, r=None, out=None), M.MOE_OK),
])
def test_norm_post_rejects(kw, want):
    a = dict(y=FAKE, yt=0, r=FAKE, rt=0, wp=FAKE, gate=None, kind=0, scale=1.0, wn=FAKE, eps=EPS, T=4, H=64, out=FAKE,
             normed=FAKE)
    a.update(kw)
    got = M.lib().moe_norm_post(a["y"], a["yt"], a["r"], a["rt"], a["wp"], a["gate"], a["kind"], a["scale"], a["wn"],
                                a["eps"], a["T"], a["H"], a["out"], a["normed"], None)
    assert got == want


def test_every_argument_may_be_named():
    """A call that names its first tensor too reaches its operator's checks."""
    z, w, f = torch.zeros(4, 64, dtype=BF), torch.zeros(64), torch.zeros(8, 64)
    gu, dn = torch.zeros(8, 64, 64, dtype=BF), torch.zeros(8, 32, 64, dtype=BF)
    q, s4 = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    layer = dict(w_router=f, bias=None, k=2)
    i8 = dict(w_gate_up=gu.to(torch.int8), s_gate_up=torch.zeros(8, 64), w_down=torch.zeros(8, 64, 32, dtype=torch.int8),
              s_down=torch.zeros(8, 64))
    for call in (lambda: M.moe_norm_pre(r=z, w=w), lambda: M.moe_norm_post(y=z, residual=z),
                 lambda: M.moe_forward_few(x=z, w_gate_up=gu, w_down=dn, e0=0, **layer),
                 lambda: M.moe_forward_few_f32(x=z, w_gate_up=gu, w_down=dn, e0=0, **layer),
                 lambda: M.moe_quantize_rows(x=z), lambda: M.moe_quantize_weights(w=gu),
                 lambda: M.moe_gemm_i8(a=q, a_scale=s4, w=q[None], w_scale=s4[None]),
                 lambda: M.moe_expert_ffn_i8(x_perm=z, offsets=torch.zeros(9, dtype=torch.int32), **i8),
                 lambda: M.moe_forward_i8(x=z, e0=0, **layer, **i8),
                 lambda: M.moe_block_forward(residual=z, w_pre=w, w_gate_up=gu, w_down=dn, **layer)):
        with pytest.raises(ValueError, match="must live on a GPU"):
            call()


def test_norms_reject_mismatched_tensors():
    y, w = torch.zeros(4, 64, dtype=BF), torch.zeros(64)
    for bad, exc, match in ((dict(r=y.double()), TypeError, "r must be"), (dict(w=w.double()), TypeError, "w must be"),
                            (dict(w=torch.zeros(72)), ValueError, "w has shape"),
                            (dict(out=torch.zeros(4, 72, dtype=BF)), ValueError, "out has shape"),
                            (dict(), ValueError, "must live on a GPU")):
        a = dict(r=y, w=w)
        a.update(bad)
        with pytest.raises(exc, match=match):
            M.moe_norm_pre(a.pop("r"), a.pop("w"), **a)
    for bad, exc, match in ((dict(residual=torch.zeros(5, 64, dtype=BF)), ValueError, "residual has shape"),
                            (dict(residual=y.half()), TypeError, "residual must be"),
                            (dict(w_post=torch.zeros(63)), ValueError, "w_post has shape"),
                            (dict(w_next=torch.zeros(63)), ValueError, "w_next has shape"),
                            (dict(gate=torch.zeros(4)), ValueError, "gate has shape"),
                            (dict(gate=torch.zeros(4, 1, dtype=BF)), TypeError, "gate must be"),
                            (dict(normed=y), ValueError, "normed is given"),
                            (dict(out=torch.zeros(4, 64)), TypeError, "out must be"),
                            (dict(w_next=w, normed=torch.zeros(4, 64)), TypeError, "normed must be"),
                            (dict(), ValueError, "must live on a GPU")):
        a = dict(y=y, residual=y.clone())
        a.update(bad)
        with pytest.raises(exc, match=match):
            M.moe_norm_post(a.pop("y"), a.pop("residual"), **a)


def test_sizes_past_31_bits_are_refused():
    """Before they reach an int argument, which would take their low 32 bits
    (meta tensors: shapes without memory)."""
    big, small = 2 ** 32 + 16, 16

    def t(*shape, dtype=BF):
        return torch.empty(shape, dtype=dtype, device="meta")
    I8 = torch.int8
    for call in (lambda: M.moe_norm_pre(t(big, 8), t(8, dtype=F32)), lambda: M.moe_norm_pre(t(1, big), t(big, dtype=F32)),
                 lambda: M.moe_norm_post(t(big, 8), t(big, 8)),
                 lambda: M.moe_forward_few(t(big, 8), t(4, 8, dtype=F32), None, t(4, 8, 16), t(4, 8, 8), 1, 0),
                 lambda: M.moe_forward_few_f32(t(1, 8), t(big, 8, dtype=F32), None, t(4, 8, 16), t(4, 8, 8), 1, 0),
                 lambda: M.moe_quantize_rows(t(1, big)), lambda: M.moe_quantize_weights(t(1, big, 8)),
                 lambda: M.moe_quantize_weights(t(1, 16, big)), lambda: M.moe_quantize_weights(t(big, 16, 8)),
                 lambda: M.moe_gemm_i8(t(1, small, dtype=I8), t(1, dtype=F32), t(1, big, small, dtype=I8), t(1, big, dtype=F32)),
                 lambda: M.moe_expert_ffn_i8(t(big, small), t(2, dtype=torch.int32), t(1, 32, small, dtype=I8),
                                             t(1, 32, dtype=F32), t(1, small, small, dtype=I8), t(1, small, dtype=F32)),
                 lambda: M.moe_forward_i8(t(big, small), t(4, small, dtype=F32), None, t(1, 32, small, dtype=I8),
                                          t(1, 32, dtype=F32), t(1, small, small, dtype=I8), t(1, small, dtype=F32), 1, 0),
                 lambda: M.moe_block_forward(t(big, 8), t(8, dtype=F32), t(4, 8, dtype=F32), None, t(4, 8, 16), t(4, 8, 8),
                                             1)):
        with pytest.raises(ValueError, match="at most 2.31 - 1, got 42949"):
            call()


# --------------------------------------------------------------------------- #
# The kernels (GPU)                                                            #
# --------------------------------------------------------------------------- #
def _rms(v, w):
    return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w.to(F64)


def _within(got, ref, slack, what):
    tol = HALF[got.dtype] * ref.abs() + slack + 1e-37
    err = (got.to(F64) - ref).abs()
    worst = float((err / tol).max()) if ref.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the tolerance"


def _inputs(T, H, yt, rt, gate, post, seed=0):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)

    def rn(*s, k=1.0):
        return torch.randn(s, generator=g, device=dev) * k

    shape = {None: None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return (rn(T, H, k=0.3).to(yt), rn(T, H).to(rt), 1 + rn(H, k=0.1) if post else None,
            None if shape is None else rn(*shape, k=0.5), 1 + rn(H, k=0.1))


def _check_post(T, H, yt, rt, gate, post, nxt, scale, **kw):
    y, r, wp, ga, wn = _inputs(T, H, yt, rt, gate, post)
    z = y.to(F64) if wp is None else _rms(y.to(F64), wp)
    if ga is not None:
        z = ga.to(F64) * z
    sr = scale * r.to(F64)
    ref = sr + z
    slack = U * (sr.abs() + z.abs())
    print(f"[gpu] norm_post T={T} H={H} y={yt} r={rt} gate={gate} post={post} next={nxt}", flush=True)
    out, normed = M.moe_norm_post(y, r, wp, gate=ga, residual_scale=scale, w_next=wn if nxt else None, eps=EPS, **kw)
    torch.cuda.synchronize()
    assert out.dtype == rt and (normed is None) == (not nxt)
    _within(out, ref, slack, "out")
    if nxt:
        n = _rms(ref, wn)
        inv = n.abs() / ref.abs().clamp_min(1e-30)
        # d n = inv * d r' directly, and through the row's norm at most the same
        # relative to the row's largest error over its rms
        rms = (ref.square().mean(-1, keepdim=True) + EPS).sqrt()
        row = (slack.square().mean(-1, keepdim=True)).sqrt() / rms
        _within(normed, n, inv * slack + n.abs() * (U + row), "normed")


@gpu
@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (3, 72), (600, 64), (1001, 2880), (517, 4104), (700, 8200), (2, 32768),
                                 (1, 16392), (530, 8192)])
@pytest.mark.parametrize("rt", [BF, F32])
def test_norm_pre(T, H, rt):
    _, r, _, _, w = _inputs(T, H, BF, rt, None, False)
    print(f"[gpu] norm_pre T={T} H={H} {rt}", flush=True)
    out = M.moe_norm_pre(r, w, EPS)
    torch.cuda.synchronize()
    ref = _rms(r.to(F64), w)
    _within(out, ref, U * ref.abs(), "out")


@gpu
@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (5, 2880), (600, 4104), (700, 8200), (2, 32768)])
@pytest.mark.parametrize("yt,rt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
def test_norm_post(T, H, yt, rt, gate):
    _check_post(T, H, yt, rt, gate, True, True, 0.7071)


@gpu
@pytest.mark.parametrize("post,nxt,scale", [(False, True, 1.0), (True, False, 0.5), (False, False, 0.0), (False, True, -2.0)])
@pytest.mark.parametrize("T,H", [(2, 1024), (520, 6144)])
def test_norm_post_parts(T, H, post, nxt, scale):
    _check_post(T, H, F32, BF, "channel", post, nxt, scale)


@gpu
def test_norm_post_no_rows():
    y, r, wp, ga, wn = _inputs(0, 64, BF, BF, "token", True)
    out, normed = M.moe_norm_post(y, r, wp, gate=ga, w_next=wn)
    assert out.shape == normed.shape == (0, 64)


@gpu
def test_norm_post_in_place_equals_apart():
    y, r, wp, ga, wn = _inputs(900, 2880, BF, BF, "full", True)
    out, normed = M.moe_norm_post(y, r, wp, gate=ga, w_next=wn, residual_scale=0.5)
    r2, y2 = r.clone(), y.clone()
    o2, n2 = M.moe_norm_post(y2, r2, wp, gate=ga, w_next=wn, residual_scale=0.5, out=r2, normed=y2)
    assert o2 is r2 and n2 is y2
    y3 = y.clone()
    o3, n3 = M.moe_norm_post(y3, r, wp, gate=ga, w_next=wn, residual_scale=0.5, out=y3)
    p = M.moe_norm_pre(r, wn)
    r4 = r.clone()
    M.moe_norm_pre(r4, wn, out=r4)
    torch.cuda.synchronize()
    for a, b in ((o2, out), (n2, normed), (o3, out), (n3, normed), (r4, p)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@gpu
@pytest.mark.parametrize("T,H", [(4, 512), (600, 5000)])
def test_norm_post_keeps_infinities_and_nans_in_their_row(T, H):
    y, r, wp, ga, wn = _inputs(T, H, F32, BF, "channel", True)
    out, normed = M.moe_norm_post(y, r, wp, gate=ga, w_next=wn)
    y2, r2 = y.clone(), r.clone()
    y2[1, 3] = math.nan
    r2[2, 5] = math.inf
    y2[3, :] = 0
    o2, n2 = M.moe_norm_post(y2, r2, wp, gate=ga, w_next=wn)
    torch.cuda.synchronize()
    assert torch.isnan(o2[1]).all() and torch.isnan(n2[1]).all()
    assert math.isinf(o2[2, 5]) and torch.isfinite(o2[2, 6:]).all() and torch.isnan(n2[2, 5])
    assert torch.equal(o2[3], r[3]) and torch.isfinite(n2[3]).all()  # a row of zeros has the norm zero
    keep = [0, *range(4, T)]
    assert torch.equal(o2[keep], out[keep]) and torch.equal(n2[keep], normed[keep])


@gpu
def test_norm_arguments_by_name_on_a_stream():
    x, w = torch.randn(5, 96, device="cuda"), torch.randn(96, device="cuda")
    want = M.moe_norm_pre(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.moe_norm_pre(r=x, w=w, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(M.moe_norm_pre(w=w, r=x), want)


@gpu
def test_small_calls_report_and_keep_what_they_are_given():
    """The calls of the extension module: the library's status as MoEError, a
    wrong number as TypeError, the caller's outputs returned as they are and
    with no reference kept."""
    x, w = torch.randn(6, 64, device="cuda", dtype=BF), torch.randn(64, device="cuda")
    flat = torch.zeros(6 * 64 + 1, device="cuda", dtype=BF)[1:].view(6, 64)  # 2 bytes past an aligned address
    i8, s = torch.zeros(6, 64, device="cuda", dtype=torch.int8), torch.ones(6, device="cuda")
    for call in (lambda: M.moe_norm_pre(x, w, -1.0), lambda: M.moe_norm_pre(flat, w), lambda: M.moe_norm_post(flat, x),
                 lambda: M.moe_norm_pre(x[:, :12].contiguous(), w[:12].contiguous()), lambda: M.moe_quantize_rows(flat),
                 lambda: M.moe_quantize_rows(x[:, :24].contiguous()),
                 lambda: M.moe_gemm_i8(i8, s, i8[None], s[None], out=torch.empty(37, device="cuda", dtype=BF)[1:].view(6, 6))):
        with pytest.raises(M.MoEError):
            call()
    for call in (lambda: M.moe_norm_pre(x, w, "1"), lambda: M.moe_norm_post(x, x, residual_scale=None)):
        with pytest.raises(TypeError):
            call()
    for call, exc in ((lambda: M.moe_norm_pre(x.t(), w), ValueError), (lambda: M.moe_norm_pre(x, w.cpu()), ValueError),
                      (lambda: M.moe_norm_pre(x, w, stream=0), AttributeError), (lambda: M.moe_norm_post(x, x.float()[:5]), ValueError),
                      (lambda: M.moe_gemm_i8(i8, s, i8.view(2, 3, 64), s.view(2, 3)), ValueError)):
        with pytest.raises(exc):
            call()
    out, normed, q = torch.empty_like(x), torch.empty_like(x), torch.empty_like(i8)
    held = [sys.getrefcount(t) for t in (x, w, out, normed, q, s)]
    for _ in range(3):
        assert M.moe_norm_pre(x, w, out=out) is out
        got = M.moe_norm_post(x, x, w, w_next=w, out=out, normed=normed)
        assert got[0] is out and got[1] is normed
        got = M.moe_quantize_rows(x, q=q, scale=s)
        assert got[0] is q and got[1] is s
    assert M.moe_norm_post(x, x)[1] is None
    del got
    assert [sys.getrefcount(t) for t in (x, w, out, normed, q, s)] == held


@gpu
def test_small_calls_refuse_tensors_without_storage():
    """A tensor that only pretends to be on the GPU has no data pointer: an
    exception, and the calls after it work."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    x, w = torch.randn(6, 64, device="cuda", dtype=BF), torch.randn(64, device="cuda")
    mode = FakeTensorMode()
    fx, fw = mode.from_tensor(x), mode.from_tensor(w)
    for call in (lambda: M.moe_norm_pre(fx, fw), lambda: M.moe_norm_pre(fx, fw, out=fx),
                 lambda: M.moe_norm_post(fx, fx, fw), lambda: M.moe_quantize_rows(fx)):
        with pytest.raises((RuntimeError, TypeError, ValueError)):
            call()
        assert torch.equal(M.moe_norm_pre(x, w), M.moe_norm_pre(x, w))


@gpu
def test_norm_replays_and_other_stream():
    y, r, wp, ga, wn = _inputs(700, 7168, F32, BF, "channel", True)
    ref, nref = M.moe_norm_post(y, r, wp, gate=ga, w_next=wn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, n = M.moe_norm_post(y, r, wp, gate=ga, w_next=wn, stream=side)
    side.synchronize()
    assert torch.equal(o, ref) and torch.equal(n, nref)
    out, normed = torch.empty_like(ref), torch.empty_like(nref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_norm_post(y, r, wp, gate=ga, w_next=wn, out=out, normed=normed)
    for _ in range(3):
        out.fill_(math.nan)
        normed.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(normed, nref)
        M.moe_norm_post(y, r, wp, gate=ga, w_next=wn)


@gpu
@pytest.mark.parametrize("T,H", [(16384, 4096), (16384, 8200), (70000, 2048)])
def test_norm_post_past_the_caches(T, H):
    """More rows than the caches hold take the loads and stores that pass them."""
    _check_post(T, H, F32, BF, "channel", True, True, 0.5)
    _check_post(T, H, BF, F32, "token", False, True, 1.0)


@gpu
def test_norm_pre_offsets_beyond_32_bits():
    T, H = 300001, 7168
    w = 1 + 0.1 * torch.randn(H, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    r = torch.zeros((T, H), dtype=BF, device="cuda")
    at = torch.tensor([0, 149796, 149797, 299593, T - 1], device="cuda")  # around 2^30 and 2^31 elements, and the ends
    r[at] = torch.randn((5, H), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    print(f"[gpu] norm_pre T={T} H={H}", flush=True)
    out = M.moe_norm_pre(r, w, EPS)
    torch.cuda.synchronize()
    ref = _rms(r[at].to(F64), w)
    _within(out[at], ref, U * ref.abs(), "out")
    assert int(out.abs().amax(1).gt(0).sum()) == 5
