"""moe_gemm (bf16 products with bias, activation and residual) against its
formula in float64, and its refusals.

Two kinds of inputs. Small integers: every partial sum is an integer below 2^24,
so z = a . w is exact in float32 in any order, and any product left out or taken
twice shows. Normal values: a sum of K products in float32 is off by at most
K x 2^-24 of the sum of their magnitudes, whatever its order.

Behind z: the bias rounds once (2^-24 of z). An activation has a slope of at most
1.2 and rounds a few times: 16 steps of 2^-24 of its value, and for its
exponential's argument's rounding 2 steps times that argument, twice (gelu: the
argument z^2 / 2 of exp(-z^2 / 2); tanh form: 2 sqrt(2 / pi) (|z| + 0.045 |z|^3)).
swiglu is silu's error times |u| plus u's times |silu(g)|. The residual's
addition rounds once, and the store once to its type.
"""
import ctypes
import math

import pytest
import torch

import expert_token_routing_amd as M
from tests.gpu_helpers import device, say

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]
gpu = pytest.mark.gpu


def act64(name, z, dz):
    """act(z) in float64 and its error bound for z off by dz."""
    az = z.abs()
    if name == "none":
        return z, dz
    if name == "relu":
        return torch.relu(z), dz
    if name == "silu":
        v, arg = z * torch.sigmoid(z), az
    elif name == "gelu":
        v, arg = 0.5 * z * torch.special.erfc(-z / math.sqrt(2)), z * z / 2
    else:
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        v, arg = z * torch.sigmoid(2 * u), 2 * math.sqrt(2 / math.pi) * (az + 0.045 * az ** 3)
    # (below the smallest normal numbers of float32 there are no steps to count)
    return v, 1.2 * dz + (16 + 4 * arg) * U * v.abs() + 2.0 ** -120


def reference(a, w, bias, offsets, act, residual, exact):
    """(value, bound before the store) [M, N] in float64; NaN bounds nowhere."""
    Mr, K = a.shape
    off = [0, Mr] if offsets is None else [min(max(o, 0), Mr) for o in offsets.tolist()]
    n = w.shape[2] // (2 if act == "swiglu" else 1)
    v = torch.full((Mr, n), math.nan, dtype=F64, device=a.device)
    tol = torch.zeros_like(v)
    for e in range(len(off) - 1):
        lo, hi = off[e], max(off[e], off[e + 1])
        if lo == hi:
            continue
        x, we = a[lo:hi].double(), w[e].double()
        z = x @ we
        dz = torch.zeros_like(z) if exact else K * U * (x.abs() @ we.abs())
        if bias is not None:
            z = z + bias[e].double()
            dz = dz + U * z.abs()
        if act == "swiglu":
            g, dg = act64("silu", z[:, :n], dz[:, :n])
            u, du = z[:, n:], dz[:, n:]
            v[lo:hi] = g * u
            tol[lo:hi] = dg * u.abs() + du * g.abs() + dg * du + U * (g * u).abs()
        else:
            v[lo:hi], tol[lo:hi] = act64(act, z, dz)
    if residual is not None:
        v = v + residual.double()
        tol = tol + U * v.abs()
    return v, tol


def inputs(Mr, K, N, act, bias, res, El, integers, seed):
    dev = device()
    g = torch.Generator(device=dev).manual_seed(seed)
    C = 2 * N if act == "swiglu" else N

    def values(*shape, scale):
        if integers:
            return torch.randint(-4, 5, shape, generator=g, device=dev).float()
        return torch.randn(shape, generator=g, device=dev) * scale
    a = values(Mr, K, scale=1.0).to(BF)
    w = values(El, K, C, scale=K ** -0.5).to(BF)
    b = values(El, C, scale=0.5) if bias else None
    r = None if res is None else values(Mr, N, scale=1.0).to(res)
    return a, w, b, r


TILES = ["few", "mid", "tall", "big", "small"]


def on_tile(tile, a, w, b, off, act, r, out, ranges=1):
    """moe_gemm on given tiles (an entry point for the tests, not of the header)."""
    fn = M.lib().moe_internal_gemm
    fn.restype = ctypes.c_int
    P, I = ctypes.c_void_p, ctypes.c_int
    fn.argtypes = [P, P, P, P, I, P, ctypes.c_int64, I, I, I, I, P, I, I, I, P, ctypes.c_size_t, P]

    def ptr(t):
        return None if t is None else t.data_ptr()
    part = torch.full((ranges, a.shape[0], w.shape[2]), math.nan, device=a.device) if ranges > 1 else None
    st = fn(ptr(a), ptr(w), ptr(b), ptr(r), int(r is not None and r.dtype == F32), ptr(off), a.shape[0], out.shape[1],
            a.shape[1], w.shape[0], ACTS.index(act), ptr(out), int(out.dtype == F32), TILES.index(tile),
            ranges, ptr(part), 0 if part is None else 4 * part.numel(), torch.cuda.current_stream(a.device).cuda_stream)
    M.check(st, f"moe_internal_gemm on {tile}")
    return out


def run(Mr, K, N, act="none", bias=False, res=None, out=BF, El=1, offsets=None, integers=False, seed=0, tile=None,
        ranges=1):
    say(f"gemm {Mr} x {K} x {N} act={act} bias={bias} res={res} out={out} El={El} offsets={offsets} integers={integers} "
        f"tile={tile} ranges={ranges}")
    a, w, b, r = inputs(Mr, K, N, act, bias, res, El, integers, seed)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=a.device)
    given = torch.full((Mr, N), -77.0, dtype=out, device=a.device)
    if tile is None:
        assert M.moe_gemm(a, w, b, off, activation=act, residual=r, out=given).data_ptr() == given.data_ptr()
    else:
        on_tile(tile, a, w, b, off, act, r, given, ranges)
    v, tol = reference(a, w, b, off, act, r, integers)
    written = ~torch.isnan(v)
    assert torch.all(given[~written] == -77.0)
    err = (given.double() - v).abs()
    bound = tol + HALF[out] * (v.abs() + tol) + 2.0 ** -133
    bad = written & ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(err[bad].max()))
    if integers and act in ("none", "relu"):
        assert torch.equal(given[written], v[written].to(out))


# --------------------------------------------------------------------------- #
# Refusals (CPU)                                                               #
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("kw,want", [
    (dict(cap=-1), M.MOE_ERR_INVALID_ARG), (dict(N=0), M.MOE_ERR_INVALID_ARG), (dict(N=12), M.MOE_ERR_INVALID_ARG),
    (dict(K=0), M.MOE_ERR_INVALID_ARG), (dict(K=20), M.MOE_ERR_INVALID_ARG), (dict(El=0), M.MOE_ERR_INVALID_ARG),
    (dict(act=6), M.MOE_ERR_INVALID_ARG), (dict(act=-1), M.MOE_ERR_INVALID_ARG), (dict(ot=2), M.MOE_ERR_INVALID_ARG),
    (dict(rt=2), M.MOE_ERR_INVALID_ARG), (dict(offsets=None, El=2), M.MOE_ERR_INVALID_ARG),
    (dict(a=None), M.MOE_ERR_INVALID_ARG), (dict(w=None), M.MOE_ERR_INVALID_ARG), (dict(out=None), M.MOE_ERR_INVALID_ARG),
    (dict(a=ODD), M.MOE_ERR_INVALID_ARG), (dict(w=ODD), M.MOE_ERR_INVALID_ARG), (dict(bias=ODD), M.MOE_ERR_INVALID_ARG),
    (dict(res=ODD), M.MOE_ERR_INVALID_ARG), (dict(out=ODD), M.MOE_ERR_INVALID_ARG),
    (dict(N=1 << 15, K=1 << 15), M.MOE_ERR_UNSUPPORTED), (dict(N=1 << 14, K=1 << 15, act=5), M.MOE_ERR_UNSUPPORTED),
    (dict(El=1025), M.MOE_ERR_UNSUPPORTED), (dict(cap=2 ** 31 - 1000), M.MOE_ERR_UNSUPPORTED),
    (dict(cap=1 << 30, N=1 << 16, K=8), M.MOE_ERR_UNSUPPORTED),
    (dict(K=1 << 20, N=8), M.MOE_ERR_UNSUPPORTED),
    (dict(K=7168), M.MOE_ERR_WORKSPACE), (dict(K=7168, ws=ODD, nws=1 << 30), M.MOE_ERR_WORKSPACE),
    (dict(K=7168, ws=FAKE, nws=1024), M.MOE_ERR_WORKSPACE),
    (dict(cap=0, a=None, w=None, out=None), M.MOE_OK),
])
def test_gemm_rejects(kw, want):
    p = dict(a=FAKE, w=FAKE, bias=FAKE, res=FAKE, rt=0, offsets=FAKE, cap=16, N=64, K=64, El=1, act=0, out=FAKE, ot=0, ws=None, nws=0)
    p.update(kw)
    assert M.lib().moe_gemm(p["a"], p["w"], p["bias"], p["res"], p["rt"], p["offsets"], p["cap"], p["N"], p["K"], p["El"],
                            p["act"], p["out"], p["ot"], p["ws"], p["nws"], None) == want


def test_gemm_rejects_mismatched_tensors():
    a, w = torch.zeros(4, 64, dtype=BF), torch.zeros(1, 64, 32, dtype=BF)
    for kw, exc, match in ((dict(a=a.float()), TypeError, "a must be"), (dict(w=w.float()), TypeError, "w must be"),
                           (dict(w=w[0]), ValueError, "w has shape"), (dict(w=torch.zeros(1, 72, 32, dtype=BF)), ValueError, "w has"),
                           (dict(w=torch.zeros(2, 64, 32, dtype=BF)), ValueError, "offsets is required"),
                           (dict(bias=torch.zeros(32)), ValueError, "bias has shape"),
                           (dict(bias=torch.zeros(1, 32, dtype=BF)), TypeError, "bias must be"),
                           (dict(offsets=torch.zeros(2)), TypeError, "offsets must be"),
                           (dict(offsets=torch.zeros(3, dtype=torch.int32)), ValueError, "offsets has shape"),
                           (dict(activation="tanh"), ValueError, "activation must be one of"),
                           (dict(activation="swiglu", w=torch.zeros(1, 64, 33, dtype=BF)), ValueError, "must be even"),
                           (dict(activation="swiglu", residual=torch.zeros(4, 32)), ValueError, "residual has shape"),
                           (dict(residual=torch.zeros(4, 32, dtype=F64)), TypeError, "residual must be"),
                           (dict(out_dtype=F64), TypeError, "out_dtype must be"),
                           (dict(out=torch.zeros(4, 32, dtype=F64)), TypeError, "out_dtype must be"),
                           (dict(out=torch.zeros(4, 32), out_dtype=BF), TypeError, "out must be"),
                           (dict(out=torch.zeros(5, 32)), ValueError, "out has shape"),
                           (dict(), ValueError, "must live on a GPU")):
        p = dict(a=a, w=w)
        p.update(kw)
        with pytest.raises(exc, match=match):
            M.moe_gemm(p.pop("a"), p.pop("w"), **p)


def test_gemm_sizes_past_31_bits_are_refused():
    big = torch.empty(2 ** 32 + 16, 16, dtype=BF, device="meta")
    with pytest.raises(ValueError, match="at most 2\\^31 - 1"):
        M.moe_gemm(big, torch.empty(1, 16, 16, dtype=BF, device="meta"))


def plan(swiglu, E_local, capacity, N, K, cus=256):
    fn = M.lib().moe_internal_gemm_plan
    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    ranges = ctypes.c_int(0)
    return TILES[fn(int(swiglu), E_local, capacity, N, K, cus, ctypes.byref(ranges))], ranges.value


def test_plan():
    """Every kind of tile is some size's, k is cut into whole ranges where tiles are few, and the
    sums of the ranges stay small."""
    assert plan(False, 1, 1, 4096, 7168) == ("tall", 8)
    assert plan(False, 1, 1, 7168, 256) == ("small", 1)
    assert plan(False, 1, 1024, 4096, 7168) == ("mid", 1)
    assert plan(True, 1, 2048, 2048, 7168) == ("tall", 1)
    assert plan(True, 1, 8192, 2048, 7168) == ("big", 1)
    assert plan(True, 32, 256, 2048, 7168) == ("few", 1)
    assert plan(False, 1, 512, 512, 2048) == ("small", 4)
    for E_local, capacity, N, K in ((1, 1, 8, 8), (1, 1, 8, (1 << 20) - 8), (1, 2 ** 31 - 2000, 8, 8), (1024, 1, 8, 8),
                                    (1024, 3, 1032, 1032), (7, 2, 16, 7168), (1, 300, 256, 65536), (300, 300, 256, 2048),
                                    (1, 128, 128, 520192)):
        for swiglu in (False, True):
            tile, ranges = plan(swiglu, E_local, capacity, N, K)
            assert 1 <= ranges <= max(1, -(-K // 64) // 2) and (ranges == 1 or tile != "big")
            nbytes = M.gemm_workspace_size(capacity, N, K, E_local, "swiglu" if swiglu else "none")
            assert nbytes == (0 if ranges == 1 else 4 * ranges * capacity * N * (2 if swiglu else 1))
            assert nbytes <= 64 << 20
    assert M.gemm_workspace_size(4, 12, 8) == 0  # (a size that the call refuses)


# --------------------------------------------------------------------------- #
# One matrix                                                                   #
# --------------------------------------------------------------------------- #
ROWS = [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 100, 128, 129, 200, 289, 600]
# ends of k: below a stage of 64, in its middle, on it, past it by one vector
DEPTHS = [8, 40, 64, 72, 128, 200, 520, 1032]
COLS = [8, 24, 32, 40, 64, 72, 136, 256, 264, 520]


@gpu
@pytest.mark.parametrize("i", range(len(ROWS)))
def test_every_edge_of_a_tile(i):
    for j, K in enumerate(DEPTHS):
        for N in (COLS[(i + j) % len(COLS)], COLS[(i + 3 * j + 5) % len(COLS)]):
            run(ROWS[i], K, N, integers=True, out=F32 if j % 2 else BF, seed=i + 31 * j)
            run(ROWS[i], K, N, act="swiglu", bias=True, integers=False, seed=i + 31 * j)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
def test_epilogues(act, res, out):
    for Mr, K, N in ((3, 136, 40), (20, 72, 88), (77, 128, 264), (300, 200, 520)):
        run(Mr, K, N, act=act, bias=True, res=res, out=out, seed=Mr)
        run(Mr, K, N, act=act, bias=False, res=res, out=out, integers=True, seed=Mr + 1)


# shapes of the layers this library knows, thinned out, and long k with few tiles
@gpu
@pytest.mark.parametrize("Mr,K,N", [(1, 7168, 256), (1, 2048, 7168), (16, 7168, 512), (32, 2880, 1536), (64, 7168, 256),
                                    (100, 7168, 520), (128, 4096, 1024), (256, 2880, 2880), (512, 7168, 512),
                                    (520, 1032, 3080), (1000, 2048, 1024), (1500, 2880, 1536), (2100, 2056, 2056),
                                    (2304, 512, 4096), (4097, 256, 2880), (8192, 264, 2048)])
def test_sizes_of_layers(Mr, K, N):
    run(Mr, K, N, integers=True, res=BF, out=F32, seed=N)
    run(Mr, K, N, act="swiglu", bias=True, res=F32, seed=K)
    run(Mr, K, N, act="silu", bias=True, seed=K + 1)


@gpu
@pytest.mark.parametrize("tile,ranges", [(t, r) for t in TILES for r in (1, 2, 3, 16) if t != "big" or r == 1])
def test_every_tile(tile, ranges):
    """Each kind of tile at sizes that the rule may give to another one: rows and columns past and
    inside a block, every end of k, more ranges than stages, several rounds of the grid."""
    for i, (Mr, K, N) in enumerate(((1, 8, 8), (5, 64, 32), (16, 72, 40), (33, 136, 72), (70, 584, 136), (130, 1032, 264),
                                    (300, 328, 520), (577, 2056, 1032))):
        run(Mr, K, N, bias=True, res=(None, BF, F32)[i % 3], out=(BF, F32)[i % 2], integers=True, seed=i, tile=tile, ranges=ranges)
        run(Mr, K, N, act="swiglu", bias=True, res=(F32, None, BF)[i % 3], out=(BF, F32)[i % 2], seed=i, tile=tile, ranges=ranges)
        run(Mr, K, N, act="gelu", bias=True, res=BF, seed=i, tile=tile, ranges=ranges)
    lens = [40, 0, 3, 100, 0, 333, 7, 1]
    off = [sum(lens[:i]) for i in range(len(lens) + 1)]
    run(off[-1] + 9, 328, 264, bias=True, res=F32, El=8, offsets=off, integers=True, tile=tile, ranges=ranges)
    run(off[-1], 128, 264, act="swiglu", bias=True, El=8, offsets=off, tile=tile, ranges=ranges)
    run(6000, 72, 2056, integers=True, tile=tile, ranges=ranges)


@gpu
@pytest.mark.parametrize("Mr,K,N", [(3826, 72, 14592), (3350, 136, 11000), (6918, 8, 11736), (5125, 64, 12504), (2901, 264, 12544)])
def test_last_round_in_halves(Mr, K, N):
    """Largest tiles, some left for the last round of a grid of 256: those go in halves, the last
    block of 6 to 242 rows among them."""
    run(Mr, K, N, bias=True, res=BF, integers=True, tile="big")
    run(Mr, K, N // 16 * 8, act="swiglu", res=F32, seed=1, tile="big")


# --------------------------------------------------------------------------- #
# Segments                                                                     #
# --------------------------------------------------------------------------- #
@gpu
@pytest.mark.parametrize("lens", [[0, 0, 0], [1], [0, 5, 0, 0, 17, 1], [16, 16, 16, 16], [40, 0, 3, 100, 0, 33, 7, 1],
                                  [300, 290, 0, 5], [1] * 70, [0] * 300 + [9] + [0] * 20 + [64], [700, 20, 600, 650, 1, 2]])
def test_segments(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    for K, N, act in ((64, 72, "none"), (136, 264, "swiglu"), (520, 40, "gelu")):
        # more rows in the buffers than the segments hold: they are left as they are
        run(off[-1] + 13, K, N, act=act, bias=True, res=BF, El=len(lens), offsets=off, integers=act == "none", seed=K)
    run(off[-1] or 1, 256, 512, act="swiglu", El=len(lens), offsets=off, seed=5)


@gpu
def test_device_offsets_out_of_range():
    """Offsets that start past 0, end past the buffers or step back: clamped, rows outside untouched."""
    for off in ([3, 10, 25], [0, 10, 99], [0, 30, 20], [-5, 10, 40], [50, 60, 70], [7, 7, 7]):
        run(40, 72, 40, act="none", bias=True, El=2, offsets=off, integers=True)
        run(40, 128, 264, act="swiglu", bias=True, El=2, offsets=off)


@gpu
@pytest.mark.parametrize("rows", [3, 40, 140, 300, 1000])
def test_segments_are_their_products_alone(rows):
    """A segment's rows by themselves, to float32 accuracy of any order."""
    dev = device()
    off = [0, rows, rows + 1, 2 * rows]
    a, w, b, r = inputs(2 * rows, 320, 264, "gelu", True, F32, 3, True, rows)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    whole = M.moe_gemm(a, w, b, o, activation="none", residual=r, out_dtype=F32)
    for e in range(3):
        s = slice(off[e], off[e + 1])
        assert torch.equal(whole[s], M.moe_gemm(a[s], w[e:e + 1], b[e:e + 1], residual=r[s].contiguous(), out_dtype=F32))


# --------------------------------------------------------------------------- #
# Non-finite values, repeats, streams, graphs, far offsets                     #
# --------------------------------------------------------------------------- #
@gpu
@pytest.mark.parametrize("Mr,K,N", [(5, 72, 40), (33, 200, 72), (70, 1032, 264), (300, 136, 520), (1200, 328, 1032)])
@pytest.mark.parametrize("act", ["none", "swiglu", "relu"])
def test_nonfinite_rows_touch_no_other(Mr, K, N, act):
    a, w, b, r = inputs(Mr, K, N, act, True, F32, 1, True, 3)
    clean = M.moe_gemm(a, w, b, activation=act, residual=r, out_dtype=F32)
    dirty = a.clone()
    rows = sorted({0, Mr // 2, Mr - 1})
    dirty[rows[0], K - 1] = math.inf
    dirty[rows[1], 0] = math.nan
    dirty[rows[-1], K // 2] = -math.inf
    say(f"nonfinite {Mr} {K} {N} {act}")
    got = M.moe_gemm(dirty, w, b, activation=act, residual=r, out_dtype=F32)
    keep = torch.ones(Mr, dtype=torch.bool, device=a.device)
    keep[rows] = False
    assert torch.equal(got[keep], clean[keep])
    z = dirty[rows].double() @ w[0].double() + b[0].double()
    v = torch.relu(z) if act == "relu" else z if act == "none" else torch.nn.functional.silu(z[:, :N]) * z[:, N:]
    v = v + r[rows].double()
    assert torch.equal(torch.isnan(got[rows]), torch.isnan(v))
    assert torch.equal(torch.isposinf(got[rows]), torch.isposinf(v))
    assert torch.equal(torch.isneginf(got[rows]), torch.isneginf(v))


@gpu
@pytest.mark.parametrize("Mr,K,N", [(3, 1032, 40), (64, 200, 264), (300, 200, 520)])
def test_infinite_weights_stay_in_their_column(Mr, K, N):
    """An infinity in the last k rows is one product's, not the padding's."""
    a, w, _, _ = inputs(Mr, K, N, "none", False, None, 2, True, 4)
    a = torch.where(a == 0, torch.ones_like(a), a)
    w[0, K - 1, 5], w[0, K - 3, 7], w[1, 0, 2] = math.inf, -math.inf, math.inf
    o = torch.tensor([0, Mr - 1, Mr], dtype=torch.int32, device=a.device)
    got = M.moe_gemm(a, w, None, o, out_dtype=F32)
    v = torch.cat([a[:-1].double() @ w[0].double(), a[-1:].double() @ w[1].double()])
    assert torch.equal(torch.isnan(got), torch.isnan(v)) and not torch.isnan(v).any()
    assert torch.equal(got.double(), v)


@gpu
@pytest.mark.parametrize("Mr,K,N", [(4, 7168, 512), (200, 1032, 520), (2000, 520, 1032)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_streams_and_repeats(Mr, K, N, dtype):
    a, w, b, r = inputs(Mr, K, N, "silu", True, dtype, 1, False, 7)
    want = M.moe_gemm(a, w, b, activation="silu", residual=r, out_dtype=dtype)
    assert torch.equal(want, M.moe_gemm(a, w, b, activation="silu", residual=r, out_dtype=dtype))
    side = torch.cuda.Stream(device=a.device)
    side.wait_stream(torch.cuda.current_stream(a.device))
    got = M.moe_gemm(a, w, b, activation="silu", residual=r, out_dtype=dtype, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    M.moe_gemm(a, w, b, activation="silu", residual=r, out=r)
    assert torch.equal(r, want)


@gpu
@pytest.mark.parametrize("Mr,K,N,El", [(3, 1032, 40, 1), (200, 520, 520, 3), (700, 256, 264, 2)])
def test_graph_replays(Mr, K, N, El):
    a, w, b, r = inputs(Mr, K, N, "swiglu", True, BF, El, False, 8)
    off = torch.tensor([Mr * e // El for e in range(El + 1)], dtype=torch.int32, device=a.device)
    M.moe_gemm(a, w, b, off, activation="swiglu", residual=r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.moe_gemm(a, w, b, off, activation="swiglu", residual=r)
    for rep in range(3):
        a.copy_(torch.randn(Mr, K, device=a.device))
        want = M.moe_gemm(a, w, b, off, activation="swiglu", residual=r)
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


@gpu
@pytest.mark.parametrize("Mr,K,N", [(300000, 8, 8192), (620000, 4096, 8)])
def test_rows_past_32_bit_offsets(Mr, K, N):
    a, w, _, _ = inputs(Mr, K, N, "none", False, None, 1, True, 9)
    say(f"far rows {Mr} {K} {N}")
    got = M.moe_gemm(a, w)
    for s in (slice(0, 50), slice(Mr // 2, Mr // 2 + 300), slice(Mr - 300, Mr)):
        assert torch.equal(got[s], (a[s].double() @ w[0].double()).to(BF))


@gpu
def test_workspaces():
    """A given workspace of any content, too small ones refused, two calls on two streams with their own."""
    dev = device()
    a, w, _, _ = inputs(2, 7168, 512, "none", False, None, 1, True, 11)
    n = M.gemm_workspace_size(2, 512, 7168)
    assert n > 0
    want = (a.double() @ w[0].double()).to(BF)
    ws = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(2)]
    with pytest.raises(ValueError, match="workspace holds"):
        M.moe_gemm(a, w, workspace=ws[0][:-256])
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    for _ in range(20):
        got = [M.moe_gemm(a, w, workspace=ws[0]), M.moe_gemm(a, w, workspace=ws[1], stream=side)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)


@gpu
def test_no_rows():
    dev = device()
    out = M.moe_gemm(torch.zeros(0, 64, dtype=BF, device=dev), torch.zeros(1, 64, 32, dtype=BF, device=dev))
    assert out.shape == (0, 32)
