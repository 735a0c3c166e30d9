"""ctypes binding of ``libmoe.so`` (the C-ABI declared in include/moe.h); the
small calls go through the extension module ``_calls.so`` (csrc/calls.cpp).

Argument marshalling only: every step of the MoE share runs in the library's
HIP kernels. PyTorch provides device memory and the current stream. There is
no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import numbers
import pathlib
import sys
from ctypes import c_float, c_int, c_int64, c_size_t, c_void_p

LIB_PATH = pathlib.Path(__file__).resolve().parent / "libmoe.so"

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_HIP = -4

# symbol -> (restype, argtypes)
_P = c_void_p
SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [c_int]),
    "moe_route_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int]),
    "moe_route": (c_int, [_P, _P, _P, c_int, c_int, c_int, c_int, c_int, _P, _P, _P, _P, c_size_t, _P]),
    "moe_dispatch_workspace_size": (c_size_t, [c_int, c_int, c_int]),
    "moe_dispatch": (c_int, [_P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int64,
                             _P, _P, _P, _P, _P, _P, c_size_t, _P]),
    "moe_expert_ffn": (c_int, [_P, _P, _P, _P, c_int, c_int, c_int, c_int64, _P, _P, _P]),
    "moe_combine": (c_int, [_P, _P, _P, c_int, c_int, c_int, _P, _P]),
    "moe_combine_f32": (c_int, [_P, _P, _P, c_int, c_int, c_int, _P, _P]),
    "moe_forward_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int]),
    "moe_forward_workspace_layout": (c_int, [c_int, c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(c_size_t)]),
    "moe_forward": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                            _P, _P, c_size_t, _P]),
    "moe_forward_f32": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                _P, _P, c_size_t, _P]),
    "moe_forward_profiled": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                     _P, _P, c_size_t, _P, _P]),
    "moe_forward_fused": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                  _P, _P, c_size_t, _P]),
    "moe_forward_fused_profiled": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                           c_int, _P, _P, c_size_t, _P, _P]),
    "moe_forward_noalloc": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                    _P, _P]),
    "moe_few_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int]),
    "moe_forward_few": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                _P, _P, c_size_t, _P]),
    "moe_forward_few_f32": (c_int, [_P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                    _P, _P, c_size_t, _P]),
    "moe_quantize_rows": (c_int, [_P, c_int64, c_int, _P, _P, _P]),
    "moe_quantize_weights": (c_int, [_P, c_int, c_int, c_int, _P, _P, _P]),
    "moe_gemm_i8": (c_int, [_P, _P, _P, _P, _P, c_int64, c_int, c_int, c_int, _P, _P]),
    "moe_expert_ffn_i8_workspace_size": (c_size_t, [c_int, c_int, c_int64]),
    "moe_expert_ffn_i8": (c_int, [_P, _P, _P, _P, _P, _P, c_int, c_int, c_int, c_int64, _P, _P, c_size_t, _P]),
    "moe_forward_i8_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int]),
    "moe_forward_i8": (c_int, [_P, _P, _P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                               _P, _P, c_size_t, _P]),
    "moe_block_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
    "moe_block_forward": (c_int, [_P, c_int, _P, _P, _P, _P, _P, _P, _P, c_int, c_float, _P, c_float, c_int, c_int,
                                  c_int, c_int, c_int, c_int, _P, _P, _P, c_size_t, _P]),
    "moe_select": (c_int, [_P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float, _P, _P, _P]),
    "moe_route_scored": (c_int, [_P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_float,
                                 _P, _P, _P, _P, c_size_t, _P]),
    "moe_gemm_workspace_size": (c_size_t, [c_int64, c_int, c_int, c_int, c_int]),
    "moe_gemm": (c_int, [_P, _P, _P, _P, c_int, _P, c_int64, c_int, c_int, c_int, c_int, _P, c_int, _P, c_size_t, _P]),
    "moe_layer_workspace_size": (c_size_t, [c_int, c_int, c_int, c_int, c_int, c_int, c_int]),
    "moe_layer_forward": (c_int, [_P, _P, _P, _P, _P, _P, _P, _P, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                  c_int, c_int, c_int, c_int, c_int, c_float, _P, c_int, _P, c_size_t, _P]),
    "moe_norm_pre": (c_int, [_P, c_int, _P, c_float, c_int, c_int, _P, _P]),
    "moe_norm_post": (c_int, [_P, c_int, _P, c_int, _P, _P, c_int, c_float, _P, c_float, c_int, c_int, _P, _P, _P]),
}

# most tokens of moe_forward_few (MOE_FEW_TOKENS)
FEW_TOKENS = 32
# bytes of the static scratch moe_forward_noalloc works in (MOE_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 128 << 20

_lib = None


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m expert_token_routing_amd.build_lib`; there is no fallback path")
        h = ctypes.CDLL(str(LIB_PATH))
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


_calls_module = None


def torch_identity() -> str:
    """The torch and the interpreter that _calls.so has to be built for: it uses
    torch's C++ ABI and both's object layouts."""
    torch = _torch()
    return f"torch {torch.__version__} {torch.version.git_version} {sys.implementation.cache_tag}"


def _calls():
    """The extension module behind the small calls (csrc/calls.cpp), which
    calls the library loaded here."""
    global _calls_module
    if _calls_module is None:
        L = lib()
        _torch()  # its libraries first
        how = "build it with `python -m expert_token_routing_amd.build_lib`; there is no fallback path"
        try:
            from . import _calls as module
        except ImportError as e:
            raise RuntimeError(f"_calls.so is missing or was built for another torch: {how}") from e
        built_for = getattr(module, "built_for", "an unnamed torch")
        if built_for != torch_identity():
            raise RuntimeError(f"_calls.so was built for {built_for}, this is {torch_identity()}: {how}")
        module.bind(*(ctypes.cast(getattr(L, n), c_void_p).value
                      for n in ("moe_norm_pre", "moe_norm_post", "moe_quantize_rows", "moe_gemm_i8",
                                "moe_expert_ffn_i8_workspace_size", "moe_expert_ffn_i8", "moe_few_workspace_size",
                                "moe_forward_few", "moe_forward_few_f32", "moe_select", "moe_gemm_workspace_size",
                                "moe_gemm")))
        _calls_module = module
    return _calls_module


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoEError(status, where)


# --------------------------------------------------------------------------- #
# torch-facing wrappers                                                        #
# --------------------------------------------------------------------------- #
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    # the handle itself: building the torch.cuda.Stream around it takes 3 us
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _need(t, dtype, name, shape=None, dev=None, min_rows=False):
    """``t`` must be a ``dtype`` tensor of ``shape`` (None entries: any size;
    with ``min_rows`` the first dimension may also be larger). The library
    sees only pointers, so a wrong size would otherwise become an
    out-of-bounds access on the GPU. Contiguity and device are checked
    afterwards by _placed, once every shape has been checked, so that a
    mismatch is reported as one whatever the tensors' device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        got = tuple(t.shape)
        ok = len(got) == len(shape)
        if ok:
            for i, want in enumerate(shape):
                if want is not None and got[i] != want and not (min_rows and i == 0 and got[i] >= want):
                    ok = False
                    break
        if not ok:
            want_s = "(" + ", ".join("*" if v is None else (f">={v}" if min_rows and i == 0 else str(v))
                                     for i, v in enumerate(shape)) + ")"
            raise ValueError(f"{name} has shape {got}, expected shape {want_s}")


def _placed(dev, **tensors):
    """Every given tensor (None: skipped) is contiguous and on the GPU dev."""
    index = dev.index
    for name, t in tensors.items():
        if t is None or (t.get_device() == index and t.is_contiguous() and t.is_cuda):
            continue
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not t.is_cuda:
            raise ValueError(f"{name} must live on a GPU (this library has no CPU path)")
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {dev}")


def _nbytes(t):
    return t.numel() * t.element_size()


def _workspace(nbytes, device, workspace, name="workspace"):
    torch = _torch()
    if workspace is None:
        return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if _nbytes(workspace) < nbytes:
        raise ValueError(f"{name} holds {_nbytes(workspace)} bytes, needs {nbytes}")
    if not workspace.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not workspace.is_cuda or workspace.device != device:
        raise ValueError(f"{name} must live on {device}")
    return workspace


def _out(t, shape, dtype, dev, name):
    """The caller's output tensor, checked, or a new one."""
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, dtype, name, shape, dev)
    _placed(dev, **{name: t})
    return t


def _check_k(k, E):
    if not isinstance(k, numbers.Integral) or k < 1 or k > E:
        raise ValueError(f"k must be an int in [1, E = {E}], got {k!r}")


def moe_route(x, w_router, bias, k, renormalize=True, *, logits=None, topk_idx=None, topk_w=None,
              workspace=None, stream=None):
    """Router logits [T,E] f32, top-k ids [T,k] i32 and combine weights [T,k] f32."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    T, H = x.shape
    dev = x.device
    _need(w_router, torch.float32, "w_router", (None, H), dev)
    E = w_router.shape[0]
    if bias is not None:
        _need(bias, torch.float32, "bias", (E,), dev)
    _check_k(k, E)
    for name, t, shp, dt in (("logits", logits, (T, E), torch.float32), ("topk_idx", topk_idx, (T, k), torch.int32),
                             ("topk_w", topk_w, (T, k), torch.float32)):
        if t is not None:
            _need(t, dt, name, shp)
    _placed(dev, x=x, w_router=w_router, bias=bias)
    logits = _out(logits, (T, E), torch.float32, dev, "logits")
    topk_idx = _out(topk_idx, (T, k), torch.int32, dev, "topk_idx")
    topk_w = _out(topk_w, (T, k), torch.float32, dev, "topk_w")
    L = lib()
    ws = _workspace(L.moe_route_workspace_size(T, H, E, k), dev, workspace)
    st = L.moe_route(_ptr(x), _ptr(w_router), _ptr(bias), T, H, E, k, int(bool(renormalize)), _ptr(logits),
                     _ptr(topk_idx), _ptr(topk_w), _ptr(ws), _nbytes(ws), _stream(stream, dev))
    check(st, "moe_route")
    return logits, topk_idx, topk_w


def moe_dispatch(x, topk_idx, E, e0, E_local, *, capacity=None, counts=None, offsets=None, perm_src=None,
                 inv=None, x_perm=None, workspace=None, stream=None):
    """counts [E], offsets [E_local+1], perm_src [cap], inv [T*k], x_perm [cap,H]."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    T, H = x.shape
    dev = x.device
    _need(topk_idx, torch.int32, "topk_idx", (T, None), dev)
    k = topk_idx.shape[1]
    if not (0 <= e0 and E_local >= 1 and e0 + E_local <= E):
        raise ValueError(f"local experts [e0, e0 + E_local) = [{e0}, {e0 + E_local}) must lie in [0, E = {E})")
    _check_k(k, E)
    cap = T * min(k, E_local) if capacity is None else int(capacity)
    if cap < T * min(k, E_local):
        raise ValueError(f"capacity {cap} < T * min(k, E_local) = {T * min(k, E_local)}")
    for name, t, shp, dt, mr in (("counts", counts, (E,), torch.int32, False),
                                 ("offsets", offsets, (E_local + 1,), torch.int32, False),
                                 ("perm_src", perm_src, (max(cap, 1),), torch.int32, True),
                                 ("inv", inv, (max(T * k, 1),), torch.int32, True),
                                 ("x_perm", x_perm, (max(cap, 1), H), torch.bfloat16, True)):
        if t is not None:
            _need(t, dt, name, shp, min_rows=mr)
    _placed(dev, x=x, topk_idx=topk_idx)
    counts = _out(counts, (E,), torch.int32, dev, "counts")
    offsets = _out(offsets, (E_local + 1,), torch.int32, dev, "offsets")
    if perm_src is None:
        perm_src = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    else:
        _placed(dev, perm_src=perm_src)
    if inv is None:
        inv = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    else:
        _placed(dev, inv=inv)
    if x_perm is None:
        x_perm = torch.empty((max(cap, 1), H), dtype=torch.bfloat16, device=dev)
    else:
        _placed(dev, x_perm=x_perm)
    L = lib()
    ws = _workspace(L.moe_dispatch_workspace_size(T, E, k), dev, workspace)
    st = L.moe_dispatch(_ptr(x), _ptr(topk_idx), T, H, E, k, e0, E_local, cap, _ptr(counts), _ptr(offsets),
                        _ptr(perm_src), _ptr(inv), _ptr(x_perm), _ptr(ws), _nbytes(ws), _stream(stream, dev))
    check(st, "moe_dispatch")
    return counts, offsets, perm_src, inv, x_perm


def moe_expert_ffn(x_perm, offsets, w_gate_up, w_down, *, h=None, out=None, stream=None):
    """h [cap, I] and expert outputs [cap, H] for the segments in ``offsets``."""
    torch = _torch()
    _need(x_perm, torch.bfloat16, "x_perm", (None, None))
    cap, H = x_perm.shape
    dev = x_perm.device
    _need(w_gate_up, torch.bfloat16, "w_gate_up", (None, H, None), dev)
    E_local, _, I2 = w_gate_up.shape
    if I2 % 2:
        raise ValueError(f"w_gate_up's last dimension 2I must be even, got {I2}")
    I = I2 // 2
    _need(w_down, torch.bfloat16, "w_down", (E_local, I, H), dev)
    _need(offsets, torch.int32, "offsets", (E_local + 1,), dev)
    if h is not None:
        _need(h, torch.bfloat16, "h", (cap, I))
    if out is not None:
        _need(out, torch.bfloat16, "out", (cap, H))
    _placed(dev, x_perm=x_perm, offsets=offsets, w_gate_up=w_gate_up, w_down=w_down)
    h = _out(h, (cap, I), torch.bfloat16, dev, "h")
    out = _out(out, (cap, H), torch.bfloat16, dev, "out")
    st = lib().moe_expert_ffn(_ptr(x_perm), _ptr(offsets), _ptr(w_gate_up), _ptr(w_down), H, I, E_local, cap,
                              _ptr(h), _ptr(out), _stream(stream, dev))
    check(st, "moe_expert_ffn")
    return h, out


def _combine(name, out_dtype, expert_out, inv, topk_w, y, stream):
    torch = _torch()
    _need(topk_w, torch.float32, "topk_w", (None, None))
    T, k = topk_w.shape
    dev = topk_w.device
    _need(expert_out, torch.bfloat16, "expert_out", (None, None), dev)
    H = expert_out.shape[1]
    if inv.dim() != 1:
        raise ValueError(f"inv has shape {tuple(inv.shape)}, expected shape ({T * k},)")
    _need(inv, torch.int32, "inv", (T * k,), dev)
    if y is not None:
        _need(y, out_dtype, "y", (T, H))
    _placed(dev, expert_out=expert_out, inv=inv, topk_w=topk_w)
    y = _out(y, (T, H), out_dtype, dev, "y")
    st = getattr(lib(), name)(_ptr(expert_out), _ptr(inv), _ptr(topk_w), T, H, k, _ptr(y), _stream(stream, dev))
    check(st, name)
    return y


def moe_combine(expert_out, inv, topk_w, *, y=None, stream=None):
    """y [T, H] bf16: weighted sum of each token's local expert outputs.
    Every inv entry that is not -1 must be a row of expert_out (the library
    cannot check device values)."""
    return _combine("moe_combine", _torch().bfloat16, expert_out, inv, topk_w, y, stream)


def moe_combine_f32(expert_out, inv, topk_w, *, y=None, stream=None):
    """y [T, H] float32: moe_combine's sums before their rounding to bf16."""
    return _combine("moe_combine_f32", _torch().float32, expert_out, inv, topk_w, y, stream)


def forward_workspace_size(T, H, I, E, k, E_local) -> int:
    return int(lib().moe_forward_workspace_size(T, H, I, E, k, E_local))


def forward_workspace_layout(T, H, I, E, k, E_local) -> dict:
    arr = (c_size_t * 9)()
    check(lib().moe_forward_workspace_layout(T, H, I, E, k, E_local, arr), "moe_forward_workspace_layout")
    names = ["logits", "topk_idx", "topk_w", "counts", "offsets", "perm_src", "inv", "x_perm", "expert_out"]
    return dict(zip(names, [int(v) for v in arr]))


def _forward_args(x, w_router, bias, w_gate_up, w_down, k, e0):
    """Checks the forward's inputs; returns (T, H, I, E, E_local, device)."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    T, H = x.shape
    dev = x.device
    _need(w_router, torch.float32, "w_router", (None, H), dev)
    E = w_router.shape[0]
    if bias is not None:
        _need(bias, torch.float32, "bias", (E,), dev)
    _need(w_gate_up, torch.bfloat16, "w_gate_up", (None, H, None), dev)
    E_local, _, I2 = w_gate_up.shape
    if I2 % 2:
        raise ValueError(f"w_gate_up's last dimension 2I must be even, got {I2}")
    I = I2 // 2
    _need(w_down, torch.bfloat16, "w_down", (E_local, I, H), dev)
    _check_k(k, E)
    if not (0 <= e0 and e0 + E_local <= E):
        raise ValueError(f"local experts [e0, e0 + E_local) = [{e0}, {e0 + E_local}) must lie in [0, E = {E})")
    return T, H, I, E, E_local, dev


def _forward_placed(dev, x, w_router, bias, w_gate_up, w_down):
    _placed(dev, x=x, w_router=w_router, bias=bias, w_gate_up=w_gate_up, w_down=w_down)


def _forward(name, out_dtype, x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y, workspace, stream):
    T, H, I, E, E_local, dev = _forward_args(x, w_router, bias, w_gate_up, w_down, k, e0)
    if y is not None:
        _need(y, out_dtype, "y", (T, H))
    _forward_placed(dev, x, w_router, bias, w_gate_up, w_down)
    y = _out(y, (T, H), out_dtype, dev, "y")
    ws = _workspace(forward_workspace_size(T, H, I, E, k, E_local), dev, workspace)
    st = getattr(lib(), name)(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up), _ptr(w_down), T, H, I, E, k,
                              e0, E_local, int(bool(renormalize)), _ptr(y), _ptr(ws), _nbytes(ws),
                              _stream(stream, dev))
    check(st, name)
    return y, ws


def moe_forward(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize=True, *, y=None, workspace=None,
                stream=None):
    """The rank's share of the MoE layer: y [T, H] bf16. ``E_local`` is
    ``w_gate_up.shape[0]``; the rank owns experts [e0, e0 + E_local)."""
    return _forward("moe_forward", _torch().bfloat16, x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y,
                    workspace, stream)


def moe_forward_f32(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize=True, *, y=None, workspace=None,
                    stream=None):
    """moe_forward with the share kept in float32 (y [T, H] float32), for
    summing the shares of several ranks before one rounding."""
    return _forward("moe_forward_f32", _torch().float32, x, w_router, bias, w_gate_up, w_down, k, e0, renormalize,
                    y, workspace, stream)


def moe_forward_fused(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize=True, *, y=None, workspace=None,
                      stream=None):
    """moe_forward with the combine of tokens that have exactly one local
    selection done in the down GEMM's epilogue; y equals moe_forward's."""
    return _forward("moe_forward_fused", _torch().bfloat16, x, w_router, bias, w_gate_up, w_down, k, e0,
                    renormalize, y, workspace, stream)


def moe_forward_profiled(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y, workspace, events,
                         stream=None, fused=False):
    """moe_forward (moe_forward_fused with ``fused``) into preallocated ``y`` /
    ``workspace``, recording the six torch.cuda.Event objects in ``events``
    (already recorded once, so they exist) around the router, dispatch,
    gate/up GEMM, down GEMM and combine."""
    torch = _torch()
    T, H, I, E, E_local, dev = _forward_args(x, w_router, bias, w_gate_up, w_down, k, e0)
    _need(y, torch.bfloat16, "y", (T, H))
    if workspace is None:
        raise ValueError("workspace is required")
    if len(events) != 6:
        raise ValueError(f"events must hold 6 events, got {len(events)}")
    _forward_placed(dev, x, w_router, bias, w_gate_up, w_down)
    _placed(dev, y=y)
    ws = _workspace(forward_workspace_size(T, H, I, E, k, E_local), dev, workspace)
    arr = (c_void_p * 6)(*[c_void_p(ev.cuda_event) for ev in events])
    name = "moe_forward_fused_profiled" if fused else "moe_forward_profiled"
    st = getattr(lib(), name)(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up), _ptr(w_down), T, H, I, E, k, e0,
                              E_local, int(bool(renormalize)), _ptr(y), _ptr(ws), _nbytes(ws), arr,
                              _stream(stream, dev))
    check(st, name)


def moe_forward_noalloc(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize=True, *, y, stream=None):
    """moe_forward with the intermediates in the library's static scratch
    (no workspace; the call allocates nothing on the device). ``y`` [T, H]
    bf16 is the caller's. Raises MoEError(MOE_ERR_WORKSPACE) when the problem
    needs more than NOALLOC_SCRATCH_BYTES."""
    torch = _torch()
    T, H, I, E, E_local, dev = _forward_args(x, w_router, bias, w_gate_up, w_down, k, e0)
    _need(y, torch.bfloat16, "y", (T, H))
    _forward_placed(dev, x, w_router, bias, w_gate_up, w_down)
    _placed(dev, y=y)
    st = lib().moe_forward_noalloc(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up), _ptr(w_down), T, H, I, E, k,
                                   e0, E_local, int(bool(renormalize)), _ptr(y), _stream(stream, dev))
    check(st, "moe_forward_noalloc")
    return y


@contextlib.contextmanager
def _current(first, stream):
    """``first``'s device, and ``stream`` where the caller gave one, as the
    current ones: what the call allocates then belongs to the stream its kernels
    run on, so the memory cannot be handed to them while another stream still
    uses it."""
    torch = _torch()
    if stream is not None and stream.device.index != first.get_device():
        raise ValueError(f"stream is on {stream.device}, the call's tensors on {first.device}")
    with torch.cuda.device(first.get_device()) if stream is None else torch.cuda.stream(stream):
        yield


def _on_stream(fn):
    """Runs ``fn`` with the device of its first tensor current and, where the
    caller gave a ``stream``, with that stream current."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        torch = _torch()
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            return fn(*args, **kw)  # refused by fn's checks
        if stream is not None or first.get_device() != torch._C._cuda_getDevice():
            with _current(first, stream):
                return fn(*args, **kw)
        return fn(*args, **kw)
    return call


def _small_call(name, args, stream, refuse):
    """The call ``name`` of the extension module. Where it does not take the
    arguments as they are, ``refuse`` says what is wrong with them, or their
    device or stream is made current first."""
    fn = getattr(_calls(), name)
    done = fn(*args) if stream is None else None
    if done is None:
        refuse()
        with _current(args[0], stream):
            done = fn(*args)
        if done is None:
            raise TypeError(f"moe_{name} does not take these tensors")
    if done.__class__ is int:
        check(done, "moe_" + name)
    return done


# --------------------------------------------------------------------------- #
# Norms before and after the block                                             #
# --------------------------------------------------------------------------- #
# element types and gate shapes (MOE_TYPE_*, MOE_GATE_*)
TYPE_BF16, TYPE_F32 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


def _need_either(t, name, shape):
    """``t`` must be a bf16 or float32 tensor of ``shape``; returns its MOE_TYPE."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = t.dtype
    kind = TYPE_BF16 if dtype == torch.bfloat16 else TYPE_F32 if dtype == torch.float32 else -1
    if kind < 0:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {dtype}")
    _need(t, dtype, name, shape)
    return kind


def _ints(*sizes):
    """Sizes that the library takes as int: ctypes would pass on a larger one's
    low 32 bits."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"sizes are at most 2^31 - 1, got {max(sizes)}")


def _plain_int(n):
    """An integer of another type (numpy's) as int; anything else as it is."""
    return n if type(n) is int else int(n) if isinstance(n, numbers.Integral) else n


def _gate_kind(gate, T, H):
    """The MOE_GATE of a float32 gate by its shape: [H], [T, 1] or [T, H]."""
    torch = _torch()
    if gate is None:
        return GATE_NONE
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    got = tuple(gate.shape)
    if got == (T, 1):
        kind = GATE_TOKEN
    elif got == (H,):
        kind = GATE_CHANNEL
    elif got == (T, H):
        kind = GATE_FULL
    else:
        raise ValueError(f"gate has shape {got}, expected shape ({H},), ({T}, 1) or ({T}, {H})")
    _need(gate, torch.float32, "gate")
    return kind


def moe_norm_pre(r, w, eps=1e-6, *, out=None, stream=None):
    """The norm before the block: out [T, H] bf16 = r / sqrt(mean(r^2) + eps) * w.
    ``r`` [T, H] is bf16 or float32, ``w`` [H] float32."""
    def refuse():
        torch = _torch()
        _need_either(r, "r", (None, None))
        T, H = r.shape
        _need(w, torch.float32, "w", (H,))
        if out is not None:
            _need(out, torch.bfloat16, "out", (T, H))
        _ints(T, H)
        _placed(r.device, r=r, w=w, out=out)
    return _small_call("norm_pre", (r, w, eps, out), stream, refuse)


def moe_norm_post(y, residual, w_post=None, *, gate=None, residual_scale=1.0, w_next=None, eps=1e-6, out=None,
                  normed=None, stream=None):
    """out = residual_scale * residual + gate * norm(y; w_post), of the
    residual's type, and with ``w_next`` also normed [T, H] bf16 =
    norm(out before its rounding; w_next). Returns (out, normed or None).

    ``y`` and ``residual`` [T, H] are bf16 or float32; ``w_post`` and
    ``w_next`` [H] float32 (``w_post`` None: y as it is). ``gate`` float32 is
    [H] (per channel), [T, 1] (per token) or [T, H]. ``out`` may be
    ``residual``."""
    def refuse():
        torch = _torch()
        _need_either(y, "y", (None, None))
        T, H = y.shape
        _need_either(residual, "residual", (T, H))
        if w_post is not None:
            _need(w_post, torch.float32, "w_post", (H,))
        _gate_kind(gate, T, H)
        if w_next is not None:
            _need(w_next, torch.float32, "w_next", (H,))
        elif normed is not None:
            raise ValueError("normed is given without w_next")
        if out is not None:
            _need(out, residual.dtype, "out", (T, H))
        if normed is not None:
            _need(normed, torch.bfloat16, "normed", (T, H))
        _ints(T, H)
        _placed(y.device, y=y, residual=residual, w_post=w_post, gate=gate, w_next=w_next, out=out, normed=normed)
    return _small_call("norm_post", (y, residual, w_post, gate, residual_scale, w_next, eps, out, normed), stream, refuse)


# --------------------------------------------------------------------------- #
# The whole share for a few tokens                                             #
# --------------------------------------------------------------------------- #
def few_workspace_size(T, H, I, E, k, E_local) -> int:
    """Bytes of workspace moe_forward_few needs (0 where T > FEW_TOKENS)."""
    return int(lib().moe_few_workspace_size(T, H, I, E, k, E_local))


def _few(name, out_dtype, x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y, workspace, stream):
    def refuse():
        T, H, I, E, E_local, dev = _forward_args(x, w_router, bias, w_gate_up, w_down, k, e0)
        if y is not None:
            _need(y, out_dtype, "y", (T, H))
        _ints(T, H, E, I)
        _placed(dev, x=x, w_router=w_router, bias=bias, w_gate_up=w_gate_up, w_down=w_down, y=y)
        if workspace is not None:
            _workspace(lib().moe_few_workspace_size(T, H, I, E, k, E_local), dev, workspace)
    return _small_call(name, (x, w_router, bias, w_gate_up, w_down, _plain_int(k), _plain_int(e0), renormalize, y,
                              workspace), stream, refuse)


def moe_forward_few(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize=True, *, y=None, workspace=None,
                    stream=None):
    """moe_forward for at most FEW_TOKENS tokens in two kernels: y [T, H] bf16,
    rounded once. Returns (y, workspace)."""
    return _few("forward_few", _torch().bfloat16, x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y,
                workspace, stream)


def moe_forward_few_f32(x, w_router, bias, w_gate_up, w_down, k, e0, renormalize=True, *, y=None, workspace=None,
                        stream=None):
    """moe_forward_few with the share kept in float32 (y [T, H] float32)."""
    return _few("forward_few_f32", _torch().float32, x, w_router, bias, w_gate_up, w_down, k, e0, renormalize, y,
                workspace, stream)


# --------------------------------------------------------------------------- #
# 8-bit integer products                                                       #
# --------------------------------------------------------------------------- #
def moe_quantize_rows(x, *, q=None, scale=None, stream=None):
    """q [M, K] int8 and scale [M] float32 of x [M, K] bf16: scale = max|x| / 127
    per row, q = x / scale to the nearest integer."""
    def refuse():
        torch = _torch()
        _need(x, torch.bfloat16, "x", (None, None))
        M, K = x.shape
        if q is not None:
            _need(q, torch.int8, "q", (M, K))
        if scale is not None:
            _need(scale, torch.float32, "scale", (M,))
        _ints(M, K)
        _placed(x.device, x=x, q=q, scale=scale)
    return _small_call("quantize_rows", (x, q, scale), stream, refuse)


@_on_stream
def moe_quantize_weights(w, *, q=None, scale=None):
    """q [E_local, N, K] int8 and scale [E_local, N] float32 of the weights w
    [E_local, K, N] bf16 (the layout of w_gate_up and w_down), a scale per
    output channel. Takes ``stream``."""
    torch = _torch()
    _need(w, torch.bfloat16, "w", (None, None, None))
    E_local, K, N = w.shape
    _ints(E_local, K, N)
    if q is not None:
        _need(q, torch.int8, "q", (E_local, N, K))
    if scale is not None:
        _need(scale, torch.float32, "scale", (E_local, N))
    dev = w.device
    _placed(dev, w=w)
    q = _out(q, (E_local, N, K), torch.int8, dev, "q")
    scale = _out(scale, (E_local, N), torch.float32, dev, "scale")
    st = lib().moe_quantize_weights(_ptr(w), E_local, K, N, _ptr(q), _ptr(scale), _stream(None, dev))
    check(st, "moe_quantize_weights")
    return q, scale


def moe_gemm_i8(a, a_scale, w, w_scale, offsets=None, *, out=None, stream=None):
    """out [M, N] bf16 = (a @ w[e].T) * a_scale[:, None] * w_scale[e] for the
    rows of segment e of ``offsets`` [E_local + 1] int32 (None: one weight
    matrix for all rows). a [M, K] and w [E_local, N, K] are int8, the scales
    [M] and [E_local, N] float32."""
    def refuse():
        torch = _torch()
        _need(a, torch.int8, "a", (None, None))
        M, K = a.shape
        _need(a_scale, torch.float32, "a_scale", (M,))
        _need(w, torch.int8, "w", (None, None, K))
        E_local, N, _ = w.shape
        _need(w_scale, torch.float32, "w_scale", (E_local, N))
        if offsets is not None:
            _need(offsets, torch.int32, "offsets", (E_local + 1,))
        elif E_local != 1:
            raise ValueError(f"w holds {E_local} matrices: offsets is required")
        if out is not None:
            _need(out, torch.bfloat16, "out", (M, N))
        _ints(M, K, E_local, N)
        _placed(a.device, a=a, a_scale=a_scale, w=w, w_scale=w_scale, offsets=offsets, out=out)
    return _small_call("gemm_i8", (a, a_scale, w, w_scale, offsets, out), stream, refuse)


def _need_ffn_i8(H, w_gate_up, s_gate_up, w_down, s_down):
    torch = _torch()
    _need(w_gate_up, torch.int8, "w_gate_up", (None, None, H))
    E_local, I2, _ = w_gate_up.shape
    if I2 % 2:
        raise ValueError(f"w_gate_up's second dimension 2I must be even, got {I2}")
    I = I2 // 2
    _need(s_gate_up, torch.float32, "s_gate_up", (E_local, I2))
    _need(w_down, torch.int8, "w_down", (E_local, H, I))
    _need(s_down, torch.float32, "s_down", (E_local, H))
    return E_local, I


def expert_ffn_i8_workspace_size(H, I, capacity) -> int:
    return int(lib().moe_expert_ffn_i8_workspace_size(H, I, capacity))


def moe_expert_ffn_i8(x_perm, offsets, w_gate_up, s_gate_up, w_down, s_down, *, out=None, workspace=None, stream=None):
    """moe_expert_ffn with 8-bit weights (moe_quantize_weights) and activations
    quantised per row: expert outputs [cap, H] bf16 for the segments in
    ``offsets``. Returns (out, workspace)."""
    def refuse():
        torch = _torch()
        _need(x_perm, torch.bfloat16, "x_perm", (None, None))
        cap, H = x_perm.shape
        E_local, I = _need_ffn_i8(H, w_gate_up, s_gate_up, w_down, s_down)
        _need(offsets, torch.int32, "offsets", (E_local + 1,))
        if out is not None:
            _need(out, torch.bfloat16, "out", (cap, H))
        _ints(cap, H, E_local, I)
        _placed(x_perm.device, x_perm=x_perm, offsets=offsets, w_gate_up=w_gate_up, s_gate_up=s_gate_up, w_down=w_down,
                s_down=s_down, out=out)
        if workspace is not None:
            _workspace(lib().moe_expert_ffn_i8_workspace_size(H, I, cap), x_perm.device, workspace)
    return _small_call("expert_ffn_i8", (x_perm, offsets, w_gate_up, s_gate_up, w_down, s_down, out, workspace), stream,
                       refuse)


def forward_i8_workspace_size(T, H, I, E, k, E_local) -> int:
    return int(lib().moe_forward_i8_workspace_size(T, H, I, E, k, E_local))


@_on_stream
def moe_forward_i8(x, w_router, bias, w_gate_up, s_gate_up, w_down, s_down, k, e0, renormalize=True, *, y=None,
                   workspace=None):
    """moe_forward with the expert MLPs of moe_expert_ffn_i8: y [T, H] bf16.
    Returns (y, workspace). Takes ``stream``."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (None, None))
    T, H = x.shape
    _need(w_router, torch.float32, "w_router", (None, H))
    E = w_router.shape[0]
    if bias is not None:
        _need(bias, torch.float32, "bias", (E,))
    E_local, I = _need_ffn_i8(H, w_gate_up, s_gate_up, w_down, s_down)
    _ints(T, H, E, E_local, I)
    _check_k(k, E)
    if not (0 <= e0 and e0 + E_local <= E):
        raise ValueError(f"local experts [e0, e0 + E_local) = [{e0}, {e0 + E_local}) must lie in [0, E = {E})")
    if y is not None:
        _need(y, torch.bfloat16, "y", (T, H))
    dev = x.device
    _placed(dev, x=x, w_router=w_router, bias=bias, w_gate_up=w_gate_up, s_gate_up=s_gate_up, w_down=w_down,
            s_down=s_down)
    y = _out(y, (T, H), torch.bfloat16, dev, "y")
    L = lib()
    ws = _workspace(L.moe_forward_i8_workspace_size(T, H, I, E, k, E_local), dev, workspace)
    st = L.moe_forward_i8(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up), _ptr(s_gate_up), _ptr(w_down),
                          _ptr(s_down), T, H, I, E, k, e0, E_local, int(bool(renormalize)), _ptr(y), _ptr(ws),
                          _nbytes(ws), _stream(None, dev))
    check(st, "moe_forward_i8")
    return y, ws


def block_workspace_size(T, H, I, E, k) -> int:
    return int(lib().moe_block_workspace_size(T, H, I, E, k))


@_on_stream
def moe_block_forward(residual, w_pre, w_router, bias, w_gate_up, w_down, k, w_post=None, *, gate=None,
                      residual_scale=1.0, w_next=None, eps=1e-6, renormalize=True, out=None, normed=None,
                      workspace=None):
    """A whole block with every expert on this GPU: moe_norm_pre of
    ``residual`` [T, H], the MoE layer, moe_norm_post. Returns (out, normed or
    None, workspace). Takes ``stream``."""
    torch = _torch()
    rt = _need_either(residual, "residual", (None, None))
    T, H = residual.shape
    _ints(T, H)
    _need(w_pre, torch.float32, "w_pre", (H,))
    _need(w_router, torch.float32, "w_router", (None, H))
    E = w_router.shape[0]
    if bias is not None:
        _need(bias, torch.float32, "bias", (E,))
    _need(w_gate_up, torch.bfloat16, "w_gate_up", (E, H, None))
    I2 = w_gate_up.shape[2]
    if I2 % 2:
        raise ValueError(f"w_gate_up's last dimension 2I must be even, got {I2}")
    I = I2 // 2
    _ints(E, I)
    _need(w_down, torch.bfloat16, "w_down", (E, I, H))
    _check_k(k, E)
    if w_post is not None:
        _need(w_post, torch.float32, "w_post", (H,))
    kind = _gate_kind(gate, T, H)
    if w_next is not None:
        _need(w_next, torch.float32, "w_next", (H,))
    elif normed is not None:
        raise ValueError("normed is given without w_next")
    if out is not None:
        _need(out, residual.dtype, "out", (T, H))
    if normed is not None:
        _need(normed, torch.bfloat16, "normed", (T, H))
    dev = residual.device
    _placed(dev, residual=residual, w_pre=w_pre, w_router=w_router, bias=bias, w_gate_up=w_gate_up, w_down=w_down,
            w_post=w_post, gate=gate, w_next=w_next)
    out = _out(out, (T, H), residual.dtype, dev, "out")
    if w_next is not None:
        normed = _out(normed, (T, H), torch.bfloat16, dev, "normed")
    L = lib()
    ws = _workspace(L.moe_block_workspace_size(T, H, I, E, k), dev, workspace)
    st = L.moe_block_forward(_ptr(residual), rt, _ptr(w_pre), _ptr(w_router), _ptr(bias), _ptr(w_gate_up), _ptr(w_down),
                             _ptr(w_post), _ptr(gate), kind, residual_scale, _ptr(w_next), eps, T, H, I, E, k,
                             int(bool(renormalize)), _ptr(out), _ptr(normed), _ptr(ws), _nbytes(ws),
                             _stream(None, dev))
    check(st, "moe_block_forward")
    return out, normed, ws


# --------------------------------------------------------------------------- #
# Routing by scores                                                            #
# --------------------------------------------------------------------------- #
# MOE_SCORE_*, MOE_GROUP_*, MOE_ACT_* by the names that the calls take
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}
# most groups of experts (MOE_MAX_GROUPS)
MAX_GROUPS = 64


def _named(names, value, what):
    try:
        return names[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {', '.join(map(repr, names))}, got {value!r}") from None


def _check_groups(E, k, n_group, topk_group):
    for name, v in (("n_group", n_group), ("topk_group", topk_group)):
        if not isinstance(v, numbers.Integral) or v < 1:
            raise ValueError(f"{name} must be an int >= 1, got {v!r}")
    if E % n_group:
        raise ValueError(f"the {E} experts do not divide into n_group = {n_group} groups")
    if topk_group > n_group:
        raise ValueError(f"topk_group = {topk_group} exceeds n_group = {n_group}")
    if k > topk_group * (E // n_group):
        raise ValueError(f"k = {k} exceeds the {topk_group * (E // n_group)} experts of topk_group = {topk_group} groups")


def moe_select(logits, k, bias=None, *, score="softmax", n_group=1, topk_group=1, group_score="max", renormalize=True,
               scale=1.0, topk_idx=None, topk_w=None, stream=None):
    """Experts of each token from its router logits [T, E] float32: topk_idx
    [T, k] int32 and topk_w [T, k] float32.

    ``score`` "softmax" or "sigmoid" of the logits; ``bias`` [E] float32 is added
    to the scores for the choice alone. The experts are ``n_group`` groups of
    consecutive ones, of which the ``topk_group`` with the largest
    ``group_score`` stay ("max": their best expert, "top2": the sum of their two
    best). The k best of these are taken in descending order, equal ones by
    lower id; their weights are the scores, with ``renormalize`` divided by
    their sum, times ``scale``."""
    rule, kind = _named(GROUP_SCORES, group_score, "group_score"), _named(SCORES, score, "score")

    def refuse():
        torch = _torch()
        _need(logits, torch.float32, "logits", (None, None))
        T, E = logits.shape
        if bias is not None:
            _need(bias, torch.float32, "bias", (E,))
        _check_k(k, E)
        _check_groups(E, k, n_group, topk_group)
        if topk_idx is not None:
            _need(topk_idx, torch.int32, "topk_idx", (T, k))
        if topk_w is not None:
            _need(topk_w, torch.float32, "topk_w", (T, k))
        _ints(T, E)
        _placed(logits.device, logits=logits, bias=bias, topk_idx=topk_idx, topk_w=topk_w)
    return _small_call("select", (logits, bias, _plain_int(k), kind, _plain_int(n_group), _plain_int(topk_group), rule,
                                  renormalize, scale, topk_idx, topk_w), stream, refuse)


@_on_stream
def moe_route_scored(x, w_router, bias, choice_bias, k, *, score="softmax", n_group=1, topk_group=1, group_score="max",
                     renormalize=True, scale=1.0, logits=None, topk_idx=None, topk_w=None, workspace=None):
    """moe_route with moe_select's choice: logits [T, E] float32 (with ``bias``,
    as moe_route computes them), topk_idx [T, k] and topk_w [T, k], chosen with
    ``choice_bias`` added to the scores. Takes ``stream``."""
    torch = _torch()
    rule, kind = _named(GROUP_SCORES, group_score, "group_score"), _named(SCORES, score, "score")
    _need(x, torch.bfloat16, "x", (None, None))
    T, H = x.shape
    _need(w_router, torch.float32, "w_router", (None, H))
    E = w_router.shape[0]
    for name, t in (("bias", bias), ("choice_bias", choice_bias)):
        if t is not None:
            _need(t, torch.float32, name, (E,))
    _ints(T, H, E)
    _check_k(k, E)
    _check_groups(E, k, n_group, topk_group)
    for name, t, shp, dt in (("logits", logits, (T, E), torch.float32), ("topk_idx", topk_idx, (T, k), torch.int32),
                             ("topk_w", topk_w, (T, k), torch.float32)):
        if t is not None:
            _need(t, dt, name, shp)
    dev = x.device
    _placed(dev, x=x, w_router=w_router, bias=bias, choice_bias=choice_bias)
    logits = _out(logits, (T, E), torch.float32, dev, "logits")
    topk_idx = _out(topk_idx, (T, k), torch.int32, dev, "topk_idx")
    topk_w = _out(topk_w, (T, k), torch.float32, dev, "topk_w")
    L = lib()
    ws = _workspace(L.moe_route_workspace_size(T, H, E, k), dev, workspace)
    st = L.moe_route_scored(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(choice_bias), T, H, E, k, kind, n_group,
                            topk_group, rule, int(bool(renormalize)), scale, _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                            _ptr(ws), _nbytes(ws), _stream(None, dev))
    check(st, "moe_route_scored")
    return logits, topk_idx, topk_w


# --------------------------------------------------------------------------- #
# bf16 products with an epilogue, and the layer with a shared expert           #
# --------------------------------------------------------------------------- #
def gemm_workspace_size(M, N, K, E_local=1, activation="none") -> int:
    """Bytes of workspace moe_gemm needs for [M, K] rows and N outputs (0: none)."""
    return int(lib().moe_gemm_workspace_size(M, N, K, E_local, _named(ACTIVATIONS, activation, "activation")))


def moe_gemm(a, w, bias=None, offsets=None, *, activation="none", residual=None, out_dtype=None, out=None,
             workspace=None, stream=None):
    """out [M, N] = act(a @ w[e] + bias[e]) + residual for the rows of segment e
    of ``offsets`` [E_local + 1] int32 (None: one weight matrix for all rows).

    a [M, K] and w [E_local, K, N] are bf16, ``bias`` [E_local, N] float32,
    ``residual`` [M, N] bf16 or float32. ``activation``: "none", "relu", "silu",
    "gelu", "gelu_tanh" or "swiglu" (w and bias then have 2 N columns, gate before
    up, as w_gate_up). ``out_dtype`` bf16 (the default, or that of ``out``) or
    float32; ``out`` may be ``residual``. Rows past the last segment are left as
    they are."""
    kind = _named(ACTIVATIONS, activation, "activation")
    torch = _torch()
    if out_dtype is None:
        out_dtype = out.dtype if isinstance(out, torch.Tensor) else torch.bfloat16
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")

    def refuse():
        _need(a, torch.bfloat16, "a", (None, None))
        M, K = a.shape
        _need(w, torch.bfloat16, "w", (None, K, None))
        E_local, _, C = w.shape
        if kind == ACTIVATIONS["swiglu"] and C % 2:
            raise ValueError(f"w's last dimension 2 N must be even, got {C}")
        N = C // 2 if kind == ACTIVATIONS["swiglu"] else C
        if bias is not None:
            _need(bias, torch.float32, "bias", (E_local, C))
        if offsets is not None:
            _need(offsets, torch.int32, "offsets", (E_local + 1,))
        elif E_local != 1:
            raise ValueError(f"w holds {E_local} matrices: offsets is required")
        if residual is not None:
            _need_either(residual, "residual", (M, N))
        if out is not None:
            _need(out, out_dtype, "out", (M, N))
        _ints(M, K, E_local, C)
        _placed(a.device, a=a, w=w, bias=bias, offsets=offsets, residual=residual, out=out)
        if workspace is not None:
            _workspace(lib().moe_gemm_workspace_size(M, N, K, E_local, kind), a.device, workspace)
    return _small_call("gemm", (a, w, bias, offsets, kind, residual,
                                TYPE_F32 if out_dtype is torch.float32 else TYPE_BF16, out, workspace), stream, refuse)


def layer_workspace_size(T, H, I, I_shared, E, k, E_local) -> int:
    return int(lib().moe_layer_workspace_size(T, H, I, I_shared, E, k, E_local))


@_on_stream
def moe_layer_forward(x, w_router, bias, choice_bias, w_gate_up, w_down, k, e0, shared_gate_up=None, shared_down=None, *,
                      score="softmax", n_group=1, topk_group=1, group_score="max", renormalize=True, scale=1.0,
                      out_dtype=None, y=None, workspace=None):
    """The rank's share of an MoE layer routed as by moe_route_scored, plus the
    expert that every token shares: swiglu(x @ shared_gate_up) @ shared_down
    ([H, 2 I_shared] and [I_shared, H] bf16; None: no shared expert). Under
    expert parallelism one of a token's ranks adds it. Returns (y [T, H] bf16 or
    float32, workspace). Takes ``stream``."""
    torch = _torch()
    rule, kind = _named(GROUP_SCORES, group_score, "group_score"), _named(SCORES, score, "score")
    T, H, I, E, E_local, dev = _forward_args(x, w_router, bias, w_gate_up, w_down, k, e0)
    if choice_bias is not None:
        _need(choice_bias, torch.float32, "choice_bias", (E,))
    _check_groups(E, k, n_group, topk_group)
    if (shared_gate_up is None) != (shared_down is None):
        raise ValueError("shared_gate_up and shared_down are given together")
    Is = 0
    if shared_gate_up is not None:
        _need(shared_gate_up, torch.bfloat16, "shared_gate_up", (H, None))
        if shared_gate_up.shape[1] % 2:
            raise ValueError(f"shared_gate_up's last dimension 2 I_shared must be even, got {shared_gate_up.shape[1]}")
        Is = shared_gate_up.shape[1] // 2
        if Is == 0:
            raise ValueError("shared_gate_up has no columns")
        _need(shared_down, torch.bfloat16, "shared_down", (Is, H))
    _ints(T, H, I, E, E_local, Is)
    if out_dtype is None:
        out_dtype = y.dtype if isinstance(y, torch.Tensor) else torch.bfloat16
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
    if y is not None:
        _need(y, out_dtype, "y", (T, H))
    _placed(dev, x=x, w_router=w_router, bias=bias, choice_bias=choice_bias, w_gate_up=w_gate_up, w_down=w_down,
            shared_gate_up=shared_gate_up, shared_down=shared_down)
    y = _out(y, (T, H), out_dtype, dev, "y")
    L = lib()
    ws = _workspace(L.moe_layer_workspace_size(T, H, I, Is, E, k, E_local), dev, workspace)
    st = L.moe_layer_forward(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(choice_bias), _ptr(w_gate_up), _ptr(w_down),
                             _ptr(shared_gate_up), _ptr(shared_down), T, H, I, Is, E, k, e0, E_local, kind, n_group,
                             topk_group, rule, int(bool(renormalize)), scale, _ptr(y),
                             TYPE_F32 if out_dtype is torch.float32 else TYPE_BF16, _ptr(ws), _nbytes(ws),
                             _stream(None, dev))
    check(st, "moe_layer_forward")
    return y, ws
