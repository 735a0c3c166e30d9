"""Row counts next to 2^31 in the grouped products: the blocks that a segment is cut
into (on the CPU), and the products that go through them (on the GPU)."""
import ctypes

import pytest
import torch

import expert_token_routing_amd as M
from tests.gpu_helpers import device, say

BF = torch.bfloat16
CAPS = [16, 32, 64, 128, 160, 192, 224, 256, 288]
gpu = pytest.mark.gpu


@pytest.mark.parametrize("cap", CAPS)
def test_blocks_cover_every_segment(cap):
    fn = M.lib().moe_internal_row_blocks
    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    top = 2 ** 31 - 1
    sizes = [1, 15, 16, 17, cap - 1, cap, cap + 1, 3 * cap + 5, 10 ** 6 + 7, 2 ** 30 + 1, 2_139_100_000, 2 ** 31 - 2000,
             2 ** 31 - 1025, top - 2 * cap, top - cap, top - cap + 1, top - 1, top]
    for rows in sizes:
        height = ctypes.c_int(-1)
        n = fn(rows, cap, ctypes.byref(height))
        h = height.value
        assert n == -(-rows // cap), rows
        assert h == (-(-rows // n) + 15) // 16 * 16 and 0 < h <= cap, rows
        # every row is in a block, and no block starts past what an int holds
        assert n * h >= rows and (n - 1) * h <= top, rows


@pytest.mark.parametrize("rows", [2 ** 31 - 1024, 2 ** 31 - 1, 2 ** 31])
def test_rows_that_blocks_do_not_take_are_refused(rows):
    p = ctypes.c_void_p(0x10000)
    L = M.lib()
    assert L.moe_expert_ffn(p, p, p, p, 32, 32, 4, rows, p, p, None) == M.MOE_ERR_UNSUPPORTED
    assert L.moe_gemm(p, p, None, None, 0, None, rows, 8, 8, 1, 0, p, 0, None, 0, None) == M.MOE_ERR_UNSUPPORTED


def far(M_rows, K, N, dtype):
    """A row pattern of 2^20 rows, repeated over `M_rows` rows."""
    dev = device()
    torch.cuda.empty_cache()
    g = torch.Generator(device=dev).manual_seed(M_rows % 1000)
    pattern = torch.randint(-4, 5, (1 << 20, K), generator=g, device=dev).to(dtype)
    a = torch.empty(M_rows, K, dtype=dtype, device=dev)
    for lo in range(0, M_rows, 1 << 20):
        n = min(1 << 20, M_rows - lo)
        a[lo:lo + n] = pattern[:n]
    w = torch.randint(-4, 5, (1, K, N), generator=g, device=dev)
    return a, pattern, w


def same_everywhere(out, want):
    for lo in range(0, out.shape[0], 1 << 20):
        n = min(1 << 20, out.shape[0] - lo)
        assert torch.equal(out[lo:lo + n], want[:n]), lo


@gpu
@pytest.mark.parametrize("segments", [1, 2])
def test_gemm_rows_next_to_31_bits(segments):
    rows = 2 ** 31 - 2000
    say(f"moe_gemm {rows} x 8 x 8 in {segments} segments")
    a, pattern, w = far(rows, 8, 8, BF)
    off = torch.tensor([0, 5, rows], dtype=torch.int32, device=a.device) if segments == 2 else None
    out = M.moe_gemm(a, w.to(BF).repeat(segments, 1, 1), None, off)
    same_everywhere(out, (pattern.float() @ w[0].float()).to(BF))
    del a, out
    torch.cuda.empty_cache()


@gpu
def test_i8_rows_next_to_31_bits():
    rows = 2 ** 31 - 2000
    say(f"moe_gemm_i8 {rows} x 16 x 8")
    a, pattern, w = far(rows, 16, 8, torch.int8)
    out = M.moe_gemm_i8(a, torch.ones(rows, device=a.device), w[0].T[None].to(torch.int8).contiguous(),
                        torch.ones(1, 8, device=a.device))
    same_everywhere(out, (pattern.float() @ w[0].float()).to(BF))
    del a, out
    torch.cuda.empty_cache()
