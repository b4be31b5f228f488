"""moe_fp8_gemm against the 64-bit product of the same codes and scales.

Tolerance: the products of codes are exact in fp32 (8-bit significands) and
are added in fp32 in any order within a block of 128, the blocks one after
another with one product of scales, one FMA each: every partial sum is at
most S = sum |x| |w|, so the error is at most (128 + nkb + 4) u S, u = 2^-24,
or twice that where a sum truncates instead of rounding; bf16 adds 2^-8 of
the result.
"""
import numpy as np
import pytest
import torch

from fp8_util import EPS32, f64, fp8_weight, padded, rows
from gpu_util import lib, status
from offloaded_expert_slot_gb300 import oes
from oracle import fp8

pytestmark = pytest.mark.gpu


def operands(T, K, N, seed=0, spread=True):
    q, s = fp8.quantize(rows(T, K, seed + T + K, spread=spread))
    codes = torch.from_numpy(q.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    xs = torch.from_numpy(s.astype(np.float32))
    w = fp8_weight(N, K, seed + N)
    return padded(codes), xs.cuda(), fp8.dequantize(q, s.astype(np.float32).astype(np.float64)), w


def product(xq, xs, K, w, N, dtype=torch.bfloat16, pad=0, stream=None):
    T = xq.shape[0]
    buf = torch.full((T + 2, N + pad), -77.0, dtype=dtype, device="cuda")
    out = buf[1:T + 1]
    st = status()
    wq, ws, _ = w
    oes.moe_fp8_gemm(xq, xq.stride(0), xs, T, K, wq, wq.stride(0), ws, N, out, N + pad, st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert (buf[0] == -77).all() and (buf[-1] == -77).all() and (buf[:, N:] == -77).all()
    return out[:, :N]


def check(out, x64, w64, K):
    want = x64 @ w64.T
    big = np.abs(x64) @ np.abs(w64).T
    tol = big * 2 * (128 + -(-K // 128) + 4) * EPS32
    if out.dtype == torch.bfloat16:
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(f64(out) - want) <= tol + 1e-37)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 40, 64, 65, 128, 200, 300])
@pytest.mark.parametrize("K,N", [(128, 128), (768, 256), (2048, 1536)])
def test_gemm(T, K, N, dtype):
    lib()
    xq, xs, x64, w = operands(T, K, N)
    check(product(xq, xs, K, w, N, dtype), x64, w[2], K)


@pytest.mark.parametrize("T,K,N,pad", [(1, 1, 1, 0), (3, 5, 7, 0), (1, 127, 129, 0), (17, 129, 127, 1),
                                       (33, 200, 300, 4), (130, 1000, 333, 0), (257, 640, 513, 3),
                                       (129, 4099, 136, 0), (5, 130, 2000, 0), (70, 384, 1, 0),
                                       (1000, 16, 24, 0), (1, 16384, 100, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_gemm_odd_sizes(T, K, N, pad, dtype):
    lib()
    xq, xs, x64, w = operands(T, K, N, seed=9)
    check(product(xq, xs, K, w, N, dtype, pad), x64, w[2], K)


@pytest.mark.parametrize("T", [20, 2500])
def test_gemm_many_tiles(T):
    """More tiles than a GPU has multiprocessors, whole and ragged."""
    lib()
    K, N = 256, 2500
    xq, xs, x64, w = operands(T, K, N, seed=3)
    check(product(xq, xs, K, w, N), x64, w[2], K)


@pytest.mark.parametrize("T,N", [(4, 300), (200, 300)])
def test_gemm_nan_codes_and_infinite_scales_stay_in_their_rows(T, N):
    lib()
    K = 256
    xq, xs, x64, w = operands(T, K, N, spread=False)
    xq[1, 200] = 0x7F
    xs[2, 1] = float("inf")
    out = product(xq, xs, K, w, N)
    bad = ~torch.isfinite(out)
    assert bad[1].all() and bad[2].all() and not bad[0].any() and not bad[3:].any()
    wq = w[0].clone()
    xq, xs, x64, _ = operands(T, K, N, spread=False)
    w2 = padded(wq.cpu())
    w2[5, 7] = 0x7F
    out = product(xq, xs, K, (w2, w[1], None), N)
    bad = ~torch.isfinite(out)
    assert bad[:, 5].all() and int(bad.sum()) == T


@pytest.mark.parametrize("T", [1, 24, 256])
def test_gemm_repeats_bit_for_bit_on_any_stream(T):
    lib()
    K, N = 2048, 640
    xq, xs, _, w = operands(T, K, N)
    first = product(xq, xs, K, w, N, torch.float32).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(product(xq, xs, K, w, N, torch.float32, stream=side), first)
    # a row's result does not depend on what the other rows hold
    xq2, xs2 = xq.clone(), xs.clone()
    if T > 1:
        xq2 = padded(torch.flip(xq.cpu(), [0]))
        xs2 = torch.flip(xs, [0]).contiguous()
        assert torch.equal(torch.flip(product(xq2, xs2, K, w, N, torch.float32), [0]), first)


def test_gemm_in_a_graph_and_empty():
    lib()
    K, N, T = 512, 384, 48
    xq, xs, x64, w = operands(T, K, N)
    out, st = torch.empty((T, N), dtype=torch.float32, device="cuda"), status()
    args = (xq, xq.stride(0), xs, T, K, w[0], w[0].stride(0), w[1], N, out, N, st)
    oes.moe_fp8_gemm(*args)
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oes.moe_fp8_gemm(*args)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    oes.moe_fp8_gemm(0, 16, 0, 0, 16, 0, 16, 0, 16, 0, 16, 0, dtype=oes.OES_BF16)   # no rows


@pytest.mark.parametrize("T", [1, 2, 3, 5, 9, 15, 16, 17, 18, 25, 31, 33])
@pytest.mark.parametrize("K,N", [(1000, 640), (1024, 2200), (1152, 1000), (2000, 384), (4200, 130)])
def test_gemm_shared_k(T, K, N):
    """Few tiles over 8 to 33 blocks of K, where several CTAs share a tile, some of
    them without rows of their own; the same bits from one call after another."""
    lib()
    xq, xs, x64, w = operands(T, K, N, seed=5)
    first = product(xq, xs, K, w, N, torch.float32).clone()
    check(first, x64, w[2], K)
    for _ in range(20):
        assert torch.equal(product(xq, xs, K, w, N, torch.float32), first)
