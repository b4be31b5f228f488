"""Shared by the tests of the 8-bit operators: seeded rows and weights, and
the checks of codes and scales against the 64-bit oracle."""
from __future__ import annotations

import numpy as np
import torch

from offloaded_expert_slot_gb300.inputs import quantize_fp8_blocks, rng
from oracle import fp8

# fp32 unit roundoff
EPS32 = 2.0 ** -24


def strided(a: np.ndarray, pad: int, dtype) -> torch.Tensor:
    """A CUDA [T, W] view with row stride W + pad; the padding is NaN."""
    T, W = a.shape
    b = torch.full((T, W + pad), float("nan"), dtype=torch.float32)
    b[:, :W] = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return b.to(dtype).cuda()[:, :W]


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def rows(T, K, seed, spread=True) -> np.ndarray:
    """N(0, 1) rows; with spread, each row has its own magnitude and some groups are zero."""
    g = rng(seed)
    x = g.standard_normal((T, K))
    if spread:
        x *= 2.0 ** g.integers(-12, 12, size=(T, 1))
        x[g.random((T, K)) < 0.05] = 0.0
        if K > 128:
            x[:: 3, 128:256] = 0.0
    return x


def check_codes(codes: torch.Tensor, scale: torch.Tensor, want: np.ndarray, rel: float,
                amax_rel: float):
    """codes [T, K] u8 and scale against the quantiser applied to `want`
    (float64), of which the kernel had values with relative error at most
    `rel`: each code is a nearest code of a ratio within 2 rel + 2^-22 of
    the exact one (the value and amax, then the division's roundings)."""
    K = want.shape[1]
    a = fp8.group_amax(want)
    s = f64(scale)
    assert s.shape == a.shape
    assert np.all(np.abs(s - a / 448.0) <= (a / 448.0) * (amax_rel + 2 * EPS32))
    q = fp8.e4m3_values()[codes.cpu().numpy()]
    r = fp8.ratios(want)
    tol = np.abs(r) * (rel + amax_rel + 4 * EPS32)
    # half the gap on the side of the ratio: the wider neighbouring gap bounds it
    half = 0.5 * fp8.e4m3_step(np.abs(r) + tol)
    assert np.all(np.abs(q - r) <= half + tol)
    assert np.all((q == 0) | (np.sign(q) == np.sign(r)))


def fp8_weight(N, K, seed):
    """codes [N, K] in rows of a multiple of 16 bytes (CUDA), scales (CUDA), float64 [N, K]."""
    w = torch.from_numpy(rng(seed).standard_normal((N, K)).astype(np.float32) * 0.05)
    q, s = quantize_fp8_blocks(w)
    return padded(q), s.cuda(), fp8.weight(q.numpy(), s.numpy())


def padded(q: torch.Tensor, extra: int = 0) -> torch.Tensor:
    """u8 [N, K] as a CUDA view whose row stride is a multiple of 16; the padding holds NaN codes."""
    ld = (q.shape[1] + 15) // 16 * 16 + extra
    b = torch.full((q.shape[0], ld), 0x7F, dtype=torch.uint8)
    b[:, : q.shape[1]] = q
    return b.cuda()[:, : q.shape[1]]
