"""SwiGLU inside moe_fp8_quantize over the whole fp32 range of its gate.

Tolerance of silu(gate) up (u = 2^-24): exp within 2 ulp, a sum, a quotient
and two products, 16 u; where exp(-|gate|) is below 2^-126 fp32 holds it in
steps of 2^-149, which adds |gate| 2^-149 to silu.
"""
import numpy as np
import pytest
import torch

from fp8_util import EPS32, f64
from gpu_util import lib
from offloaded_expert_slot_gb300 import oes
from oracle import fp8

pytestmark = pytest.mark.gpu

F32_MAX = float(np.finfo(np.float32).max)


def swiglu(gate, up, K, dtype=torch.float32):
    """Codes' values and scales of rows [gate, up] of K each (0 past what is given)."""
    T, n = gate.shape
    x = torch.zeros((T, 2 * K))
    x[:, :n] = torch.from_numpy(np.asarray(gate, np.float32))
    x[:, K:K + n] = torch.from_numpy(np.asarray(up, np.float32))
    x = x.to(dtype).cuda()
    q = torch.empty((T, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((T, -(-K // 128)), device="cuda")
    oes.moe_fp8_quantize(x, 2 * K, T, K, oes.OES_ACT_SWIGLU, q, K, s)
    torch.cuda.synchronize()
    return fp8.e4m3_values()[q.cpu().numpy()], f64(s), f64(x)


@pytest.mark.parametrize("K", [128, 127])
def test_silu_at_every_size_of_the_gate(K):
    """One value a row, so that the row's scale is |silu(gate) up| / 448."""
    lib()
    g = np.concatenate([np.linspace(-104, 104, 4000), 2.0 ** np.linspace(-30, 127, 1200),
                        -(2.0 ** np.linspace(-30, 6.5, 300)), [F32_MAX, 2.36e38, 3e38, -88.0, -87.4, -88.7]])
    g = g.astype(np.float32).astype(np.float64)
    e = np.exp(-np.abs(g))
    silu = np.where(g < 0, g * e, g) / (1 + e)
    # a power of two that brings the product into fp32's normal range
    up = 2.0 ** np.clip(-np.floor(np.log2(np.abs(silu))), -20, 100)
    q, s, _ = swiglu(g[:, None], up[:, None], K)
    h = np.abs(silu * up)
    tol = h * 18 * EPS32 + np.abs(g) * 2.0 ** -149 * up
    assert np.all(h >= 2.0 ** -60) and np.all(h < F32_MAX)
    assert np.all(np.abs(s[:, 0] * 448 - h) <= tol)
    assert np.array_equal(q[:, 0], np.sign(g) * 448)


@pytest.mark.parametrize("K", [384, 385])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_swiglu_special_values(K, dtype):
    """Values of silu(gate) up that are infinite make their group's scale infinite;
    NaN takes no part in amax and gets a NaN code; what is finite stays so."""
    lib()
    inf, nan = np.inf, np.nan
    #        gate   up     silu(gate) up
    cases = [(inf, 1.0, inf), (inf, -2.0, -inf), (3e38, 1.0, 3e38), (3e38, -0.5, -1.5e38), (3e38, 2.0, inf),
             (1.0, inf, inf), (-88.0, 2.0 ** 40, -88.0 * np.exp(-88.0) * 2.0 ** 40), (-3e38, 1.0, 0.0),
             (-3e38, -1e30, 0.0), (-inf, 1.0, nan), (nan, 1.0, nan), (1.0, nan, nan), (nan, nan, nan), (inf, nan, nan)]
    T = len(cases)
    g, u = np.random.default_rng(4).standard_normal((2, T, K))
    at = 131                                      # in the second group
    for t, (a, b, _) in enumerate(cases):
        g[t, at], u[t, at] = a, b
    q, s, x = swiglu(g, u, K, dtype)
    x[:, at], x[:, K + at] = 0.0, 0.0             # the others' values, as the kernel had them
    h = x[:, :K] / (1 + np.exp(-x[:, :K])) * x[:, K:]
    for t, (_, _, want) in enumerate(cases):
        rest = fp8.group_amax(h[t:t + 1])[0] / 448
        assert np.allclose(np.delete(s[t], 1), np.delete(rest, 1), rtol=18 * EPS32, atol=0), cases[t]
        if np.isinf(want):
            assert np.isinf(s[t, 1]), cases[t]
            with np.errstate(invalid="ignore"):
                assert np.isnan(q[t, 128:256] * s[t, 1]).all(), cases[t]
            continue
        assert np.isnan(q[t, at]) == np.isnan(want), cases[t]
        assert int(np.isnan(q[t]).sum()) == int(np.isnan(want)), cases[t]
        amax = max(abs(want) / 448, rest[1]) if want == want else rest[1]
        assert np.isclose(s[t, 1], amax, rtol=2.0 ** -7 if dtype == torch.bfloat16 else 18 * EPS32), cases[t]
        if abs(want) > 1e30:
            assert q[t, at] == np.sign(want) * 448, cases[t]
