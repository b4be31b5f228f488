"""moe_fp8_quantize and moe_block_norm against 64-bit references.

Tolerances, from the operations (u = 2^-24):
* quantize without activation: the values are exact, so from bf16 the codes
  equal the 64-bit definition's bit for bit (a ratio of integers below 2^20
  is an exact midpoint or at least 2^-13 away from one, relatively; from
  fp32 a code may be either neighbour within 4 u of a midpoint).
* SwiGLU: exp within 2 ulp, a sum, a quotient and two products: 16 u.
* norm: a mean of squares over H <= 16384 values added in at most 32 + 10
  steps a thread and tree: 64 u on the mean, half of it after the root, 8 u
  for the rest; so 48 u relative for v and u, plus, for r', u on each term of
  the sum.  bf16 outputs add 2^-8.
"""
import numpy as np
import pytest
import torch

from fp8_util import EPS32, check_codes, f64, rows, strided
from gpu_util import lib
from offloaded_expert_slot_gb300 import oes
from oracle import fp8

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def quantize(x, K, act=oes.OES_ACT_NONE, q_pad=0, stream=None):
    T = x.shape[0]
    qb = torch.full((T + 2, K + q_pad), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((T + 2, -(-K // 128)), -7.0, device="cuda")
    q, s = qb[1:T + 1], sb[1:T + 1]
    oes.moe_fp8_quantize(x, x.stride(0), T, K, act, q, K + q_pad, s, stream=stream)
    torch.cuda.synchronize()
    assert (qb[0] == 0xA5).all() and (qb[-1] == 0xA5).all() and (qb[:, K:] == 0xA5).all()
    assert (sb[0] == -7).all() and (sb[-1] == -7).all()
    return q[:, :K], s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,pad,q_pad", [(1, 1, 0, 0), (3, 127, 0, 0), (5, 128, 0, 0), (7, 129, 0, 3),
                                           (33, 768, 8, 8), (17, 777, 3, 0), (300, 2048, 0, 0),
                                           (2, 8200, 0, 0), (1001, 64, 0, 0)])
def test_quantize(dtype, T, K, pad, q_pad):
    lib()
    x = strided(rows(T, K, 31 * T + K), pad, DTYPES[dtype])
    q, s = quantize(x, K, q_pad=q_pad)
    if dtype == "bf16":
        want, _ = fp8.quantize(f64(x))
        assert np.array_equal(fp8.e4m3_values()[q.cpu().numpy()], want)
    check_codes(q, s, f64(x), 0.0, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,pad", [(1, 64, 0), (5, 131, 0), (32, 768, 0), (9, 640, 5), (200, 1024, 8)])
def test_quantize_swiglu(dtype, T, K, pad):
    lib()
    x = strided(rows(T, 2 * K, 7 * T + K, spread=False) * 2, pad, DTYPES[dtype])
    q, s = quantize(x, K, act=oes.OES_ACT_SWIGLU)
    v = f64(x)
    h = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
    check_codes(q, s, h, 16 * EPS32, 16 * EPS32)


@pytest.mark.parametrize("K", [384, 385])
def test_quantize_special_values(K):
    """NaN, infinities, zeros, the largest and the smallest values."""
    lib()
    x = rows(6, K, 5, spread=False)
    x[0, 3] = np.nan
    x[1, 130] = np.inf
    x[2] = 0.0
    x[3] = 3.0e38 * np.sign(x[3])
    x[4] = 1e-38 * x[4]
    x[5, :128] = np.nan
    t = strided(x, 0, torch.float32)
    q, s = quantize(t, K)
    got = fp8.e4m3_values()[q.cpu().numpy()]
    scale = f64(s)
    assert np.isnan(got[0, 3]) and np.isfinite(np.delete(got[0], 3)).all() and np.isfinite(scale[0]).all()
    read = got * fp8.spread(scale, K)
    assert np.isinf(scale[1, 1]) and np.isnan(read[1, 128:256]).all()
    assert np.isfinite(read[1, :128]).all() and np.isfinite(read[1, 256:]).all()
    assert not got[2].any() and np.all(scale[2] > 0)
    assert np.all(np.abs(got[3]) == 448) and np.isfinite(scale[3]).all()
    assert not got[4].any()                       # far below the floor of a group
    assert np.isnan(got[5, :128]).all() and np.isfinite(scale[5]).all()


def test_quantize_exact_midpoints():
    """448 x / amax a midpoint between two codes in every place: ties to even."""
    lib()
    v = np.unique(np.abs(fp8.e4m3_values()[np.isfinite(fp8.e4m3_values())]))
    mid = ((v[:-1] + v[1:]) / 2)[-100:]
    for amax in (448.0, 1.0, 3.5, 2.0 ** -40 * 1.75):
        x = np.zeros((2, 128))
        x[:, 0] = amax
        x[0, 1:101] = mid * amax / 448
        x[1, 1:101] = -mid * amax / 448
        x = x.astype(np.float32).astype(np.float64)
        exact = 448 * x / amax == np.concatenate([[[448.0], [448.0]], np.stack([mid, -mid]),
                                                  np.zeros((2, 27))], axis=1)
        q, _ = quantize(strided(x, 0, torch.float32), 128)
        got = fp8.e4m3_values()[q.cpu().numpy()]
        want = fp8.e4m3_round(448 * x / amax)
        assert exact.mean() > 0.3
        assert np.array_equal(got[exact], want[exact])


def test_quantize_on_another_stream_and_empty():
    lib()
    x = strided(rows(64, 512, 3), 0, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = quantize(x, 512, stream=side)
    q0, s0 = quantize(x, 512)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    oes.moe_fp8_quantize(0, 512, 0, 512, 0, 0, 512, 0, dtype=oes.OES_BF16)   # no rows: nothing to do


# -------------------------------------------------------------------- norm
GATES = {"none": oes.OES_GATE_NONE, "token": oes.OES_GATE_TOKEN, "channel": oes.OES_GATE_CHANNEL,
         "element": oes.OES_GATE_ELEMENT}


def norm_case(T, H, res="bf16", gate="none", sigmoid=True, y=True, post=True, pre=True, quant=True,
              pad=0, scale=0.5, offset=0.0, eps=1e-6, in_place=False, stream=None):
    g = np.random.Generator(np.random.PCG64(T * 1000 + H))
    dt = DTYPES[res]
    r = strided(rows(T, H, 1 + T + H, spread=False) * 3, pad, dt)
    yt = strided(rows(T, H, 2 + T + H), pad, torch.bfloat16) if y else None
    w = [torch.from_numpy((1 - offset + 0.2 * g.standard_normal(H)).astype(np.float32)).to(torch.bfloat16).cuda()
         for _ in range(2)]
    gt, gate_ld = None, 0
    if gate == "token":
        gt = torch.from_numpy(g.standard_normal((T, 3)).astype(np.float32)).cuda()[:, 1]  # a column
        gate_ld = 3
    elif gate == "channel":
        gt = torch.from_numpy(g.standard_normal(H).astype(np.float32)).to(torch.bfloat16).cuda()
    elif gate == "element":
        gt = strided(g.standard_normal((T, H)), pad, torch.bfloat16)
        gate_ld = gt.stride(0)
    r64, y64 = f64(r), f64(yt) if y else None
    mag = np.abs(r64)
    if y:
        v = y64
        if post:
            v = v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * (offset + f64(w[0]))
        if gate != "none":
            a = f64(gt)
            a = a[:, None] if gate == "token" else a
            v = v * (1 / (1 + np.exp(-a)) if sigmoid else a)
        want_r = r64 + scale * v
        mag = mag + np.abs(scale * v)
    else:
        want_r = r64
    u = want_r
    if pre:
        inv = 1 / np.sqrt((u * u).mean(1, keepdims=True) + eps)
        u = u * inv * (offset + f64(w[1]))
        mag_u = mag * inv * np.abs(offset + f64(w[1]))
    else:
        mag_u = mag
    r_out = r if in_place else torch.empty((T, H + pad), dtype=dt, device="cuda")[:, :H]
    out = torch.empty((T, H + pad), dtype=torch.bfloat16, device="cuda")[:, :H]
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda") if quant else None
    s = torch.empty((T, -(-H // 128)), device="cuda") if quant else None
    args = oes.block_norm(T, H, r, r.stride(0), y=yt, y_ld=yt.stride(0) if y else None,
                          post_weight=w[0] if post and y else None, pre_weight=w[1] if pre else None,
                          gate=gt, gate_kind=GATES[gate], gate_ld=gate_ld, gate_sigmoid=sigmoid,
                          residual_scale=scale, weight_offset=offset, eps=eps, out_residual=r_out,
                          out_residual_ld=r_out.stride(0), out=out, out_ld=out.stride(0), out_q=q,
                          out_scale=s)
    oes.moe_block_norm(args, stream=stream)
    torch.cuda.synchronize()
    rel = 48 * EPS32
    half = 2.0 ** -8 if res == "bf16" else 0.0
    tol = mag * 2 * rel
    assert np.all(np.abs(f64(r_out) - want_r) <= np.abs(want_r) * half + tol + 1e-37)
    tol_u = mag_u * 4 * rel
    assert np.all(np.abs(f64(out) - u) <= np.abs(u) * 2.0 ** -8 + tol_u + 1e-37)
    if quant:
        # the error of u relative to its group's amax decides codes and scales
        a = fp8.spread(fp8.group_amax(u), H)
        e = (tol_u / a).max()
        qv = fp8.e4m3_values()[q.cpu().numpy()]
        assert np.all(np.abs(f64(s) - fp8.group_amax(u) / 448) <= fp8.group_amax(u) / 448 * (e + 4 * EPS32))
        rt = fp8.ratios(u)
        d = 448 * 2 * e + np.abs(rt) * 8 * EPS32
        assert np.all(np.abs(qv - rt) <= 0.5 * fp8.e4m3_step(np.abs(rt) + d) + d)
    return r_out, out, q, s


@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("T,H,pad", [(1, 2048, 0), (5, 256, 0), (7, 499, 0), (3, 512, 8), (40, 1999, 3)])
def test_norm_gates(res, gate, T, H, pad):
    lib()
    norm_case(T, H, res=res, gate=gate, pad=pad)


@pytest.mark.parametrize("T,H", [(1, 1), (2, 7), (4, 8), (2, 4096), (2, 4104), (2, 5000), (2, 8192),
                                 (3, 8200), (2, 16384), (2, 16383), (700, 64), (9000, 128)])
@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_norm_widths(res, T, H):
    lib()
    norm_case(T, H, res=res, gate="token")


@pytest.mark.parametrize("kw", [dict(y=False), dict(y=False, pre=False), dict(post=False), dict(pre=False),
                                dict(post=False, pre=False, gate="element"), dict(sigmoid=False, gate="token"),
                                dict(sigmoid=False, gate="channel"), dict(offset=1.0, gate="none"),
                                dict(scale=-1.5), dict(quant=False), dict(in_place=True, gate="channel")],
                         ids=str)
@pytest.mark.parametrize("H", [384, 391])
def test_norm_forms(H, kw):
    lib()
    norm_case(11, H, **kw)


@pytest.mark.parametrize("kw", [dict(post=False), dict(pre=False), {}], ids=str)
@pytest.mark.parametrize("T,H", [(6000, 1024), (3000, 2040), (2000, 1999), (700, 5001), (400, 12001)])
def test_norm_many_rows_a_cta(T, H, kw):
    """Each CTA walks many rows, with one reduction a row or two."""
    lib()
    norm_case(T, H, pad=1, **kw)
    norm_case(T, H, **kw)


def test_norm_outputs_may_be_left_out_and_stand_in_place():
    lib()
    T, H = 37, 640
    r = strided(rows(T, H, 8, spread=False), 0, torch.bfloat16)
    y = strided(rows(T, H, 9, spread=False), 0, torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    full = [torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, s = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 5), device="cuda")
    oes.moe_block_norm(oes.block_norm(T, H, r, y=y, post_weight=w, pre_weight=w, out_residual=full[0],
                                      out=full[1], out_q=q, out_scale=s))
    only_q, only_s = torch.empty_like(q), torch.empty_like(s)
    oes.moe_block_norm(oes.block_norm(T, H, r, y=y, post_weight=w, pre_weight=w, out_q=only_q, out_scale=only_s))
    only_r = torch.empty_like(full[0])
    oes.moe_block_norm(oes.block_norm(T, H, r, y=y, post_weight=w, pre_weight=w, out_residual=only_r))
    oes.moe_block_norm(oes.block_norm(T, H, r, y=y, post_weight=w, pre_weight=w, out_residual=r, out=y))
    torch.cuda.synchronize()
    assert torch.equal(only_q, q) and torch.equal(only_s, s) and torch.equal(only_r, full[0])
    assert torch.equal(r, full[0]) and torch.equal(y, full[1])


def test_norm_rows_with_nan_do_not_reach_others():
    lib()
    T, H = 9, 768
    x = rows(T, H, 4, spread=False)
    x[4, 100] = np.nan
    r = strided(x, 0, torch.float32)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    oes.moe_block_norm(oes.block_norm(T, H, r, pre_weight=w, out=out))
    torch.cuda.synchronize()
    bad = torch.isnan(out).any(1).cpu().numpy()
    assert np.array_equal(np.nonzero(bad)[0], [4]) and torch.isnan(out[4]).all()


def test_norm_on_another_stream_and_empty():
    lib()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm_case(64, 2048, gate="token", stream=side)
    z = torch.empty(1, dtype=torch.bfloat16, device="cuda")
    oes.moe_block_norm(oes.block_norm(0, 2048, z, out=z))
