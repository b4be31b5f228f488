"""The 8-bit oracle's product, expert MLP and expert rows by brute force (CPU
only): plain loops over rows, blocks and K, from the row's bytes on."""
import numpy as np
import pytest
import torch

from offloaded_expert_slot_gb300.configs import C2, fp8_offsets, scaled
from offloaded_expert_slot_gb300.inputs import expert_rows, rng
from oracle import fp8


def e4m3(byte):
    """One code, digit by digit."""
    sign = -1.0 if byte & 0x80 else 1.0
    e, m = (byte >> 3) & 15, byte & 7
    assert byte & 0x7F != 0x7F
    return sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


CODES = sorted({e4m3(b) for b in range(127)})       # the values of the positive codes


def nearest(v):
    """The nearest code's value, ties to the even one."""
    a = abs(v)
    i = min(range(len(CODES)), key=lambda n: (abs(CODES[n] - a), n % 2))
    return CODES[i] if v >= 0 else -CODES[i]


def product_row(x, codes, scale_row):
    """sum_b scale[b] sum_{k in b} x[k] w[k] for one row of weights."""
    s = 0.0
    for k in range(len(x)):
        s += x[k] * e4m3(int(codes[k])) * float(scale_row[k // 128])
    return s


def quantised(v):
    """A row's values as their codes and scales stand for them."""
    out = []
    for b in range(0, len(v), 128):
        part = v[b:b + 128]
        amax = max([2.0 ** -100] + [abs(a) for a in part])
        out += [nearest(448 * a / amax) * (amax / 448) for a in part]
    return out


@pytest.mark.parametrize("H,I", [(64, 64), (192, 64), (128, 192), (64, 320)])
def test_expert_mlp_by_loops(H, I):
    """Short last blocks, gate and up scales in halves of their own, h in groups of 128."""
    g = rng(H * I)
    o, hb, ib = fp8_offsets(H, I), -(-H // 128), -(-I // 128)
    row = g.integers(0, 256, size=o["end"]).astype(np.uint8)
    w = row[:o["w13s"]]
    w[(w & 0x7F) == 0x7F] = 0x31
    for name, n in (("w13s", 2 * ib * hb), ("w2s", hb * ib)):
        row[o[name]:o[name] + 4 * n] = (g.random(n).astype(np.float32) * 0.01 + 0.001).view(np.uint8)
    x = g.standard_normal((2, H))
    got = fp8.expert_mlp(x, row, H, I)
    w13, w2 = row[:o["w2q"]].reshape(2 * I, H), row[o["w2q"]:o["w13s"]].reshape(H, I)
    s13 = row[o["w13s"]:o["w13s"] + 8 * ib * hb].view(np.float32).reshape(2, ib, hb)
    s2 = row[o["w2s"]:o["w2s"] + 4 * ib * hb].view(np.float32).reshape(hb, ib)
    for t in range(2):
        h = []
        for i in range(I):
            gate = product_row(x[t], w13[i], s13[0][i // 128])
            up = product_row(x[t], w13[I + i], s13[1][i // 128])
            h.append(gate / (1 + np.exp(-gate)) * up)
        h = quantised(h)
        want = np.array([product_row(h, w2[n], s2[n // 128]) for n in range(H)])
        assert np.allclose(got[t], want, rtol=1e-9, atol=1e-9 * np.abs(want).max())


def test_dequantise_and_weight_by_loops():
    g = rng(12)
    q, s = np.array(CODES)[g.integers(0, len(CODES), size=(3, 200))], g.random((3, 2))
    d = fp8.dequantize(q, s)
    codes, ws = g.integers(0, 127, size=(130, 200)).astype(np.uint8), g.random((2, 2)).astype(np.float32)
    w = fp8.weight(codes, ws)
    for t in range(3):
        for k in range(200):
            assert d[t, k] == q[t, k] * s[t, k // 128]
    for n in range(130):
        for k in range(200):
            assert w[n, k] == e4m3(int(codes[n, k])) * float(ws[n // 128, k // 128])


def test_expert_rows_hold_zero_only_where_the_ratio_rounds_to_it():
    """A code is 0 where the weight is at most half the smallest code, 2^-10, of its
    block's scale (the tie goes to the even code), and nowhere else."""
    cfg = scaled(C2, name="fp8_zero", T=4, k=2, E=4, H=192, I=192, S=4, L=1, prefill=0, wfmt="fp8")
    row = expert_rows(cfg, 0, [1])[0].numpy()
    raw = expert_rows(scaled(cfg, wfmt="bf16"), 0, [1])[0].view(torch.bfloat16).to(torch.float64).numpy()
    H, I, o = cfg.H, cfg.I, fp8_offsets(cfg.H, cfg.I)
    s13 = row[o["w13s"]:o["w13s"] + 32].view(np.float32).astype(np.float64).reshape(2, 2, 2)
    s2 = row[o["w2s"]:o["w2s"] + 16].view(np.float32).astype(np.float64).reshape(2, 2)
    spread = lambda s, N, K: np.repeat(np.repeat(s, 128, 0)[:N], 128, 1)[:, :K]  # noqa: E731
    scale = np.concatenate([spread(s13[0], I, H).ravel(), spread(s13[1], I, H).ravel(), spread(s2, H, I).ravel()])
    got = np.concatenate([m.ravel() for m in fp8.expert_weights(row, H, I)])
    ratio = np.abs(raw) / scale
    assert (ratio <= 2.0 ** -10).sum() > 0
    assert np.array_equal(got == 0, ratio <= 2.0 ** -10)
    assert np.all(np.sign(got[got != 0]) == np.sign(raw[got != 0]))
