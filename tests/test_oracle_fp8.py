"""Pins of the 8-bit oracle and of the FP8 expert row (CPU only)."""
import numpy as np
import pytest
import torch

from offloaded_expert_slot_gb300.configs import C2, expert_row_bytes, fp8_offsets, scaled
from offloaded_expert_slot_gb300.inputs import expert_rows
from oracle import fp8


def test_e4m3_values_are_torchs():
    b = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    want = b.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(fp8.e4m3_values(), want, equal_nan=True)


def test_rounding_to_the_nearest_code_ties_to_even():
    v = fp8.e4m3_values()
    v = np.unique(np.abs(v[np.isfinite(v)]))   # code order
    assert np.array_equal(fp8.e4m3_round(v), v)
    mid = (v[:-1] + v[1:]) / 2
    got = fp8.e4m3_round(mid)
    lo = np.arange(len(mid))
    want = np.where(lo % 2 == 0, v[:-1], v[1:])      # the even code of the two
    assert np.array_equal(got, want)
    assert np.array_equal(fp8.e4m3_round(np.nextafter(mid, np.inf)), v[1:])
    assert np.array_equal(fp8.e4m3_round(np.nextafter(mid, 0)), v[:-1])
    assert fp8.e4m3_round(np.array([1e9]))[0] == 448 and fp8.e4m3_round(np.array([-460.0]))[0] == -448


def test_quantize_by_hand():
    x = np.zeros((1, 130))
    x[0, :4] = [448.0, -224.0, 1.0, 0.3]
    x[0, 128:] = [2.0, 1.0]
    q, s = fp8.quantize(x)
    assert np.array_equal(s, [[1.0, 2.0 / 448.0]])
    assert np.array_equal(q[0, :4], [448.0, -224.0, 1.0, 0.3125])
    assert np.array_equal(q[0, 128:], [448.0, 224.0])
    z, sz = fp8.quantize(np.zeros((2, 5)))
    assert not z.any() and np.all(sz == 2.0 ** -100 / 448.0)
    n = np.array([[np.nan, 1.0, 0.5]])
    qn, sn = fp8.quantize(n)
    assert np.isnan(qn[0, 0]) and qn[0, 1] == 448 and sn[0, 0] == 1 / 448


@pytest.mark.parametrize("H,I", [(128, 64), (192, 320), (2048, 768)])
def test_row_layout(H, I):
    o, c = fp8.row_offsets(H, I), fp8_offsets(H, I)
    assert (o["w2"], o["s13"], o["s2"], o["end"]) == (c["w2q"], c["w13s"], c["w2s"], c["end"])
    assert expert_row_bytes("fp8", H, I) == o["end"] and all(v % 16 == 0 for v in o.values())


def test_expert_rows_decode_near_their_bf16_weights():
    """An e4m3 code is within 2^-4 of its value, or half a subnormal step of its block."""
    cfg = scaled(C2, name="fp8_row", T=4, k=2, E=4, H=192, I=64, S=4, L=1, prefill=0, wfmt="fp8")
    b = scaled(cfg, wfmt="bf16")
    row = expert_rows(cfg, 0, [1])[0].numpy()
    raw = expert_rows(b, 0, [1])[0].view(torch.bfloat16).to(torch.float64).numpy()
    gate, up, w2 = fp8.expert_weights(row, cfg.H, cfg.I)
    got = np.concatenate([gate.ravel(), up.ravel(), w2.ravel()])
    amax = np.abs(raw).max()
    assert np.all(np.abs(got - raw) <= np.abs(raw) * 2.0 ** -4 + amax / 448 * 2.0 ** -10 + 1e-9)
    assert np.array_equal(got == 0, np.abs(got) == 0)
