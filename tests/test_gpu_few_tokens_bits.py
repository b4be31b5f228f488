"""How many bits moe_layer_few_tokens holds between its products: cases whose results are exact when the sums are
fp32 and h keeps its bits, and far off when either is rounded to fewer."""
import numpy as np
import pytest
import torch

from gpu_util import lib
from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.inputs import rng

pytestmark = pytest.mark.gpu

WFMT = {"bf16": oes.OES_WFMT_BF16, "fp8": oes.OES_WFMT_FP8, "nvfp4": oes.OES_WFMT_NVFP4}
E4M3 = {0.0: 0x00, 1.0: 0x38, -1.0: 0xB8, 4.0: 0x48}
E2M1 = {0.0: 0x0, 1.0: 0x2, -1.0: 0xA, 4.0: 0x6}


def up16(n):
    return (n + 15) // 16 * 16


def encode(fmt, w13, w2):
    """An expert's row of bytes from its matrices, [2I, H] and [H, I]; scales of 1 (for the 8- and 4-bit formats
    values of 0, 1, -1 and 4)."""
    H, I = w2.shape
    if fmt == "bf16":
        return torch.cat([torch.from_numpy(m).to(torch.bfloat16).reshape(-1) for m in (w13, w2)]).view(torch.uint8).numpy()

    def codes(m, table):
        c = np.zeros(m.shape, np.uint8)
        for v, code in table.items():
            c[m == v] = code
        return c

    if fmt == "fp8":
        n = -(-H // 128) * -(-I // 128)
        s13, s2 = np.zeros(up16(8 * n), np.uint8), np.zeros(up16(4 * n), np.uint8)
        s13.view(np.float32)[: 2 * n] = 1
        s2.view(np.float32)[:n] = 1
        return np.concatenate([codes(w13, E4M3).reshape(-1), codes(w2, E4M3).reshape(-1), s13, s2])
    parts = []
    for m in (w13, w2):
        c = codes(m, E2M1).reshape(m.shape[0], -1, 2)
        parts += [(c[..., 0] | c[..., 1] << 4).reshape(-1), np.full(m.size // 16, 0x38, np.uint8)]
    return np.concatenate([*parts, np.array([1, 1, 0, 0], np.float32).view(np.uint8)])


def run(fmt, experts, x, ids, w):
    """experts: [(w13, w2)]; x: fp32 rows -> out, float64."""
    lib()
    rows = np.stack([encode(fmt, *e) for e in experts])
    H, I = experts[0][1].shape
    T, k = ids.shape
    pool, e2s = torch.from_numpy(rows).cuda(), torch.arange(len(experts), dtype=torch.int32, device="cuda")
    view = oes.routed_experts(0, len(experts), e2s, WFMT[fmt], pool, rows.shape[1], len(experts), H, I)
    nb = oes.moe_layer_few_tokens_workspace_size(view, T, k)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    xb = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    assert torch.equal(xb.cpu().float(), torch.from_numpy(x.astype(np.float32)))
    out = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    oes.moe_layer_few_tokens(view, xb, T, k, torch.from_numpy(ids.astype(np.int32)).cuda(),
                             torch.from_numpy(w.astype(np.float32)).cuda(), ws, nb, out, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out.double().cpu().numpy()


@pytest.mark.parametrize("H,I", [(128, 128), (64, 192), (192, 64)])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 12, 16])
@pytest.mark.parametrize("fmt", list(WFMT))
def test_h_keeps_its_bits(fmt, T, H, I):
    """h_i = 64 u_i, u_i a number of n bits (23; 22 for the 8- and 4-bit formats, what two f16 numbers hold)
    whose bits are the row's weights and whose places are x's powers of two, so that every sum is exact; a row of
    the output is the difference of two h that differ in their last bits, a number of eight bits: all exact."""
    n = 23 if fmt == "bf16" else 22
    g = rng(T + H)
    experts, u = [], []
    for _ in range(2):
        top = g.integers(1 << (n - 1), 1 << n, size=I) & ~127
        v = top + g.integers(0, 64, size=I)
        v[1::2] = top[::2] + g.integers(0, 64, size=(I + 1) // 2)[: len(v[1::2])]
        w13, w2 = np.zeros((2 * I, H)), np.zeros((H, I))
        w13[:I, n] = 4.0                                            # gate: 4 x_n = 64
        w13[I:, :n] = (v[:, None] >> np.arange(n - 1, -1, -1)) & 1
        pair = g.integers(0, I // 2, size=H)
        sign = g.choice([-1.0, 1.0], size=H)
        w2[np.arange(H), 2 * pair], w2[np.arange(H), 2 * pair + 1] = sign, -sign
        experts.append((w13, w2))
        u.append(v.astype(np.float64))
    x = np.zeros((T, H))
    x[:, n] = 16.0
    scale = 2.0 ** -(np.arange(T) % 4 + n - 1.0)                    # of u's last bit
    x[:, :n] = scale[:, None] * 2.0 ** np.arange(n - 1, -1, -1)
    ids = np.tile([0, 1], (T, 1))
    ids[T // 2] = [1, -1]
    w = np.tile([1.0, 2.0], (T, 1))
    want = np.zeros((T, H))
    for t, j in np.argwhere(ids >= 0):
        want[t] += w[t, j] * (experts[ids[t, j]][1] @ (64.0 * scale[t] * u[ids[t, j]]))
    assert np.array_equal(torch.from_numpy(want).to(torch.bfloat16).double().numpy(), want) and np.abs(want).max() > 0
    assert np.array_equal(run(fmt, experts, x, ids, w), want)


def test_sums_over_x_are_fp32():
    """1 and 255 x 64 numbers of 2^-28 (whose sixteens are half a unit of 1's last place) add up to 1 + 255 2^-22, as
    the other row has it from two numbers: their difference is 0."""
    H, I = 16384, 64
    x = np.full((1, H), 2.0 ** -14)
    x[0, 0], x[0, 2] = 1.0, 16.0
    w13, w2 = np.zeros((2 * I, H)), np.zeros((H, I))
    w13[:I, 2] = 4.0
    w13[I:, 0] = 1.0
    w13[I::2, 64:] = 2.0 ** -14
    w13[I + 1::2, 1] = 255 * 2.0 ** -8
    w2[:, 0], w2[:, 1] = 1.0, -1.0
    assert not run("bf16", [(w13, w2)], x, np.array([[0]]), np.ones((1, 1))).any()


def test_sums_over_h_are_fp32():
    """The same along I, as the difference of two experts."""
    H, I = 64, 4096
    x = np.zeros((1, H))
    x[0, 0], x[0, 2] = 1.0, 16.0
    w13 = np.zeros((2 * I, H))
    w13[:I, 2], w13[I:, 0] = 4.0, 1.0                               # h = 64
    a, b = np.zeros((H, I)), np.zeros((H, I))
    a[:, 0] = b[:, 0] = 1.0
    a[:, 64:] = 2.0 ** -28
    b[:, 1] = 63 * 2.0 ** -22
    assert not run("bf16", [(w13, a), (w13, b)], x, np.array([[0, 1]]), np.array([[1.0, -1.0]])).any()


@pytest.mark.parametrize("fmt", list(WFMT))
def test_an_infinite_h_stays_one(fmt):
    """h = 64 x 2^127 in one place: infinite results of its weights' signs, and not what its parts' differences are."""
    H, I = 256, 128
    x = np.zeros((2, H))
    x[:, 0], x[:, 200] = 2.0 ** 127, 16.0           # in different groups of 128
    w13, w2 = np.zeros((2 * I, H)), np.zeros((H, I))
    w13[:I, 200] = 4.0
    w13[I + 5, 0] = w13[I + 6, 200] = 1.0
    w2[:, 5] = np.where(np.arange(H) % 3, 1.0, -1.0)
    w2[:, 6] = 1.0
    out = run(fmt, [(w13, w2)], x, np.array([[0], [-1]]), np.ones((2, 1)))
    assert np.array_equal(out[0], w2[:, 5] * np.inf) and not out[1].any()
