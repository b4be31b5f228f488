"""moe_int8_quantize and moe_int8_gemm: codes, scales and products against exact
integers, and a shared expert's products with the few-token layer beside them."""
import numpy as np
import pytest
import torch

from fp8_util import EPS32, f64, rows, strided
from gpu_util import lib
from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.inputs import rng
from oracle.expert_mlp import silu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    lib()


def quantize(x, K, act=oes.OES_ACT_NONE, q_pad=0, stream=None):
    """x: CUDA rows -> (codes [T, K], scales [T], the codes' whole buffer)."""
    T = x.shape[0]
    buf = torch.full((T + 1, K + q_pad), 99, dtype=torch.int8, device="cuda")
    s = torch.full((T + 1,), 5.0, dtype=torch.float32, device="cuda")
    oes.moe_int8_quantize(x, x.stride(0), T, K, act, buf, buf.stride(0), s, stream=stream)
    torch.cuda.synchronize()
    assert bool((buf[T] == 99).all()) and bool((buf[:, K:] == 99).all()) and float(s[T]) == 5.0
    return buf[:T, :K].cpu().numpy().astype(np.int64), s[:T].cpu().numpy()


def codes_of(v):
    """The definition, in 64 bits.  v: fp32 values.  127 v is exact in float64; its
    quotient by amax is a tie only if the real one is (any other is further from a
    tie than float64 rounds), so np.round decides as the real number does."""
    a = np.maximum(np.abs(v).max(1), 2.0 ** -100)
    return np.round(v * 127.0 / a[:, None]).astype(np.int64), (a.astype(np.float32) / np.float32(127.0))


SIZES = [(1, 1), (1, 2048), (3, 7), (5, 128), (2, 1999), (700, 256), (700, 2048), (640, 1000), (641, 33), (9, 2056),
         (4, 16384), (650, 5000), (2, 40000), (3, 9001)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_are_exact(size, dtype):
    T, K = size
    x = strided(rows(T, K, T + K), (T + K) % 3 * 4, dtype)
    q, s = quantize(x, K, q_pad=K % 5)
    want, scale = codes_of(f64(x))
    assert np.array_equal(q, want)
    assert np.array_equal(s, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_even(dtype):
    """amax = 127 2^e makes every odd multiple of 2^(e-1) a tie; bf16 numbers beside them are not."""
    for e in (-90, -3, 0, 60, 120):
        v = np.arange(-254, 255, dtype=np.float64) / 2
        v = np.concatenate([v, v * (1 + 2.0 ** -7), v * (1 - 2.0 ** -8)])
        v = v[np.abs(v) <= 127.0]
        x = torch.from_numpy((v * 2.0 ** e)[None, :].astype(np.float32)).to(dtype).cuda()
        x[0, 0] = 127.0 * 2.0 ** e
        q, s = quantize(x, x.shape[1])
        want, scale = codes_of(f64(x))
        assert np.array_equal(q, want) and np.array_equal(s, scale)


def test_next_to_ties():
    """fp32 values one unit on either side of a tie, for amax of all kinds."""
    g = rng(3)
    a = (1 + g.random((64, 1))).astype(np.float32)
    m = g.integers(0, 127, size=(64, 300))
    v = ((2 * m + 1) * a.astype(np.float64) / 254).astype(np.float32)
    v = np.concatenate([v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(0)), a], 1)
    x = torch.from_numpy(v * np.where(g.random(v.shape) < 0.5, -1, 1).astype(np.float32)).cuda()
    q, s = quantize(x, x.shape[1])
    want, scale = codes_of(f64(x))
    assert np.array_equal(q, want) and np.array_equal(s, scale)


def test_small_zero_and_odd_rows():
    x = torch.zeros((8, 300), device="cuda")
    x[1] = 2.0 ** -110
    x[2, 5] = -(2.0 ** -149)
    x[3, 7], x[3, 8] = float("nan"), 1.0
    x[4, 9], x[4, 1] = float("-inf"), 2.0
    x[5, 299] = 3.4e38
    x[5, 3] = -1.7e38
    x[6, 0] = -0.0
    x[7] = 2.0 ** -100
    q, s = quantize(x, 300)
    finite = [0, 1, 2, 5, 6, 7]
    want, scale = codes_of(f64(x)[finite])
    assert np.array_equal(q[finite], want) and np.array_equal(s[finite], scale)
    assert np.isnan(s[[3, 4]]).all() and not q[[3, 4]].any()


@pytest.mark.parametrize("T,K", [(1, 768), (32, 768), (700, 640), (5, 1001), (800, 77), (3, 12000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu(T, K, dtype):
    """v is off by at most 18 units of 2^-24 (silu 17, the product's rounding), so
    a ratio by twice that and the code by half a step more; scale by one more."""
    x = strided(rows(T, 2 * K, T * K, spread=False) * 2, (T % 2) * 8, dtype)
    q, s = quantize(x, K, act=oes.OES_ACT_SWIGLU)
    x = f64(x)
    v = silu(x[:, :K]) * x[:, K:]
    a = np.abs(v).max(1)
    r = 127.0 * v / a[:, None]
    assert np.all(np.abs(q - r) <= 0.5 + np.abs(r) * 38 * EPS32)
    assert np.all(np.abs(s - a / 127.0) <= a / 127.0 * 20 * EPS32)


def product(xq, xs, wq, ws, out_dtype):
    """fp32(sum) * xs * ws, each rounded, then to out's type: the definition bit for bit."""
    sums = xq.astype(np.float64) @ wq.astype(np.float64).T      # below 2^53: exact
    o = sums.astype(np.float32) * xs[:, None]
    return torch.from_numpy(o * ws[None, :]).to(out_dtype)


def gemm_inputs(T, K, N, seed, pad=0):
    g = rng(seed)

    def codes(n):
        ld = (K + 15) // 16 * 16 + pad
        b = torch.full((n, ld), 77, dtype=torch.int8)
        c = g.integers(-128, 128, size=(n, K)).astype(np.int8)
        b[:, :K] = torch.from_numpy(c)
        return b.cuda()[:, :K], c

    xq, xn = codes(T)
    wq, wn = codes(N)
    xs = (2.0 ** g.integers(-9, 4, size=T) * (1 + g.random(T))).astype(np.float32)
    ws = (2.0 ** g.integers(-12, 2, size=N) * (1 + g.random(N)) * g.choice([-1, 1], size=N)).astype(np.float32)
    return xq, xn, torch.from_numpy(xs).cuda(), xs, wq, wn, torch.from_numpy(ws).cuda(), ws


def run_gemm(xq, xs, wq, ws, K, out_dtype, out_pad=0, stream=None, work=None):
    T, N = xq.shape[0], wq.shape[0]
    nb = oes.moe_int8_gemm_workspace_size(T, K, N)
    work = torch.full((nb + 256,), 0x7F, dtype=torch.uint8, device="cuda") if work is None else work
    out = torch.full((T + 1, N + out_pad), 3.0, dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    oes.moe_int8_gemm(xq, xq.stride(0), xs, T, K, wq, wq.stride(0), ws, N, out, out.stride(0), work, nb, status,
                      stream=stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert bool((out[T] == 3.0).all()) and bool((out[:, N:] == 3.0).all())
    assert work.numel() > nb + 256 or bool((work[nb:] == 0x7F).all())
    return out[:T, :N].cpu()


# few rows: one token to 32, a chunk of K or many, tiles of one row to many, tiles of 32
# tokens; more rows: tiles of 64, 128 and 256 weight rows, one sum of 1024 of K or several
GEMMS = [(1, 1, 1), (1, 2048, 1536), (7, 100, 64), (8, 768, 2048), (9, 129, 300), (16, 4096, 200), (17, 1000, 333),
         (32, 768, 2048), (32, 1990, 77), (32, 4096, 500), (33, 64, 64), (1, 65536, 40), (5, 65536, 33), (20, 65536, 65),
         (200, 768, 2048), (129, 1025, 257), (601, 1999, 1001), (128, 2048, 128), (300, 63, 1500), (1, 127, 5000),
         (2, 3000, 40000), (1500, 1100, 4000), (40, 9000, 9001), (33, 2049, 1000), (100, 5000, 300), (4096, 250, 256), (255, 512, 512), (64, 700, 20000),
         (600, 1500, 2600), (257, 4100, 4100), (1030, 2050, 1700), (2049, 1500, 1030),
         (2100, 2100, 2500), (2305, 4096, 2047)]


@pytest.mark.parametrize("size", GEMMS, ids=str)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_are_exact(size, out):
    T, K, N = size
    xq, xn, xs, xsn, wq, wn, ws, wsn = gemm_inputs(T, K, N, T + K + N, pad=(K % 3) * 16)
    got = run_gemm(xq, xs, wq, ws, K, out, out_pad=N % 2 * 3)
    assert torch.equal(got, product(xn, xsn, wn, wsn, out))


@pytest.mark.parametrize("T", [3, 24, 150, 1300])
@pytest.mark.parametrize("K", [1024, 1025, 5000, 65536])
def test_largest_sums(T, K):
    """All codes -128, and rows that cancel after sums far past 2^24: exact all the same."""
    N = 4000 if T > 1000 else 70
    if K == 65536 and T > 1000:
        N = 4000
    x = torch.full((T, (K + 15) // 16 * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((N, (K + 15) // 16 * 16), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1::2, K // 2:] = 127
    x[:, K - 1] = 1
    ones = torch.ones(max(T, N), device="cuda")
    got = run_gemm(x, ones[:T], w, ones[:N], K, torch.float32)
    xn, wn = x[:1].cpu().numpy().astype(np.int64), w[:2].cpu().numpy().astype(np.int64)
    want = (xn @ wn.T).astype(np.float32)
    assert bool((got[:, 0::2] == float(want[0, 0])).all()) and bool((got[:, 1::2] == float(want[0, 1])).all())


def test_scales_of_any_value():
    xq, xn, xs, xsn, wq, wn, ws, wsn = gemm_inputs(40, 320, 130, 1)
    xs[3], xs[4], ws[7] = float("nan"), 0.0, float("inf")
    xsn, wsn = xs.cpu().numpy(), ws.cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = product(xn, xsn, wn, wsn, torch.float32)
    for T in (5, 40):
        got = run_gemm(xq[:T], xs[:T], wq, ws, 320, torch.float32)
        assert torch.equal(torch.isnan(got), torch.isnan(want[:T]))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want[:T]))


def test_unaligned_output_rows():
    xq, xn, xs, xsn, wq, wn, ws, wsn = gemm_inputs(1400, 256, 300, 2)
    for T in (6, 140, 1400):
        nb = oes.moe_int8_gemm_workspace_size(T, 256, 300)
        work = torch.empty(nb + 1, dtype=torch.uint8, device="cuda")
        flat = torch.full((T * 301 + 7,), 3.0, dtype=torch.bfloat16, device="cuda")
        oes.moe_int8_gemm(xq, xq.stride(0), xs, T, 256, wq, wq.stride(0), ws, 300, flat[1:], 301, work, nb)
        got = flat[1:1 + T * 301].view(T, 301)
        assert torch.equal(got[:, :300].cpu(), product(xn[:T], xsn[:T], wn, wsn, torch.bfloat16))
        assert float(flat[0]) == 3.0 and bool((got[:, 300] == 3.0).all()) and bool((flat[1 + T * 301:] == 3.0).all())


def test_no_rows():
    e = torch.empty(0, device="cuda")
    oes.moe_int8_gemm(0, 16, 0, 0, 16, 0, 16, 0, 4, e, 4)
    oes.moe_int8_quantize(e, 16, 0, 16, 0, 0, 16, 0)
    assert oes.moe_int8_gemm_workspace_size(0, 16, 4) == 0


def test_streams_and_two_calls_at_once():
    a, b = gemm_inputs(900, 768, 2048, 5), gemm_inputs(700, 640, 3000, 6)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    keep = []
    for _ in range(5):
        for s, m, (T, K, N) in ((sa, a, (900, 768, 2048)), (sb, b, (700, 640, 3000))):
            with torch.cuda.stream(s):
                nb = oes.moe_int8_gemm_workspace_size(T, K, N)
                work = torch.empty(nb, dtype=torch.uint8, device="cuda")
                out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
                oes.moe_int8_gemm(m[0], m[0].stride(0), m[2], T, K, m[4], m[4].stride(0), m[6], N, out, N, work, nb)
                keep.append(work)
                outs.append((m, out))
    torch.cuda.synchronize()
    for m, out in outs:
        assert torch.equal(out.cpu(), product(m[1], m[3], m[5], m[7], torch.bfloat16))


@pytest.mark.parametrize("T", [1, 32, 200, 1500])
def test_linear_replayed_from_a_graph(T):
    """Rows to codes and the product, captured once and replayed on new rows; two
    graphs share the workspace."""
    K, N = 1024, 768
    g = rng(T)
    _, _, _, _, wq, wn, ws, wsn = gemm_inputs(1, K, N, 9)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    nb = oes.moe_int8_gemm_workspace_size(T, K, N)
    work = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")

    def step():
        oes.moe_int8_quantize(x, K, T, K, 0, q, K, s)
        oes.moe_int8_gemm(q, K, s, T, K, wq, wq.stride(0), ws, N, out, N, work, nb)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    for i in range(4):
        x.copy_(torch.from_numpy(g.standard_normal((T, K)).astype(np.float32)))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        want, scale = codes_of(f64(x))
        assert torch.equal(out.cpu(), product(want, scale, wn, wsn, torch.bfloat16))


@pytest.mark.parametrize("T", [1, 5, 16])
def test_decode_block(T):
    """A decode step's MoE block, its operators run one after another: norm, router
    logits, the routed experts (moe_layer_few_tokens) and an int8 shared expert
    beside them, residual update.  Against 64 bits, by the sizes of the roundings:
    u 2^-8 and out 2^-8 in bf16, h 2^-8, codes 1/254 of a row's largest value, which
    is at most 8 sigma of the values here."""
    from test_gpu_few_tokens import Layer, weights_of
    k, E, H, I, J = 4, 16, 512, 256, 384
    m = Layer("fp8", T, k, E, H, I)
    g = rng(T)

    def bf(*shape, std=1.0):
        return torch.from_numpy((g.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16).cuda()

    r, y, gate, pre = bf(T, H), bf(T, H), bf(H, E, std=0.05), bf(H, std=0.1) + 1
    w13, w2 = bf(2 * J, H, std=0.04).float(), bf(H, J, std=0.04).float()
    q13, s13 = (torch.empty((2 * J, H), dtype=torch.int8, device="cuda"), torch.empty(2 * J, device="cuda"))
    q2, s2 = (torch.empty((H, J), dtype=torch.int8, device="cuda"), torch.empty(H, device="cuda"))
    oes.moe_int8_quantize(w13, H, 2 * J, H, 0, q13, H, s13)       # weights: a scale for each channel
    oes.moe_int8_quantize(w2, J, H, J, 0, q2, J, s2)
    r0 = f64(r)
    logits = torch.empty((T, E), device="cuda")
    xq, xs = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    hq, hs = torch.empty((T, J), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    h13, s = torch.empty((T, 2 * J), dtype=torch.float32, device="cuda"), bf(T, H)
    nb = max(oes.moe_int8_gemm_workspace_size(T, H, 2 * J), oes.moe_int8_gemm_workspace_size(T, J, H))
    work = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
    n1 = oes.block_norm(T, H, r, y=y, pre_weight=pre, out_residual=r, out=m.x)
    n2 = oes.block_norm(T, H, r, y=m.out, out_residual=r)
    n3 = oes.block_norm(T, H, r, y=s, out_residual=r)
    oes.moe_block_norm(n1)
    oes.moe_gate_logits(m.x, gate, T, H, E, logits)
    m.call(logits=logits)
    oes.moe_int8_quantize(m.x, H, T, H, 0, xq, H, xs)
    oes.moe_int8_gemm(xq, H, xs, T, H, q13, H, s13, 2 * J, h13, 2 * J, work, nb)
    oes.moe_int8_quantize(h13, 2 * J, T, J, oes.OES_ACT_SWIGLU, hq, J, hs)
    oes.moe_int8_gemm(hq, J, hs, T, J, q2, J, s2, H, s, H, work, nb)
    oes.moe_block_norm(n2)
    oes.moe_block_norm(n3)
    routed = m.check()
    u = f64(m.x)
    r1 = r0 + f64(y)
    uw = r1 / np.sqrt((r1 * r1).mean(1, keepdims=True) + 1e-6) * f64(pre)
    assert np.all(np.abs(u - uw) <= 2.0 ** -8 * np.abs(uw) + 2.0 ** -7 * np.abs(uw))   # r1 rounded, then u
    # the shared expert from its own codes, in 64 bits
    def deq(q, sc):
        return q.cpu().numpy().astype(np.float64) * f64(sc)[:, None]
    a = deq(xq, xs) @ deq(q13, s13).T
    assert np.all(np.abs(f64(h13) - a) <= 4 * EPS32 * np.abs(a) + 1e-30)
    sh = deq(hq, hs) @ deq(q2, s2).T
    assert np.all(np.abs(f64(s) - sh) <= (2.0 ** -8 + 4 * EPS32) * np.abs(sh))
    # and against the unquantised expert: each code is off by at most half a step
    full = (silu(u @ f64(w13)[:J].T) * (u @ f64(w13)[J:].T)) @ f64(w2).T
    assert np.linalg.norm(sh - full) <= 0.05 * np.linalg.norm(full)
    r_want = r1 + routed + f64(s)
    tol = 2.0 ** -8 * (np.abs(r1) + np.abs(r1 + routed) + np.abs(r_want)) * 1.02
    assert np.all(np.abs(f64(r) - r_want) <= tol)
