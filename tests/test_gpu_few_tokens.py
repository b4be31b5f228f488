"""moe_layer_few_tokens against the layer in 64 bits: formats, sizes, masks,
routing, faults of the inputs, streams and graphs."""
import numpy as np
import pytest
import torch

from gpu_util import lib
from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.configs import C2, scaled
from offloaded_expert_slot_gb300.inputs import expert_layer_rows, rng
from oracle import expert_mlp, fp8
from oracle.router import route_topk

pytestmark = pytest.mark.gpu

WFMT = {"bf16": oes.OES_WFMT_BF16, "fp8": oes.OES_WFMT_FP8, "nvfp4": oes.OES_WFMT_NVFP4}


def weights_of(row, fmt, H, I):
    if fmt == "fp8":
        g, u, w2 = fp8.expert_weights(row, H, I)
        return np.concatenate([g, u]), w2
    return expert_mlp.expert_weights(row, fmt, H, I)


class Layer:
    """A layer's experts in a pool at shuffled slots, and the call's buffers."""

    def __init__(self, fmt, T, k, E, H, I, seed=0, extra_slots=3):
        lib()
        self.fmt, self.T, self.k, self.E, self.H, self.I = fmt, T, k, E, H, I
        cfg = scaled(C2, name="few", T=max(T, 1), k=k, E=E, H=H, I=I, S=E + extra_slots, L=1, prefill=0, wfmt=fmt,
                     seed=seed)
        self.rows = expert_layer_rows(cfg, 0).numpy()
        g = rng(seed + 1)
        self.S = E + extra_slots
        slots = g.permutation(self.S)[:E].astype(np.int32)
        pool = np.full((self.S, self.rows.shape[1]), 0x7F, np.uint8)       # slots without an expert: NaN patterns
        pool[slots] = self.rows
        self.pool, self.e2s = torch.from_numpy(pool).cuda(), torch.from_numpy(slots).cuda()
        self.x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
        self.view = oes.routed_experts(0, E, self.e2s, WFMT[fmt], self.pool, self.rows.shape[1], self.S, H, I)
        self.bytes = oes.moe_layer_few_tokens_workspace_size(self.view, T, k)
        self.ws = torch.full((self.bytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
        self.ids = torch.full((max(T, 1), k), -9, dtype=torch.int32, device="cuda")
        self.w = torch.zeros((max(T, 1), k), dtype=torch.float32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def set_routes(self, ids, w):
        self.ids.copy_(torch.from_numpy(np.asarray(ids, np.int32).reshape(self.T, self.k)))
        self.w.copy_(torch.from_numpy(np.asarray(w, np.float32).reshape(self.T, self.k)))

    def call(self, logits=None, stream=None):
        oes.moe_layer_few_tokens(self.view, self.x, self.T, self.k, self.ids, self.w, self.ws, self.bytes, self.out,
                                 self.status, logits=logits, stream=stream)

    def check(self, status=0, skip=()):
        """out against 64 bits, with the routing the call wrote or read.  Bound
        of each element: every fp32 sum of n products, in any order, is off by at
        most (n / 16 + 18) units of 2^-23 of the sum of the products' sizes (an
        instruction adds 16 of them at a time to the sum before, and sixteen warps'
        sums are added); silu is off by 17 x 2^-24 of itself and its slope is
        below 1.1; h rounds by half a step (of the second of two bf16 numbers; of f16,
        whose smallest steps are 2^-39 of the largest value nearby), and out."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        x = self.x.double().cpu().numpy()
        ids, w = self.ids.cpu().numpy(), self.w.double().cpu().numpy()
        H, I = self.H, self.I
        eh = 2.0 ** -16 if self.fmt == "bf16" else 2.0 ** -11
        e13, e2 = (H / 16 + 18) * 2.0 ** -23, (I / 16 + 18 + 4 * self.k) * 2.0 ** -23
        want, tol = np.zeros((self.T, H)), np.zeros((self.T, H))
        for e in np.unique(ids):
            if e < 0 or e >= self.E or e in skip:
                continue
            w13, w2 = weights_of(self.rows[e], self.fmt, H, I)
            for t, j in np.argwhere(ids == e):
                g, u = w13[:I] @ x[t], w13[I:] @ x[t]
                dg, du = (e13 * (np.abs(m) @ np.abs(x[t])) for m in (w13[:I], w13[I:]))
                s = expert_mlp.silu(g)
                h = s * u
                dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * (du + 20 * 2.0 ** -24 * np.abs(u))
                dh += eh * (np.abs(h) + dh) + 2.0 ** -38 * np.abs(h).max()
                want[t] += w[t, j] * (w2 @ h)
                tol[t] += abs(w[t, j]) * (np.abs(w2) @ (dh + e2 * (np.abs(h) + dh)))
        got = self.out[: self.T].double().cpu().numpy()
        tol += 2.0 ** -8 * (np.abs(want) + tol) + 1e-38
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
        # what is not the call's stays as it was
        assert bool((self.out[self.T:] == 7.0).all())
        assert bool((self.ws[self.bytes:] == 0xFF).all())
        return got


SIZES = [(1, 10, 64, 256, 128), (1, 1, 1, 64, 64), (3, 2, 8, 64, 192), (8, 4, 16, 1088, 704), (9, 3, 12, 192, 64),
         (16, 10, 24, 320, 448), (5, 6, 40, 2432, 64), (2, 8, 8, 128, 1024)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("fmt", list(WFMT))
def test_given_routes(fmt, size):
    T, k, E, H, I = size
    m = Layer(fmt, T, k, E, H, I, seed=hash(size) % 1000)
    g = rng(5)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    ids[g.random((T, k)) < 0.15] = -1
    m.set_routes(ids, g.random((T, k)) * 2 - 0.5)
    m.call()
    m.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt,T,k,E", [("fp8", 1, 10, 512), ("bf16", 4, 4, 33), ("nvfp4", 16, 8, 100), ("fp8", 9, 1, 7),
                                       ("bf16", 2, 3, 600), ("fp8", 16, 32, 64), ("nvfp4", 3, 2, 4096)])
def test_routed_from_logits(fmt, T, k, E, dtype):
    m = Layer(fmt, T, k, E, 128, 64, seed=E)
    logits = torch.from_numpy(rng(E + 1).standard_normal((T, E)).astype(np.float32))
    logits[:, E // 2:] = logits[:, : E - E // 2].flip(1)      # pairs of equal logits
    logits[0, 0] = float("nan")
    logits = logits.to(dtype).cuda()
    m.call(logits=logits)
    ids, w = torch.empty_like(m.ids), torch.empty_like(m.w)
    oes.moe_route_topk(logits, T, E, k, ids, w)
    m.check()
    assert torch.equal(ids, m.ids) and torch.equal(w, m.w)      # the router's, bit for bit


@pytest.mark.parametrize("E,k", [(512, 32), (512, 10), (40, 5), (33, 32), (5, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_odd_logits_are_routed_as_the_router_does(E, k, dtype):
    """Equal rows, rows with nothing, one or a few numbers above -inf, NaN rows, infinities, zeros of both signs,
    masks of the type's lowest value."""
    T = 12
    z = rng(21).standard_normal((T, E)).astype(np.float32)
    z[0] = 1.5
    z[1] = -np.inf
    z[2] = np.nan
    z[3] = -np.inf
    z[3, E - 1] = -3.0
    z[4, 2:] = -np.inf
    z[5, ::2] = np.inf
    z[6] = np.where(np.arange(E) % 3, 0.0, -0.0)
    z[7, 3:] = torch.finfo(dtype).min
    z[8, ::2] = np.nan
    z[9] = torch.finfo(dtype).min
    z[10] = np.arange(E) % 2
    logits = torch.from_numpy(z).to(dtype).cuda()
    m = Layer("fp8", T, k, E, 64, 64)
    m.call(logits=logits)
    ids, w = torch.empty_like(m.ids), torch.empty_like(m.w)
    oes.moe_route_topk(logits, T, E, k, ids, w)
    torch.cuda.synchronize()
    assert torch.equal(ids, m.ids) and torch.equal(w.view(torch.int32), m.w.view(torch.int32))


def test_routing_matches_the_oracle():
    m = Layer("fp8", 6, 8, 128, 64, 64)
    logits = rng(3).standard_normal((6, 128)).astype(np.float32)
    m.call(logits=torch.from_numpy(logits).cuda())
    torch.cuda.synchronize()
    ids, w = route_topk(logits, 8)
    assert np.array_equal(m.ids.cpu().numpy(), ids)
    assert np.abs(m.w.cpu().numpy() - w).max() <= 2e-6


@pytest.mark.parametrize("fmt", list(WFMT))
def test_masked_tokens_and_ids_out_of_range(fmt):
    """Tokens without a route get exact zeros; ids outside [0, E) count for nothing."""
    m = Layer(fmt, 11, 4, 9, 192, 128)
    g = rng(1)
    ids = g.integers(0, 9, size=(11, 4))
    ids[::3] = -1
    ids[1] = [9, -2 ** 31, 2 ** 31 - 1, 3]
    ids[4] = [12, -1, -7, 1 << 20]
    m.set_routes(ids, g.random((11, 4)))
    m.call()
    got = m.check()
    assert not got[::3].any() and not got[4].any() and got[1].any()
    m.set_routes(np.full((11, 4), -1), np.full((11, 4), np.nan))     # weights of absent routes are not used
    m.call()
    assert not m.check().any()


@pytest.mark.parametrize("fmt", list(WFMT))
def test_one_expert_many_times(fmt):
    """A token may list an expert several times, and all tokens the same ones."""
    m = Layer(fmt, 16, 32, 3, 128, 64)
    g = rng(2)
    ids = g.integers(0, 3, size=(16, 32))
    ids[3] = 2
    ids[4] = 2
    m.set_routes(ids, g.random((16, 32)) / 8)
    m.call()
    m.check()


def test_largest_tables():
    """512 routes to 512 experts: the most blocks a call can have."""
    m = Layer("nvfp4", 16, 32, 512, 64, 64)
    m.set_routes(rng(4).permutation(512).reshape(16, 32), rng(5).random((16, 32)))
    m.call()
    m.check()


@pytest.mark.parametrize("fmt,T,H", [("bf16", 16, 16384), ("fp8", 7, 16384), ("nvfp4", 16, 6144), ("bf16", 16, 4096),
                                     ("fp8", 16, 4736)])
def test_wide_rows(fmt, T, H):
    """Rows of x that do not fit beside the queues, or only beside short ones; tiles of several rows a CTA."""
    m = Layer(fmt, T, 2, 3, H, 64)
    ids = np.stack([rng(t).permutation(3)[:2] for t in range(T)])
    m.set_routes(ids, rng(6).random((T, 2)))
    m.call()
    m.check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("T,H,I", [(16, 128, 64), (9, 192, 1024), (16, 64, 4096)])
def test_experts_of_early_late_and_all_tokens(fmt, T, H, I):
    """Experts that only tokens before the ninth chose, only tokens from there on, both, and one token alone; a NaN
    of one token's row stays in its own result."""
    m = Layer(fmt, T, 3, 6, H, I)
    ids = np.array([[0 if t < 8 else 1, 2, 3 if t == 2 else 4 if t == 8 else 5 if t % 5 == 0 else -1] for t in range(T)])
    m.set_routes(ids, rng(12).random((T, 3)) + 0.1)
    m.call()
    m.check()
    clean = m.out.clone()
    m.x[T - 1, 5] = float("nan")
    m.call()
    torch.cuda.synchronize()
    assert torch.isnan(m.out[T - 1].float()).all()
    assert torch.equal(m.out[: T - 1], clean[: T - 1])


def test_wide_rows_from_logits_in_groups():
    m = Layer("bf16", 16, 2, 4, 16384, 64)
    logits = torch.from_numpy(rng(9).standard_normal((16, 4)).astype(np.float32)).cuda()
    m.call(logits=logits)
    m.check()


@pytest.mark.parametrize("fmt,I", [("bf16", 4096), ("fp8", 4160), ("nvfp4", 8192)])
def test_wide_experts(fmt, I):
    m = Layer(fmt, 2, 1, 2, 64, I)
    m.set_routes([[0], [1]], [[1.0], [0.5]])
    m.call()
    m.check()


@pytest.mark.parametrize("bad", [-1, 11, 1 << 30, -(1 << 31)])
def test_expert_without_a_slot(bad):
    m = Layer("fp8", 4, 3, 8, 128, 128)
    ids = np.array([[0, 1, 2], [3, 0, 1], [2, 2, 2], [7, 6, 5]])
    m.set_routes(ids, np.ones((4, 3)))
    m.e2s[2] = bad
    m.call()
    got = m.check(status=oes.OES_DEV_BAD_ID, skip=(2,))
    assert not got[2].any()


@pytest.mark.parametrize("fmt", list(WFMT))
def test_nan_stays_with_its_token(fmt):
    """A NaN in a token's row, and in an expert's weights, reaches the tokens that use them and no others."""
    m = Layer(fmt, 5, 2, 6, 128, 128)
    m.set_routes([[0, 1], [1, 2], [3, 4], [5, 3], [0, 4]], np.full((5, 2), 0.5))
    m.call()
    clean = m.check()
    m.x[1, 77] = float("nan")
    m.call()
    torch.cuda.synchronize()
    got = m.out[:5].double().cpu().numpy()
    assert np.isnan(got[1]).all()
    assert np.array_equal(got[[0, 2, 3, 4]], clean[[0, 2, 3, 4]])
    m.x[1, 77] = 0.0
    row = m.pool[int(m.e2s[5])]
    if fmt == "bf16":
        row.view(torch.bfloat16)[3] = float("nan")                   # gate, row 0
    elif fmt == "fp8":
        row[3] = 0x7F
    else:
        row[-16:-12].view(torch.float32)[0] = float("nan")           # the global scale of w13
    m.call()
    torch.cuda.synchronize()
    got = m.out[:5].double().cpu().numpy()
    assert np.isnan(got[3]).any()
    assert np.array_equal(got[[0, 2, 4]], clean[[0, 2, 4]])


@pytest.mark.parametrize("fmt", list(WFMT))
def test_large_values_keep_their_range(fmt):
    """Activations far beyond f16: 1e13 in, about 1e25 out."""
    m = Layer(fmt, 2, 1, 2, 128, 64)
    m.x.mul_(1e13)
    m.set_routes([[0], [1]], [[1.0], [1.0]])
    m.call()
    assert np.abs(m.check()).max() > 1e20


def test_no_tokens():
    m = Layer("fp8", 0, 2, 4, 64, 64)
    assert m.bytes == 0
    m.call()
    m.check()


def test_repeats_streams_and_shared_workspace():
    """Calls in a row over one workspace, on another stream, give the same bytes."""
    m = Layer("bf16", 8, 4, 32, 512, 256)
    logits = torch.from_numpy(rng(8).standard_normal((8, 32)).astype(np.float32)).cuda()
    m.call(logits=logits)
    want = m.check()
    n = Layer("fp8", 3, 2, 8, 128, 64, seed=4)
    n.ws, n.bytes = m.ws, m.bytes
    n.set_routes([[0, 1], [2, 3], [4, 5]], np.ones((3, 2)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            m.out.fill_(7.0)
            m.call(logits=logits)
            n.call()
    torch.cuda.synchronize()
    assert np.array_equal(m.check(), want)
    n.check()


def test_inputs_of_the_kernel_before():
    """Logits, ids and x written by the launches right before, call after call:
    nothing of an earlier call is read."""
    T, k, E, H = 4, 2, 16, 256
    m = Layer("bf16", T, k, E, H, 128)
    g = rng(11)
    xs = [torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(6)]
    gate = torch.from_numpy(g.standard_normal((H, E)).astype(np.float32)).to(torch.bfloat16).cuda()
    logits = torch.zeros((T, E), device="cuda")
    outs = []
    for x in xs:
        m.x.copy_(x)
        oes.moe_gate_logits(m.x, gate, T, H, E, logits)
        m.call(logits=logits)
        outs.append((m.out[:T].clone(), m.ids.clone(), m.w.clone()))
    for x, (out, ids, w) in zip(xs, outs):
        m.x.copy_(x)
        m.ids.copy_(ids)
        m.w.copy_(w)
        m.call()
        torch.cuda.synchronize()
        assert torch.equal(out, m.out[:T])
        m.check()


def test_graph_replay_on_new_tokens():
    """Captured once, replayed on other tokens, logits and a moved expert; a
    second graph shares the workspace."""
    T, k, E, H = 5, 3, 20, 320
    m = Layer("nvfp4", T, k, E, H, 192)
    n = Layer("fp8", 2, 2, 6, 128, 128, seed=3)
    n.ws, n.bytes = m.ws, m.bytes
    n.set_routes([[0, 1], [2, 3]], np.ones((2, 2)))
    logits = torch.zeros((T, E), device="cuda")
    m.call(logits=logits)
    n.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga, stream=s):
        m.call(logits=logits)
    with torch.cuda.graph(gb, stream=s):
        n.call()
    g = rng(12)
    for i in range(4):
        m.x.copy_(torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)))
        logits.copy_(torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)))
        if i == 2:      # expert 0 moves to the free slot
            free = (set(range(m.S)) - set(m.e2s.tolist())).pop()
            m.pool[free] = m.pool[int(m.e2s[0])]
            m.pool[int(m.e2s[0])] = 0x7F
            m.e2s[0] = free
        ga.replay()
        gb.replay()
        m.check()
        n.check()


@pytest.mark.parametrize("T", [1, 16])
def test_layers_in_a_row(T):
    """Each call's result is the next one's input, through one workspace, without a wait in between and from a
    graph, as with one."""
    k, E, H = 2, 8, 512
    a, b = Layer("bf16", T, k, E, H, 256), Layer("nvfp4", T, k, E, H, 128, seed=2)
    first, x, y = a.x.clone(), a.x.clone(), torch.empty_like(a.x)
    z = torch.from_numpy(rng(31).standard_normal((T, E)).astype(np.float32)).cuda()

    def run(wait):
        x.copy_(first)
        for _ in range(6):
            for m, i, o in ((a, x, y), (b, y, x)):
                oes.moe_layer_few_tokens(m.view, i, T, k, m.ids, m.w, a.ws, a.bytes, o, m.status, logits=z)
                if wait:
                    torch.cuda.synchronize()

    run(True)
    want = x.clone()
    run(False)
    torch.cuda.synchronize()
    assert torch.equal(x.view(torch.int16), want.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run(False)
    for _ in range(3):
        x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.view(torch.int16), want.view(torch.int16))


def test_two_calls_at_once():
    """Two streams, two workspaces, at the same time."""
    a, b = Layer("bf16", 8, 4, 24, 1024, 512), Layer("fp8", 16, 4, 24, 1024, 512, seed=5)
    for m in (a, b):
        m.set_routes(np.stack([rng(t).permutation(24)[:4] for t in range(m.T)]), rng(7).random((m.T, 4)))
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        a.call(stream=sa)
        b.call(stream=sb)
    a.check()
    b.check()


def test_beside_the_grouped_gemm():
    """The same layer through moe_grouped_gemm_slots: both within their bars of each other (bf16 weights)."""
    T, k, E, H, I = 12, 4, 32, 512, 256
    m = Layer("bf16", T, k, E, H, I)
    logits = torch.from_numpy(rng(13).standard_normal((T, E)).astype(np.float32)).cuda()
    m.call(logits=logits)
    got = m.check()
    B = oes.oes_tile_plan(T * k, E)
    cap = oes.align_capacity(T * k, E, B)

    def i32(n):
        return torch.empty(n, dtype=torch.int32, device="cuda")

    srt, blk, npad = i32(cap), i32(cap // B), i32(1)
    nb = oes.moe_align_workspace_size(T * k, E, B)
    aws = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")
    oes.moe_align_block_size(m.ids, T * k, E, B, 1, srt, blk, npad, m.status, aws, nb)
    gb = oes.moe_grouped_gemm_workspace_size(m.view, T, k)
    gws = torch.empty(gb, dtype=torch.uint8, device="cuda")
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    oes.moe_grouped_gemm_slots(m.view, m.x, T, k, m.ids, m.w, srt, blk, npad, B, gws, gb, out, m.status)
    torch.cuda.synchronize()
    other = out.double().cpu().numpy()
    assert np.linalg.norm(got - other) <= 5e-3 * np.linalg.norm(other)
