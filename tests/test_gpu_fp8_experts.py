"""The FP8 expert format: the grouped GEMM, step by step and end to end,
against the 64-bit oracle, and the layer paths over it.

Tolerances (u = 2^-24): the sums of one product are within
2 (128 + nkb + 4) u S of the exact ones, S = sum |x| |w|; h = silu(g) u then
within |h| 16 u plus what the sums' errors give (|silu'| <= 1.1); its codes
are nearest codes of ratios that far off.  y is checked from the GPU's own
codes of h, so a code on the other side of a midpoint does not count twice.
out adds each route's bf16 y (2^-8) and its own rounding (2^-8).
"""
import numpy as np
import pytest
import torch

from fp8_util import EPS32, f64
from gpu_util import Workload, bits16, cuda, i32, lib, scratch, status
from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.configs import C2, C5, scaled
from offloaded_expert_slot_gb300.inputs import expert_rows, f32_to_bf16_bits, rng
from oracle import fp8

pytestmark = pytest.mark.gpu


def case(name, T, k, E, H, I, **kw):
    return scaled(C2, name=name, T=T, k=k, E=E, H=H, I=I, S=kw.pop("S", E + 3), L=kw.pop("L", 1),
                  prefill=kw.pop("prefill", 0), wfmt="fp8", **kw)


def sum_tol(K):
    return 2 * (128 + -(-K // 128) + 4) * EPS32


class Experts:
    """A pool of random experts in shuffled slots and one call of the grouped GEMM over it."""

    def __init__(self, cfg, ids=None, seed=3):
        lib()
        self.cfg = cfg
        g = rng(seed)
        T, k, E, H, I = cfg.T, cfg.k, cfg.E, cfg.H, cfg.I
        self.rows = expert_rows(cfg, 0, range(E)).numpy()
        self.slot = g.permutation(cfg.S)[:E].astype(np.int32)
        pool = np.full((cfg.S, cfg.row_bytes), 0x7F, np.uint8)
        pool[self.slot] = self.rows
        self.pool, self.e2s = cuda(pool), cuda(self.slot)
        x = g.standard_normal((T, H)) * 2.0 ** g.integers(-3, 4, size=(T, 1))
        self.x = bits16(f32_to_bf16_bits(x.astype(np.float32)))
        self.x64 = f64(self.x.view(torch.bfloat16))
        if ids is None:
            ids = np.stack([g.permutation(E)[:k] for _ in range(max(T, 1))])[:T]
        self.ids = np.ascontiguousarray(ids, np.int32).reshape(T, k)
        self.w = g.random((T, k)).astype(np.float32)

    def run(self, stream=None, e2s=None):
        cfg = self.cfg
        T, k, E, H, I = cfg.T, cfg.k, cfg.E, cfg.H, cfg.I
        R = T * k
        self.B = B = oes.oes_tile_plan(R, E)
        self.cap = cap = oes.align_capacity(R, E, B)
        ids, w = cuda(self.ids.reshape(-1)) if R else i32(1), cuda(self.w.reshape(-1)) if R else i32(1)
        st = status()
        self.sorted, be, npad = i32(cap), i32(max(cap // B, 1)), i32(1)
        wsb = oes.moe_align_workspace_size(R, E, B)
        aws = scratch(wsb)
        view = oes.routed_experts(0, E, self.e2s if e2s is None else e2s, oes.OES_WFMT_FP8, self.pool,
                                  cfg.row_bytes, cfg.S, H, I)
        self.gb = oes.moe_grouped_gemm_workspace_size(view, T, k)
        self.ws = torch.full((max(self.gb, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        self.views = oes.moe_grouped_gemm_workspace_views(view, T, k, self.ws)
        buf = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        oes.moe_align_block_size(ids, R, E, B, 1, self.sorted, be, npad, st, aws, wsb, stream=stream)
        oes.moe_grouped_gemm_slots(view, self.x, T, k, ids, w, self.sorted, be, npad, B, self.ws, self.gb,
                                   buf[1:T + 1], st, stream=stream)
        torch.cuda.synchronize()
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        self.status = int(st.item())
        return buf[1:T + 1]

    def part(self, ptr, nbytes, dtype, shape):
        o = ptr - self.ws.data_ptr()
        return self.ws[o:o + nbytes].cpu().numpy().view(dtype).reshape(shape)

    def steps(self):
        """(x codes, x scales, h codes, h scales, y) of the last call."""
        cfg = self.cfg
        T, H, I, cap, R = cfg.T, cfg.H, cfg.I, self.cap, cfg.T * cfg.k
        up = lambda n: (n + 255) // 256 * 256  # noqa: E731
        hb, ib = -(-H // 128), -(-I // 128)
        v = self.views
        return (self.part(v["x16"], T * H, np.uint8, (T, H)),
                self.part(v["x16"] + up(T * H), T * hb * 4, np.float32, (T, hb)),
                self.part(v["h"], cap * I, np.uint8, (cap, I)),
                self.part(v["h"] + up(cap * I), cap * ib * 4, np.float32, (cap, ib)),
                self.ws[v["y"] - self.ws.data_ptr():][:R * H * 2].view(torch.bfloat16).reshape(R, H))

    def check(self, out):
        cfg = self.cfg
        k, H, I = cfg.k, cfg.H, cfg.I
        val = fp8.e4m3_values()
        qx, sx, qh, sh, y = self.steps()
        want_q, want_s = fp8.quantize(self.x64)
        assert np.array_equal(val[qx], want_q)
        assert np.allclose(sx, want_s, rtol=2 * EPS32, atol=0)
        xd = fp8.dequantize(want_q, sx.astype(np.float64))
        place = {int(r): i for i, r in enumerate(self.sorted.cpu().numpy()) if r < cfg.T * k}
        y64 = f64(y)
        total, big = np.zeros((cfg.T, H)), np.zeros((cfg.T, H))
        for e in range(cfg.E):
            t, j = np.nonzero(self.ids == e)
            if not len(t):
                continue
            gate, up, w2 = fp8.expert_weights(self.rows[e], H, I)
            gv, uv = xd[t] @ gate.T, xd[t] @ up.T
            gt, ut = sum_tol(H) * (np.abs(xd[t]) @ np.abs(gate).T), sum_tol(H) * (np.abs(xd[t]) @ np.abs(up).T)
            h = gv / (1 + np.exp(-gv)) * uv
            err = np.abs(h) * 16 * EPS32 + 1.1 * gt * (np.abs(uv) + ut) + np.abs(gv) * ut
            at = [place[int(a) * k + int(b)] for a, b in zip(t, j)]
            a = fp8.group_amax(h)
            e_rel = (fp8.group_amax(err) / a).max()
            s = sh[at].astype(np.float64)
            assert np.all(np.abs(s - a / 448) <= fp8.group_amax(err) / 448 + a / 448 * 4 * EPS32)
            r = fp8.ratios(h)
            d = 448 * err / fp8.spread(a, I) + np.abs(r) * (e_rel + 8 * EPS32)
            q = val[qh[at]]
            assert np.all(np.abs(q - r) <= 0.5 * fp8.e4m3_step(np.abs(r) + d) + d)
            hd = fp8.dequantize(q, s)
            yw, yb = hd @ w2.T, np.abs(hd) @ np.abs(w2).T
            got = y64[t * k + j]
            assert np.all(np.abs(got - yw) <= sum_tol(I) * yb + np.abs(yw) * 2.0 ** -8 + 1e-37)
            wj = self.w[t, j].astype(np.float64)[:, None]
            np.add.at(total, t, wj * got)
            np.add.at(big, t, np.abs(wj * got))
        o = f64(out)
        assert np.all(np.abs(o - total) <= big * (k + 2) * EPS32 + np.abs(total) * 2.0 ** -8 + 1e-37)


CASES = [case("one_token", 1, 4, 16, 256, 192), case("one_route", 1, 1, 1, 128, 64),
         case("few", 7, 3, 16, 192, 320), case("swap", 40, 3, 16, 256, 192),
         case("narrow", 5, 2, 8, 64, 64), case("wide_blocks", 160, 8, 12, 128, 128),
         case("ragged", 96, 4, 16, 320, 192), case("one_expert", 300, 1, 1, 256, 128),
         case("two_full_blocks", 256, 1, 1, 128, 320), case("long_k", 3, 2, 4, 4096, 128),
         case("long_i", 130, 2, 4, 128, 2048), case("many_units", 64, 8, 64, 1152, 384),
         # K shared by a cluster in both products, blocks part full and full
         case("shared_k", 3, 2, 4, 1600, 2048), case("shared_k_full", 16, 1, 1, 2048, 1600),
         case("shared_k_two", 24, 2, 8, 1536, 1536)]


@pytest.mark.parametrize("cfg", CASES, ids=lambda c: c.name)
def test_grouped_gemm(cfg):
    e = Experts(cfg)
    out = e.run()
    assert e.status == 0
    e.check(out)


@pytest.mark.parametrize("T", [8, 80])
def test_masked_routes_and_empty_rows(T):
    """Routes with ids out of range give nothing; a token with none left gives zeros."""
    cfg = case("masked", T, 3, 8, 192, 128)
    g = rng(1)
    ids = np.stack([g.permutation(cfg.E)[:3] for _ in range(T)])
    ids[g.random(ids.shape) < 0.3] = -1
    ids[2] = -1
    ids[5] = [cfg.E, 1, 2 ** 30]
    e = Experts(cfg, ids=ids)
    out = e.run()
    assert e.status == 0 and not out[2].any()
    e.check(out)


@pytest.mark.parametrize("T", [6, 90])
def test_all_routes_on_one_expert(T):
    cfg = case("hot", T, 1, 32, 256, 192)
    e = Experts(cfg, ids=np.full((T, 1), 17))
    e.check(e.run())


@pytest.mark.parametrize("T", [4, 64])
def test_expert_without_a_slot_gives_zeros_and_a_status(T):
    cfg = case("missing", T, 2, 4, 192, 320)
    ids = np.tile([0, 3], (T, 1))
    e = Experts(cfg, ids=ids)
    full = e.run().clone()
    assert e.status == 0
    e2s = e.e2s.clone()
    e2s[3] = -1
    out = e.run(e2s=e2s)
    assert e.status == oes.OES_DEV_BAD_ID
    keep = Experts(cfg, ids=np.tile([0, -1], (T, 1)))
    keep.w = e.w
    assert torch.equal(out, keep.run()) and not torch.equal(out, full)


@pytest.mark.parametrize("T", [8, 128])
def test_the_slots_do_not_change_a_bit_and_calls_repeat(T):
    """Slots, streams and what else the pool holds change no bit of the result."""
    cfg = case("slots", T, 4, 16, 512, 256, S=40)
    a = Experts(cfg)
    first = a.run().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(a.run(stream=side), first)
    pool = np.zeros((cfg.S, cfg.row_bytes), np.uint8)
    order = rng(77).permutation(cfg.S)[:cfg.E].astype(np.int32)
    pool[order] = a.rows
    a.pool, a.e2s = cuda(pool), cuda(order)
    assert torch.equal(a.run(), first)


def test_pool_past_4_gib():
    """Slots whose bytes lie past 2^32: 64-bit offsets."""
    cfg = case("far", 16, 2, 4, 2048, 768)
    e = Experts(cfg)
    near = e.run().clone()
    S = (1 << 32) // cfg.row_bytes + 40
    pool = torch.empty((S, cfg.row_bytes), dtype=torch.uint8, device="cuda")
    slots = np.array([S - 1, S - 30, 3, S - 17], np.int32)
    pool[torch.from_numpy(slots).long().cuda()] = cuda(e.rows)
    e.pool, e.e2s, e.cfg = pool, cuda(slots), scaled(cfg, S=S)
    assert torch.equal(e.run(), near)
    assert e.status == 0


@pytest.mark.parametrize("T", [5, 70])
def test_nan_and_infinity_stay_with_their_token(T):
    cfg = case("nan", T, 2, 4, 256, 192)
    e = Experts(cfg)
    clean = e.run().clone()
    e.x[1, 7] = 0x7FC0            # NaN
    e.x[3, 200] = 0x7F80          # infinity
    out = e.run()
    assert e.status == 0
    bad = torch.isnan(out.float()).any(1)
    assert bad[1] and bad[3] and int(bad.sum()) == 2
    keep = ~bad
    assert torch.equal(out[keep], clean[keep])


def test_no_tokens():
    cfg = case("none", 0, 2, 4, 256, 192)
    lib()
    view = oes.routed_experts(0, 4, 16, oes.OES_WFMT_FP8, 16, cfg.row_bytes, cfg.S, 256, 192)
    oes.moe_grouped_gemm_slots(view, 16, 0, 2, 16, 16, 16, 16, 16, oes.oes_tile_plan(0, 4), 256, 1 << 20, 16, 0)
    torch.cuda.synchronize()


# ------------------------------------------------------------- layer paths
def layer_desc(cfg):
    return oes.layer_desc(cfg.E, cfg.H, cfg.I, oes.OES_WFMT_FP8)


def chunk_of(w, desc, logits=None):
    cfg = w.cfg
    wsb = oes.moe_layer_workspace_size(desc, cfg.T, cfg.k)
    ws = scratch(wsb)
    out = torch.zeros((cfg.T, cfg.H), dtype=torch.bfloat16, device="cuda")
    st = status()
    return oes.chunk(w.x, cfg.T, cfg.k, out, st, ws, wsb, logits=w.logits if logits is None else logits), out, st, ws


LAYERS = [case("decode", 4, 3, 16, 256, 192, S=24, L=2, prefill=14),
          case("swap", 40, 3, 16, 256, 192, S=40, L=2, prefill=20),
          case("blocks", 96, 4, 16, 320, 128, S=40, L=2, prefill=20),
          case("queries", 120, 4, 300, 128, 64, S=320, L=2, prefill=100)]


def oracle_layer(w, layer):
    cfg = w.cfg
    x = fp8.dequantize(*fp8.quantize(f64(w.x.view(torch.bfloat16))))
    lg = w.rin["logits"].astype(np.float64)
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :cfg.k]
    top = np.take_along_axis(lg, ids, 1)
    p = np.exp(top - top.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out = np.zeros((cfg.T, cfg.H))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        out_e = fp8.expert_mlp(x[t], w.source_row(layer, e), cfg.H, cfg.I)
        np.add.at(out, t, p[t, j][:, None] * out_e)
    return out


@pytest.mark.parametrize("cfg", LAYERS, ids=lambda c: c.name)
def test_slot_path_streamed_path_and_staged_layers_agree(cfg):
    """Byte for byte with one another; against the oracle within the bf16
    roundings of y and out (2^-8 each) and a rare code of h on the
    other side of a midpoint, under 1 % of the norm together."""
    lib()
    w = Workload(cfg, gen_device="cpu", extra_rows=2 * cfg.E)
    desc = layer_desc(cfg)
    buf = torch.empty((cfg.E, cfg.row_bytes), dtype=torch.uint8, device="cuda")
    streamed = []
    for layer in range(cfg.L):
        ch, out, st, ws = chunk_of(w, desc)
        oes.moe_layer_forward_stream(w.src, buf, layer, desc, ch, copy_stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        streamed.append(out)
        want = oracle_layer(w, layer)
        err = np.linalg.norm(f64(out) - want) / np.linalg.norm(want)
        assert err <= 1e-2, err
    plan = oes.oes_stage_plan_create(w.cache, [0, 1], True)
    cs = [chunk_of(w, desc) for _ in range(2)]
    oes.moe_layers_forward_staged(plan, w.src, w.pool_all, desc, [c[0] for c in cs],
                                  copy_stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for layer in range(2):
        assert int(cs[layer][2].item()) == 0
        assert torch.equal(cs[layer][1].view(torch.int16), streamed[layer].view(torch.int16))
    oes.oes_stage_plan_destroy(plan)
    for layer in (0, 1, 0):
        ch, out, st, ws = chunk_of(w, desc)
        oes.moe_layer_forward_slots(w.cache, w.src, w.pool, layer, desc, ch, 1)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert torch.equal(out.view(torch.int16), streamed[layer].view(torch.int16))
    w.close()


def test_decode_step_in_a_graph():
    lib()
    cfg = LAYERS[0]
    w = Workload(cfg, gen_device="cpu")
    desc = layer_desc(cfg)
    ch, out, st, ws = chunk_of(w, desc)
    oes.moe_layer_forward_slots(w.cache, w.src, w.pool, 0, desc, ch, 1)
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oes.moe_layer_forward_slots(w.cache, w.src, w.pool, 0, desc, ch, 1)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and int(st.item()) == 0
    w.close()
