"""FP8 expert products with more units of work (block x weight tile) than a CTA
keeps in its table, in both kernels, unfiltered and filtered.

Checked against the same routes in calls small enough for the table, byte for
byte (each route's row y, from the workspace), and a few tokens against the
64-bit oracle within bf16's roundings of y and out and a rare code of h on the
other side of a midpoint: under 1 % of the norm together.
"""
import numpy as np
import pytest
import torch

from fp8_util import f64
from gpu_util import bits16, cuda, i32, lib, scratch, status
from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.configs import C2, scaled
from offloaded_expert_slot_gb300.inputs import expert_rows, f32_to_bf16_bits, rng
from oracle import fp8

pytestmark = pytest.mark.gpu

TABLE = 256       # units of a CTA's table
ROWS = 4          # different experts; the others are copies of them


def sizes(kernel, H, I):
    """(T, k, E) whose blocks x 128 tiles pass every CTA's table; H or I is 16384."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = TABLE * sms // 128 + 48
    if kernel == "weight-major":          # one block of 16 an expert
        return blocks, 1, blocks
    return 128 * (blocks // 16), 16, 16   # blocks of 128, every token through 16 experts


def inputs(T, k, E, H, I):
    cfg = scaled(C2, name="units", T=T, k=k, E=E, H=H, I=I, S=E, L=1, prefill=0, wfmt="fp8")
    g = rng(T + H)
    rows = expert_rows(cfg, 0, range(ROWS)).numpy()
    x = bits16(f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32)))
    ids = np.stack([np.roll(np.arange(E), t)[:k] for t in range(T)]).astype(np.int32)
    w = g.random((T, k)).astype(np.float32)
    return cfg, rows, x, ids, w


class Call:
    def __init__(self, cfg, rows, x, w):
        self.cfg, self.x, self.w = cfg, x, cuda(w.reshape(-1))
        self.pool = cuda(rows)
        self.e2s = cuda((np.arange(cfg.E) % ROWS).astype(np.int32))

    def run(self, ids):
        c = self.cfg
        R = c.T * c.k
        B = oes.oes_tile_plan(R, c.E)
        cap = oes.align_capacity(R, c.E, B)
        view = oes.routed_experts(0, c.E, self.e2s, oes.OES_WFMT_FP8, self.pool, c.row_bytes, ROWS, c.H, c.I)
        ab, gb = oes.moe_align_workspace_size(R, c.E, B), oes.moe_grouped_gemm_workspace_size(view, c.T, c.k)
        srt, be, npad, st, aws = i32(cap), i32(cap // B), i32(1), status(), scratch(ab)
        ws = torch.zeros(gb, dtype=torch.uint8, device="cuda")
        out = torch.zeros((c.T, c.H), dtype=torch.bfloat16, device="cuda")
        dids = cuda(ids.reshape(-1))
        oes.moe_align_block_size(dids, R, c.E, B, 1, srt, be, npad, st, aws, ab)
        oes.moe_grouped_gemm_slots(view, self.x, c.T, c.k, dids, self.w, srt, be, npad, B, ws, gb, out, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        o = oes.moe_grouped_gemm_workspace_views(view, c.T, c.k, ws)["y"] - ws.data_ptr()
        return out, ws[o:o + R * c.H * 2].view(torch.int16).reshape(R, c.H), int(npad.item()) // B, B


@pytest.mark.parametrize("H,I", [(16384, 64), (64, 16384)])
@pytest.mark.parametrize("kernel", ["weight-major", "token-major"])
def test_more_units_than_the_table(kernel, H, I):
    lib()
    T, k, E = sizes(kernel, H, I)
    cfg, rows, x, ids, w = inputs(T, k, E, H, I)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    call = Call(cfg, rows, x, w)
    out, y, blocks, B = call.run(ids)
    assert B == (16 if kernel == "weight-major" else 128)
    assert blocks * 128 > TABLE * sms
    for half in (0, 1):
        keep = (ids % 2) == half
        part, yp, n, _ = call.run(np.where(keep, ids, -1))
        assert n * 128 <= TABLE * sms
        at = torch.from_numpy(np.nonzero(keep.reshape(-1))[0]).cuda()
        assert torch.equal(y[at], yp[at])
        del yp
    xd = fp8.dequantize(*fp8.quantize(f64(x.view(torch.bfloat16)[[0, T // 2, T - 1]])))
    for i, t in enumerate((0, T // 2, T - 1)):
        want = sum(float(w[t, j]) * fp8.expert_mlp(xd[i:i + 1], rows[ids[t, j] % ROWS], H, I)[0] for j in range(k))
        got = f64(out[t])
        assert np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)


@pytest.mark.parametrize("kernel", ["weight-major", "token-major"])
def test_more_units_than_the_table_among_hits_and_misses(kernel):
    """The slot path, whose launches take the experts found and the experts copied
    apart, gives the streamed path's bytes: with every expert missing, with
    every expert found, and with some of each."""
    lib()
    H, I = 16384, 64
    T, k, E = sizes(kernel, H, I)
    cfg, rows, x, ids, w = inputs(T, k, E, H, I)
    src = torch.empty((E, cfg.row_bytes), dtype=torch.uint8, pin_memory=True)
    for e in range(E):
        src[e] = torch.from_numpy(rows[e % ROWS])
    source = oes.oes_expert_source_create([src, src], E, cfg.row_bytes)
    logits = torch.full((T, E), -30.0)
    logits.scatter_(1, torch.from_numpy(ids).long(), torch.from_numpy(w) * 4)
    logits = logits.cuda()
    desc = oes.layer_desc(E, H, I, oes.OES_WFMT_FP8)
    wsb = oes.moe_layer_workspace_size(desc, T, k)
    ws = scratch(wsb)

    def chunk():
        out, st = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), status()
        return oes.chunk(x, T, k, out, st, ws, wsb, logits=logits), out, st

    buf = torch.empty((E, cfg.row_bytes), dtype=torch.uint8, device="cuda")
    ch, want, st = chunk()
    oes.moe_layer_forward_stream(source, buf, 0, desc, ch, copy_stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and want.abs().max() > 0
    cache = oes.slot_cache_create(E + E // 4, 2, E)
    pool = torch.empty((E + E // 4, cfg.row_bytes), dtype=torch.uint8, device="cuda")
    # layer 0 missing, found; layer 1 missing (evicts most of layer 0); layer 0 part found
    for layer in (0, 0, 1, 0):
        ch, out, st = chunk()
        oes.moe_layer_forward_slots(cache, source, pool, layer, desc, ch, 1)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    oes.slot_cache_destroy(cache)
    oes.oes_expert_source_destroy(source)
