"""An MoE block with 8-bit experts, run through the library's calls as a model
would: the norms around it, the router, the routed experts over the slot cache
and a shared expert beside them.

One step, for the residual stream r and the output a of the block before:

    r, u, uq = moe_block_norm       r += post_norm(a);  u = pre_norm(r), and u in 8 bits
    logits   = moe_gate_logits      the router's, and one gate a token for the shared expert
    e        = moe_layer_forward_slots   routed experts (OES_WFMT_FP8) from the slot cache
    s        = moe_fp8_gemm, moe_fp8_quantize (SwiGLU), moe_fp8_gemm
    r        = moe_block_norm       r += sigmoid(gate) s
    r, u'    = moe_block_norm       r += scale * post_norm(e);  u' = pre_norm(r) of the next block

`python -m offloaded_expert_slot_gb300.fp8_block` runs a small block on the
GPU, checks it against the same steps in 64 bits on the CPU (the `oracle`
package) and times it.
"""
from __future__ import annotations

import numpy as np
import torch

from . import oes
from .configs import C2, LayerConfig, scaled
from .inputs import expert_layer_rows, quantize_fp8_blocks

EPS = 1e-6
SCALE = 0.5          # of the routed experts' update


def small_config(T: int = 40) -> LayerConfig:
    return scaled(C2, name="fp8_block", T=T, k=4, E=16, H=512, I=256, S=24, L=1, prefill=0, wfmt="fp8")


class Fp8Block:
    """Weights, slot cache and buffers of one block; step() runs it."""

    def __init__(self, cfg: LayerConfig, shared_I: int | None = None, seed: int = 0):
        oes.load()
        self.cfg = cfg
        T, k, E, H, I = cfg.T, cfg.k, cfg.E, cfg.H, cfg.I
        self.shared_I = J = shared_I or I
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16

        def randn(*shape, std=0.02):
            return (torch.randn(*shape, generator=g) * std).cuda()

        self.post_a, self.pre_u, self.post_e, self.pre_next = [(1 + randn(H, std=0.1)).to(bf) for _ in range(4)]
        self.gate, self.shared_gate = randn(H, E).to(bf), randn(H, 1).to(bf)
        self.s13, self.s13_scale = quantize_fp8_blocks(randn(2 * J, H))
        self.s2, self.s2_scale = quantize_fp8_blocks(randn(H, J))
        self.rows = expert_layer_rows(cfg, 0).pin_memory()
        self.source = oes.oes_expert_source_create([self.rows], E, cfg.row_bytes)
        self.cache = oes.slot_cache_create(cfg.S, 1, E)
        self.pool = torch.empty((cfg.S, cfg.row_bytes), dtype=torch.uint8, device="cuda")
        self.desc = oes.layer_desc(E, H, I, oes.OES_WFMT_FP8)
        wsb = oes.moe_layer_workspace_size(self.desc, T, k)
        self.ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")

        def new(shape, dtype=bf):
            return torch.empty(shape, dtype=dtype, device="cuda")

        hb, jb = -(-H // 128), -(-J // 128)
        self.r, self.a, self.u, self.e = new((T, H)), new((T, H)), new((T, H)), new((T, H))
        self.uq, self.us = new((T, H), torch.uint8), new((T, hb), torch.float32)
        self.logits, self.token_gate = new((T, E), torch.float32), new((T, 1), torch.float32)
        self.h13, self.hq, self.hs = new((T, 2 * J)), new((T, J), torch.uint8), new((T, jb), torch.float32)
        self.s, self.u_next = new((T, H)), new((T, H))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.chunk = oes.chunk(self.u, T, k, self.e, self.status, self.ws, wsb, logits=self.logits)
        self.n1 = oes.block_norm(T, H, self.r, y=self.a, post_weight=self.post_a, pre_weight=self.pre_u, eps=EPS,
                                 out_residual=self.r, out=self.u, out_q=self.uq, out_scale=self.us)
        self.n2 = oes.block_norm(T, H, self.r, y=self.s, gate=self.token_gate, gate_kind=oes.OES_GATE_TOKEN,
                                 gate_ld=1, gate_sigmoid=True, eps=EPS, out_residual=self.r)
        self.n3 = oes.block_norm(T, H, self.r, y=self.e, post_weight=self.post_e, pre_weight=self.pre_next,
                                 residual_scale=SCALE, eps=EPS, out_residual=self.r, out=self.u_next)

    def step(self, stream=None):
        """One step over the residual in self.r and the previous block's output
        in self.a; leaves the residual in self.r and its norm in self.u_next."""
        c, J = self.cfg, self.shared_I
        T, H = c.T, c.H
        oes.moe_block_norm(self.n1, stream=stream)
        oes.moe_gate_logits(self.u, self.gate, T, H, c.E, self.logits, stream=stream)
        oes.moe_gate_logits(self.u, self.shared_gate, T, H, 1, self.token_gate, stream=stream)
        oes.moe_layer_forward_slots(self.cache, self.source, self.pool, 0, self.desc, self.chunk, 1, stream=stream)
        oes.moe_fp8_gemm(self.uq, H, self.us, T, H, self.s13, H, self.s13_scale, 2 * J, self.h13, 2 * J, self.status,
                         stream=stream)
        oes.moe_fp8_quantize(self.h13, 2 * J, T, J, oes.OES_ACT_SWIGLU, self.hq, J, self.hs, stream=stream)
        oes.moe_fp8_gemm(self.hq, J, self.hs, T, J, self.s2, J, self.s2_scale, H, self.s, H, self.status,
                         stream=stream)
        oes.moe_block_norm(self.n2, stream=stream)
        oes.moe_block_norm(self.n3, stream=stream)

    def close(self):
        oes.slot_cache_destroy(self.cache)
        oes.oes_expert_source_destroy(self.source)


def reference(block: Fp8Block, r: np.ndarray, a: np.ndarray, ids: np.ndarray, weights: np.ndarray,
              u_gpu: np.ndarray):
    """The step in 64 bits; routing (ids and weights) and the bf16 u that the
    experts quantise are taken from the GPU, so that a near tie does not send a
    token, or a code, elsewhere."""
    from oracle import fp8
    c, J = block.cfg, block.shared_I

    def f64(t):
        return t.detach().to(torch.float64).cpu().numpy()

    def norm(v, w):
        return v / np.sqrt((v * v).mean(1, keepdims=True) + EPS) * f64(w)

    r1 = r + norm(a, block.post_a)
    u = norm(r1, block.pre_u)
    x = fp8.dequantize(*fp8.quantize(u_gpu))
    e = np.zeros_like(r)
    for i in np.unique(ids):
        t, j = np.nonzero(ids == i)
        np.add.at(e, t, weights[t, j][:, None] * fp8.expert_mlp(x[t], block.rows[int(i)].numpy(), c.H, c.I))
    xu = fp8.dequantize(*fp8.quantize(u))
    w13 = fp8.weight(block.s13.cpu().numpy(), f64(block.s13_scale))
    w2 = fp8.weight(block.s2.cpu().numpy(), f64(block.s2_scale))
    s = fp8.dequantize(*fp8.quantize(fp8.hidden(xu, w13[:J], w13[J:]))) @ w2.T
    gate = 1 / (1 + np.exp(-(u_gpu @ f64(block.shared_gate))))
    r3 = r1 + gate * s + SCALE * norm(e, block.post_e)
    return u, r3, norm(r3, block.pre_next)


def run_and_check(T: int = 40, seed: int = 0):
    """One step against the reference; returns (block, relative errors of u, r and the next u)."""
    block = Fp8Block(small_config(T), seed=seed)
    c = block.cfg
    g = torch.Generator().manual_seed(seed + 1)
    block.r.copy_(torch.randn((c.T, c.H), generator=g))
    block.a.copy_(torch.randn((c.T, c.H), generator=g))
    r0, a0 = (t.to(torch.float64).cpu().numpy() for t in (block.r, block.a))
    block.step()
    torch.cuda.synchronize()
    if int(block.status.item()):
        raise RuntimeError(f"fp8_block: device status {int(block.status.item())}")
    v = oes.moe_layer_workspace_views(block.desc, c.T, c.k, block.ws)
    n, base = c.T * c.k * 4, block.ws.data_ptr()
    ids, w = (block.ws[v[f] - base:v[f] - base + n].cpu().numpy().view(d).reshape(c.T, c.k)
              for f, d in (("ids", np.int32), ("weights", np.float32)))
    got = [t.to(torch.float64).cpu().numpy() for t in (block.u, block.r, block.u_next)]
    want = reference(block, r0, a0, ids, w.astype(np.float64), got[0])
    return block, [float(np.linalg.norm(x - y) / np.linalg.norm(y)) for x, y in zip(got, want)]


def main():
    block, err = run_and_check()
    print("against 64 bits: u %.2g, residual %.2g, next u %.2g" % tuple(err))
    for _ in range(3):
        block.step()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(20):
        block.step()
    b.record()
    torch.cuda.synchronize()
    c = block.cfg
    print("%d tokens, top-%d of %d experts, H %d, I %d: %.1f us a step" % (c.T, c.k, c.E, c.H, c.I, a.elapsed_time(b) * 50))
    block.close()


if __name__ == "__main__":
    main()
