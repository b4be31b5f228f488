"""The top-k combine at every k: out[t] = sum_j w[t, j] y[t, j] in fp32, in j
order, rounded once, from the y the call leaves in its workspace.

Tolerance (u = 2^-24): k fp32 steps on sums of at most big = sum |w y|, so (k +
2) u big, and half a bf16 step, 2^-8 |out| at most.
"""
import numpy as np
import pytest
import torch

from fp8_util import EPS32, f64
from gpu_util import bits16, cuda, i32, lib, scratch, status
from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.configs import C2, scaled
from offloaded_expert_slot_gb300.inputs import expert_rows, f32_to_bf16_bits, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 130])
@pytest.mark.parametrize("k", list(range(1, 19)) + [24, 25, 31, 32])
def test_combine(k, T):
    lib()
    E, H, I = 36, 128, 64
    cfg = scaled(C2, name="combine", T=T, k=k, E=E, H=H, I=I, S=E, L=1, prefill=0, wfmt="bf16")
    g = rng(k * 1000 + T)
    pool, e2s = cuda(expert_rows(cfg, 0, range(E)).numpy()), cuda(np.arange(E, dtype=np.int32))
    x = bits16(f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32)))
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[g.random(ids.shape) < 0.2] = -1
    w = g.standard_normal((T, k)).astype(np.float32)
    R = T * k
    B = oes.oes_tile_plan(R, E)
    cap = oes.align_capacity(R, E, B)
    view = oes.routed_experts(0, E, e2s, oes.OES_WFMT_BF16, pool, cfg.row_bytes, E, H, I)
    srt, be, npad, st = i32(cap), i32(cap // B), i32(1), status()
    ab, gb = oes.moe_align_workspace_size(R, E, B), oes.moe_grouped_gemm_workspace_size(view, T, k)
    aws, ws = scratch(ab), scratch(gb)
    out = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    dids, dw = cuda(ids.reshape(-1)), cuda(w.reshape(-1))
    oes.moe_align_block_size(dids, R, E, B, 1, srt, be, npad, st, aws, ab)
    oes.moe_grouped_gemm_slots(view, x, T, k, dids, dw, srt, be, npad, B, ws, gb, out[1:T + 1], st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (out[0] == 7).all() and (out[-1] == 7).all()
    v = oes.moe_grouped_gemm_workspace_views(view, T, k, ws)
    y = f64(ws[v["y"] - ws.data_ptr():][:R * H * 2].view(torch.bfloat16).reshape(T, k, H))
    terms = np.where((ids >= 0)[:, :, None], w.astype(np.float64)[:, :, None] * np.where(np.isfinite(y), y, 0), 0.0)
    want, big = terms.sum(1), np.abs(terms).sum(1)
    assert np.abs(terms).max() > 0
    assert np.all(np.abs(f64(out[1:T + 1]) - want) <= big * (k + 2) * EPS32 + np.abs(want) * 2.0 ** -8 + 1e-37)
