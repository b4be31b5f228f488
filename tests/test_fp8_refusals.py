"""What the 8-bit calls and the block norm refuse, on the host (no GPU)."""
import ctypes as C

import pytest

from offloaded_expert_slot_gb300 import build, oes

P = 4096          # an aligned address; nothing is launched


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return oes.load()


def refused(call, *a, code=oes.OES_ERR_INVALID_ARG, **kw):
    with pytest.raises(oes.OesError) as e:
        call(*a, stream=0, **kw)
    assert e.value.code == code and call.__name__ in str(e.value)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(K=0), dict(K=(1 << 28) + 1), dict(act=2), dict(act=-1),
                                dict(x=0), dict(q=0), dict(scale=0), dict(x_ld=127), dict(q_ld=127),
                                dict(act=1, x_ld=255), dict(x=P + 1), dict(scale=P + 2), dict(dtype=2),
                                dict(dtype=oes.OES_F32, x=P + 2)], ids=str)
def test_quantize_refuses(kw):
    a = dict(x=P, x_ld=128, T=4, K=128, act=0, q=P, q_ld=128, scale=P, dtype=oes.OES_BF16)
    a.update(kw)
    dtype = a.pop("dtype")
    refused(oes.moe_fp8_quantize, *a.values(), dtype=dtype)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(K=0), dict(N=0), dict(K=(1 << 24) + 1), dict(N=(1 << 24) + 1),
                                dict(xq=0), dict(xs=0), dict(wq=0), dict(ws=0), dict(out=0), dict(xq=P + 8),
                                dict(wq=P + 4), dict(xq_ld=136), dict(wq_ld=200), dict(xq_ld=112), dict(wq_ld=0),
                                dict(out_ld=63), dict(xs=P + 1), dict(ws=P + 2), dict(out=P + 1), dict(dtype=5),
                                dict(dtype=oes.OES_F32, out=P + 2)], ids=str)
def test_gemm_refuses(kw):
    a = dict(xq=P, xq_ld=128, xs=P, T=4, K=128, wq=P, wq_ld=128, ws=P, N=64, out=P, out_ld=64, status=0,
             dtype=oes.OES_BF16)
    a.update(kw)
    dtype = a.pop("dtype")
    refused(oes.moe_fp8_gemm, *a.values(), dtype=dtype)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=0), dict(residual=0), dict(residual_ld=255), dict(y_ld=255),
                                dict(out=0, out_residual=0), dict(out_q=P), dict(out_scale=P), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(gate=P), dict(gate_kind=oes.OES_GATE_TOKEN),
                                dict(gate=P, gate_kind=4), dict(gate=P, gate_kind=oes.OES_GATE_ELEMENT, gate_ld=255),
                                dict(gate=P, gate_kind=oes.OES_GATE_TOKEN, gate_ld=0), dict(y=0),
                                dict(y=0, post_weight=0, gate=P, gate_kind=oes.OES_GATE_CHANNEL),
                                dict(out_ld=255), dict(out_residual_ld=1), dict(out_q=P, out_scale=P, out_q_ld=9),
                                dict(residual=P + 1), dict(out=P + 1), dict(dtype=7), dict(pre_weight=P + 1),
                                dict(dtype=oes.OES_F32, residual=P + 2),
                                dict(gate=P + 2, gate_kind=oes.OES_GATE_TOKEN, gate_ld=1)], ids=str)
def test_norm_refuses(kw):
    a = dict(T=4, H=256, residual=P, y=P, post_weight=P, pre_weight=P, out=P, out_residual=P, dtype=oes.OES_BF16)
    a.update(kw)
    for name in ("y", "post_weight", "out", "out_residual"):
        a[name] = a[name] or None
    refused(oes.moe_block_norm, oes.block_norm(**a))


def test_norm_refuses_wide_rows_and_null():
    refused(oes.moe_block_norm, oes.block_norm(1, 16385, P, out=P, dtype=oes.OES_BF16), code=oes.OES_ERR_UNSUPPORTED)
    assert oes.load().moe_block_norm(None, None) == oes.OES_ERR_INVALID_ARG


def test_arrays_of_another_type_are_refused_by_the_binding():
    import torch
    t = torch.zeros(4, dtype=torch.float16)
    with pytest.raises(TypeError):
        oes.moe_fp8_quantize(t, 4, 1, 4, 0, P, 4, P, stream=0)
    with pytest.raises(TypeError):
        oes.moe_fp8_gemm(P, 16, P, 1, 16, P, 16, P, 4, t, 4, stream=0)
    with pytest.raises(TypeError):
        oes.block_norm(1, 4, P)


@pytest.mark.parametrize("kw", [dict(H=96), dict(I=32), dict(row_bytes=-16), dict(pool=P + 8), dict(wfmt=4), dict(B=32)],
                         ids=str)
def test_grouped_gemm_refuses(kw):
    H, I = kw.get("H", 256), kw.get("I", 128)
    from offloaded_expert_slot_gb300.configs import expert_row_bytes
    rb = expert_row_bytes("fp8", H, I) + kw.get("row_bytes", 0)
    view = oes.routed_experts(0, 8, P, kw.get("wfmt", oes.OES_WFMT_FP8), kw.get("pool", P), rb, 8, H, I)
    refused(oes.moe_grouped_gemm_slots, view, P, 4, 2, P, P, P, P, P, kw.get("B", 16), P, 1 << 30, P, P)


def test_grouped_gemm_refuses_a_short_workspace():
    from offloaded_expert_slot_gb300.configs import expert_row_bytes
    view = oes.routed_experts(0, 8, P, oes.OES_WFMT_FP8, P, expert_row_bytes("fp8", 256, 128), 8, 256, 128)
    need = oes.moe_grouped_gemm_workspace_size(view, 4, 2)
    assert need > 0
    refused(oes.moe_grouped_gemm_slots, view, P, 4, 2, P, P, P, P, P, 16, P, need - 1, P, P)


def test_struct_matches_the_header():
    """The ctypes structure has the header's size: 5 ints, 3 floats, then 8-byte fields."""
    assert C.sizeof(oes.BlockNorm) == 8 * 4 + 15 * 8
