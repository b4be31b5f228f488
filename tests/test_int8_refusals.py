"""What the 8-bit integer calls refuse, on the host (no GPU)."""
import pytest

from offloaded_expert_slot_gb300 import build, oes

P = 4096          # an aligned address; nothing is launched
MANY = dict(T=4096, K=4096, N=4096, xq_ld=4096, wq_ld=4096, out_ld=4096)      # a size that needs a workspace


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return oes.load()


def refused(call, *a, **kw):
    with pytest.raises(oes.OesError) as e:
        call(*a, stream=0, **kw)
    assert e.value.code == oes.OES_ERR_INVALID_ARG and call.__name__ in str(e.value)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(K=0), dict(K=(1 << 28) + 1), dict(act=2), dict(act=-1), dict(x=0),
                                dict(q=0), dict(scale=0), dict(x_ld=127), dict(q_ld=127), dict(act=1, x_ld=255),
                                dict(x=P + 1), dict(scale=P + 2), dict(dtype=2), dict(dtype=oes.OES_F32, x=P + 2)],
                         ids=str)
def test_quantize_refuses(kw):
    a = dict(x=P, x_ld=128, T=4, K=128, act=0, q=P, q_ld=128, scale=P, dtype=oes.OES_BF16)
    a.update(kw)
    dtype = a.pop("dtype")
    refused(oes.moe_int8_quantize, *a.values(), dtype=dtype)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=(1 << 28) + 1), dict(K=0), dict(N=0), dict(K=65537),
                                dict(N=(1 << 24) + 1), dict(xq=0),
                                dict(xs=0), dict(wq=0), dict(ws=0), dict(out=0), dict(xq=P + 8), dict(wq=P + 4),
                                dict(xq_ld=136), dict(wq_ld=200), dict(xq_ld=112), dict(wq_ld=0), dict(out_ld=63),
                                dict(xs=P + 1), dict(ws=P + 2), dict(out=P + 1), dict(dtype=5), dict(status=P + 2),
                                dict(dtype=oes.OES_F32, out=P + 2), MANY, dict(MANY, workspace=P),
                                dict(MANY, workspace=P + 16, bytes=1 << 30),
                                dict(MANY, workspace=P, bytes=2 * (4096 + 4096) * 4096 - 1)], ids=str)
def test_gemm_refuses(kw):
    a = dict(xq=P, xq_ld=128, xs=P, T=4, K=128, wq=P, wq_ld=128, ws=P, N=64, out=P, out_ld=64, workspace=0, bytes=0,
             status=0, dtype=oes.OES_BF16)
    a.update(kw)
    dtype = a.pop("dtype")
    refused(oes.moe_int8_gemm, *a.values(), dtype=dtype)


def test_workspace_sizes():
    assert oes.moe_int8_gemm_workspace_size(1, 2048, 1536) == 0                     # few rows
    assert oes.moe_int8_gemm_workspace_size(4096, 4096, 4096) >= 2 * 4096 * (4096 + 4096)
    for T, K, N in ((-1, 16, 16), (4, 0, 16), (4, 65537, 16), (4, 16, 0), (4, 16, (1 << 24) + 1), (0, 16, 16)):
        assert oes.moe_int8_gemm_workspace_size(T, K, N) == 0


def test_arrays_of_another_type_are_refused_by_the_binding():
    import torch
    t = torch.zeros(4, dtype=torch.float16)
    with pytest.raises(TypeError):
        oes.moe_int8_quantize(t, 4, 1, 4, 0, P, 4, P, stream=0)
    with pytest.raises(TypeError):
        oes.moe_int8_gemm(P, 16, P, 1, 16, P, 16, P, 4, t, 4, stream=0)
