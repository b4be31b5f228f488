"""What moe_layer_few_tokens refuses, on the host (no GPU)."""
import pytest

from offloaded_expert_slot_gb300 import build, oes
from offloaded_expert_slot_gb300.configs import expert_row_bytes

P = 4096          # an aligned address; nothing is launched


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return oes.load()


def view(**kw):
    a = dict(layer=0, E=8, e2s=P, wfmt=oes.OES_WFMT_FP8, pool=P, row_bytes=None, S=8, H=256, I=128)
    a.update(kw)
    if a["row_bytes"] is None:
        name = {oes.OES_WFMT_BF16: "bf16", oes.OES_WFMT_NVFP4: "nvfp4"}.get(a["wfmt"], "fp8")
        a["row_bytes"] = expert_row_bytes(name, 256, 128)
    return oes.routed_experts(*a.values())


def call(v, **kw):
    a = dict(x=P, T=4, k=2, ids=P, weights=P, workspace=P, workspace_bytes=1 << 20, out=P, status=P, logits=P, dtype=0)
    a.update(kw)
    return oes.moe_layer_few_tokens(v, stream=0, **a)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(T=17), 2), (dict(k=0), 1), (dict(k=33), 1), (dict(k=9), 1), (dict(x=0), 1), (dict(ids=0), 1),
    (dict(weights=0), 1), (dict(workspace=0), 1), (dict(out=0), 1), (dict(x=P + 8), 1), (dict(workspace=P + 8), 1),
    (dict(ids=P + 2), 1), (dict(weights=P + 1), 1), (dict(out=P + 1), 1), (dict(status=P + 2), 1),
    (dict(logits=P + 2), 1), (dict(logits=P + 1, dtype=1), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1),
    (dict(workspace_bytes=4 * 2 * 128 * 4 - 1), 1)], ids=str)
def test_call_refuses(kw, code):
    with pytest.raises(oes.OesError) as e:
        call(view(), **kw)
    assert e.value.code == code and "moe_layer_few_tokens" in str(e.value)


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), 1), (dict(E=4097), 1), (dict(S=0), 1), (dict(H=96), 1), (dict(I=32), 1), (dict(H=16448), 1),
    (dict(I=16448), 1), (dict(H=0), 1), (dict(wfmt=4), 1), (dict(wfmt=-1), 1), (dict(wfmt=oes.OES_WFMT_NVFP4_W4A4), 2),
    (dict(pool=0), 1), (dict(e2s=0), 1), (dict(pool=P + 8), 1), (dict(e2s=P + 2), 1),
    (dict(row_bytes=expert_row_bytes("fp8", 256, 128) - 16), 1),
    (dict(row_bytes=expert_row_bytes("fp8", 256, 128) + 8), 1),
    (dict(wfmt=oes.OES_WFMT_BF16, row_bytes=expert_row_bytes("bf16", 256, 128) - 16), 1),
    (dict(wfmt=oes.OES_WFMT_NVFP4, row_bytes=expert_row_bytes("nvfp4", 256, 128) - 16), 1)], ids=str)
def test_view_refuses(kw, code):
    with pytest.raises(oes.OesError) as e:
        call(view(**kw))
    assert e.value.code == code and "moe_layer_few_tokens" in str(e.value)


def test_null_view_and_sizes():
    assert oes.load().moe_layer_few_tokens(None, P, 1, 1, P, 0, P, P, P, 1 << 20, P, P, None) == oes.OES_ERR_INVALID_ARG
    assert oes.load().moe_layer_few_tokens_workspace_size(None, 1, 1) == 0
    v = view()
    assert oes.moe_layer_few_tokens_workspace_size(v, 4, 2) >= 4 * 2 * 128 * 4
    for T, k in ((17, 2), (-1, 2), (4, 0), (4, 33)):
        assert oes.moe_layer_few_tokens_workspace_size(v, T, k) == 0
    assert oes.moe_layer_few_tokens_workspace_size(view(wfmt=oes.OES_WFMT_NVFP4_W4A4), 4, 2) == 0


def test_logits_of_another_type_are_refused_by_the_binding():
    import torch
    with pytest.raises(TypeError):
        call(view(), logits=torch.zeros(4, dtype=torch.float16), dtype=None)


def test_no_tokens_are_a_no_op():
    call(view(), T=0, x=0, ids=0, weights=0, workspace=0, out=0, logits=0, workspace_bytes=0)
