"""moe_layer_few_tokens from logits that choose experts without a slot."""
import numpy as np
import pytest
import torch

from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.inputs import rng
from test_gpu_few_tokens import WFMT, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(WFMT))
@pytest.mark.parametrize("bad", [-1, "S", 1 << 30])
@pytest.mark.parametrize("T", [1, 4, 16])
def test_a_chosen_expert_without_a_slot(fmt, T, bad):
    """From logits: the routing is the router's all the same, the expert's routes give 0, the status says so."""
    k, E = 3, 20
    m = Layer(fmt, T, k, E, 192, 128, seed=T)
    logits = torch.from_numpy(rng(T + 50).standard_normal((T, E)).astype(np.float32)).cuda()
    ids, w = torch.empty_like(m.ids), torch.empty_like(m.w)
    oes.moe_route_topk(logits, T, E, k, ids, w)
    lost = int(ids[T // 2, 1])
    m.e2s[lost] = m.S if bad == "S" else bad
    m.call(logits=logits)
    m.check(status=oes.OES_DEV_BAD_ID, skip=(lost,))
    assert torch.equal(ids, m.ids) and torch.equal(w, m.w)


@pytest.mark.parametrize("T", [1, 16])
def test_no_chosen_expert_has_a_slot(T):
    m = Layer("bf16", T, 4, 12, 128, 64)
    m.e2s.fill_(-1)
    m.call(logits=torch.from_numpy(rng(3).standard_normal((T, 12)).astype(np.float32)).cuda())
    assert not m.check(status=oes.OES_DEV_BAD_ID, skip=range(12)).any()
