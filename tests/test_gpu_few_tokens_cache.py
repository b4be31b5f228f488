"""moe_layer_few_tokens as an offloaded layer uses it: behind the slot cache's own ensure and copies, on its own
slot map."""
import numpy as np
import pytest
import torch

from offloaded_expert_slot_gb300 import oes
from offloaded_expert_slot_gb300.inputs import rng
from test_gpu_few_tokens import WFMT, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(WFMT))
@pytest.mark.parametrize("T,k,E,S", [(1, 4, 24, 9), (4, 3, 24, 14), (16, 2, 40, 33)])
def test_behind_the_slot_cache(fmt, T, k, E, S):
    """Steps of route, distinct, ensure, copy and layer, two layers in one cache smaller than both: hits, misses,
    evicted slots taken again. The layer reads the cache's map of the routing's ids, the stream alone orders it."""
    H, I, L, steps = 256, 128, 2, 6
    layers = [Layer(fmt, T, k, E, H, I, seed=100 * i) for i in range(L)]      # for their rows and their check
    row_bytes = layers[0].rows.shape[1]
    host = [torch.from_numpy(m.rows).pin_memory() for m in layers]
    src = oes.oes_expert_source_create([h.data_ptr() for h in host], E, row_bytes)
    cache = oes.slot_cache_create(S, L, E)
    pool = torch.full((S, row_bytes), 0x7F, dtype=torch.uint8, device="cuda")
    g = rng(T)

    def i32(n):
        return torch.zeros(n, dtype=torch.int32, device="cuda")

    distinct, count, miss, n_miss, status = i32(T * k), i32(1), i32(3 * oes.OES_QUERY_MAX), i32(1), i32(1)
    try:
        seen = 0
        for step in range(steps):
            for i, m in enumerate(layers):
                logits = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32)).cuda()
                m.x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
                oes.moe_route_topk(logits, T, E, k, m.ids, m.w)
                oes.moe_distinct_experts(m.ids, T * k, E, distinct, count)
                n = int(count.item())
                oes.slot_cache_ensure(cache, i, distinct, n, True, miss, n_miss, status)
                seen += int(n_miss.item())
                oes.slot_cache_copy_misses(src, pool, S, miss, n_miss, n, status)
                m.view = oes.routed_experts(i, E, oes.slot_cache_layer_map(cache, i), WFMT[fmt], pool, row_bytes, S, H, I)
                m.call()
                m.check()
                if step % 2:        # the same call from the logits, on the same map
                    given = m.out.clone()
                    m.call(logits=logits)
                    m.check()
                    assert torch.equal(given, m.out)
        assert int(status.item()) == 0
        state = oes.slot_cache_read_state(cache, S, L, E)
        assert seen > S and state["hits"] > 0 and state["evictions"] > 0
    finally:
        torch.cuda.synchronize()
        oes.slot_cache_destroy(cache)
        oes.oes_expert_source_destroy(src)
