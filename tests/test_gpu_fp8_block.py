"""The 8-bit MoE block end to end (offloaded_expert_slot_gb300/fp8_block.py).

u is one bf16 rounding from the reference (2^-8 at most, a third of that in
the norm); the residual takes three bf16 roundings and its updates those of
y, out and the shared expert's rows (2^-8 each) and rare codes on the other
side of a midpoint: 1.5 % of the norm covers all of them.
"""
import pytest
import torch

from gpu_util import lib
from offloaded_expert_slot_gb300 import fp8_block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 150])
def test_block_against_64_bits(T):
    lib()
    block, (u, r, nxt) = fp8_block.run_and_check(T)
    assert u <= 2.0 ** -8 and r <= 1.5e-2 and nxt <= 1.5e-2, (u, r, nxt)
    block.close()


def test_block_in_a_graph():
    lib()
    block, _ = fp8_block.run_and_check(8)
    r0, a0 = torch.randn_like(block.r), torch.randn_like(block.a)
    block.a.copy_(a0)
    block.r.copy_(r0)
    block.step()
    torch.cuda.synchronize()
    want = block.r.clone(), block.u_next.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block.step()
    block.r.copy_(r0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(block.r, want[0]) and torch.equal(block.u_next, want[1])
    assert int(block.status.item()) == 0
    block.close()
