"""8-bit integer products whose waits run out, each kernel of its own: that the paths which end a CTA, or a pair
of them, after a wait gave up are reached, and that calls after it are right."""
import pytest
import torch

from offloaded_expert_slot_gb300 import oes
from test_gpu_fp8_give_up import both
from test_gpu_int8 import gemm_inputs
from test_gpu_int8_give_up import impatient  # noqa: F401  (the build with one poll a wait)

pytestmark = pytest.mark.gpu
# tiles of one SM: fewer than 76 pairs' tiles; pairs of SMs: more, and K of 2048 or more
CASES = {"tile": [(700, 4096, 6000, torch.bfloat16), (500, 8192, 8192, torch.float32), (130, 8192, 20000, torch.bfloat16)],
         "pair": [(1300, 2500, 4100, torch.bfloat16), (2300, 2100, 3000, torch.float32), (4096, 8192, 2048, torch.bfloat16)]}
ran_out = {kernel: [] for kernel in CASES}      # the status bits that each case saw


@pytest.mark.parametrize("kernel,case", [(k, c) for k, cs in CASES.items() for c in cs], ids=str)
def test_products(impatient, kernel, case):  # noqa: F811
    T, K, N, dtype = case
    xq, _, xs, _, wq, _, ws, _ = gemm_inputs(T, K, N, 7)
    nb = oes.moe_int8_gemm_workspace_size(T, K, N)
    work = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.empty((T, N), dtype=dtype, device="cuda")
    ran_out[kernel].append(both(impatient, lambda st: oes.moe_int8_gemm(
        xq, xq.stride(0), xs, T, K, wq, wq.stride(0), ws, N, out, N, work, nb, st), out))


@pytest.mark.parametrize("kernel", list(CASES))
def test_waits_ran_out(kernel):
    """The cases above, where all have run, reached the path that they are for."""
    seen = ran_out[kernel]
    assert len(seen) < len(CASES[kernel]) or oes.OES_DEV_TIMEOUT in seen, seen
