"""8-bit integer products whose waits run out: a build that gives up after one poll
ends with OES_DEV_TIMEOUT (or is done), frees what it held, and leaves the
context usable."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from gpu_util import lib
from offloaded_expert_slot_gb300 import build, oes
from test_gpu_fp8_give_up import both
from test_gpu_int8 import gemm_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """The library with one poll a wait in the integer products."""
    lib()
    d = tmp_path_factory.mktemp("impatient8")
    src, obj, so = os.path.join(build.CSRC, "gemm_int8.cu"), str(d / "gemm_int8.o"), str(d / "liboes_impatient8.so")
    objs = [os.path.join(build.OUT_DIR, os.path.basename(s)[:-3] + ".o") for s in build._sources() if s != src]
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-DOES_FP8_WAIT_POLLS=1", "-c", src, "-o", obj], check=True)
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-o", so, obj, *objs], check=True)
    handle = C.CDLL(so)
    for name, (res, args) in oes._SIGS.items():
        f = getattr(handle, name)
        f.restype, f.argtypes = res, args
    return handle


@pytest.mark.parametrize("T,K,N", [(900, 768, 2048), (700, 4096, 6000), (1300, 2500, 4100), (300, 4096, 4096), (2300, 2100, 3000)])
def test_products(impatient, T, K, N):
    xq, _, xs, _, wq, _, ws, _ = gemm_inputs(T, K, N, 7)
    nb = oes.moe_int8_gemm_workspace_size(T, K, N)
    work = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    seen = both(impatient, lambda st: oes.moe_int8_gemm(xq, xq.stride(0), xs, T, K, wq, wq.stride(0), ws, N, out, N,
                                                        work, nb, st), out)
    assert seen in (0, oes.OES_DEV_TIMEOUT)
