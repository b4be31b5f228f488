"""FP8 products whose waits run out: a build of the kernels that give up after one
poll.  The calls then end with OES_DEV_TIMEOUT in the status word (or are done,
where no wait was that long), the context stays usable, and what the kernels
held (tensor memory, shared memory with copies on their way) is free again:
further calls, of both builds, run and are right.
"""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

from fp8_util import fp8_weight, padded, rows
from gpu_util import bits16, cuda, i32, lib, scratch, status
from offloaded_expert_slot_gb300 import build, oes
from offloaded_expert_slot_gb300.configs import C2, scaled
from offloaded_expert_slot_gb300.inputs import expert_rows, f32_to_bf16_bits, rng
from oracle import fp8

pytestmark = pytest.mark.gpu
ran_out = []      # the status bits that each case saw


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """The library with one poll a wait in the FP8 products."""
    lib()
    d = tmp_path_factory.mktemp("impatient")
    src, obj, so = os.path.join(build.CSRC, "gemm_fp8.cu"), str(d / "gemm_fp8.o"), str(d / "liboes_impatient.so")
    objs = [os.path.join(build.OUT_DIR, os.path.basename(s)[:-3] + ".o") for s in build._sources() if s != src]
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-DOES_FP8_WAIT_POLLS=1", "-c", src, "-o", obj], check=True)
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-o", so, obj, *objs], check=True)
    handle = C.CDLL(so)
    for name, (res, args) in oes._SIGS.items():
        f = getattr(handle, name)
        f.restype, f.argtypes = res, args
    return handle


def both(impatient, call, out, times=20):
    """Status bits that `call` left in the impatient build; it and the library in turn."""
    st = status()
    call(st)
    torch.cuda.synchronize()
    want = out.clone()
    assert int(st.item()) == 0
    seen, normal = 0, oes._lib
    for _ in range(times):
        st = status()
        try:
            oes._lib = impatient
            oes._funcs.clear()
            call(st)
            call(st)
            torch.cuda.synchronize()
        finally:
            oes._lib = normal
            oes._funcs.clear()
        bits = int(st.item())
        assert bits in (0, oes.OES_DEV_TIMEOUT)
        assert bits or torch.equal(out, want)
        seen |= bits
        st = status()
        call(st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(out, want)
    return seen


# shared K (clusters of 8 and 4), one wave without, token-major tiles
@pytest.mark.parametrize("T,K,N", [(1, 2048, 1536), (9, 1536, 2200), (2, 32768, 1024), (60, 512, 4096),
                                   (700, 4096, 6000)])
def test_dense(impatient, T, K, N):
    q, s = fp8.quantize(rows(T, K, T + K))
    xq = padded(torch.from_numpy(q.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8))
    xs = torch.from_numpy(s.astype(np.float32)).cuda()
    wq, ws, _ = fp8_weight(N, K, 7)
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    seen = both(impatient, lambda st: oes.moe_fp8_gemm(xq, xq.stride(0), xs, T, K, wq, wq.stride(0), ws, N, out, N,
                                                       st), out)
    ran_out.append(seen)


# one token (shared K, the second with a down product that waits long for h), weight-major, token-major
@pytest.mark.parametrize("T,k,E,H,I", [(1, 4, 16, 2048, 768), (1, 1, 2, 8192, 8192), (64, 4, 64, 1024, 512), (600, 4, 64, 1024, 512)])
def test_experts(impatient, T, k, E, H, I):
    cfg = scaled(C2, name="give_up", T=T, k=k, E=E, H=H, I=I, S=E, L=1, prefill=0, wfmt="fp8")
    g = rng(T)
    pool, e2s = cuda(expert_rows(cfg, 0, range(E), device="cuda").cpu().numpy()), cuda(np.arange(E, dtype=np.int32))
    x = bits16(f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32)))
    ids = cuda(np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32).reshape(-1))
    w = cuda(g.random(T * k).astype(np.float32))
    R = T * k
    B = oes.oes_tile_plan(R, E)
    cap = oes.align_capacity(R, E, B)
    view = oes.routed_experts(0, E, e2s, oes.OES_WFMT_FP8, pool, cfg.row_bytes, E, H, I)
    srt, be, npad = i32(cap), i32(cap // B), i32(1)
    ab, gb = oes.moe_align_workspace_size(R, E, B), oes.moe_grouped_gemm_workspace_size(view, T, k)
    aws, gws = scratch(ab), scratch(gb)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")

    def call(st):
        oes.moe_align_block_size(ids, R, E, B, 1, srt, be, npad, st, aws, ab)
        oes.moe_grouped_gemm_slots(view, x, T, k, ids, w, srt, be, npad, B, gws, gb, out, st)

    ran_out.append(both(impatient, call, out))


def test_waits_ran_out():
    """The cases above, where all have run, reached the path that they are for."""
    assert len(ran_out) < 9 or oes.OES_DEV_TIMEOUT in ran_out, ran_out
