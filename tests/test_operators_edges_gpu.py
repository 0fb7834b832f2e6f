"""Calls at the edges of the epilogue, gated and norm operators: norms that are
switched off with pointers left in them, outputs that share their storage,
overlapping tensors, groups whose inputs were written just before, and the
accuracy of the activations in fp32 outputs.

Tolerances count roundings, u = 2^-24 (half an fp32 step), with CUDA's
documented error bounds of expf (2 ulp = 4 u) and normcdff (5 ulp = 10 u).
"""
import ctypes
import math

import pytest
import torch

from test_operators_gpu import BF, F32, Weight, check_norm, quantize, randn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    from sparse_gemm_wanda_b200 import build, patch
    build.build()
    patch.load_library()
    return patch


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(23)
    return g


# ------------------------------------------------------------------ norms
@pytest.mark.parametrize("M,C", [(64, 4096), (300, 1001), (4096, 4096), (2048, 8192)])
def test_a_norm_that_is_off_ignores_its_parameters(P, gen, M, C):
    # the same call with and without vectors in a norm of kind NONE, on every size of kernel
    lib = P.load_library()
    b, r = randn(gen, M, C, dtype=BF), randn(gen, M, C, dtype=BF)
    w, off = randn(gen, C, dtype=BF), randn(gen, C, spread=7.0, dtype=BF)
    h, z = torch.empty_like(b), torch.empty_like(b)

    def run(post, pre):
        h.fill_(float("nan"))
        z.fill_(float("nan"))
        a = P.PatchBlockNormArgs()
        a.branch, a.residual, a.h, a.z = b.data_ptr(), r.data_ptr(), h.data_ptr(), z.data_ptr()
        a.z_type, a.scale, a.gate_tokens, a.post, a.pre = P.Z_TYPES["bf16"], 0.5, 1, post, pre
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.patch_block_norm(ctypes.byref(a), M, C, ctypes.c_void_p(stream)) == 0
        return h.clone(), z.clone()

    none = P.PatchNorm(0, 0, None, None, 0.0)
    stray = P.PatchNorm(0, 0, off.data_ptr(), off.data_ptr(), 0.0)
    rms = P.PatchNorm(1, 0, w.data_ptr(), None, 1e-5)
    for clean, left in (((none, rms), (stray, rms)), ((rms, none), (rms, stray)), ((none, none), (stray, stray))):
        for got, want in zip(run(*left), run(*clean)):
            assert torch.equal(got, want)
