"""Refusals of the epilogue, gated and norm calls that need no GPU: the C ABI
checks its arguments before touching the device, the binding its tensors."""
import ctypes

import pytest
import torch

FAKE = 0x1000  # never dereferenced: checks fail first


@pytest.fixture(scope="module")
def P():
    from sparse_gemm_wanda_b200 import build, patch
    build.build()
    patch.load_library()
    return patch


def norm_args(P, **kw):
    d = dict(branch=FAKE, residual=FAKE + 0x1000, h=FAKE + 0x2000, z=FAKE + 0x3000, z_type=1, gate_tokens=1, scale=1.0)
    pre = P.PatchNorm(1, 0, None, None, 1e-5)
    a = P.PatchBlockNormArgs()
    a.pre = pre
    for k, v in {**d, **kw}.items():
        setattr(a, k, v)
    return a


def norm_call(P, M=4, C=64, **kw):
    return P.load_library().patch_block_norm(ctypes.byref(norm_args(P, **kw)), M, C, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(M=1 << 31), dict(C=0), dict(branch=None), dict(h=None, z=None, z_type=0), dict(z=None),
    dict(z_type=0), dict(z_type=4), dict(z_type=3), dict(branch=FAKE + 1), dict(residual_is_fp32=1, residual=FAKE + 2),
    dict(branch_stride=63), dict(residual_stride=-64), dict(h_stride=1), dict(z_stride=63), dict(gate=FAKE, gate_tokens=0),
    dict(gate=FAKE, gate_stride=3), dict(branch_is_fp32=2), dict(h=FAKE, h_is_fp32=1), dict(h=FAKE, h_stride=65),
    dict(z=FAKE, z_type=2), dict(h=FAKE + 0x3000), dict(z_type=3, z_scales=FAKE + 2),
], ids=str)
def test_block_norm_refuses(P, kw):
    assert norm_call(P, **kw) == 1


@pytest.mark.parametrize("norm", [(3, 0, 1e-5), (-1, 0, 1e-5), (1, 2, 1e-5), (1, 0, -1.0), (2, 0, float("nan"))])
def test_block_norm_refuses_norms(P, norm):
    kind, fp32, eps = norm
    for where in ("post", "pre"):
        assert norm_call(P, **{where: P.PatchNorm(kind, fp32, None, None, eps)}) == 1
    assert norm_call(P, pre=P.PatchNorm(1, 1, FAKE + 2, None, 1e-5)) == 1


def test_block_norm_width_limit_and_empty_batch(P):
    assert norm_call(P, C=P.NORM_MAX_C + 1) == 2
    assert norm_call(P, M=0) == 0
    assert norm_call(P, M=0, branch=None, h=None, z=None) == 0


def test_products_refuse_null_handles_and_counts(P):
    lib = P.load_library()
    vp = ctypes.c_void_p
    hs, ys = (vp * 9)(), (vp * 9)(*[FAKE] * 9)
    assert lib.patch_hybrid_linear(None, FAKE, None, 1, FAKE, 0, None, None) == 1
    assert lib.patch_hybrid_linear_group(hs, 2, FAKE, None, 1, ys, 0, None, None) == 1
    assert lib.patch_hybrid_linear_group(None, 1, FAKE, None, 1, ys, 0, None, None) == 1
    assert lib.patch_hybrid_linear_group(hs, 0, FAKE, None, 1, ys, 0, None, None) == 1
    assert lib.patch_hybrid_linear_group(hs, 9, FAKE, None, 1, ys, 0, None, None) == 1
    assert lib.patch_hybrid_gated(None, None, FAKE, None, 1, FAKE, 0, 0, None, None, 0, 4, None) == 1


def test_struct_sizes_match_the_header(P, tmp_path):
    import os
    import subprocess
    from sparse_gemm_wanda_b200 import build
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "patch.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu",'
                   "sizeof(patch_epilogue), sizeof(patch_norm), sizeof(patch_block_norm_args),"
                   "offsetof(patch_block_norm_args, post), offsetof(patch_block_norm_args, z_type),"
                   "offsetof(patch_epilogue, alpha)); }\n")
    exe = os.path.join(tmp_path, "sizes")
    subprocess.run(["gcc", "-I", build.INCLUDE, str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    A = P.PatchBlockNormArgs
    assert got == [ctypes.sizeof(P.PatchEpilogue), ctypes.sizeof(P.PatchNorm), ctypes.sizeof(A), A.post.offset,
                   A.z_type.offset, P.PatchEpilogue.alpha.offset]


def test_binding_refuses_host_tensors(P):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        P.patch_block_norm(x, pre=("rms", None, None, 1e-5))
    pk = P.PackedWeight(0, (128, 64, 64, 64), 0)
    with pytest.raises(ValueError, match="CUDA"):
        P.patch_hybrid_linear(pk, x)
    with pytest.raises(ValueError, match="CUDA"):
        P.patch_hybrid_gated(pk, pk, x)
    with pytest.raises(ValueError, match="CUDA"):
        P.patch_hybrid_linear_group([pk, pk], x, biases=[None])
    for bad in (None, 3, [x]):
        with pytest.raises(ValueError, match="tensor"):
            P.patch_block_norm(bad)
    with pytest.raises(ValueError, match="1 to 8"):
        P.patch_hybrid_linear_group([], x)
    with pytest.raises(ValueError, match="z_type"):
        P.patch_block_norm(x, z_type="fp16")
    with pytest.raises(ValueError, match="activation"):
        P.patch_hybrid_gated(pk, pk, x, activation="tanh")


def test_binding_fails_loudly_without_its_native_module(P, monkeypatch, tmp_path):
    monkeypatch.setattr(P, "_native", None)
    monkeypatch.setattr(P, "_HERE", str(tmp_path))
    with pytest.raises(P.PatchLibraryError):
        P.patch_block_norm(torch.zeros(2, 64, dtype=torch.bfloat16))
