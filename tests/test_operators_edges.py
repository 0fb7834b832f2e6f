"""Edges of the epilogue, gated and norm calls that need no GPU: which tensors
overlap, what the norm call refuses for it, and when the native modules are built."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_gemm_wanda_b200", "csrc")
BASE = 0x100000  # never dereferenced: refused before the device is asked for


@pytest.fixture(scope="module")
def P():
    from sparse_gemm_wanda_b200 import build, patch
    build.build()
    patch.load_library()
    return patch


# ------------------------------------------------------------ overlapping rows
@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    src = d / "overlap.cpp"
    src.write_text('#include "overlap.h"\n'
                   'extern "C" int overlap(long a, long an, long as, long aw, long b, long bn, long bs, long bw) {\n'
                   "    return patchk::overlap({(void *)a, an, as, aw}, {(void *)b, bn, bs, bw});\n}\n")
    lib = str(d / "overlap.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).overlap
    fn.argtypes = [ctypes.c_long] * 8
    return lambda a, b: fn(*a, *b) != 0


def byte_set(at, count, stride, width):
    return {at + i * stride + k for i in range(count) for k in range(width)}


def test_overlap_is_that_of_the_bytes(overlap):
    rng = random.Random(5)
    hits = 0
    for _ in range(30000):
        rows = []
        stride = rng.randint(1, 20)
        for _ in range(2):
            if rng.random() < 0.5:
                stride = rng.randint(1, 20)
            rows.append((rng.randint(100, 190), rng.randint(0, 6), stride, rng.randint(1, stride)))
        want = bool(byte_set(*rows[0]) & byte_set(*rows[1]))
        hits += want
        assert overlap(*rows) == want and overlap(*rows[::-1]) == want, rows
    assert 6000 < hits < 24000


def test_overlap_of_large_strides(overlap):
    big = 1 << 61
    assert not overlap((8, 1 << 31, big, 8), (16, 1 << 31, big, 8))
    assert overlap((8, 1 << 31, big, 16), (16, 1 << 31, big, 8))
    assert not overlap((8, 3, big, 8), (16, 1, 1 << 40, 1 << 40))
    assert overlap((1 << 40, 1, 8, 8), (8, 1 << 31, 1 << 20, 1 << 20))
    assert not overlap((0, 3, 8, 8), (0, 3, 8, 8))  # null: absent


# ------------------------------------------------- what the norm call refuses
def norm_status(P, M, C, **kw):
    a = P.PatchBlockNormArgs()
    for k, v in dict(dict(branch=BASE, residual=BASE + 0x10000, h=BASE + 0x20000, z=BASE + 0x30000, z_type=1, gate_tokens=1,
                          scale=1.0, pre=P.PatchNorm(1, 0, None, None, 1e-5)), **kw).items():
        setattr(a, k, v)
    return P.load_library().patch_block_norm(ctypes.byref(a), M, C, None)


H, Z = BASE + 0x20000, BASE + 0x30000
OVERLAPS = [
    dict(h=BASE + 2), dict(h=BASE + 4 * 128 - 2), dict(z=BASE + 0x10000 + 16), dict(z=H + 64), dict(h=Z + 2 * 63),
    dict(h=BASE + 64, h_stride=128, branch_stride=65), dict(gate=H, gate_tokens=4), dict(gate=Z + 300, gate_tokens=1),
    dict(gate=H - 200, gate_tokens=2, gate_stride=100), dict(pre=(1, 0, H + 30, None, 1e-5)),
    dict(post=(2, 0, None, Z - 2, 1e-5)), dict(post=(1, 1, H - 252, None, 1e-5)), dict(pre=(1, 0, Z, None, 1e-5)),
    dict(z_type=3, z_scales=H + 4), dict(z_type=3, z_scales=BASE + 8), dict(z_type=3, z_scales=Z + 252),
    dict(z_type=3, z=H + 511, z_scales=BASE + 0x50000), dict(z_type=3, z=BASE, z_scales=BASE + 0x50000),
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that were not refused would run on made-up addresses")
@pytest.mark.parametrize("kw", OVERLAPS, ids=str)
def test_block_norm_refuses_overlaps(P, kw):
    norms = {k: P.PatchNorm(*v) for k, v in kw.items() if isinstance(v, tuple)}
    assert norm_status(P, 4, 64, **{**kw, **norms}) == 1


NEIGHBOURS = [
    dict(), dict(h=BASE), dict(h=BASE + 0x10000), dict(z=BASE, h=None), dict(h=BASE, z=BASE + 0x10000),
    dict(h=BASE + 512), dict(z=H + 512), dict(h=BASE + 128, h_stride=128, branch_stride=128),
    dict(gate=H - 128, gate_tokens=4), dict(pre=(1, 0, Z + 512, Z - 128, 1e-5)),
    dict(z_type=3, z_scales=Z + 256), dict(post=(0, 0, H, Z, 0.0)),
    dict(h=BASE + 128, h_stride=192, branch_stride=192, z=BASE + 256, z_stride=192),
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("kw", NEIGHBOURS, ids=str)
def test_block_norm_takes_neighbours_and_in_place(P, kw):
    # past every check of the arguments: the device is asked for, and missing
    norms = {k: P.PatchNorm(*v) for k, v in kw.items() if isinstance(v, tuple)}
    assert norm_status(P, 4, 64, **{**kw, **norms}) in (2, 3)


# ------------------------------------------------------ building the native modules
@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    """The build module over a folder of its own; compilers that only leave their output file."""
    from sparse_gemm_wanda_b200 import build
    ran, fail = [], set()

    def run(cmd, **_):
        tool = os.path.basename(cmd[0])
        ran.append(tool)
        if tool not in fail:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(tool in fail), "", "no such header")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setenv("CXX", "g++")
    for name, leaf in (("OUT", "lib.so"), ("BINDING_OUT", "binding.so"), ("BUILD_DIR", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / leaf))
    return build, ran, fail


def test_the_library_is_built_without_the_binding(fake_build):
    build, ran, fail = fake_build
    fail.add("g++")
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.OUT) and not os.path.exists(build.BINDING_OUT)


def test_a_binding_for_another_torch_is_rebuilt(fake_build, monkeypatch):
    build, ran, _ = fake_build
    build.build()
    assert "nvcc" in ran and ran[-1] == "g++"
    ran.clear()
    build.build()
    assert ran == []
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert ran == ["g++"]
    build.build()
    assert ran == ["g++"]


def test_a_binding_for_another_torch_is_not_loaded(P, monkeypatch):
    from sparse_gemm_wanda_b200 import build
    monkeypatch.setattr(P, "_native", None)
    monkeypatch.setattr(build, "binding_target", lambda: "torch 0.0.1, cpython-30")
    with pytest.raises(P.PatchLibraryError, match="0.0.1"):
        P.patch_block_norm(torch.zeros(2, 64, dtype=torch.bfloat16))
