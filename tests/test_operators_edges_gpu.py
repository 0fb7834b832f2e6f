"""Calls at the edges of the epilogue, gated and norm operators: norms that are
switched off with pointers left in them, outputs that share their storage,
overlapping tensors, groups whose inputs were written just before, and the
accuracy of the activations in fp32 outputs.

Tolerances count roundings, u = 2^-24 (half an fp32 step), with the documented
error bounds of the instructions and functions used.
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


@pytest.mark.parametrize("M,C", [(4096, 4096), (3001, 5120), (900, 16384)])
def test_norms_of_many_rows_with_every_parameter_in_bf16(P, gen, M, C):
    # the parts of the shared-memory ring: a gate with a weightless post norm
    # and no pre norm, e4m3 output behind weights, no residual, z in fp32
    bf = dict(dtype=BF)
    b, r = randn(gen, M, C, **bf), randn(gen, M, C, **bf)
    rms = lambda: ("rms", randn(gen, C, spread=0.2, **bf) + 1, None, 1e-5)  # noqa: E731
    check_norm(P, b, r, gate=randn(gen, 1, C, **bf), post=("rms", None, None, 1e-5), pre=None)
    check_norm(P, b, r, post=rms(), pre=rms(), z_type="e4m3")
    check_norm(P, b, r, pre=rms(), z_type="e4m3")
    check_norm(P, b, None, gate=randn(gen, C, **bf), post=rms(), pre=("rms", None, None, 1e-5), z_type="fp32")


@pytest.mark.parametrize("M,C", [(64, 4096), (300, 1032), (33, 999), (4096, 4096)])
def test_codes_behind_a_norm_are_the_rounded_quotients(P, gen, M, C):
    # the codes are those of the normed fp32 row divided by its scale, bit for bit
    for dtype in (BF, F32):
        b, pre = randn(gen, M, C, dtype=dtype), ("rms", randn(gen, C, dtype=dtype), None, 1e-5)
        z = P.patch_block_norm(b, pre=pre, z_type="fp32")["z"]
        e = P.patch_block_norm(b, pre=pre, z_type="e4m3")
        q, s = quantize(z)
        assert torch.equal(e["scales"], s)
        assert torch.equal(e["z"], q.view(torch.uint8))


# ------------------------------------------- outputs that share their storage
def test_an_output_that_is_a_lazy_clone_leaves_its_origin_alone(P, gen):
    M, N = 40, 256
    wg, wu = Weight(P, gen, N, 256), Weight(P, gen, N, 256)
    x, res = randn(gen, M, 256, dtype=BF), randn(gen, M, N, dtype=BF)
    pre = ("rms", None, None, 1e-5)

    def fresh(origin):
        return torch._lazy_clone(origin), origin.clone()

    calls = [
        (lambda o: P.patch_hybrid_linear(wg.packed, x, residual=res, out=o),
         lambda: P.patch_hybrid_linear(wg.packed, x, residual=res)),
        (lambda o: P.patch_hybrid_gated(wg.packed, wu.packed, x, out=o),
         lambda: P.patch_hybrid_gated(wg.packed, wu.packed, x)),
        (lambda o: P.patch_hybrid_linear_group([wg.packed, wu.packed], x, outs=[None, o])[1],
         lambda: P.patch_hybrid_linear_group([wg.packed, wu.packed], x)[1]),
        (lambda o: P.patch_block_norm(res, pre=pre, out_h=o)["h"], lambda: P.patch_block_norm(res, pre=pre)["h"]),
        (lambda o: P.patch_block_norm(res, pre=pre, out_z=o)["z"], lambda: P.patch_block_norm(res, pre=pre)["z"]),
    ]
    for into, plain in calls:
        origin = torch.zeros(M, N, dtype=BF, device="cuda")
        out, keep = fresh(origin)
        got, want = into(out), plain()
        assert torch.equal(got, want) and torch.equal(out, want)
        assert torch.equal(origin, keep)


def test_an_in_place_update_of_a_lazy_clone(P, gen):
    M, N = 40, 256
    w = Weight(P, gen, N, 256)
    x, origin = randn(gen, M, 256, dtype=BF), randn(gen, M, N, dtype=BF)
    keep, stream = origin.clone(), torch._lazy_clone(origin)
    P.patch_hybrid_linear(w.packed, x, residual=stream, out=stream)
    assert torch.equal(stream, P.patch_hybrid_linear(w.packed, x, residual=keep)) and torch.equal(origin, keep)
    stream = torch._lazy_clone(origin)
    P.patch_block_norm(stream, residual=keep, out_h=stream)
    assert torch.equal(stream, P.patch_block_norm(keep, residual=keep)["h"]) and torch.equal(origin, keep)


# ----------------------------------------------- activations in fp32 outputs
def identity(P, n, nm=(2, 4)):
    """A packed n x n identity of dense tiles: every sum is one value of X, exactly."""
    w = torch.eye(n, dtype=BF, device="cuda")
    return P.patch_pack(w, torch.full((n, n // 32), 0x44444444, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), tile_n=128, tile_k=128, nm=nm)


def value_and_bound(v, kind):
    """act(v) in 64 bits and the error that the header states, from v (exact).

    silu: e = __expf(-v) is off by 2 + floor(|1.173 v|) ulp of 2 u, 1 + e by u,
      __fdividef by 2 ulp (4 u): (9 + 2.35 |v|) u; a quotient over 2^126 may be 0.
    tanh GELU: the same behind y = v (c0 + c1 v^2), which has two rounded
      constants and three roundings, 5 u |y| in the exponent.
    GELU: erff is off by 2 ulp (2 u below 1), its argument by 2 u (worth 1 u: x
      erf'(x) <= 0.49), 1 + erf by u: 4 u of 0.5 |v|, and one rounded product."""
    if kind == "gelu":
        want = 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
        return want, 3 * U * v.abs()
    y = v if kind == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)
    want = v * torch.sigmoid(y)
    return want, (10 + (2.4 if kind == "silu" else 7.4) * y.abs()) * U * want.abs() + 2.0 ** -118


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_activations_of_fp32_outputs(P, gen, kind, M):
    n = 256
    w = identity(P, n)
    span = torch.linspace(-12, 12, M * n, device="cuda")[torch.randperm(M * n, generator=gen, device="cuda")]
    x = span.to(BF).view(M, n)
    v = x.double()
    want, tol = value_and_bound(v, kind)
    got = P.patch_hybrid_linear(w, x, activation=kind, out_fp32=True).double()
    err = (got - want).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    # the gated pair: the same value times the up projection's, one more rounding
    got = P.patch_hybrid_gated(w, w, x, activation=kind, out_fp32=True).double()
    err = (got - want * v).abs()
    assert (err <= tol * v.abs() + 2 * U * (want * v).abs() + 2.0 ** -118).all()


def test_activations_of_fp32_outputs_far_out(P):
    # no infinity, NaN or early zero where an exponential over- or underflows
    n = 256
    w = identity(P, n)
    for M in (2, 100, 300):
        x = (torch.linspace(-100, 100, M * n, device="cuda")).to(BF).view(M, n)
        for kind in ("silu", "gelu", "gelu_tanh"):
            want, tol = value_and_bound(x.double(), kind)
            got = P.patch_hybrid_linear(w, x, activation=kind, out_fp32=True).double()
            assert ((got - want).abs() <= tol).all()


# --------------------------------------------- overlapping tensors are refused
def test_overlapping_outputs_and_inputs_are_refused(P, gen):
    # refused before anything is enqueued: every tensor keeps its bits
    N, K, M = 256, 512, 20
    packed = [Weight(P, gen, N, K).packed for _ in range(2)]
    big = randn(gen, M + 2, 1024, dtype=BF)
    keep = big.clone()
    x = randn(gen, M, K, dtype=BF)
    rows = lambda c, r=0: big[r:r + M, c:c + N]  # noqa: E731
    flat = big.view(-1)
    at = lambda i, n, m: flat[i:i + m * n].view(m, n)  # noqa: E731
    ok = P.patch_hybrid_linear_group(packed, x, outs=[rows(0), rows(256)], residuals=[rows(512), rows(768)])
    want = P.patch_hybrid_linear_group(packed, x, residuals=[keep[:M, 512:768], keep[:M, 768:]])
    assert all(torch.equal(a, b) for a, b in zip(ok, want))
    big.copy_(keep)
    refused = [
        lambda: P.patch_hybrid_linear_group(packed, x, outs=[rows(0), rows(128)]),
        lambda: P.patch_hybrid_linear_group(packed, x, outs=[rows(0), rows(0, 1)]),
        lambda: P.patch_hybrid_linear_group(packed, x, outs=[rows(0), rows(512)], residuals=[None, rows(255)]),
        lambda: P.patch_hybrid_linear(packed[0], x, out=rows(0), residual=rows(8)),
        lambda: P.patch_hybrid_linear(packed[0], x, out=rows(0), residual=rows(0, 1)),
        lambda: P.patch_hybrid_linear(packed[0], x, out=rows(0), bias=flat[64:64 + N]),
        lambda: P.patch_hybrid_linear(packed[0], at(1024, K, M), out=at(1024 + K, N, M)),
        lambda: P.patch_hybrid_gated(packed[0], packed[1], at(0, K, M), out=at(K, N, M)),
        lambda: P.patch_hybrid_gated(packed[0], packed[1], x, out=rows(256), bias_up=flat[400:400 + N]),
    ]
    for call in refused:
        with pytest.raises(P.PatchError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(big, keep)


# --------------------------------- members side by side and their late inputs
@pytest.mark.parametrize("kind", ["2:4", "4:8", "fp8"])
@pytest.mark.parametrize("M", [20, 100, 300])
def test_members_side_by_side_read_what_was_just_written(P, gen, kind, M):
    # X, its scales, the residuals and the biases are all rewritten by the
    # kernels right before the group, with other values in every pass
    N, K = 384, 640
    ws = [Weight(P, gen, n, K, kind) for n in (N, 128, N)]
    packed = [w.packed for w in ws]
    sets = []
    for _ in range(3):
        q, s = quantize(randn(gen, M, K))
        sets.append({"x": q.view(torch.uint8) if kind == "fp8" else randn(gen, M, K, dtype=BF), "s": s,
                     "r": randn(gen, M, N, dtype=BF), "t": randn(gen, M, N), "b": randn(gen, N)})
    live = {k: torch.empty_like(v) for k, v in sets[0].items()}

    def group(d):
        return P.patch_hybrid_linear_group(packed, d["x"], x_scales=d["s"] if kind == "fp8" else None,
                                           activation="silu", residuals=[d["r"], None, d["t"]], biases=[None, None, d["b"]])

    want = []
    for d in sets:
        torch.cuda.synchronize()
        want.append([y.clone() for y in group(d)])
        torch.cuda.synchronize()
    pick = torch.zeros(1, dtype=torch.long, device="cuda")
    stacked = {k: torch.stack([d[k] for d in sets]) for k in live}

    def step():
        for k, v in live.items():
            torch.index_select(stacked[k], 0, pick, out=v.unsqueeze(0))
        # the last kernel before the group writes a residual: 0.5 * (2 r), exactly r
        P.patch_block_norm(2 * live["r"], scale=0.5, out_h=live["r"])
        return group(live)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for k in range(30):
        pick.fill_(k % 3)
        graph.replay()
        pick.fill_((k + 1) % 3)
        eager = step()
        torch.cuda.synchronize()
        for i, got in ((k % 3, captured), ((k + 1) % 3, eager)):
            for y, y1 in zip(got, want[i]):
                assert torch.equal(y, y1)
    for w in packed:
        assert P.patch_get_status(w) == 0


# ------------------------------------------------ exceptions at the C boundary
def test_no_exception_leaves_the_first_call_out_of_host_memory(tmp_path):
    # the first call of a process notes the device's properties, which allocates
    import os
    import subprocess
    import sys
    src = tmp_path / "shim.cpp"
    src.write_text("""
#include <cstdlib>
#include <new>
static thread_local int failing = 0;
extern "C" void fail_new(int on) { failing = on; }
static void *get(std::size_t n) {
    void *p = failing ? nullptr : std::malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void *operator new(std::size_t n) { return get(n); }
void *operator new[](std::size_t n) { return get(n); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete[](void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
void operator delete[](void *p, std::size_t) noexcept { std::free(p); }
""")
    shim = str(tmp_path / "shim.so")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", str(src), "-o", shim], check=True)
    code = """
import ctypes, sys, torch
from sparse_gemm_wanda_b200 import patch as P
shim, lib = ctypes.CDLL(sys.argv[1]), P.load_library()
x = torch.randn(4, 64, device="cuda").bfloat16()
h = torch.zeros_like(x)
a = P.PatchBlockNormArgs()
a.branch, a.h, a.scale = x.data_ptr(), h.data_ptr(), 1.0
arg, M, C, stream, run = ctypes.byref(a), 4, 64, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), lib.patch_block_norm
fail = shim.fail_new
fail(1)
status = run(arg, M, C, stream)
fail(0)
assert P.STATUS_NAMES[status] == "PATCH_ERR_OOM", status
assert run(arg, M, C, stream) == 0
torch.cuda.synchronize()
assert torch.equal(x, h)
print("returned")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code, shim], cwd=root, env={**os.environ, "LD_PRELOAD": shim},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "returned" in r.stdout, r.stderr[-2000:]
