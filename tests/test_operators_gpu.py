"""The epilogue, gated and norm calls against plain 64-bit implementations.

Tolerances are derived, never fitted:

* a product's sum of K terms is added by the tensor core in fp32, truncating
  after every instruction of 16 terms: with K / 16 + 32 additions (the split-K
  joins included) each off by at most 2^-23 of the sum of |terms|,
  t_sum = (K / 16 + 32) * 2^-23 * sum |x w|; FP8 scales add 2 * 2^-24 relative;
* an activation has slope at most 1.13 and is computed by functions good to a
  few 2^-24 relative on arguments with as many, so it adds 2^-20 |v|;
* the rest of the epilogue is at most four fp32 roundings, 2^-22 of the
  magnitudes added;
* the output is off by half a step: 2^-8 (bf16) or 2^-24 (fp32) relative, and
  a subnormal's half step where the result is that small.
"""
import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines, skipped there
    pytest.skip("needs a CUDA device", allow_module_level=True)

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    from sparse_gemm_wanda_b200 import build, patch
    build.build()
    patch.load_library()
    return patch


@pytest.fixture
def gen():
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    return g


def randn(g, *shape, spread=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * spread).to(dtype)


def quantize(x):
    x = x.float()
    amax = x.abs().amax(1)
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / s[:, None]).to(torch.float8_e4m3fn), s


class Weight:
    """One packed weight and its W_eff (64 bits) from seeded random codes and map."""

    def __init__(self, P, g, N, K, kind="2:4", tn=128, tk=128, f=0.5):
        self.w = randn(g, N, K, spread=0.05, dtype=BF)
        size = 8 if kind == "4:8" else 4
        order = torch.rand(N, K // size, size, generator=g, device="cuda").argsort(-1)
        keep = order < size // 2
        at = torch.arange(size, device="cuda")
        if size == 8:
            code = (keep.long() << at).sum(-1)
        else:
            first = keep.to(torch.int8).argmax(-1)
            code = first | ((3 - keep.flip(-1).to(torch.int8).argmax(-1)) << 2)
        per = 32 // size
        meta = (code.view(N, K // 32, per) << (size * torch.arange(per, device="cuda"))).sum(-1).to(torch.int32)
        tiles = (N // tn) * (K // tk)
        sparse = torch.zeros(-(-tiles // 32) * 32, dtype=torch.long, device="cuda")
        sparse[torch.randperm(tiles, generator=g, device="cuda")[: int(f * tiles)]] = 1
        tmap = (sparse.view(-1, 32) << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
        wide = sparse[:tiles].view(N // tn, K // tk).repeat_interleave(tn, 0).repeat_interleave(tk, 1).bool()
        weff = torch.where(wide & ~keep.view(N, K), torch.zeros_like(self.w), self.w)
        self.kind, self.N, self.K = kind, N, K
        if kind == "fp8":
            q, s = quantize(weff)
            self.weff = q.double() * s.double()[:, None]
            self.packed = P.patch_pack_fp8(self.w, meta, tmap, tile_n=tn, tile_k=tk)
        else:
            self.weff = weff.double()
            self.packed = P.patch_pack(self.w, meta, tmap, tile_n=tn, tile_k=tk, nm=(4, 8) if size == 8 else (2, 4))

    def sums(self, x, x_scales=None):
        """(sums, their tolerance) in 64 bits."""
        if self.kind == "fp8":
            q, s = (x.view(torch.float8_e4m3fn), x_scales) if x_scales is not None else quantize(x)
            x = q.double() * s.double()[:, None]
        x = x.double()
        y, size = x @ self.weff.t(), x.abs() @ self.weff.abs().t()
        return y, (self.K / 16 + 32) * 2.0 ** -23 * size + 2.0 ** -22 * y.abs()


def act64(v, kind):
    if kind == "relu":
        return v.clamp_min(0)
    if kind == "gelu":
        return v * torch.special.ndtr(v)
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if kind == "silu":
        return v * torch.sigmoid(v)
    return v


def activated(y, tol, bias, kind):
    b = torch.zeros_like(y) if bias is None else bias.double().expand_as(y)
    v = y + b
    tol = tol + 2.0 ** -23 * v.abs()
    return act64(v, kind), (1.13 * tol if kind else tol) + (2.0 ** -20 * v.abs() if kind else 0)


def close(got, want, tol):
    half = HALF_STEP[got.dtype]
    bound = tol + half * (want.abs() + tol) + 2.0 ** -130
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} beyond the bound, worst " \
        f"{((got.double() - want).abs() / bound).max().item():.2f} of it"


def check_linear(got, w, x, x_scales=None, bias=None, act=None, alpha=1.0, residual=None):
    y, tol = w.sums(x, x_scales)
    y, tol = activated(y, tol, bias, act)
    y, tol = alpha * y, abs(alpha) * tol
    r = torch.zeros_like(y) if residual is None else residual.double()
    close(got, r + y, tol + 2.0 ** -22 * (r.abs() + y.abs()))


def check_gated(got, wg, wu, x, x_scales=None, bg=None, bu=None, act="silu"):
    a, ta = activated(*wg.sums(x, x_scales), bg, act)
    b, tb = activated(*wu.sums(x, x_scales), bu, None)
    close(got, a * b, ta * b.abs() + tb * a.abs() + ta * tb + 2.0 ** -23 * (a * b).abs())


def x_of(g, w, M, codes=False):
    x = randn(g, M, w.K, dtype=BF)
    if not codes:
        return x, None
    q, s = quantize(x)
    return q.view(torch.uint8), s


SHAPES = [  # kind, N, K, tile_n, tile_k, f
    ("2:4", 256, 256, 128, 128, 0.5),
    ("2:4", 384, 640, 64, 64, 0.5),      # an odd band count, fine tiles
    ("2:4", 128, 8448, 128, 128, 0.6),   # one band, K beyond the split-K range above 16 tokens
    ("4:8", 256, 384, 128, 64, 0.6),
    ("fp8", 256, 512, 128, 128, 0.5),
    ("fp8", 384, 384, 128, 128, 1.0),    # odd band and k-step counts
]
TOKENS = [1, 3, 16, 17, 64, 65, 128, 129, 300]


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(P, gen, shape, M):
    kind, N, K, tn, tk, f = shape
    w = Weight(P, gen, N, K, kind, tn, tk, f)
    x, xs = x_of(gen, w, M, codes=kind == "fp8" and M % 2 == 1)
    bias = randn(gen, N, dtype=BF if M % 2 else F32)
    res = randn(gen, M, N, dtype=F32 if M % 3 else BF)
    act = [None, "relu", "gelu", "gelu_tanh", "silu"][TOKENS.index(M) % 5]
    got = P.patch_hybrid_linear(w.packed, x, x_scales=xs, bias=bias, activation=act, alpha=0.75, residual=res,
                                out_fp32=M % 2 == 0)
    check_linear(got, w, x, xs, bias, act, 0.75, res)
    # no epilogue at all is the plain product, at decode token counts bit for bit
    if xs is None and M <= 64:
        assert torch.equal(P.patch_hybrid_linear(w.packed, x), P.patch_hybrid_gemm(w.packed, x))
    assert P.patch_get_status(w.packed) == 0


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated(P, gen, shape, M):
    kind, N, K, tn, tk, f = shape
    wg, wu = Weight(P, gen, N, K, kind, tn, tk, f), Weight(P, gen, N, K, kind, tn, tk, 1 - f)
    x, xs = x_of(gen, wg, M, codes=kind == "fp8" and M % 2 == 0)
    bg = randn(gen, N, dtype=BF) if M % 2 else None
    bu = randn(gen, N, dtype=BF) if M % 3 else None
    act = [None, "relu", "gelu", "gelu_tanh", "silu"][TOKENS.index(M) % 5]
    got = P.patch_hybrid_gated(wg.packed, wu.packed, x, x_scales=xs, bias_gate=bg, bias_up=bu, activation=act,
                               out_fp32=M % 2 == 0)
    check_gated(got, wg, wu, x, xs, bg, bu, act)
    assert P.patch_get_status(wg.packed) == 0 and P.patch_get_status(wu.packed) == 0


@pytest.mark.parametrize("kernel", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", ["2:4", "fp8"])
def test_each_prefill_kernel(P, gen, kind, kernel):
    wg, wu = Weight(P, gen, 512, 512, kind, f=0.5), Weight(P, gen, 512, 512, kind, f=0.75)
    M = 700  # several token tiles, the last one ragged
    x, xs = x_of(gen, wg, M, codes=kind == "fp8")
    bias, res = randn(gen, 512), randn(gen, M, 512, dtype=BF)
    P.test_prefill_kernel(kernel)
    try:
        y = P.patch_hybrid_linear(wg.packed, x, x_scales=xs, bias=bias, activation="silu", residual=res)
        z = P.patch_hybrid_gated(wg.packed, wu.packed, x, x_scales=xs, bias_up=bias, activation="gelu")
        ys = P.patch_hybrid_linear_group([wg.packed, wu.packed], x, x_scales=xs, biases=[None, bias],
                                         residuals=[res, None], activation="relu")
    finally:
        P.test_prefill_kernel(0)
    check_linear(y, wg, x, xs, bias, "silu", 1.0, res)
    check_gated(z, wg, wu, x, xs, None, bias, "gelu")
    check_linear(ys[0], wg, x, xs, None, "relu", 1.0, res)
    check_linear(ys[1], wu, x, xs, bias, "relu")


@pytest.mark.parametrize("M", [1, 8, 40, 100, 400])
@pytest.mark.parametrize("kinds", [("2:4", "2:4", "2:4"), ("fp8", "fp8"), ("2:4", "4:8"), ("fp8", "2:4")], ids=str)
def test_group(P, gen, kinds, M):
    sizes = [256, 512, 128][: len(kinds)]
    ws = [Weight(P, gen, n, 512, k) for n, k in zip(sizes, kinds)]
    codes = set(kinds) == {"fp8"} and M != 8
    x, xs = x_of(gen, ws[0], M, codes=codes)
    biases = [randn(gen, n) if i else None for i, n in enumerate(sizes)]
    residuals = [randn(gen, M, n, dtype=BF if i % 2 else F32) if i != 1 else None for i, n in enumerate(sizes)]
    got = P.patch_hybrid_linear_group([w.packed for w in ws], x, x_scales=xs, biases=biases, residuals=residuals,
                                      activation="gelu_tanh", alpha=-2.0)
    for y, w, b, r in zip(got, ws, biases, residuals):
        check_linear(y, w, x, xs, b, "gelu_tanh", -2.0, r)


@pytest.mark.parametrize("kind", ["2:4", "fp8", "4:8"])
def test_the_same_handle_twice(P, gen, kind):
    w = Weight(P, gen, 256, 512, kind)
    for M in (4, 40, 300):
        x, _ = x_of(gen, w, M)
        b = randn(gen, 256)
        one, two = P.patch_hybrid_linear_group([w.packed, w.packed], x, biases=[b, None])
        check_linear(one, w, x, bias=b)
        check_linear(two, w, x)
        check_gated(P.patch_hybrid_gated(w.packed, w.packed, x), w, w, x)


@pytest.mark.parametrize("M", [1, 17, 100, 300])
@pytest.mark.parametrize("kind", ["2:4", "fp8", "4:8"])
def test_strided_rows_in_place_and_rows_behind(P, gen, kind, M):
    # Y is the left part of wider rows, with rows behind the batch; the
    # residual is updated in place and nothing around it moves
    w = Weight(P, gen, 384, 512, kind)
    x, _ = x_of(gen, w, M)
    for dtype in (BF, F32):
        wide = randn(gen, M + 3, 384 + 5, dtype=dtype)
        before = wide.clone()
        y = wide[:M, :384]
        got = P.patch_hybrid_linear(w.packed, x, residual=y, out=y, activation="silu", out_fp32=dtype == F32)
        assert got.data_ptr() == wide.data_ptr()
        check_linear(got, w, x, act="silu", residual=before[:M, :384])
        assert torch.equal(wide[:, 384:], before[:, 384:]) and torch.equal(wide[M:], before[M:])
        # an offset that is not 16-byte aligned
        z = wide[1:M + 1, 1:385]
        before = wide.clone()
        P.patch_hybrid_gated(w.packed, w.packed, x, out=z, out_fp32=dtype == F32)
        check_gated(z, w, w, x)
        assert torch.equal(wide[:, 385:], before[:, 385:]) and torch.equal(wide[:, :1], before[:, :1])
        assert torch.equal(wide[0], before[0]) and torch.equal(wide[M + 1:], before[M + 1:])


@pytest.mark.parametrize("M", [5, 90, 200])
def test_not_a_number_stays_in_its_row(P, gen, M):
    w = Weight(P, gen, 256, 256)
    x, _ = x_of(gen, w, M)
    clean = P.patch_hybrid_linear(w.packed, x, activation="relu")
    x[2, 7] = float("nan")
    got = P.patch_hybrid_linear(w.packed, x, activation="relu")
    rows = torch.arange(M, device="cuda") != 2
    assert torch.equal(got[rows], clean[rows])
    hit = w.weff[:, 7] != 0
    assert torch.isnan(got[2][hit]).all()


def test_large_arguments_of_the_activations(P, gen):
    # sums of a thousand and more: no infinity or NaN out of exp and tanh
    w = Weight(P, gen, 128, 256)
    x = randn(gen, 4, 256, spread=4000.0, dtype=BF)
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        got = P.patch_hybrid_linear(w.packed, x, activation=act, out_fp32=True)
        assert torch.isfinite(got).all()
        check_linear(got, w, x, act=act)


def test_empty_batch(P, gen):
    for kind in ("2:4", "fp8"):
        w = Weight(P, gen, 256, 256, kind)
        x = torch.empty(0, 256, dtype=BF, device="cuda")
        assert P.patch_hybrid_linear(w.packed, x, activation="silu").shape == (0, 256)
        assert P.patch_hybrid_gated(w.packed, w.packed, x).shape == (0, 256)
        assert P.patch_block_norm(x, pre=("rms", None, None, 1e-5))["z"].shape == (0, 256)


def test_refusals(P, gen):
    w, other, f8 = Weight(P, gen, 256, 256), Weight(P, gen, 256, 512), Weight(P, gen, 256, 256, "fp8")
    tall = Weight(P, gen, 384, 256)
    x, _ = x_of(gen, w, 4)
    q, s = quantize(x)
    bad = [dict(bias=randn(gen, 255)), dict(bias=randn(gen, 256).half()), dict(activation="tanh"),
           dict(residual=randn(gen, 3, 256)), dict(residual=randn(gen, 256, 4).t()), dict(x_scales=s),
           dict(out=torch.empty(4, 256, device="cuda")), dict(out=torch.empty(1, 256, dtype=BF, device="cuda").expand(4, 256)),
           dict(bias=torch.zeros(256))]
    for kw in bad:
        with pytest.raises(ValueError):
            P.patch_hybrid_linear(w.packed, x, **kw)
    for args in ((other.packed, x), (w.packed, x.t().contiguous().t()), (f8.packed, q), (w.packed, x.float())):
        with pytest.raises(ValueError):
            P.patch_hybrid_linear(*args)
    with pytest.raises(ValueError):
        P.patch_hybrid_linear(f8.packed, q, x_scales=s[:3])
    with pytest.raises(ValueError, match="one per handle"):
        P.patch_hybrid_linear_group([w.packed, w.packed], x, biases=[None])
    closed = Weight(P, gen, 256, 256).packed
    closed.close()
    with pytest.raises(P.PatchError):
        P.patch_hybrid_linear(closed, x)
    with pytest.raises(ValueError):
        P.patch_hybrid_gated(w.packed, tall.packed, x)
    with pytest.raises(ValueError):
        P.patch_hybrid_gated(f8.packed, w.packed, q, x_scales=s)
    # Y at the residual's address with another stride
    wide = torch.zeros(8, 512, dtype=BF, device="cuda")
    with pytest.raises(P.PatchError):
        P.patch_hybrid_linear(w.packed, x, residual=wide[:4, :256], out=wide.view(-1)[:1024].view(4, 256))
    # members of a group that write what another writes or reads
    r = torch.zeros(4, 256, dtype=BF, device="cuda")
    with pytest.raises(P.PatchError):
        P.patch_hybrid_linear_group([w.packed, w.packed], x, outs=[r, r])
    with pytest.raises(P.PatchError):
        P.patch_hybrid_linear_group([w.packed, w.packed], x, outs=[r, None], residuals=[r, r])
    # through the C ABI: bad flags, strides and alignment are errors, nothing runs
    lib, y = P.load_library(), torch.full((4, 256), 7.0, dtype=BF, device="cuda")

    def call(x_ptr=None, y_ptr=None, M=4, **kw):
        e = P.PatchEpilogue(alpha=1.0)
        for k, v in kw.items():
            setattr(e, k, v)
        return lib.patch_hybrid_linear(w.packed.handle, x_ptr or x.data_ptr(), None, M, y_ptr or y.data_ptr(), 0,
                                       ctypes.byref(e), P._stream(None))

    assert call(activation=5) == 1 and call(activation=-1) == 1 and call(y_stride=255) == 1
    assert call(residual=y.data_ptr() + 512, residual_stride=10) == 1 and call(bias=y.data_ptr() + 1) == 1
    assert call(bias_is_fp32=3) == 1 and call(x_ptr=x.data_ptr() + 2) == 1 and call(y_ptr=y.data_ptr() + 1) == 1
    assert call(M=-1) == 1 and call(M=1 << 31) == 1
    torch.cuda.synchronize()
    assert (y == 7).all()
    assert call() == 0


# ------------------------------------------------------------------- norms
def norm64(v, spec):
    kind, weight, bias, eps = spec
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / (v.pow(2).mean(1, keepdim=True) + eps).sqrt()
    v = v if weight is None else v * weight.double()
    return v if bias is None else v + bias.double()


def check_norm(P, branch, residual=None, gate=None, scale=1.0, post=None, pre=None, z_type="bf16", h_fp32=False, **kw):
    """Runs the call and holds it to the definition.

    fp32 sums of C squares, each added at most ~C / 32 times in a row per
    thread and then over 10 levels, are off by (C / 32 + 16) * 2^-24 relative;
    half of that reaches the quotient, the mean's share is as large in units of
    the row's mean |v|.  Each elementwise step adds 2^-24: with two norms,
    e = (C / 32 + 48) * 2^-24 of the magnitudes involved."""
    M, C = branch.shape
    b0, r0 = branch.clone(), None if residual is None else residual.clone()
    got = P.patch_block_norm(branch, residual=residual, gate=gate, scale=scale, post=post, pre=pre, z_type=z_type,
                             h_fp32=h_fp32, **kw)
    e = (C / 32 + 48) * 2.0 ** -24
    v = b0.double()
    size = v.abs()
    if post:
        top = v.abs().mean(1, keepdim=True) if post[0] == "layer" else 0
        n = norm64(v, (post[0], None, None, post[3]))
        inv = 1 / ((v - (v.mean(1, keepdim=True) if post[0] == "layer" else 0)).pow(2).mean(1, keepdim=True) + post[3]).sqrt()
        wt = 1 if post[1] is None else post[1].double().abs()
        size = (n.abs() + (size + top) * inv) * wt + (0 if post[2] is None else post[2].double().abs())
        v = norm64(v, post)
    gated = v * scale
    size = size * abs(scale)
    if gate is not None:
        gm = gate.double().view(-1, C).repeat_interleave(M // (1 if gate.dim() == 1 else gate.shape[0]), 0)
        gated, size = gated * gm, size * gm.abs()
    h = gated if r0 is None else gated + r0.double()
    size = size + h.abs() + (0 if r0 is None else r0.double().abs())
    tol_h = e * size
    close(got["h"], h, tol_h)
    if got["z"] is None:
        return got
    z, tol_z = h, tol_h
    if pre:
        layer = pre[0] == "layer"
        mean = h.mean(1, keepdim=True) if layer else torch.zeros_like(h[:, :1])
        inv = 1 / ((h - mean).pow(2).mean(1, keepdim=True) + pre[3]).sqrt()
        wt = 1 if pre[1] is None else pre[1].double().abs()
        rms_tol = tol_h.pow(2).mean(1, keepdim=True).sqrt()  # what h's error does to the mean and the norm
        n = (h - mean) * inv
        tol_n = (tol_h + rms_tol + e * (h.abs() + h.abs().mean(1, keepdim=True))) * inv + n.abs() * (rms_tol * inv + e)
        z = norm64(h, pre)
        tol_z = tol_n * wt + 2.0 ** -23 * (n.abs() * wt + (0 if pre[2] is None else pre[2].double().abs()))
    if z_type != "e4m3":
        close(got["z"], z, tol_z)
        return got
    amax = z.abs().amax(1)
    s = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    close(got["scales"], s, tol_z.amax(1) / 448)
    # a code is within half a step (2^-4 relative, 2^-10 below the normals) of
    # z over the scale that was written
    scaled = z / got["scales"].double()[:, None]
    codes = got["z"].view(torch.float8_e4m3fn).double()
    t = tol_z / got["scales"].double()[:, None] + 2.0 ** -23 * scaled.abs()
    assert ((codes - scaled).abs() <= t + torch.maximum(2.0 ** -4 * (scaled.abs() + t), torch.full_like(t, 2.0 ** -10))).all()
    return got


WIDTHS = [1, 2, 7, 8, 33, 64, 100, 256, 1000, 1001, 2048, 4096, 5120, 11008, 16384, 32768]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("M", [1, 2, 37, 300])
def test_norm_widths(P, gen, C, M):
    wt = randn(gen, C, spread=0.2) + 1
    check_norm(P, randn(gen, M, C, dtype=BF), randn(gen, M, C, dtype=BF), pre=("rms", wt.to(BF), None, 1e-5))
    check_norm(P, randn(gen, M, C) + 3, pre=("layer", wt, randn(gen, C), 1e-6), z_type="fp32", h_fp32=True)
    check_norm(P, randn(gen, M, C, dtype=BF), randn(gen, M, C), scale=0.5, gate=randn(gen, C), post=("rms", wt, None, 1e-5),
               pre=("layer", None, None, 1e-5), z_type="e4m3", h_fp32=True)


@pytest.mark.parametrize("z_type", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("types", [(BF, BF, BF), (F32, BF, F32), (BF, F32, BF), (F32, F32, F32)], ids=str)
@pytest.mark.parametrize("kinds", [(None, "rms"), ("rms", "rms"), ("layer", "layer"), ("rms", None), ("layer", "rms")], ids=str)
def test_norm_types(P, gen, kinds, types, z_type):
    M, C = 24, 520
    b, r, p = types
    spec = [None if k is None else (k, randn(gen, C, dtype=p), randn(gen, C, dtype=p), 1e-5) for k in kinds]
    for gate in (None, randn(gen, C, dtype=p), randn(gen, 8, C, dtype=b), randn(gen, M, C, dtype=p)):
        check_norm(P, randn(gen, M, C, dtype=b), randn(gen, M, C, dtype=r), gate, -0.5, *spec, z_type=z_type,
                   h_fp32=p == F32)


@pytest.mark.parametrize("shift", [0, 1])
def test_norm_strides_and_rows_behind(P, gen, shift):
    M, C = 19, 264
    big = [randn(gen, M + 2, C + 40 + shift, dtype=BF) for _ in range(4)]
    keep = [t.clone() for t in big]
    view = [t[1:M + 1, 8 + shift:8 + shift + C] for t in big]
    wt = randn(gen, 2 * C + shift, dtype=BF)[C + shift:]
    check_norm(P, view[0], view[1], pre=("rms", wt, None, 1e-5), out_h=view[2], out_z=view[3])
    assert torch.equal(big[0], keep[0]) and torch.equal(big[1], keep[1])
    for t, k in zip(big[2:], keep[2:]):
        k[1:M + 1, 8 + shift:8 + shift + C] = t[1:M + 1, 8 + shift:8 + shift + C]
        assert torch.equal(t, k)


@pytest.mark.parametrize("M,C", [(3, 1000), (40, 77), (4096, 4096)])
def test_norm_alone(P, gen, M, C):
    # no residual stream is written: a plain norm, and a plain quantisation
    b = randn(gen, M, C, dtype=BF)
    pre = ("rms", randn(gen, C, dtype=BF), None, 1e-5)
    got = P.patch_block_norm(b, pre=pre, want_h=False)
    assert got["h"] is None and torch.equal(got["z"], P.patch_block_norm(b, pre=pre)["z"])
    if C % 8 == 0:
        e = P.patch_block_norm(b, z_type="e4m3", want_h=False)
        q, s = P.patch_quantize_fp8(b)
        assert torch.equal(e["z"], q) and torch.equal(e["scales"], s)
    with pytest.raises(P.PatchError):
        P.patch_block_norm(b, want_h=False)


def test_norm_in_place(P, gen):
    M, C = 33, 1000
    pre = ("rms", randn(gen, C, dtype=BF), None, 1e-5)
    b, r = randn(gen, M, C, dtype=BF), randn(gen, M, C, dtype=BF)
    want = P.patch_block_norm(b, residual=r, pre=pre)
    got = P.patch_block_norm(b, residual=r, pre=pre, out_h=r, out_z=b)
    assert got["h"] is r and torch.equal(r, want["h"]) and torch.equal(b, want["z"])


def test_norm_special_rows(P, gen):
    M, C = 6, 512
    b = randn(gen, M, C, dtype=BF)
    b[1] = 0
    b[2, 5] = float("inf")
    b[3, 6] = float("nan")
    b[4] = 3e38
    b[5] = 1e-30
    clean = P.patch_block_norm(b[:1].clone(), pre=("rms", None, None, 1e-5))
    for kind in ("rms", "layer"):
        got = P.patch_block_norm(b, pre=(kind, None, None, 1e-5))
        assert torch.isfinite(got["z"][[0, 1, 5]].float()).all() and (got["z"][1] == 0).all()
        assert torch.isnan(got["z"][3].float()).all()
        # one multiplication by 1: every value as it was (which NaN a NaN becomes is not defined)
        assert ((got["h"] == b) | (torch.isnan(got["h"]) & torch.isnan(b))).all()
    assert torch.equal(P.patch_block_norm(b, pre=("rms", None, None, 1e-5))["z"][:1], clean["z"])
    e = P.patch_block_norm(torch.zeros(2, C, dtype=BF, device="cuda"), pre=("rms", None, None, 1e-5), z_type="e4m3")
    assert (e["z"] == 0).all() and (e["scales"] == 1).all()
    # a constant row has no variance: the layer norm is the bias, exactly
    bias = randn(gen, C)
    flat = P.patch_block_norm(torch.full((2, C), 0.375, device="cuda"), pre=("layer", None, bias, 1e-5), z_type="fp32")
    assert torch.equal(flat["z"], bias.expand(2, C))


def test_norm_large_mean_keeps_its_variance(P, gen):
    # a mean of 1000 with a spread of 1: E[v^2] - E[v]^2 in fp32 would lose it
    b = randn(gen, 8, 4096) + 1000
    check_norm(P, b, pre=("layer", None, None, 1e-5), z_type="fp32", h_fp32=True)


def test_norm_codes_feed_the_fp8_products(P, gen):
    w = [Weight(P, gen, 256, 512, "fp8") for _ in range(3)]
    for M in (1, 33, 260):
        b, r = randn(gen, M, 512, dtype=BF), randn(gen, M, 512, dtype=BF)
        n = check_norm(P, b, r, pre=("rms", randn(gen, 512, dtype=BF), None, 1e-5), z_type="e4m3")
        for y, v in zip(P.patch_hybrid_linear_group([v.packed for v in w], n["z"], x_scales=n["scales"]), w):
            check_linear(y, v, n["z"], n["scales"])


def test_quantised_input_equals_the_library_s_own(P, gen):
    # the codes patch_quantize_fp8 writes give bit for bit what a bf16 X gives
    w = Weight(P, gen, 512, 512, "fp8")
    for M in (2, 70, 300):
        x = randn(gen, M, 512, dtype=BF)
        q, s = P.patch_quantize_fp8(x)
        assert torch.equal(P.patch_hybrid_linear(w.packed, q, x_scales=s), P.patch_hybrid_linear(w.packed, x))
        assert torch.equal(P.patch_hybrid_gated(w.packed, w.packed, q, x_scales=s),
                           P.patch_hybrid_gated(w.packed, w.packed, x))


# ---------------------------------------------------------- used together
class Block:
    """An MLP block as a program runs it: norm, gated pair, down projection into the residual stream."""

    def __init__(self, P, g, kind, D=256, H=512):
        self.P, self.kind = P, kind
        self.gate, self.up, self.down = Weight(P, g, H, D, kind), Weight(P, g, H, D, kind), Weight(P, g, D, H, kind)
        self.pre = ("rms", randn(g, D, spread=0.2, dtype=BF) + 1, None, 1e-5)
        self.post = ("rms", randn(g, D, spread=0.2, dtype=BF) + 1, None, 1e-5)

    def __call__(self, attn, stream):
        P = self.P
        n = P.patch_block_norm(attn, residual=stream, post=self.post, pre=self.pre,
                               z_type="e4m3" if self.kind == "fp8" else "bf16", out_h=stream)
        m = P.patch_hybrid_gated(self.gate.packed, self.up.packed, n["z"], x_scales=n["scales"])
        y = P.patch_hybrid_linear(self.down.packed, m, residual=stream, out=stream, alpha=0.5)
        return n, m, y


@pytest.mark.parametrize("kind", ["2:4", "fp8", "4:8"])
@pytest.mark.parametrize("M", [1, 9, 50, 100, 333])
def test_block(P, gen, kind, M):
    block = Block(P, gen, kind)
    attn, res = randn(gen, M, 256, dtype=BF), randn(gen, M, 256, dtype=BF)
    check_norm(P, attn, res, post=block.post, pre=block.pre)
    stream = res.clone()
    n, m, y = block(attn, stream)
    h = P.patch_block_norm(attn, residual=res, post=block.post)["h"]
    check_gated(m, block.gate, block.up, n["z"], n["scales"])
    check_linear(y, block.down, m, alpha=0.5, residual=h)
    assert y.data_ptr() == stream.data_ptr()


@pytest.mark.parametrize("kind", ["2:4", "fp8"])
@pytest.mark.parametrize("M", [1, 100, 300])
def test_captured_and_replayed(P, gen, kind, M):
    # a graph of the block replays on new inputs, between eager calls
    block = Block(P, gen, kind)
    attn, res = randn(gen, M, 256, dtype=BF), randn(gen, M, 256, dtype=BF)
    block(attn, res.clone())
    a, s = torch.empty_like(attn), torch.empty_like(res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _, m, y = block(a, s)
    for k in range(3):
        attn, res = randn(gen, M, 256, dtype=BF), randn(gen, M, 256, dtype=BF)
        a.copy_(attn)
        s.copy_(res)
        graph.replay()
        got = [m.clone(), y.clone()]
        _, m1, y1 = block(attn, res)
        assert torch.equal(got[0], m1) and torch.equal(got[1], y1)


def test_other_stream(P, gen):
    # the work and its outputs belong to the stream that is given
    block = Weight(P, gen, 512, 512)
    side = torch.cuda.Stream()
    x = randn(gen, 200, 512, dtype=BF)
    want = P.patch_hybrid_linear(block.packed, x, activation="silu")
    n0 = P.patch_block_norm(x, pre=("rms", None, None, 1e-5))["z"]
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        y = P.patch_hybrid_linear(block.packed, x, activation="silu", stream=side)
        z = P.patch_block_norm(y, pre=("rms", None, None, 1e-5), stream=side)["z"]
        n = P.patch_block_norm(x, pre=("rms", None, None, 1e-5), stream=side)["z"]
        del y  # its memory goes back to the side stream, not to this one
        junk = torch.full((200, 512), float("nan"), dtype=BF, device="cuda")
    side.synchronize()
    del junk
    assert torch.equal(n, n0)
    assert torch.equal(z, P.patch_block_norm(want, pre=("rms", None, None, 1e-5))["z"])


def test_results_do_not_depend_on_the_run(P, gen):
    # no atomics in any sum: every run gives the same bits
    block = Block(P, gen, "2:4", D=512, H=1024)
    for M in (1, 16, 64, 100, 300):
        attn, res = randn(gen, M, 512, dtype=BF), randn(gen, M, 512, dtype=BF)
        first = [t.clone() for t in block(attn, res.clone())[1:]]
        for _ in range(3):
            again = block(attn, res.clone())[1:]
            assert all(torch.equal(u, v) for u, v in zip(first, again))


@pytest.mark.parametrize("spread", [1.0, 1e-30, 1e-36, 1e25])
def test_norm_codes_are_the_rounded_quotients(P, gen, spread):
    # the codes are those of the fp32 row divided by its scale, bit for bit
    for M, C in ((64, 4096), (300, 1032), (33, 999)):
        b = randn(gen, M, C) * spread
        z = P.patch_block_norm(b, pre=("rms", randn(gen, C), None, 0.0), z_type="fp32", h_fp32=True)["z"]
        e = P.patch_block_norm(b, pre=("rms", randn(gen, C), None, 0.0), z_type="e4m3", h_fp32=True)
        raw = P.patch_block_norm(b, z_type="e4m3", h_fp32=True)
        for codes, row in ((raw, b),):
            q, s = quantize(row)
            assert torch.equal(codes["scales"], s)
            assert torch.equal(codes["z"], q.view(torch.uint8))
        assert z.shape == e["z"].shape


def test_first_call_inside_a_capture():
    # a program whose first norm of a kind runs inside a stream capture
    import subprocess
    import sys
    code = """
import torch
from sparse_gemm_wanda_b200 import patch as P
x = torch.randn(64, 4096, device="cuda").bfloat16()
big = torch.randn(4096, 4096, device="cuda").bfloat16()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    z = P.patch_block_norm(x, pre=("rms", None, None, 1e-5))["z"]
    y = P.patch_block_norm(big, residual=big, pre=("rms", None, None, 1e-5))["z"]
graph.replay()
torch.cuda.synchronize()
for got, row in ((z, x.double()), (y, 2 * big.double())):
    want = row / (row.pow(2).mean(1, keepdim=True) + 1e-5).sqrt()
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()
print("replayed")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("M,C", [(4096, 4096), (3001, 5120), (1500, 8192), (900, 16384), (20000, 1024)])
def test_norm_many_rows(P, gen, M, C):
    # the sizes that run through the shared-memory ring, with every part of it present and absent
    bf = dict(dtype=BF)
    b, r = randn(gen, M, C, **bf), randn(gen, M, C, **bf)
    rms = lambda: ("rms", randn(gen, C, spread=0.2, **bf) + 1, None, 1e-5)  # noqa: E731
    check_norm(P, b, r, pre=rms())
    check_norm(P, b, None, pre=("rms", None, None, 1e-5), scale=0.5)
    check_norm(P, b, r, gate=randn(gen, C, **bf), scale=-0.5, post=rms(), pre=rms())
    check_norm(P, b, r, gate=randn(gen, 1, C), post=("rms", None, None, 1e-5), pre=None)
    check_norm(P, b, r, post=("rms", randn(gen, C), None, 1e-5), pre=("rms", randn(gen, C), None, 1e-5), z_type="e4m3")
    # rows further apart than C, in place
    wide_b, wide_r = randn(gen, M, C + 8, **bf), randn(gen, M, C + 16, **bf)
    want = P.patch_block_norm(wide_b[:, :C].contiguous(), residual=wide_r[:, :C].contiguous(), pre=rms())
    keep = wide_r[:, C:].clone()
    got = P.patch_block_norm(wide_b[:, :C], residual=wide_r[:, :C], out_h=wide_r[:, :C])
    assert torch.equal(got["h"], want["h"]) and torch.equal(wide_r[:, C:], keep)


@pytest.mark.parametrize("kind,kernel,M", [("2:4", 0, 8), ("fp8", 0, 8), ("2:4", 1, 300), ("2:4", 2, 300), ("2:4", 3, 300),
                                           ("4:8", 0, 100)])
def test_a_wait_that_runs_out_raises_the_status(P, gen, kind, kernel, M):
    # a k-step that never lands ends every form of a product through its
    # bounded waits; the status is read and cleared, and the next call is right
    # (the kernels that have the hook: all but the FP8 prefill ones)
    wg, wu = Weight(P, gen, 512, 512, kind), Weight(P, gen, 512, 512, kind)
    x, _ = x_of(gen, wg, M)
    res = randn(gen, M, 512, dtype=BF)

    def calls():
        yield P.patch_hybrid_linear(wg.packed, x, activation="silu", residual=res)
        yield P.patch_hybrid_gated(wg.packed, wu.packed, x)

    P.test_prefill_kernel(kernel)
    try:
        for i in range(2):
            P.test_stall_first_kstep(True)
            try:
                next(c for k, c in enumerate(calls()) if k == i)
            finally:
                P.test_stall_first_kstep(False)
            assert P.patch_get_status(wg.packed) == 5  # PATCH_ERR_TIMEOUT
            P.patch_get_status(wu.packed)
        y, z = calls()
        torch.cuda.synchronize()
    finally:
        P.test_prefill_kernel(0)
    assert P.patch_get_status(wg.packed) == 0 and P.patch_get_status(wu.packed) == 0
    check_linear(y, wg, x, act="silu", residual=res)
    check_gated(z, wg, wu, x)


@pytest.mark.parametrize("kernel", [1, 3])
@pytest.mark.parametrize("kind", ["2:4", "fp8"])
def test_rows_beyond_32_bit_offsets(P, gen, kind, kernel):
    # rows so far apart that the last ones start above 2^31 elements
    M, N, step = 2100, 256, (1 << 20) + 8
    wg, wu = Weight(P, gen, N, 256, kind), Weight(P, gen, N, 256, kind)
    x, _ = x_of(gen, wg, M)
    stream = torch.empty(M * step, dtype=BF, device="cuda").view(M, step)[:, 16:16 + N]
    res = randn(gen, M, N, dtype=BF)
    stream.copy_(res)
    P.test_prefill_kernel(kernel)
    try:
        check_linear(P.patch_hybrid_linear(wg.packed, x, residual=stream, out=stream), wg, x, residual=res)
        check_gated(P.patch_hybrid_gated(wg.packed, wu.packed, x, out=stream), wg, wu, x)
    finally:
        P.test_prefill_kernel(0)
    del stream
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,C,step", [(2100, 520, (1 << 20) + 8), (2100, 333, (1 << 20) + 5), (10000, 1024, 1 << 18)])
def test_norm_rows_beyond_32_bit_offsets(P, gen, M, C, step):
    b, r = randn(gen, M, C, dtype=BF), randn(gen, M, C, dtype=BF)
    pre = ("rms", randn(gen, C, dtype=BF), None, 1e-5)
    wide = torch.empty(M * step, dtype=BF, device="cuda").view(M, step)
    views = [wide[:, i * C:(i + 1) * C] for i in range(3)] if C % 8 else [wide[:, i * 2048:i * 2048 + C] for i in range(3)]
    views[0].copy_(b)
    views[1].copy_(r)
    check_norm(P, views[0], views[1], pre=pre, out_h=views[1], out_z=views[2])
    del wide, views
    torch.cuda.empty_cache()


@pytest.mark.parametrize("shift", [4, 8])
def test_norm_fp32_rows_on_16_and_32_byte_boundaries(P, gen, shift):
    M, C = 9, 256
    big = [randn(gen, M, C + 16) for _ in range(4)]
    b, r, h, z = [t[:, shift:shift + C] for t in big]
    wt = randn(gen, C + 8)[shift:shift + C]
    check_norm(P, b, r, post=("rms", wt, None, 1e-5), pre=("layer", wt, wt, 1e-5), z_type="fp32", h_fp32=True, out_h=h,
               out_z=z)


@pytest.mark.parametrize("kind", ["2:4", "fp8"])
@pytest.mark.parametrize("M", [1, 50, 100, 300])
def test_eight_members(P, gen, kind, M):
    ws = [Weight(P, gen, 128 * (1 + i % 3), 256, kind) for i in range(8)]
    x, _ = x_of(gen, ws[0], M)
    biases = [randn(gen, w.N) for w in ws]
    for y, w, b in zip(P.patch_hybrid_linear_group([w.packed for w in ws], x, biases=biases, activation="relu"), ws, biases):
        check_linear(y, w, x, bias=b, act="relu")


@pytest.mark.parametrize("kind", ["2:4", "fp8", "4:8"])
@pytest.mark.parametrize("M", [4, 300])
def test_two_streams_at_once(P, gen, kind, M):
    # different handles on different streams share nothing
    blocks = [Block(P, gen, kind) for _ in range(2)]
    attn, res = randn(gen, M, 256, dtype=BF), randn(gen, M, 256, dtype=BF)
    want = [[t.clone() for t in b(attn, res.clone())[1:]] for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (b, s) in enumerate(zip(blocks, streams)):
            with torch.cuda.stream(s):
                got[i].append(b(attn, res.clone())[1:])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(u, v) for u, v in zip(w, run))


def test_an_output_on_top_of_the_input_is_refused(P, gen):
    w = Weight(P, gen, 256, 256)
    for M in (3, 300):
        x, _ = x_of(gen, w, M)
        keep = x.clone()
        for call in (lambda: P.patch_hybrid_linear(w.packed, x, out=x), lambda: P.patch_hybrid_gated(w.packed, w.packed, x, out=x),
                     lambda: P.patch_hybrid_linear_group([w.packed, w.packed], x, outs=[None, x])):
            with pytest.raises(P.PatchError):
                call()
        torch.cuda.synchronize()
        assert torch.equal(x, keep)


@pytest.mark.parametrize("C", [515, 1001, 4100, 5247, 8186, 8193, 13491, 16381, 16385, 30001, 32761, 32767])
@pytest.mark.parametrize("M", [1, 11, 300])
def test_norm_rows_between_boundaries(P, gen, C, M):
    # rows that start at every place between two 16-byte boundaries
    bf = dict(dtype=BF)
    rms = ("rms", randn(gen, C, spread=0.2, **bf) + 1, None, 1e-5)
    layer = ("layer", randn(gen, C, **bf), randn(gen, C, **bf), 1e-5)
    check_norm(P, randn(gen, M, C, **bf), randn(gen, M, C, **bf), pre=rms)
    check_norm(P, randn(gen, M, C, **bf), randn(gen, M, C), gate=randn(gen, C, **bf), post=layer, pre=rms, z_type="e4m3",
               h_fp32=True)
    f32 = ("rms", randn(gen, C), None, 1e-5)
    check_norm(P, randn(gen, M, C), randn(gen, M, C), post=f32, pre=rms, z_type="fp32")
    check_norm(P, randn(gen, M, C), None, gate=randn(gen, M, C, **bf), pre=layer)


@pytest.mark.parametrize("C,step", [(1001, 1003), (1000, 1003), (5000, 5001), (9001, 9008)])
def test_norm_wide_rows_between_boundaries_in_place(P, gen, C, step):
    # in place, rows further apart than C, nothing around them moves; the
    # tensors' places agree in the first two calls and differ in the third
    M = 21
    pre = ("rms", randn(gen, C, dtype=BF), None, 1e-5)
    for shifts in ((0, 0, 0), (3, 3, 3), (3, 1, 2)):
        big = [randn(gen, M + 1, step + 8 - step % 8 + step % 8, dtype=BF).view(-1)[: M * step + 8] for _ in range(3)]
        view = [t[k: k + M * step].view(M, step)[:, :C] for t, k in zip(big, shifts)]
        keep = [t.clone() for t in big]
        check_norm(P, view[0], view[1], scale=0.5, pre=pre, out_h=view[1], out_z=view[2])
        assert torch.equal(big[0], keep[0])
        for i in (1, 2):
            keep[i][shifts[i]: shifts[i] + M * step].view(M, step)[:, :C] = view[i]
            assert torch.equal(big[i], keep[i])


@pytest.mark.parametrize("kind", ["2:4", "4:8", "fp8"])
@pytest.mark.parametrize("M", [20, 100, 300])
def test_members_side_by_side_read_a_finished_input(P, gen, kind, M):
    # products that run one after another as single kernels may overlap: each
    # reads the X that the kernel before the group has just written
    ws = [Weight(P, gen, n, 640, kind) for n in (384, 128, 384)]
    packed = [w.packed for w in ws]
    rows = [randn(gen, M, 640, dtype=BF) for _ in range(2)]
    z = torch.empty(M, 640, dtype=torch.uint8 if kind == "fp8" else BF, device="cuda")
    res = randn(gen, M, 384, dtype=BF)

    def step(i):
        n = P.patch_block_norm(rows[i], pre=("layer", None, None, 1e-5), z_type="e4m3" if kind == "fp8" else "bf16",
                               want_h=False, out_z=z)
        ys = P.patch_hybrid_linear_group(packed, z, x_scales=n["scales"], activation="silu", residuals=[res, None, res])
        g = P.patch_hybrid_gated(packed[0], packed[2], z, x_scales=n["scales"])
        # reads the group's outputs at once
        return *ys, g, P.patch_block_norm(g, residual=ys[2], want_h=True)["h"], n["scales"]

    want = []
    for i in range(2):
        n = P.patch_block_norm(rows[i], pre=("layer", None, None, 1e-5), z_type="e4m3" if kind == "fp8" else "bf16",
                               want_h=False)
        torch.cuda.synchronize()
        one = P.patch_hybrid_linear_group(packed, n["z"], x_scales=n["scales"], activation="silu", residuals=[res, None, res])
        torch.cuda.synchronize()
        want.append((n, one))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(0)
    for k in range(30):
        graph.replay()
        got = [step(1), step(0), step(1)]
        torch.cuda.synchronize()
        for i, g in ((0, captured), (1, got[0]), (0, got[1]), (1, got[2])):
            n, one = want[i]
            for y, y1, w, r in zip(g, one, ws, (res, None, res)):
                assert torch.equal(y, y1)  # the same kernels on the same X
                if k == 0:
                    check_linear(y, w, n["z"], n["scales"], act="silu", residual=r)
            if k == 0:
                check_gated(g[3], ws[0], ws[2], n["z"], n["scales"])
            h = g[3].double() + g[2].double()
            assert ((g[4].double() - h).abs() <= 2.0 ** -8 * h.abs() + 1e-6).all()


@pytest.mark.parametrize("kind", ["2:4", "fp8"])
@pytest.mark.parametrize("bands", [1, 149, 200, 297, 700])
def test_short_k_and_many_bands(P, gen, kind, bands):
    # bands of one chunk: more of them than blocks, claimed at run time, call after call
    w = Weight(P, gen, 128 * bands, 256, kind)
    other = Weight(P, gen, 256, 256, kind)
    for M in (3, 40):
        x, _ = x_of(gen, w, M)
        b, r = randn(gen, w.N), randn(gen, M, w.N, dtype=BF)
        first = P.patch_hybrid_linear(w.packed, x, bias=b, residual=r, activation="silu")
        check_linear(first, w, x, bias=b, residual=r, act="silu")
        for _ in range(3):
            assert torch.equal(P.patch_hybrid_linear(w.packed, x, bias=b, residual=r, activation="silu"), first)
            ys = P.patch_hybrid_linear_group([w.packed, other.packed, w.packed], x, biases=[b, None, b], activation="silu",
                                             residuals=[r, None, r])
            assert torch.equal(ys[0], first) and torch.equal(ys[2], first)
            check_linear(ys[1], other, x, act="silu")
        # the plain product shares the handle's counter
        plain = P.patch_hybrid_gemm(w.packed, x, out_fp32=True)
        assert torch.equal(P.patch_hybrid_linear(w.packed, x, out_fp32=True), plain)
        assert torch.equal(P.patch_hybrid_gemm(w.packed, x, out_fp32=True), plain)
