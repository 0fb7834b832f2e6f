"""Measured cases of the operators that surround the tile-hybrid linear layers.

Three operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and, where ``own`` is set, as the calls a user makes
of the library:

* ``linear``: Y_i = residual_i + alpha * act(X W_eff_i^T + bias_i) for one
  packed weight, or for several that read the same X (q/k/v);
* ``gated``: Y = act(X W_gate^T + b_gate) * (X W_up^T + b_up), the gated pair
  of an MLP;
* ``norm``: h = residual + scale * gate * norm_post(branch), z = norm_pre(h),
  the boundary between two sublayers, z in bf16, fp32 or e4m3 codes with a
  scale per token (the input of an FP8 linear layer).

W_eff is W with the pruned entries of its 2:4 (or 4:8) tiles set to zero; FP8
weights and activations are e4m3 codes with one scale per row, s = amax / 448.
"""
from __future__ import annotations

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


# ------------------------------------------------------------------- cases
def _linear(name, N, K, M, **kw):
    case = {"name": name, "op": "linear", "N": N, "K": K, "M": M, "f": 0.6, "tn": 128, "tk": 128, "kind": "2:4",
            "codes": False, "group": 1, "act": "none", "bias": "", "residual": "", "alpha": 1.0}
    case.update(kw)
    return case


def _gated(name, N, K, M, **kw):
    case = {"name": name, "op": "gated", "N": N, "K": K, "M": M, "f": 0.6, "tn": 128, "tk": 128, "kind": "2:4",
            "codes": False, "act": "silu", "bias": ""}
    case.update(kw)
    return case


def _norm(name, M, C, **kw):
    case = {"name": name, "op": "norm", "M": M, "C": C, "residual": "bf16", "h": "bf16", "branch": "bf16",
            "gate": 0, "scale": 1.0, "post": "", "pre": "rms", "weight": "bf16", "z": "bf16"}
    case.update(kw)
    return case


def listed():
    return [
        # one decoded token: the attention output projection added to the residual stream
        _linear("o_residual_m1", 4096, 4096, 1, residual="bf16"),
        # q/k/v of an FP8 layer for a batch of 16 decoded tokens, with biases, on the codes a norm wrote
        _linear("qkv_fp8_codes_m16", 4096, 4096, 16, kind="fp8", codes=True, group=3, bias="bf16"),
        # a small encoder layer with fine tiles and a ragged batch: bias and GELU
        _linear("fc1_gelu_m300", 1024, 2048, 300, f=0.5, tn=64, tk=64, act="gelu", bias="fp32"),
        # the MLP's down projection of a short prefill, scaled, into the residual stream
        _linear("down_residual_m512", 4096, 11008, 512, residual="bf16", alpha=0.5),
        # the largest: a 13B-shaped down projection of a long prefill
        _linear("down13b_residual_m4096", 5120, 13824, 4096, f=0.75, residual="bf16", bias="bf16"),
        # the gated pair for a batch of 8 decoded tokens
        _gated("gated_m8", 11008, 4096, 8),
        # the gated pair of a short prefill
        _gated("gated_m512", 11008, 4096, 512),
        # the gated pair of an FP8 layer, prefill, tanh GELU
        _gated("gated_fp8_m2048", 11008, 4096, 2048, kind="fp8", act="gelu_tanh"),
        # one decoded token between attention and MLP: residual add and RMS norm
        _norm("norm_m1", 1, 4096),
        # prefill with norms before and after the block, a learned gate and a residual scale
        _norm("norm_sandwich_m4096", 4096, 5120, post="rms", gate=1, scale=0.7),
        # prefill into an FP8 layer, the residual stream held in 32 bits
        _norm("norm_e4m3_m2048", 2048, 4096, residual="fp32", h="fp32", z="e4m3"),
        # layer norms of an odd width, a gate per sample of three, 32-bit parameters
        _norm("norm_layer_odd", 777, 1001, post="layer", pre="layer", gate=3, weight="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "gated", "norm"))
    if op == "norm":
        M = _log(rng, 1, 6000)
        C = min(_log(rng, 64, 16384), 40_000_000 // M)
        if rng.random() < 0.6:
            C = max(8, C // 8 * 8)
        pre = rng.choice(("rms", "layer"))
        gate = rng.choice((0, 0, 1, M))
        return {"op": "norm", "M": M, "C": C, "residual": rng.choice(("", "bf16", "bf16", "fp32")),
                "h": rng.choice(("bf16", "fp32")), "branch": rng.choice(("bf16", "bf16", "fp32")), "gate": gate,
                "scale": rng.choice((1.0, 0.5)), "post": rng.choice(("", "", "rms", "layer")), "pre": pre,
                "weight": rng.choice(("bf16", "fp32")),
                "z": rng.choice(("bf16", "bf16", "fp32", "e4m3")) if C % 8 == 0 else rng.choice(("bf16", "fp32"))}
    kind = rng.choice(("2:4", "2:4", "2:4", "fp8", "fp8", "4:8"))
    M = _log(rng, 1, 4096)
    N = 128 * _log(rng, 1, 108)
    K = 128 * _log(rng, 1, 108)
    while (2 if op == "gated" else 1) * M * N * K > 4096 * 5120 * 13824:
        M = (M + 1) // 2
    case = {"op": op, "N": N, "K": K, "M": M, "f": rng.choice((0.0, 0.25, 0.5, 0.6, 0.75, 1.0)),
            "tn": rng.choice((64, 128, 128)), "tk": rng.choice((64, 128, 128)), "kind": kind,
            "codes": kind == "fp8" and rng.random() < 0.5, "act": rng.choice(ACTS), "bias": rng.choice(("", "bf16", "fp32"))}
    if op == "linear":
        case |= {"group": rng.choice((1, 1, 2, 3)) if M * N * K < 1 << 36 else 1,
                 "residual": rng.choice(("", "bf16", "fp32")), "alpha": rng.choice((1.0, 0.5))}
    return case


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """N(0, 1) with one channel in a hundred scaled by 20 (the outlier channels of decoder layers)."""
    x = _randn(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 20
    return x.to(torch.bfloat16)


def _quantize(x):
    """Row-wise e4m3: s = amax / 448 (1 for a zero row), q = e4m3(x / s), the quotient in 32 bits."""
    x = x.float()
    amax = x.abs().amax(dim=1)
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / s[:, None]).to(torch.float8_e4m3fn), s


def _weight(g, case):
    """W, its pattern codes and tile map in the library's layouts, and W_eff.

    Of every 4 (8) consecutive weights of a row the 2 (4) of highest |w| times
    a channel norm are kept; floor(f * tiles) random tiles are sparse."""
    N, K, tn, tk = case["N"], case["K"], case["tn"], case["tk"]
    w = (_randn(g, N, K) * 0.02).to(torch.bfloat16)
    norm = _randn(g, K).abs() + 0.5
    size = 8 if case["kind"] == "4:8" else 4
    score = (w.float().abs() * norm).view(N, K // size, size)
    at = torch.arange(size, device="cuda")
    ahead = torch.zeros_like(score, dtype=torch.int8)
    for j in range(size):
        sj = score[..., j:j + 1]
        ahead += (sj > score) | ((sj == score) & (j < at))
    keep = ahead < size // 2
    if size == 8:
        code = (keep.long() << at).sum(-1)
    else:
        first = keep.to(torch.int8).argmax(-1)
        last = 3 - keep.flip(-1).to(torch.int8).argmax(-1)
        code = first | (last << 2)
    words = code.view(N, K // 32, 32 // size) << (size * torch.arange(32 // size, device="cuda"))
    meta = words.sum(-1).to(torch.int32)
    tiles = (N // tn) * (K // tk)
    sparse = torch.zeros(-(-tiles // 32) * 32, dtype=torch.long, device="cuda")
    sparse[torch.randperm(tiles, generator=g, device="cuda")[: int(math.floor(case["f"] * tiles))]] = 1
    tmap = (sparse.view(-1, 32) << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
    wide = sparse[:tiles].view(N // tn, K // tk).repeat_interleave(tn, 0).repeat_interleave(tk, 1).bool()
    weff = torch.where(wide & ~keep.view(N, K), torch.zeros_like(w), w)
    return w, meta, tmap, weff


def _vector(g, kind, n, spread):
    return (_randn(g, n) * spread).to(_dtype(kind)) if kind else None


def _inputs(case, seed):
    """Every input of the case, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] == "norm":
        M, C = case["M"], case["C"]
        d = {"branch": (_randn(g, M, C) * 1.5 + 0.2).to(_dtype(case["branch"])), "residual": None, "gate": None}
        if case["residual"]:
            d["residual"] = (_activations(g, M, C).float() * 0.7).to(_dtype(case["residual"]))
        if case["gate"]:
            gate = (_randn(g, case["gate"], C) * 0.2 + 0.8).to(_dtype(case["weight"]))
            d["gate"] = gate[0] if case["gate"] == 1 else gate
        for which in ("post", "pre"):
            kind = case[which]
            d[which] = None
            if kind:
                weight = (_randn(g, C) * 0.2 + 1).to(_dtype(case["weight"]))
                d[which] = (kind, weight, _vector(g, case["weight"] if kind == "layer" else "", C, 0.2), EPS)
        return d
    M, N, K = case["M"], case["N"], case["K"]
    d = {"X": _activations(g, M, K), "x_scales": None, "weights": []}
    for _ in range(2 if case["op"] == "gated" else case["group"]):
        w, meta, tmap, weff = _weight(g, case)
        e = {"W": w, "meta": meta, "map": tmap, "weff": weff, "bias": _vector(g, case["bias"], N, 0.5)}
        if case["kind"] == "fp8":
            e["weff"], e["w_scales"] = _quantize(weff)
        if case.get("residual"):
            e["residual"] = _randn(g, M, N).to(_dtype(case["residual"]))
        d["weights"].append(e)
    if case["codes"]:
        d["X"], d["x_scales"] = _quantize(d["X"])
    return d


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own and case["op"] != "norm":
        # a program packs its weights once, when it loads them
        from sparse_gemm_wanda_b200 import patch as P
        if case["codes"]:
            state["X"] = state["X"].view(torch.uint8)
        for e in state["weights"]:
            if case["kind"] == "fp8":
                e["packed"] = P.patch_pack_fp8(e["W"], e["meta"], e["map"], tile_n=case["tn"], tile_k=case["tk"])
            else:
                nm = (4, 8) if case["kind"] == "4:8" else (2, 4)
                e["packed"] = P.patch_pack(e["W"], e["meta"], e["map"], tile_n=case["tn"], tile_k=case["tk"], nm=nm)
    return state


# --------------------------------------------------------------- operators
def _act(v, kind):
    if kind == "relu":
        return v.clamp_min(0)
    if kind == "gelu":
        return 0.5 * v * (1 + torch.erf(v * (0.5 ** 0.5)))
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _product(state, e):
    """X W_eff^T (+ bias) in 32 bits."""
    if state["case"]["kind"] == "fp8":
        xq, sx = (state["X"], state["x_scales"]) if state["case"]["codes"] else _quantize(state["X"])
        y = (xq.float() @ e["weff"].float().t()) * e["w_scales"] * sx[:, None]
    else:
        y = state["X"].float() @ e["weff"].float().t()
    return y if e["bias"] is None else y + e["bias"].float()


def _normed(v, spec):
    kind, weight, bias, eps = spec
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps) * weight.float()
    return v if bias is None else v + bias.float()


def _plain_norm(state):
    case = state["case"]
    h = state["branch"].float()
    if state["post"]:
        h = _normed(h, state["post"])
    h = h * case["scale"]
    if state["gate"] is not None:
        gate = state["gate"].float().view(-1, case["C"])
        h = h * gate.repeat_interleave(case["M"] // gate.shape[0], 0)
    if state["residual"] is not None:
        h = h + state["residual"].float()
    z = _normed(h, state["pre"])
    out = {"h": h.to(_dtype(case["h"]))}
    if case["z"] == "e4m3":
        out["z"], out["scales"] = _quantize(z)
    else:
        out["z"] = z.to(_dtype(case["z"]))
    return out


def _own_norm(state):
    from sparse_gemm_wanda_b200 import patch as P
    case = state["case"]
    r = P.patch_block_norm(state["branch"], residual=state["residual"], gate=state["gate"], scale=case["scale"],
                           post=state["post"], pre=state["pre"], z_type=case["z"], h_fp32=case["h"] == "fp32")
    out = {"h": r["h"], "z": r["z"]}
    if case["z"] == "e4m3":
        out["z"], out["scales"] = r["z"].view(torch.float8_e4m3fn), r["scales"]
    return out


def _own_products(state):
    from sparse_gemm_wanda_b200 import patch as P
    case, ws = state["case"], state["weights"]
    if case["op"] == "gated":
        return P.patch_hybrid_gated(ws[0]["packed"], ws[1]["packed"], state["X"], x_scales=state["x_scales"],
                                    bias_gate=ws[0]["bias"], bias_up=ws[1]["bias"], activation=case["act"])
    if len(ws) == 1:
        return [P.patch_hybrid_linear(ws[0]["packed"], state["X"], x_scales=state["x_scales"], bias=ws[0]["bias"],
                                      activation=case["act"], alpha=case["alpha"], residual=ws[0].get("residual"))]
    return P.patch_hybrid_linear_group([e["packed"] for e in ws], state["X"], x_scales=state["x_scales"],
                                       biases=[e["bias"] for e in ws], activation=case["act"], alpha=case["alpha"],
                                       residuals=[e.get("residual") for e in ws])


def run(state):
    case = state["case"]
    if case["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if own:
        return _own_products(state)
    if case["op"] == "gated":
        gate, up = state["weights"]
        return (_act(_product(state, gate), case["act"]) * _product(state, up)).to(torch.bfloat16)

    def one(e):
        y = _act(_product(state, e), case["act"]) * case["alpha"]
        return (y if e.get("residual") is None else y + e["residual"].float()).to(torch.bfloat16)

    return [one(e) for e in state["weights"]]


# ------------------------------------------------- the definition in 64 bits
def _exact_norm(case, d):
    M, C = case["M"], case["C"]

    def norm(rows, spec):
        kind, weight, bias, eps = spec
        mean = rows.sum(1, keepdim=True) / C if kind == "layer" else torch.zeros_like(rows[:, :1])
        var = ((rows - mean) ** 2).sum(1, keepdim=True) / C
        out = (rows - mean) * (var + eps) ** -0.5 * weight.double()
        return out + bias.double() if bias is not None else out

    b = d["branch"].double()
    if d["post"]:
        b = norm(b, d["post"])
    gate = d["gate"].double().view(-1, 1, C) if d["gate"] is not None else torch.ones(1, 1, C, dtype=torch.double, device="cuda")
    h = (case["scale"] * b.view(gate.shape[0], -1, C) * gate).reshape(M, C)
    if d["residual"] is not None:
        h = h + d["residual"].double()
    z = norm(h, d["pre"])
    if case["z"] != "e4m3":
        return {"h": h, "z": z}
    top = z.abs().max(dim=1).values
    scales = torch.where(top > 0, top / 448, torch.ones_like(top))
    return {"h": h, "z": z / scales[:, None], "scales": scales}


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, d)
    x = d["X"]
    if case["kind"] == "fp8":
        # the codes are part of the definition: one quotient in 32 bits, rounded to e4m3
        q, s = (x, d["x_scales"]) if case["codes"] else _quantize(x)
        x = q.double() * s.double()[:, None]
    x = x.double()
    outs = []
    for e in d["weights"]:
        w = e["weff"].double()
        if case["kind"] == "fp8":
            w = w * e["w_scales"].double()[:, None]
        y = torch.einsum("mk,nk->mn", x, w)
        if e["bias"] is not None:
            y += e["bias"].double()
        outs.append(y)

    def activate(v):
        if case["act"] == "relu":
            return torch.where(v > 0, v, torch.zeros_like(v))
        if case["act"] == "gelu":
            return v * torch.special.ndtr(v)
        if case["act"] == "gelu_tanh":
            return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
        if case["act"] == "silu":
            return v * torch.sigmoid(v)
        return v

    if case["op"] == "gated":
        return activate(outs[0]) * outs[1]
    for i, e in enumerate(d["weights"]):
        outs[i] = activate(outs[i]) * case["alpha"]
        if e.get("residual") is not None:
            outs[i] = outs[i] + e["residual"].double()
    return outs


# -------------------------------------------------------------------- work
def _bytes_of(name):
    return {"": 0, "bf16": 2, "fp32": 4, "e4m3": 1}[name]


def work(case):
    M = case["M"]
    if case["op"] == "norm":
        C = case["C"]
        each = _bytes_of(case["branch"]) + _bytes_of(case["residual"]) + _bytes_of(case["h"]) + _bytes_of(case["z"])
        once = _bytes_of(case["weight"]) * (case["gate"] + sum({"": 0, "rms": 1, "layer": 2}[case[k]] for k in ("post", "pre")))
        return {"bytes": M * C * each + once * C + (4 * M if case["z"] == "e4m3" else 0),
                "flops": M * C * (6 + 4 * (case["post"] != "") + 2 * (case["gate"] > 0))}
    N, K, f = case["N"], case["K"], case["f"]
    count = 2 if case["op"] == "gated" else case["group"]
    # values and pattern bits of a weight: 2:4 and 4:8 tiles keep half the values and one bit a weight
    value = 1 if case["kind"] == "fp8" else 2
    weights = N * K * (value * (1 - f) + (value / 2 + 0.125) * f) + (4 * N if case["kind"] == "fp8" else 0)
    x = M * K * (1 if case["codes"] else 2) + (4 * M if case["codes"] else 0)
    per = N * _bytes_of(case["bias"]) + M * N * _bytes_of(case.get("residual", ""))
    y = 2 * M * N * (1 if case["op"] == "gated" else count)
    return {"bytes": count * (weights + per) + x + y, "flops": count * 2 * M * N * K * (1 - f / 2)}
