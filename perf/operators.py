"""Cases that time and check the operators around the ternary product: the RMS norm with its residual addition and int8
output, the product with bias, activation and residual in its epilogue, the backward passes of both, and the clipping of
many gradients by their global norm.

Each case names an operator (`op`), sizes, a type (`kind`: bf16 or f32) and what the call is given.  `run` computes it with
elementary torch operations in 32 bits, or, with `own` set, through the framework's entry points; `exact` computes it in 64
bits.  int8 results are returned as the values they stand for (q times its row's scale, in bfloat16).

The sizes are the framework's own: widths 243, 729, 1280, 3456 and 16384, batches of 1, 27, 1782, 4096 and 16384 rows.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
MAX_NORM = 1.0
CLIP_EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "relu2", "silu", "gelu_tanh")
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # one token of a decode step enters a block: the norm of the residual stream and the int8 row the product takes
        {"name": "norm 1x1280 bf16", "op": "norm", "rows": 1, "cols": 1280, "kind": "bf16", "residual": True, "train": False},
        # a training batch enters a block; the normed values and 1/rms are kept for the backward pass
        {"name": "norm 16384x1280 bf16", "op": "norm", "rows": 16384, "cols": 1280, "kind": "bf16", "residual": True, "train": True},
        # the small trainer's rows and its odd width, float32, no gradient from a residual branch
        {"name": "norm_bwd 27x243 f32", "op": "norm_bwd", "rows": 27, "cols": 243, "kind": "f32", "residual": False},
        # the backward of a wide norm over a training batch, the residual branch's gradient added
        {"name": "norm_bwd 16384x3456 bf16", "op": "norm_bwd", "rows": 16384, "cols": 3456, "kind": "bf16", "residual": True},
        # one token through an up projection
        {"name": "product 1x3456x1280 relu2", "op": "product", "rows": 1, "n": 3456, "k": 1280, "kind": "bf16", "bias": True,
         "act": "relu2", "residual": False, "train": False},
        # 27 rows through a weight that has to come from memory, added to the residual stream
        {"name": "product 27x16384x16384", "op": "product", "rows": 27, "n": 16384, "k": 16384, "kind": "bf16", "bias": False,
         "act": "none", "residual": True, "train": False},
        # the down projection of a training batch into a float32 residual stream
        {"name": "product 4096x1280x3456 f32", "op": "product", "rows": 4096, "n": 1280, "k": 3456, "kind": "f32", "bias": True,
         "act": "none", "residual": True, "train": False},
        # the up projection of the largest batch with its activation, the pre-activation kept for the backward pass
        {"name": "product 16384x3456x1280 gelu", "op": "product", "rows": 16384, "n": 3456, "k": 1280, "kind": "bf16",
         "bias": True, "act": "gelu_tanh", "residual": False, "train": True},
        # the small trainer's backward batch at its odd width
        {"name": "product_bwd 1782x729 f32", "op": "product_bwd", "rows": 1782, "cols": 729, "kind": "f32", "act": "silu"},
        # the activation's backward over the largest batch: the int8 rows for dX, the values for dW, the bias gradient
        {"name": "product_bwd 16384x3456 bf16", "op": "product_bwd", "rows": 16384, "cols": 3456, "kind": "bf16", "act": "gelu_tanh"},
        # all gradients of the small trainer: seven small tensors a layer
        {"name": "clip 2 layers of 243 f32", "op": "clip", "layers": 2, "d": 243, "f": 729, "embed": 256, "kind": "f32"},
        # the gradients of a few layers of the wide model and its embedding
        {"name": "clip 4 layers of 1280 bf16", "op": "clip", "layers": 4, "d": 1280, "f": 3456, "embed": 16384, "kind": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "product", "product_bwd", "clip"))
    kind = rng.choice(("bf16", "f32"))
    if op == "clip":
        return {"op": op, "layers": rng.randint(1, 4), "d": _log(rng, 64, 1280), "f": _log(rng, 128, 3456),
                "embed": _log(rng, 64, 16384), "kind": kind}
    rows = _log(rng, 1, 16384)
    if op == "product":
        n = _log(rng, 16, 4096)
        k = _log(rng, 64, 4096)
        k -= k % rng.choice((4, 64))   # rows of the stored weights are whole bytes
        rows = min(rows, 16384 * 3456 * 1280 // (n * k))
        return {"op": op, "rows": rows, "n": n, "k": max(k, 64), "kind": kind, "bias": rng.random() < 0.5,
                "act": rng.choice(ACTS), "residual": rng.random() < 0.5, "train": rng.random() < 0.5}
    cols = _log(rng, 64, 16384)
    if rng.random() < 0.5:
        cols -= cols % 8
    rows = max(1, min(rows, 16384 * 3456 // (cols * (2 if kind == "f32" else 1))))
    case = {"op": op, "rows": rows, "cols": cols, "kind": kind}
    if op == "norm":
        case |= {"residual": rng.random() < 0.7, "train": rng.random() < 0.5}
    elif op == "norm_bwd":
        case |= {"residual": rng.random() < 0.7}
    else:
        case |= {"act": rng.choice(ACTS)}
    return case


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _clip_shapes(c):
    d, f = c["d"], c["f"]
    layer = [(d, d), (d, d), (f, d), (d, f), (d,), (d,), (f,)]
    return layer * c["layers"] + [(c["embed"], d)]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE)

    dt = DTYPE[case["kind"]]
    op = case["op"]
    if op == "clip":
        shapes = _clip_shapes(case)
        n = sum(math.prod(x) for x in shapes)
        # gradients whose global norm is about 3, the tensors' own sizes spread over a decade
        s["grads"] = [(normal(*x) * (3.0 / math.sqrt(n)) * 10.0 ** (uniform(1) - 0.5)).to(dt) for x in shapes]
        s["out"] = [torch.empty_like(x) for x in s["grads"]]
        return s
    R = case["rows"]
    if op == "product":
        N, K = case["n"], case["k"]
        # int8 rows as the row quantizer leaves them: the largest magnitude of a row is 127
        a = normal(R, K).clamp_(-4, 4)
        a[:, 0] = 4.0
        s["A"] = (a * (127 / 4)).round_().to(torch.int8)
        s["a_scale"] = 0.005 + 0.05 * uniform(R)
        codes = torch.randint(0, 3, (N, K // 4, 4), generator=g, device=DEVICE, dtype=torch.uint8)
        s["W"] = codes[..., 0] | (codes[..., 1] << 2) | (codes[..., 2] << 4) | (codes[..., 3] << 6)
        s["w_scale"] = 1.0 / math.sqrt(K)
        s["bias"] = normal(N) * 0.1 if case["bias"] else None
        s["residual"] = normal(R, N).to(dt) if case["residual"] else None
        return s
    C = case["cols"]
    if op == "product_bwd":
        s["dY"] = (normal(R, C) * 1e-3).to(dt)
        s["Z"] = (normal(R, C) * 1.5).to(dt)
        s["values"] = torch.empty(R, C, dtype=torch.bfloat16, device=DEVICE)
        return s
    # activations with a few channels far larger than the rest, and rows of padding that are all zero
    channel = 0.5 + uniform(C) + 6.0 * (uniform(C) < 0.01)
    padding = (torch.arange(R, device=DEVICE) % 61 != 60).float()[:, None]
    s["gain"] = 1.0 + 0.1 * normal(C)
    h = normal(R, C) * channel * padding
    if op == "norm":
        s["X"] = h.to(dt)
        s["residual"] = (normal(R, C) * channel * padding).to(dt) if case["residual"] else None
        s["values"] = torch.empty(R, C, dtype=torch.bfloat16, device=DEVICE)
    else:
        s["H"] = h.to(dt)
        s["rstd"] = (s["H"].double().square().mean(1) + EPS).rsqrt().float()
        s["dY"] = (normal(R, C) * 1e-3).to(dt)
        s["dH"] = (normal(R, C) * 1e-3).to(dt) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from ternary_weight_int8_amd import binding as B
    c = s["case"]
    op = c["op"]
    if op == "norm":
        Q, scale, H, Y, rstd = B.ternary_rmsnorm_quantize(s["X"], s["gain"], EPS, residual=s["residual"], save=c["train"])
        return _norm_outputs(c, torch.mul(Q, scale[:, None], out=s["values"]), scale, H, Y, rstd)
    if op == "norm_bwd":
        dX, dgain = B.ternary_rmsnorm_backward(s["dY"], s["H"], s["gain"], s["rstd"], dH=s["dH"])
        return {"dX": dX, "dgain": dgain}
    if op == "product":
        Y, Z = B.ternary_gemm_s8_epilogue(s["A"], s["W"], s["a_scale"], s["w_scale"], bias=s["bias"], act=c["act"],
                                          residual=s["residual"], out_dtype=DTYPE[c["kind"]], save=c["train"])
        return {"Y": Y, "Z": Z} if c["train"] else {"Y": Y}
    if op == "product_bwd":
        dZ, dbias, Q, scale = B.ternary_epilogue_backward(s["dY"], s["Z"], act=c["act"])
        return {"dZ": dZ, "dbias": dbias, "values": torch.mul(Q, scale[:, None], out=s["values"]), "scale": scale}
    out, norm = B.ternary_clip_grad_norm(s["grads"], MAX_NORM, out=s["out"])
    return {"grads": out, "norm": norm}


def _norm_outputs(c, values, scale, H, Y, rstd):
    out = {"values": values, "scale": scale}
    if c["residual"]:
        out["H"] = H
    if c["train"]:
        out |= {"Y": Y, "rstd": rstd}
    return out


def _quantized(y):
    scale = y.abs().amax(1) / 127
    q = torch.round(y / scale[:, None]).clamp(-127, 127)
    q = torch.where(scale[:, None] > 0, q, torch.zeros_like(q))
    return (q * scale[:, None]).to(torch.bfloat16), scale


def _plain_norm(s):
    c = s["case"]
    dt = s["X"].dtype
    H = s["X"]
    if s["residual"] is not None:
        H = (s["X"].float() + s["residual"].float()).to(dt)   # the residual stream is kept in its own type, and the norm is of what is kept
    h = H.float()
    rstd = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * s["gain"]
    values, scale = _quantized(y)
    return _norm_outputs(c, values, scale, H, y.to(dt), rstd)


def _plain_norm_bwd(s):
    dy, xhat, rstd = s["dY"].float(), s["H"].float() * s["rstd"][:, None], s["rstd"]
    t = dy * s["gain"]
    dx = rstd[:, None] * (t - xhat * (t * xhat).mean(1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    return {"dX": dx.to(s["H"].dtype), "dgain": (dy * xhat).sum(0)}


def _activation(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu2":
        return torch.clamp(z, min=0).square()
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(GELU_A * (z + GELU_B * z * z * z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "relu2":
        return 2 * torch.clamp(z, min=0)
    if act == "none":
        return torch.ones_like(z)
    u, du = (z, 1.0) if act == "silu" else (GELU_A * (z + GELU_B * z * z * z), GELU_A * (1 + 3 * GELU_B * z * z))
    p = torch.sigmoid(u)
    return p + z * p * torch.sigmoid(-u) * du


def _plain_product(s):
    c = s["case"]
    dt = DTYPE[c["kind"]]
    shifts = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=s["W"].device)
    code = (s["W"][:, :, None] >> shifts) & 3
    w = ((code & 1).float() - (code >> 1).float()).reshape(c["n"], c["k"])
    z = s["A"].float() @ w.t()    # whole numbers below 2^24: exact in 32 bits in any order
    z = z * s["a_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _activation(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"Y": y.to(dt), "Z": z.to(dt)} if c["train"] else {"Y": y.to(dt)}


def _plain_product_bwd(s):
    dz = s["dY"].float() * _slope(s["Z"].float(), s["case"]["act"])
    values, scale = _quantized(dz)
    return {"dZ": dz.to(s["dY"].dtype), "dbias": dz.sum(0), "values": values, "scale": scale}


def _plain_clip(s):
    norm = torch.stack([x.double().square().sum() for x in s["grads"]]).sum().sqrt().float()
    f = torch.clamp(MAX_NORM / (norm + CLIP_EPS), max=1.0)
    return {"grads": [(x.float() * f).to(x.dtype) for x in s["grads"]], "norm": norm.reshape(1)}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "product": _plain_product, "product_bwd": _plain_product_bwd,
          "clip": _plain_clip}


# ---------------------------------------------------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    e = 2 if case["kind"] == "bf16" else 4
    op = case["op"]
    if op == "clip":
        # read once, written once; a list beyond the caches is read a second time, since the norm comes before the scaling
        n = sum(math.prod(x) for x in _clip_shapes(case))
        return {"bytes": 2 * n * e, "flops": 3 * n}
    if op == "product":
        R, N, K = case["rows"], case["n"], case["k"]
        out = R * N * e * (1 + (1 if case["train"] else 0) + (1 if case["residual"] else 0))
        return {"bytes": R * K + N * K // 4 + 4 * R + (4 * N if case["bias"] else 0) + out, "flops": 2 * R * N * K}
    n, R, C = case["rows"] * case["cols"], case["rows"], case["cols"]
    if op == "norm":
        moved = n * e * (1 + 2 * case["residual"] + case["train"]) + n + 4 * C + 4 * R * (1 + case["train"])
        return {"bytes": moved, "flops": 8 * n}
    if op == "norm_bwd":
        return {"bytes": n * e * (3 + case["residual"]) + 8 * C + 4 * R, "flops": 10 * n}
    return {"bytes": n * e * 3 + n + 4 * C + 4 * R, "flops": 20 * n}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _rows_int8(v):
    top = v.abs().max(dim=1, keepdim=True).values
    step = top / 127
    q = (v / step.clamp_min(1e-300)).round().clamp(min=-127, max=127)
    return q * step, step.flatten()


def _act64(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act in ("relu", "relu2"):
        p = z.clamp_min(0)
        return (p, (z > 0).double()) if act == "relu" else (p * p, 2 * p)
    if act == "silu":
        e = torch.exp(-z)
        return z / (1 + e), (1 + e + z * e) / (1 + e) ** 2
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + GELU_B * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * GELU_B * z * z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["X"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(DTYPE[case["kind"]]).double()
        inv = 1 / torch.sqrt((h ** 2).sum(1) / case["cols"] + EPS)
        y = h * inv[:, None] * s["gain"].double()
        values, step = _rows_int8(y)
        return _norm_outputs(case, values, step, h, y, inv)
    if op == "norm_bwd":
        h, gy, inv = s["H"].double(), s["dY"].double(), s["rstd"].double()[:, None]
        gg = gy * s["gain"].double()
        dx = inv * gg - inv ** 3 * h * (gg * h).sum(1, keepdim=True) / case["cols"]
        if case["residual"]:
            dx = dx + s["dH"].double()
        return {"dX": dx, "dgain": (gy * h * inv).sum(0)}
    if op == "product":
        # the codes of place i in every byte meet columns i, i + 4, ... of A
        z = 0
        for i in range(4):
            code = torch.div(s["W"], 4 ** i, rounding_mode="floor") % 4
            w = (code == 1).double() - (code == 2).double()
            z = z + torch.matmul(s["A"][:, i::4].double(), w.t())
        z = z * (s["a_scale"].double()[:, None] * s["w_scale"])
        if case["bias"]:
            z = z + s["bias"].double()
        y = _act64(z, case["act"])[0]
        if case["residual"]:
            y = y + s["residual"].double()
        return {"Y": y, "Z": z} if case["train"] else {"Y": y}
    if op == "product_bwd":
        dz = s["dY"].double() * _act64(s["Z"].double(), case["act"])[1]
        values, step = _rows_int8(dz)
        return {"dZ": dz, "dbias": dz.sum(dim=0), "values": values, "scale": step}
    norm = sum(float(torch.sum(x.double() ** 2)) for x in s["grads"]) ** 0.5
    f = min(1.0, MAX_NORM / (norm + CLIP_EPS))
    return {"grads": [x.double() * f for x in s["grads"]], "norm": torch.tensor([norm], dtype=torch.float64)}
