"""Cases that time and check the operators of a gated block with a layer norm and an 8-bit head: both projections of a gated
feed-forward layer with the activation and the product, its backward pass, the product of int8 rows with int8 weights of one
scale a channel, the layer norm into int8 rows, and its backward pass.

Each case names an operator (`op`), sizes, a type (`kind`: bf16 or f32) and what the call is given.  `run` computes it with
elementary torch operations in 32 bits, or, with `own` set, through the framework's entry points; `exact` computes it in 64
bits.  int8 results are returned as the values they stand for (q times its row's scale, in bfloat16).

The sizes are the framework's own: widths 243, 729, 1280, 3456 and 16384, batches of 1, 27, 1782, 4096 and 16384 rows.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "relu2", "silu", "gelu_tanh")
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715
# scales of the two weight matrices of a gated layer, in units of 1 / sqrt(k)
GATE_SCALE, UP_SCALE = 1.25, 0.9


def listed():
    return [
        # one token through both projections of a gated layer
        {"name": "gated 1x3456x1280 silu", "op": "gated", "rows": 1, "n": 3456, "k": 1280, "kind": "bf16", "bias": False,
         "act": "silu", "train": False},
        # a prompt, float32 activations, with biases
        {"name": "gated 1782x3456x1280 gelu f32", "op": "gated", "rows": 1782, "n": 3456, "k": 1280, "kind": "f32",
         "bias": True, "act": "gelu_tanh", "train": False},
        # the largest training batch, both pre-activations kept for the backward pass
        {"name": "gated 16384x3456x1280 silu", "op": "gated", "rows": 16384, "n": 3456, "k": 1280, "kind": "bf16",
         "bias": False, "act": "silu", "train": True},
        # the small trainer's backward batch at its odd width
        {"name": "gated_bwd 27x729 f32", "op": "gated_bwd", "rows": 27, "cols": 729, "kind": "f32", "act": "gelu_tanh",
         "bias": True},
        # the gated layer's backward over the largest batch: the int8 rows for dX, the values for dW, the biases' gradients
        {"name": "gated_bwd 16384x3456 bf16", "op": "gated_bwd", "rows": 16384, "cols": 3456, "kind": "bf16", "act": "silu",
         "bias": True},
        # one token's logits from an 8-bit head
        {"name": "s8s8 1x16384x1280 f32", "op": "s8s8", "rows": 1, "n": 16384, "k": 1280, "kind": "f32", "channels": True,
         "bias": False, "act": "none", "residual": False, "train": False},
        # a down projection of a backward batch into the residual stream
        {"name": "s8s8 1782x1280x3456", "op": "s8s8", "rows": 1782, "n": 1280, "k": 3456, "kind": "bf16", "channels": True,
         "bias": True, "act": "none", "residual": True, "train": False},
        # an 8-bit first layer over the largest batch, the pre-activation kept
        {"name": "s8s8 16384x3456x1280 gelu", "op": "s8s8", "rows": 16384, "n": 3456, "k": 1280, "kind": "bf16",
         "channels": True, "bias": True, "act": "gelu_tanh", "residual": False, "train": True},
        # one token of a decode step enters a block
        {"name": "layernorm 1x1280 bf16", "op": "layernorm", "rows": 1, "cols": 1280, "kind": "bf16", "residual": True,
         "beta": True, "train": False},
        # a training batch enters a block; the normed values, the means and 1 / deviation are kept
        {"name": "layernorm 16384x1280 bf16", "op": "layernorm", "rows": 16384, "cols": 1280, "kind": "bf16",
         "residual": True, "beta": True, "train": True},
        # the small trainer's rows and its odd width, float32, no gradient from a residual branch
        {"name": "layernorm_bwd 27x243 f32", "op": "layernorm_bwd", "rows": 27, "cols": 243, "kind": "f32",
         "residual": False, "beta": True},
        # the backward of a wide norm over a training batch, the residual branch's gradient added
        {"name": "layernorm_bwd 16384x3456 bf16", "op": "layernorm_bwd", "rows": 16384, "cols": 3456, "kind": "bf16",
         "residual": True, "beta": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gated", "gated_bwd", "s8s8", "layernorm", "layernorm_bwd"))
    kind = rng.choice(("bf16", "f32"))
    rows = _log(rng, 1, 16384)
    if op in ("gated", "s8s8"):
        n, k = _log(rng, 16, 4096 if op == "gated" else 16384), _log(rng, 64, 4096)
        if op == "gated":
            k -= k % rng.choice((4, 64))   # rows of the stored weights are whole bytes
        elif rng.random() < 0.7:
            k -= k % rng.choice((16, 64))  # else a contraction of any length
        rows = max(1, min(rows, 16384 * 3456 * 1280 // (n * k), 16384 * 3456 // (n * (2 if kind == "f32" else 1))))
        case = {"op": op, "rows": rows, "n": n, "k": k, "kind": kind, "bias": rng.random() < 0.5, "act": rng.choice(ACTS),
                "train": rng.random() < 0.5}
        if op == "s8s8":
            case |= {"channels": rng.random() < 0.8, "residual": rng.random() < 0.5}
        return case
    cols = _log(rng, 64, 8192 if op == "gated_bwd" else 16384)
    if rng.random() < 0.5:
        cols -= cols % 8
    rows = max(1, min(rows, 16384 * 3456 // (cols * (2 if kind == "f32" else 1))))
    case = {"op": op, "rows": rows, "cols": cols, "kind": kind}
    if op == "gated_bwd":
        case |= {"act": rng.choice(ACTS), "bias": rng.random() < 0.7}
    else:
        case |= {"residual": rng.random() < 0.7, "beta": rng.random() < 0.7}
        if op == "layernorm":
            case |= {"train": rng.random() < 0.5}
    return case


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE)

    def int8_rows(r, c):
        # as the row quantizer leaves them: the largest magnitude of a row is 127
        a = normal(r, c).clamp_(-4, 4)
        a[:, 0] = 4.0
        return (a * (127 / 4)).round_().to(torch.int8)

    dt = DTYPE[case["kind"]]
    op, R = case["op"], case["rows"]
    if op in ("gated", "s8s8"):
        N, K = case["n"], case["k"]
        s["A"] = int8_rows(R, K)
        s["a_scale"] = 0.005 + 0.05 * uniform(R)
        if op == "gated":
            # the gate's weights, then the up projection's, stored as the ternary products store theirs
            codes = torch.randint(0, 3, (2 * N, K // 4, 4), generator=g, device=DEVICE, dtype=torch.uint8)
            s["W"] = codes[..., 0] | (codes[..., 1] << 2) | (codes[..., 2] << 4) | (codes[..., 3] << 6)
            s["gate_scale"], s["up_scale"] = GATE_SCALE / math.sqrt(K), UP_SCALE / math.sqrt(K)
            s["bias"] = normal(2 * N) * 0.1 if case["bias"] else None
            return s
        s["W"] = int8_rows(N, K)
        s["w_scale"] = (0.5 + uniform(N)) * (4 / 127 / math.sqrt(K)) if case["channels"] else None
        if not case["channels"]:
            s["a_scale"] *= 4 / 127 / math.sqrt(K)
        s["bias"] = normal(N) * 0.1 if case["bias"] else None
        s["residual"] = normal(R, N).to(dt) if case["residual"] else None
        return s
    C = case["cols"]
    if op == "gated_bwd":
        s["dY"] = (normal(R, C) * 1e-3).to(dt)
        s["Z"] = (normal(R, 2 * C) * 1.5).to(dt)
        s["gate_scale"], s["up_scale"] = GATE_SCALE / 36, UP_SCALE / 36
        s["values"] = torch.empty(R, 2 * C, dtype=torch.bfloat16, device=DEVICE)
        return s
    # activations with a few channels far larger than the rest, each about a value of its own, and rows of padding
    channel = 0.5 + uniform(C) + 6.0 * (uniform(C) < 0.01)
    padding = (torch.arange(R, device=DEVICE) % 61 != 60).float()[:, None]
    s["gain"] = 1.0 + 0.1 * normal(C)
    s["beta"] = 0.1 * normal(C) if case["beta"] else None
    h = (normal(R, C) + 0.5 * normal(C)) * channel * padding
    if op == "layernorm":
        s["X"] = h.to(dt)
        s["residual"] = (normal(R, C) * channel * padding).to(dt) if case["residual"] else None
        s["values"] = torch.empty(R, C, dtype=torch.bfloat16, device=DEVICE)
    else:
        s["H"] = h.to(dt)
        hd = s["H"].double()
        mean = hd.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = ((hd - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
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
    if op == "gated":
        Y, Z = B.ternary_gemm_s8_gated(s["A"], s["W"], s["a_scale"], s["gate_scale"], s["up_scale"], bias=s["bias"],
                                       act=c["act"], out_dtype=DTYPE[c["kind"]], save=c["train"])
        return {"Y": Y, "Z": Z} if c["train"] else {"Y": Y}
    if op == "gated_bwd":
        dZ, dbias, Q, scale = B.ternary_gated_backward(s["dY"], s["Z"], s["gate_scale"], s["up_scale"], act=c["act"],
                                                       bias=c["bias"])
        return _bwd_outputs(c, dZ, dbias, torch.mul(Q, scale[:, None], out=s["values"]), scale)
    if op == "s8s8":
        Y, Z = B.ternary_gemm_s8s8_epilogue(s["A"], s["W"], s["a_scale"], s["w_scale"], bias=s["bias"], act=c["act"],
                                            residual=s["residual"], out_dtype=DTYPE[c["kind"]], save=c["train"])
        return {"Y": Y, "Z": Z} if c["train"] else {"Y": Y}
    if op == "layernorm":
        Q, scale, H, Y, mean, rstd = B.ternary_layernorm_quantize(s["X"], s["gain"], s["beta"], EPS, residual=s["residual"],
                                                                  save=c["train"])
        return _norm_outputs(c, torch.mul(Q, scale[:, None], out=s["values"]), scale, H, Y, mean, rstd)
    dX, dgain, dbeta = B.ternary_layernorm_backward(s["dY"], s["H"], s["gain"], s["mean"], s["rstd"], dH=s["dH"],
                                                    beta=c["beta"])
    return {"dX": dX, "dgain": dgain, "dbeta": dbeta} if c["beta"] else {"dX": dX, "dgain": dgain}


def _bwd_outputs(c, dZ, dbias, values, scale):
    out = {"dZ": dZ, "values": values, "scale": scale}
    if c["bias"]:
        out["dbias"] = dbias
    return out


def _norm_outputs(c, values, scale, H, Y, mean, rstd):
    out = {"values": values, "scale": scale}
    if c["residual"]:
        out["H"] = H
    if c["train"]:
        out |= {"Y": Y, "mean": mean, "rstd": rstd}
    return out


def _quantized(y):
    scale = y.abs().amax(1) / 127
    q = torch.round(y / scale[:, None]).clamp(-127, 127)
    q = torch.where(scale[:, None] > 0, q, torch.zeros_like(q))
    return (q * scale[:, None]).to(torch.bfloat16), scale


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


def _plain_gated(s):
    c = s["case"]
    dt, N = DTYPE[c["kind"]], c["n"]
    shifts = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=s["W"].device)
    code = (s["W"][:, :, None] >> shifts) & 3
    w = ((code & 1).float() - (code >> 1).float()).reshape(2 * N, c["k"])
    z = s["A"].float() @ w.t()    # whole numbers below 2^24: exact in 32 bits in any order
    z = z * s["a_scale"][:, None]
    z = torch.cat((z[:, :N] * s["gate_scale"], z[:, N:] * s["up_scale"]), 1)
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _activation(z[:, :N], c["act"]) * z[:, N:]
    return {"Y": y.to(dt), "Z": z.to(dt)} if c["train"] else {"Y": y.to(dt)}


def _plain_gated_bwd(s):
    c = s["case"]
    C, dy = c["cols"], s["dY"].float()
    gate, up = s["Z"][:, :C].float(), s["Z"][:, C:].float()
    dgate, dup = dy * up * _slope(gate, c["act"]), dy * _activation(gate, c["act"])
    dz = torch.cat((dgate, dup), 1)
    # the rows that the product with the stored weights takes: each half times its matrix's scale
    values, scale = _quantized(torch.cat((dgate * s["gate_scale"], dup * s["up_scale"]), 1))
    return _bwd_outputs(c, dz.to(s["dY"].dtype), dz.sum(0), values, scale)


def _plain_s8s8(s):
    c = s["case"]
    dt = DTYPE[c["kind"]]
    # products of whole numbers below 2^14: 512 of them add up exactly in 32 bits, the parts' sums are added in 64
    z = 0
    for k in range(0, c["k"], 512):
        z = z + (s["A"][:, k:k + 512].float() @ s["W"][:, k:k + 512].float().t()).double()
    z = z.float() * s["a_scale"][:, None]
    if s["w_scale"] is not None:
        z = z * s["w_scale"]
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _activation(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"Y": y.to(dt), "Z": z.to(dt)} if c["train"] else {"Y": y.to(dt)}


def _plain_layernorm(s):
    c = s["case"]
    dt = s["X"].dtype
    H = s["X"]
    if s["residual"] is not None:
        H = (s["X"].float() + s["residual"].float()).to(dt)   # the residual stream is kept in its own type, and the norm is of what is kept
    h = H.float()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None] * s["gain"]
    if s["beta"] is not None:
        y = y + s["beta"]
    values, scale = _quantized(y)
    return _norm_outputs(c, values, scale, H, y.to(dt), mean, rstd)


def _plain_layernorm_bwd(s):
    c = s["case"]
    dy = s["dY"].float()
    xhat = (s["H"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    t = dy * s["gain"]
    dx = s["rstd"][:, None] * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    out = {"dX": dx.to(s["H"].dtype), "dgain": (dy * xhat).sum(0)}
    return out | {"dbeta": dy.sum(0)} if c["beta"] else out


_PLAIN = {"gated": _plain_gated, "gated_bwd": _plain_gated_bwd, "s8s8": _plain_s8s8, "layernorm": _plain_layernorm,
          "layernorm_bwd": _plain_layernorm_bwd}


# ---------------------------------------------------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    e = 2 if case["kind"] == "bf16" else 4
    op, R = case["op"], case["rows"]
    if op == "gated":
        N, K = case["n"], case["k"]
        out = R * N * e * (1 + 2 * case["train"])
        return {"bytes": R * K + N * K // 2 + 4 * R + 8 * N * case["bias"] + out, "flops": 4 * R * N * K}
    if op == "s8s8":
        N, K = case["n"], case["k"]
        out = R * N * e * (1 + case["train"] + case["residual"])
        return {"bytes": R * K + N * K + 4 * R + 4 * N * (case["bias"] + case["channels"]) + out, "flops": 2 * R * N * K}
    C = case["cols"]
    n = R * C
    if op == "gated_bwd":
        return {"bytes": n * e * 5 + 2 * n + 8 * C * case["bias"] + 4 * R, "flops": 30 * n}
    if op == "layernorm":
        moved = n * e * (1 + 2 * case["residual"] + case["train"]) + n + 4 * C * (1 + case["beta"])
        return {"bytes": moved + 4 * R * (1 + 2 * case["train"]), "flops": 11 * n}
    return {"bytes": n * e * (3 + case["residual"]) + 4 * C * (2 + case["beta"]) + 8 * R, "flops": 14 * n}


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
    if op == "gated":
        n = case["n"]
        # the codes of place i in every byte meet columns i, i + 4, ... of A
        acc = 0
        for i in range(4):
            code = torch.div(s["W"], 4 ** i, rounding_mode="floor") % 4
            w = (code == 1).double() - (code == 2).double()
            acc = acc + torch.matmul(s["A"][:, i::4].double(), w.t())
        parts = []
        for i, scale in enumerate((s["gate_scale"], s["up_scale"])):
            z = acc[:, i * n:i * n + n] * (s["a_scale"].double()[:, None] * scale)
            parts.append(z if s["bias"] is None else z + s["bias"][i * n:i * n + n].double())
        y = _act64(parts[0], case["act"])[0] * parts[1]
        return {"Y": y, "Z": torch.cat(parts, dim=1)} if case["train"] else {"Y": y}
    if op == "gated_bwd":
        gy = s["dY"].double()
        gate, up = s["Z"].double().chunk(2, dim=1)
        a, slope = _act64(gate, case["act"])
        dg, du = gy * slope * up, gy * a
        values, step = _rows_int8(torch.cat((s["gate_scale"] * dg, s["up_scale"] * du), dim=1))
        dz = torch.cat((dg, du), dim=1)
        return _bwd_outputs(case, dz, dz.sum(dim=0), values, step)
    if op == "s8s8":
        z = torch.matmul(s["A"].double(), s["W"].double().t())
        z = torch.mul(z, s["a_scale"].double().unsqueeze(1))
        if case["channels"]:
            z = torch.mul(z, s["w_scale"].double().unsqueeze(0))
        if case["bias"]:
            z = z + s["bias"].double()
        y = _act64(z, case["act"])[0]
        if case["residual"]:
            y = y + s["residual"].double()
        return {"Y": y, "Z": z} if case["train"] else {"Y": y}
    if op == "layernorm":
        h = s["X"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(DTYPE[case["kind"]]).double()
        var, mu = torch.var_mean(h, dim=1, correction=0)
        inv = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(torch.zeros_like(h) if s["beta"] is None else s["beta"].double().expand_as(h),
                          (h - mu[:, None]) * inv[:, None], s["gain"].double().expand_as(h))
        values, step = _rows_int8(y)
        return _norm_outputs(case, values, step, h, y, mu, inv)
    h, gy, inv = s["H"].double() - s["mean"].double()[:, None], s["dY"].double(), s["rstd"].double()[:, None]
    gg = gy * s["gain"].double()
    c = case["cols"]
    dx = inv * gg - inv * gg.sum(1, keepdim=True) / c - inv ** 3 * h * (gg * h).sum(1, keepdim=True) / c
    if case["residual"]:
        dx = dx + s["dH"].double()
    out = {"dX": dx, "dgain": (gy * h * inv).sum(0)}
    return out | {"dbeta": gy.sum(0)} if case["beta"] else out
