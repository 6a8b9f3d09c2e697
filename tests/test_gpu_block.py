"""GPU parity of the operators around the product (norm, epilogue, backward
passes, clipping) with their definitions in 64 bits, at the sizes, widths,
alignments and rows where they can go wrong."""
import sys
import zlib

import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "relu2", "silu", "gelu_tanh")


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def gen(*seed):
    return torch.Generator(device=DEV).manual_seed(zlib.crc32(repr(seed).encode()))


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


class Placed:
    """Matrices at an offset inside larger buffers whose other bytes must stay."""

    def __init__(self, offset):
        self.offset, self.made = offset, []

    def __call__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        esz = torch.empty(0, dtype=dtype).element_size()
        raw = torch.full(((n + 2 * self.offset + 16) * esz,), 0x5A, dtype=torch.uint8, device=DEV)
        self.made.append((raw, self.offset * esz, (self.offset + n) * esz))
        return raw.view(dtype)[self.offset:self.offset + n].view(shape)

    def check(self):
        for raw, lo, hi in self.made:
            assert bool((raw[:lo] == 0x5A).all()) and bool((raw[hi:] == 0x5A).all()), "bytes outside an output changed"


def placed_copy(place, t):
    out = place(tuple(t.shape), t.dtype)
    out.copy_(t)
    return out


# (R, C): one element; narrower than a vector; every register width of the row
# kernels with its neighbours; odd widths; rows past what a workgroup holds;
# more rows than workgroups
ROWS = [(1, 1), (1, 3), (3, 7), (1, 1280), (27, 243), (65, 511), (64, 512), (5, 513), (200, 729), (33, 1280), (61, 2047),
        (9, 2049), (130, 3456), (7, 4104), (3, 8191), (4, 8200), (2, 16384), (3, 16401), (2, 40000), (5000, 64),
        (2600, 320)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", ROWS)
def test_norm(R, C, kind):
    say(f"norm {R}x{C} {kind}")
    dt, g = KINDS[kind], gen(R, C, kind)
    X, res = normal(g, R, C, dtype=dt, scale=3.0), normal(g, R, C, dtype=dt)
    gain = 1 + normal(g, C, scale=0.1)
    if R > 2:
        X[1], res[1] = 0, 0                   # a row of padding
        X[2] = -res[2]                        # a sum that cancels
    for residual, save in ((res, True), (None, True), (res, False), (None, False)):
        Q, s, H, Y, rstd = B.ternary_rmsnorm_quantize(X, gain, 1e-5, residual=residual, save=save)
        if residual is None:
            assert H is X
        else:
            want = X.double() + res.double()
            ref.check(H, want, ref.rounded(want, ref.U * want.abs(), dt), "H")
        r, rel, y, e = ref.norm(H.double(), gain.double(), float(torch.tensor(1e-5)))
        ref.check_int8(Q, s, y, e, "norm")
        if save:
            ref.check(rstd, r, rel * r, "rstd")
            ref.check(Y, y, ref.rounded(y, e, dt), "Y")
            if dt == torch.float32:           # the int8 rows are the row quantizer's of the same values
                q2, s2 = B.ternary_quantize_rows(Y)
                assert torch.equal(q2, Q) and torch.equal(s2, s)
        else:
            assert Y is None and rstd is None


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C,offset", [(5, 243, 1), (37, 1280, 3), (3, 3456, 1), (4, 16384, 5), (3, 40000, 1)])
def test_norm_misaligned_and_in_place(R, C, kind, offset):
    say(f"norm at offset {offset}: {R}x{C} {kind}")
    dt, g = KINDS[kind], gen(R, C, offset)
    X, res, gain = normal(g, R, C, dtype=dt), normal(g, R, C, dtype=dt), 1 + normal(g, C, scale=0.1)
    want = B.ternary_rmsnorm_quantize(X, gain, 1e-6, residual=res, save=True)
    for into in ("X", "residual", "own"):
        p = Placed(offset)
        Xp, rp, gp = placed_copy(p, X), placed_copy(p, res), placed_copy(p, gain)
        H = {"X": Xp, "residual": rp, "own": p((R, C), dt)}[into]
        got = B.ternary_rmsnorm_quantize(Xp, gp, 1e-6, residual=rp, save=True, H=H, Y=p((R, C), dt),
                                         rstd=p((R,), torch.float32), Q=p((R, C), torch.int8),
                                         scale=p((R,), torch.float32))
        torch.cuda.synchronize()
        p.check()
        for a, b in zip(got, want):
            assert torch.equal(a, b), into


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [5, 1280, 5000, 40000])
def test_norm_rows_that_are_not_finite_stay_by_themselves(C, kind):
    say(f"norm not finite {C} {kind}")
    dt, g = KINDS[kind], gen(C, 9)
    X, gain = normal(g, 6, C, dtype=dt), 1 + normal(g, C, scale=0.1)
    clean = B.ternary_rmsnorm_quantize(X, gain, save=True)
    Xb = X.clone()
    Xb[1, C - 1], Xb[4, 0] = float("nan"), float("inf")
    Q, s, _, Y, rstd = B.ternary_rmsnorm_quantize(Xb, gain, save=True)
    for r in (1, 4):
        assert not bool(torch.isfinite(s[r])) and bool((Q[r] == 0).all())
    assert bool(torch.isnan(rstd[1])) and float(rstd[4]) == 0
    keep = [0, 2, 3, 5]
    for a, b in ((Q, clean[0]), (s, clean[1]), (Y, clean[3]), (rstd, clean[4])):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", ROWS + [(1782, 729), (600, 3456)])
def test_norm_backward(R, C, kind):
    say(f"norm backward {R}x{C} {kind}")
    dt, g = KINDS[kind], gen(R, C, kind, 1)
    H, dY, dH = (normal(g, R, C, dtype=dt, scale=x) for x in (2.0, 1e-3, 1e-3))
    if R > 2:
        H[1] = 0
    gain = 1 + normal(g, C, scale=0.1)
    rstd = (H.double().square().mean(1) + 1e-5).rsqrt().float()
    for up in (dH, None):
        dX, dgain = B.ternary_rmsnorm_backward(dY, H, gain, rstd, dH=up)
        dx, e, dg, eg = ref.norm_backward(dY.double(), H.double(), gain.double(), rstd.double(),
                                          None if up is None else up.double())
        ref.check(dX, dx, ref.rounded(dx, e, dt), "dX")
        ref.check(dgain, dg, eg, "dgain")
        again = B.ternary_rmsnorm_backward(dY, H, gain, rstd, dH=up)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dgain)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C,offset", [(5, 243, 1), (300, 1280, 3), (9, 3456, 1), (4, 16384, 5), (3, 40000, 1)])
def test_norm_backward_misaligned_and_in_place(R, C, kind, offset):
    say(f"norm backward at offset {offset}: {R}x{C} {kind}")
    dt, g = KINDS[kind], gen(R, C, offset, 1)
    H, dY, dH = (normal(g, R, C, dtype=dt, scale=x) for x in (2.0, 1e-3, 1e-3))
    gain = 1 + normal(g, C, scale=0.1)
    rstd = (H.double().square().mean(1) + 1e-5).rsqrt().float()
    want = B.ternary_rmsnorm_backward(dY, H, gain, rstd, dH=dH)
    for in_place in (True, False):
        p = Placed(offset)
        args = [placed_copy(p, t) for t in (dY, H, gain, rstd, dH)]
        got = B.ternary_rmsnorm_backward(*args[:4], dH=args[4], dX=args[4] if in_place else p((R, C), dt),
                                         dgain=p((C,), torch.float32))
        torch.cuda.synchronize()
        p.check()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("R,C", [(1, 1), (3, 7), (27, 243), (65, 511), (200, 729), (33, 1280), (9, 2049), (600, 3456),
                                 (3, 8191), (2, 16384), (3, 16401), (2, 40000), (5000, 64)])
def test_epilogue_backward(R, C, act, kind):
    say(f"epilogue backward {R}x{C} {act} {kind}")
    dt, g = KINDS[kind], gen(R, C, kind, act)
    dY, Z = normal(g, R, C, dtype=dt, scale=1e-2), normal(g, R, C, dtype=dt, scale=2.0)
    Z[0, 0], Z[-1, -1] = 0, 60
    if R > 2:
        dY[1] = 0
        Z[2] = -150                            # every slope of the row is 0 (or 1 without an activation)
    dz, e, db, eb = ref.epilogue_backward(dY.double(), Z.double(), act)
    dZ, dbias, Q, s = B.ternary_epilogue_backward(dY, Z, act=act)
    ref.check(dZ, dz, ref.rounded(dz, e, dt), "dZ")
    ref.check(dbias, db, eb, "dbias")
    ref.check_int8(Q, s, dz, e, "dZ")
    if dt == torch.float32:
        q2, s2 = B.ternary_quantize_rows(dZ)
        assert torch.equal(q2, Q) and torch.equal(s2, s)
    alone = B.ternary_epilogue_backward(dY, Z, act=act, bias=False)
    assert alone[1] is None
    for i in (0, 2, 3):
        assert torch.equal(alone[i], (dZ, dbias, Q, s)[i])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C,offset", [(5, 243, 1), (300, 1280, 3), (9, 3456, 1), (4, 16384, 5), (3, 40000, 1)])
def test_epilogue_backward_misaligned(R, C, kind, offset):
    say(f"epilogue backward at offset {offset}: {R}x{C} {kind}")
    dt, g = KINDS[kind], gen(R, C, offset, 2)
    dY, Z = normal(g, R, C, dtype=dt, scale=1e-2), normal(g, R, C, dtype=dt, scale=2.0)
    want = B.ternary_epilogue_backward(dY, Z, act="silu")
    p = Placed(offset)
    got = B.ternary_epilogue_backward(placed_copy(p, dY), placed_copy(p, Z), act="silu", dZ=p((R, C), dt),
                                      dbias=p((C,), torch.float32), Q=p((R, C), torch.int8),
                                      scale=p((R,), torch.float32))
    torch.cuda.synchronize()
    p.check()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ACTS)
def test_epilogue_backward_far_and_not_finite(act):
    say(f"epilogue backward far values {act}")
    z = torch.tensor([-3e38, -1e20, -300.0, -88.5, -87.0, -0.0, 0.0, 87.0, 88.5, 300.0, 1e20, 3e38], device=DEV)
    Z = z.repeat(3, 1)
    dY = torch.full_like(Z, 0.5)
    dY[1, 3] = float("nan")
    Z[2, 5] = float("nan")
    dZ, dbias, Q, s = B.ternary_epilogue_backward(dY, Z, act=act)
    want = {"none": lambda v: torch.ones_like(v), "relu": lambda v: (v > 0).double(), "relu2": lambda v: 2 * v.clamp_min(0)}
    d = want.get(act, lambda v: (v > 0).double() + 0.5 * (v == 0).double())(z.double())
    ref.check(dZ[0], 0.5 * d, 1e-6 * d.abs() + 1e-30, "dZ")
    assert bool(torch.isnan(dZ[1, 3])) and bool(torch.isnan(s[1])) and bool((Q[1] == 0).all())
    if act != "none":
        assert bool(torch.isnan(dZ[2, 5])) and bool(torch.isnan(s[2])) and bool((Q[2] == 0).all())


# (M, N, K): the few-row kernel in its column widths and row blocks; contractions
# that end inside a step; packed rows that are not whole dwords; every tile; the
# persistent kernel, even and ragged
PRODUCTS = [(1, 3456, 1280), (5, 16, 64), (9, 243, 320), (27, 8200, 256), (32, 17, 64), (1, 1, 4), (3, 5, 8),
            (27, 243, 244), (100, 33, 84), (200, 729, 244), (300, 272, 96), (1000, 130, 68), (2050, 900, 80), (512, 2305, 128),
            (1782, 1280, 192), (4096, 1280, 64), (8192, 2304, 64), (8191, 2305, 128), (7700, 2400, 192)]


def product_inputs(M, N, K, dt, *seed):
    g = gen(M, N, K, *seed)
    A = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    Wp = torch.randint(0, 256, (N, K // 4), generator=g, device=DEV, dtype=torch.uint8)
    rs = 0.001 + 0.02 * torch.rand(M, generator=g, device=DEV)
    return A, Wp, rs, 1.5 / K ** 0.5, normal(g, N, scale=0.3), normal(g, M, N, dtype=dt)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_epilogue(M, N, K, kind):
    say(f"product epilogue {M}x{N}x{K} {kind}")
    dt = KINDS[kind]
    A, Wp, rs, ws, bias, res = product_inputs(M, N, K, dt, kind)
    wsf = float(torch.tensor(ws))
    for act, b, r, save in (("none", None, None, False), ("none", bias, res, True), ("relu", bias, None, True),
                            ("relu2", None, res, False), ("silu", bias, None, False), ("silu", None, res, True),
                            ("gelu_tanh", bias, res, True), ("gelu_tanh", bias, None, False)):
        what = f"{act}{' bias' if b is not None else ''}{' residual' if r is not None else ''}"
        z, ez, y, ey = ref.product(A, Wp, rs, wsf, b, act, r)
        Y, Z = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=b, act=act, residual=r, out_dtype=dt, save=save)
        ref.check(Y, y, ref.rounded(y, ey, dt), f"{what}: Y")
        if save:
            ref.check(Z, z, ref.rounded(z, ez, dt), f"{what}: Z")
        else:
            assert Z is None
        if act == "none" and b is None and r is None:
            assert torch.equal(Y, B.ternary_gemm_s8_scaled(A, Wp, rs, ws, dt))
        if r is not None:                     # into the residual stream itself
            Yi = r.clone()
            B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=b, act=act, residual=Yi, out_dtype=dt, Y=Yi)
            assert torch.equal(Yi, Y), what


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K,offset", [(1, 243, 320, 1), (27, 1280, 256, 3), (200, 729, 244, 1), (1000, 130, 128, 2),
                                          (2050, 900, 80, 5), (8191, 2305, 64, 1)])
def test_product_epilogue_misaligned(M, N, K, kind, offset):
    say(f"product epilogue at offset {offset}: {M}x{N}x{K} {kind}")
    dt = KINDS[kind]
    A, Wp, rs, ws, bias, res = product_inputs(M, N, K, dt, kind, offset)
    for act in ("relu", "gelu_tanh"):
        want = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=bias, act=act, residual=res, out_dtype=dt, save=True)
        for whole in (False, True):           # the outputs alone, and the operands too
            p = Placed(offset)
            ops = [placed_copy(p, t) for t in (A, Wp, rs, bias, res)] if whole else [A, Wp, rs, bias, res]
            got = B.ternary_gemm_s8_epilogue(ops[0], ops[1], ops[2], ws, bias=ops[3], act=act, residual=ops[4],
                                             out_dtype=dt, save=True, Y=p((M, N), dt), Z=p((M, N), dt))
            torch.cuda.synchronize()
            p.check()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (act, whole)


# the persistent kernel with ragged last tiles, and the one of mid-size outputs
# over many steps, ragged and not
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(15001, 2301, 128), (14900, 2304, 64), (3001, 1250, 1088), (4096, 1280, 3456), (2048, 2048, 320)])
def test_product_epilogue_large(M, N, K, kind):
    say(f"product epilogue {M}x{N}x{K} {kind}")
    dt = KINDS[kind]
    A, Wp, rs, ws, bias, res = product_inputs(M, N, K, dt, kind, 7)
    p = Placed(8)
    for act, r, save in (("relu2", res, True), ("gelu_tanh", None, True), ("silu", res, False)):
        z, ez, y, ey = ref.product(A, Wp, rs, float(torch.tensor(ws)), bias, act, r)
        Y, Z = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=bias, act=act, residual=r, out_dtype=dt, save=save,
                                          Y=p((M, N), dt), Z=p((M, N), dt) if save else None)
        torch.cuda.synchronize()
        p.check()
        p.made.clear()
        ref.check(Y, y, ref.rounded(y, ey, dt), f"{act}: Y")
        if save:
            ref.check(Z, z, ref.rounded(z, ez, dt), f"{act}: Z")


def test_product_epilogue_not_finite_stays_by_itself():
    say("product epilogue not finite")
    M, N, K = 40, 48, 64
    A, Wp, rs, ws, bias, _ = product_inputs(M, N, K, torch.float32, 5)
    for act in ACTS:
        clean = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=bias, act=act, out_dtype=torch.float32)[0]
        b = bias.clone()
        b[7], b[9] = float("nan"), float("inf")
        Y = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=b, act=act, out_dtype=torch.float32)[0]
        assert bool(torch.isnan(Y[:, 7]).all()), act
        assert bool((Y[:, 9] == float("inf")).all()), act
        keep = [c for c in range(N) if c not in (7, 9)]
        assert torch.equal(Y[:, keep], clean[:, keep])


LISTS = {
    "one": [(1,)], "empty among others": [(0,), (5, 3), (0, 7)], "odd": [(7,), (243, 243), (1,), (729, 243), (16385,)],
    "many": [(1 + 37 * i,) for i in range(150)], "large": [(3456, 1280), (1280,), (16384, 320)],
    "all empty": [(0,)],
}


@pytest.mark.parametrize("kind", list(KINDS) + ["mixed"])
@pytest.mark.parametrize("name", LISTS)
def test_clip(name, kind):
    say(f"clip {name} {kind}")
    g = gen(len(name), kind)
    dts = [torch.float32 if kind == "f32" or (kind == "mixed" and i % 2) else torch.bfloat16
           for i in range(len(LISTS[name]))]
    grads = [normal(g, *s, dtype=d, scale=0.1) for s, d in zip(LISTS[name], dts)]
    keep = [x.clone() for x in grads]
    total = sum(float(x.double().square().sum()) for x in grads) ** 0.5
    for limit in (1.0, 1e6, 0.0):
        out, norm = B.ternary_clip_grad_norm(grads, limit)
        assert abs(float(norm) - total) <= 2 * ref.U * total
        f = min(1.0, limit / (total + float(torch.tensor(1e-6))))
        for o, x, d in zip(out, grads, dts):
            w = x.double() * f
            assert o.shape == x.shape and o.dtype == d
            ref.check(o, w, ref.rounded(w, 6 * ref.U * w.abs(), d), "out")
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    out, norm = B.ternary_clip_grad_norm(keep, 1.0, out=keep)      # in place
    want = B.ternary_clip_grad_norm(grads, 1.0)
    assert torch.equal(norm, want[1]) and all(torch.equal(a, b) for a, b in zip(keep, want[0]))


@pytest.mark.parametrize("offset", [1, 3])
def test_clip_misaligned(offset):
    say(f"clip at offset {offset}")
    g = gen(offset)
    shapes = [(5,), (243, 243), (1,), (70001,)]
    for dt in KINDS.values():
        grads = [normal(g, *s, dtype=dt) for s in shapes]
        want = B.ternary_clip_grad_norm(grads, 1.0)
        p = Placed(offset)
        got = B.ternary_clip_grad_norm([placed_copy(p, x) for x in grads], 1.0, out=[p(s, dt) for s in shapes])
        torch.cuda.synchronize()
        p.check()
        # the sum's order may follow the alignment; double sums agree to float32 all the same
        assert abs(float(got[1]) - float(want[1])) <= 2 * ref.U * float(want[1])
        for a, b in zip(got[0], want[0]):
            ref.check(a, b.double(), 4 * ref.U * b.double().abs() + (torch.finfo(dt).eps if dt != torch.float32 else 0) * b.double().abs(), "out")


def test_clip_norms_at_the_ends_of_the_range():
    say("clip ends of the range")
    big = torch.full((1000,), 1e30, device=DEV)                    # squares past float32
    out, norm = B.ternary_clip_grad_norm([big], 1.0)
    assert abs(float(norm) / (1e30 * 1000 ** 0.5) - 1) < 1e-6
    ref.check(out[0], torch.full((1000,), 1000 ** -0.5, device=DEV).double(), torch.tensor(1e-8, device=DEV), "out")
    small = torch.full((1000,), 1e-30, device=DEV)                 # squares below it
    out, norm = B.ternary_clip_grad_norm([small], 1.0)
    assert abs(float(norm) / (1e-30 * 1000 ** 0.5) - 1) < 1e-6 and torch.equal(out[0], small)
    for bad in (float("inf"), float("nan")):
        x = torch.ones(1000, device=DEV)
        x[500] = bad
        out, norm = B.ternary_clip_grad_norm([x, torch.ones(3, device=DEV)], 1.0)
        n = float(norm)
        assert n == bad or (n != n and bad != bad)
        assert bool(torch.isnan(out[0][500])) and (bool((out[1] == 0).all()) if bad == float("inf") else bool(torch.isnan(out[1]).all()))


def everything(t, stream=None):
    """Every operator once into kept outputs, on inputs t."""
    o = t["o"]
    B.ternary_rmsnorm_quantize(t["X"], t["gain"], residual=t["res"], save=True, H=o["H"], Y=o["Y"], rstd=o["rstd"],
                               Q=o["Q"], scale=o["s"], stream=stream)
    B.ternary_gemm_s8_epilogue(o["Q"], t["Wp"], o["s"], 0.05, bias=t["bias"], act="gelu_tanh", out_dtype=t["X"].dtype,
                               save=True, Y=o["U"], Z=o["Z"], stream=stream)
    B.ternary_epilogue_backward(t["dU"], o["Z"], act="gelu_tanh", dZ=o["dZ"], dbias=o["db"], Q=o["Qz"], scale=o["sz"],
                                workspace=t["ws"], stream=stream)
    B.ternary_rmsnorm_backward(t["dY"], o["H"], t["gain"], o["rstd"], dH=t["res"], dX=o["dX"], dgain=o["dg"],
                               workspace=t["ws"], stream=stream)
    B.ternary_clip_grad_norm([o["dX"], o["dg"], o["db"]], 0.1, out=[o["c0"], o["c1"], o["c2"]], norm=o["n"],
                             workspace=t["ws"], stream=stream)


def everything_inputs(R, C, N, dt):
    g = gen(R, C, N)
    e = lambda *s, d=dt: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    f = torch.float32
    return {"X": normal(g, R, C, dtype=dt), "res": normal(g, R, C, dtype=dt), "gain": 1 + normal(g, C, scale=0.1),
            "Wp": torch.randint(0, 256, (N, C // 4), generator=g, device=DEV, dtype=torch.uint8),
            "bias": normal(g, N), "dU": normal(g, R, N, dtype=dt), "dY": normal(g, R, C, dtype=dt),
            "ws": torch.empty(64 << 20, dtype=torch.uint8, device=DEV),
            "o": {"H": e(R, C), "Y": e(R, C), "rstd": e(R, d=f), "Q": e(R, C, d=torch.int8), "s": e(R, d=f),
                  "U": e(R, N), "Z": e(R, N), "dZ": e(R, N), "db": e(N, d=f), "Qz": e(R, N, d=torch.int8),
                  "sz": e(R, d=f), "dX": e(R, C), "dg": e(C, d=f), "c0": e(R, C), "c1": e(C, d=f), "c2": e(N, d=f),
                  "n": e(1, d=f)}}


@pytest.mark.parametrize("R,C,N", [(27, 1280, 3456), (2048, 320, 729)])
def test_graph_replays_and_other_streams_match(R, C, N):
    say(f"graph {R}x{C}x{N}")
    t = everything_inputs(R, C, N, torch.bfloat16)
    everything(t)
    torch.cuda.synchronize()
    eager = {k: v.clone() for k, v in t["o"].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for v in t["o"].values():
        v.zero_()
    side.wait_stream(torch.cuda.current_stream())
    everything(t, stream=side)                # named, while another stream is current
    side.synchronize()
    for k, v in t["o"].items():
        assert torch.equal(v, eager[k]), f"side stream: {k}"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        everything(t, stream=side)
    other = everything_inputs(5, 64, 96, torch.bfloat16)
    for rep in range(3):
        for v in t["o"].values():
            v.zero_()
        everything(other)                     # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        say(f"replay {rep}")
        for k, v in t["o"].items():
            assert torch.equal(v, eager[k]), f"replay {rep}: {k}"


def test_more_than_32_bit_elements():
    # rows whose offsets pass 2^32 elements: the last rows against the same rows alone
    say("offsets past 32 bits")
    R, C = (1 << 32) // 16384 + 8, 16384
    dt = torch.bfloat16
    X = torch.empty((R, C), dtype=dt, device=DEV)
    row = normal(gen(3), 1, C, dtype=dt)
    X[:] = row
    X[-3:] = normal(gen(4), 3, C, dtype=dt)
    gain = torch.ones(C, device=DEV)
    Q, s, _, Y, rstd = B.ternary_rmsnorm_quantize(X, gain, save=True)
    few = B.ternary_rmsnorm_quantize(X[-3:].clone(), gain, save=True)
    for a, b in ((Q, few[0]), (s, few[1]), (Y, few[3]), (rstd, few[4])):
        assert torch.equal(a[-3:], b)
    del Q, s
    dX, dgain = B.ternary_rmsnorm_backward(Y, X, gain, rstd)
    few = B.ternary_rmsnorm_backward(Y[-3:].clone(), X[-3:].clone(), gain, rstd[-3:].clone())
    assert torch.equal(dX[-3:], few[0])
