"""GPU parity of the layer norm and its backward pass, and of the gated
product's backward pass, with their definitions in 64 bits, at the sizes,
widths, alignments and rows where they can go wrong."""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
import gated_ref as gref  # noqa: E402
from test_gpu_block import ACTS, DEV, KINDS, ROWS, Placed, gen, normal, placed_copy, say  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = float(torch.tensor(1e-5))
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", ROWS + [(1100, 1280), (1024, 2000), (2500, 3120), (2100, 1301), (1100, 5000), (1030, 7001), (4200, 1540), (520, 6001)])
def test_layernorm(R, C, kind):
    say(f"layernorm {R}x{C} {kind}")
    dt, g = KINDS[kind], gen("ln", R, C, kind)
    X, res = (normal(g, R, C, scale=3.0) + 5 * normal(g, C)).to(dt), normal(g, R, C, dtype=dt)
    gain, beta = 1 + normal(g, C, scale=0.1), normal(g, C, scale=0.1)
    if R > 3:
        X[1], res[1] = 0, 0                   # a row of padding
        X[2] = -res[2]                        # a sum that cancels
        X[3], res[3] = 1000, 0                # a row of one value: its variance is what rounding leaves
    for residual, b, save in ((res, beta, True), (None, None, True), (res, None, False), (None, beta, False)):
        Q, s, H, Y, mean, rstd = B.ternary_layernorm_quantize(X, gain, b, EPS, residual=residual, save=save)
        if residual is None:
            assert H is X
        else:
            want = X.double() + res.double()
            ref.check(H, want, ref.rounded(want, ref.U * want.abs(), dt), "H")
        mu, em, r, rel, y, e = gref.layernorm(H.double(), gain.double(), None if b is None else b.double(), EPS)
        ref.check_int8(Q, s, y, e, "layernorm")
        if save:
            ref.check(mean, mu, em, "mean")
            ref.check(rstd, r, rel * r, "rstd")
            ref.check(Y, y, ref.rounded(y, e, dt), "Y")
            if dt == torch.float32:           # the int8 rows are the row quantizer's of the same values
                q2, s2 = B.ternary_quantize_rows(Y)
                assert torch.equal(q2, Q) and torch.equal(s2, s)
        else:
            assert Y is None and mean is None and rstd is None


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C,offset", [(5, 243, 1), (37, 1280, 3), (3, 3456, 1), (1025, 1001, 1), (4, 16384, 5), (3, 40000, 1)])
def test_layernorm_misaligned_and_in_place(R, C, kind, offset):
    say(f"layernorm at offset {offset}: {R}x{C} {kind}")
    dt, g = KINDS[kind], gen("ln", R, C, offset)
    X, res, gain, beta = normal(g, R, C, dtype=dt), normal(g, R, C, dtype=dt), 1 + normal(g, C, scale=0.1), normal(g, C)
    want = B.ternary_layernorm_quantize(X, gain, beta, residual=res, save=True)
    for into in ("X", "residual", "own"):
        p = Placed(offset)
        Xp, rp, gp, bp = (placed_copy(p, t) for t in (X, res, gain, beta))
        H = {"X": Xp, "residual": rp, "own": p((R, C), dt)}[into]
        got = B.ternary_layernorm_quantize(Xp, gp, bp, residual=rp, save=True, H=H, Y=p((R, C), dt),
                                           mean=p((R,), torch.float32), rstd=p((R,), torch.float32),
                                           Q=p((R, C), torch.int8), scale=p((R,), torch.float32))
        torch.cuda.synchronize()
        p.check()
        for a, b in zip(got, want):
            assert torch.equal(a, b), into


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [5, 1280, 5000, 40000])
def test_layernorm_rows_that_are_not_finite_stay_by_themselves(C, kind):
    say(f"layernorm not finite {C} {kind}")
    dt, g = KINDS[kind], gen("ln", C, 9)
    X, gain, beta = normal(g, 6, C, dtype=dt), 1 + normal(g, C, scale=0.1), normal(g, C)
    clean = B.ternary_layernorm_quantize(X, gain, beta, save=True)
    Xb = X.clone()
    Xb[1, C - 1], Xb[4, 0] = NAN, INF
    Q, s, _, Y, mean, rstd = B.ternary_layernorm_quantize(Xb, gain, beta, save=True)
    for r in (1, 4):
        assert not bool(torch.isfinite(s[r])) and bool((Q[r] == 0).all()) and bool(torch.isnan(Y[r].float()).any())
    assert bool(torch.isnan(mean[1])) and float(mean[4]) == INF and bool(torch.isnan(rstd[1])) and bool(torch.isnan(rstd[4]))
    keep = [0, 2, 3, 5]
    for a, b in ((Q, clean[0]), (s, clean[1]), (Y, clean[3]), (mean, clean[4]), (rstd, clean[5])):
        assert torch.equal(a[keep], b[keep])


def test_layernorm_of_a_mean_far_larger_than_the_deviation():
    """Rows about 4096 that deviate by 1/4 lose the variance to a difference of sums in float32, not to this."""
    g = gen("far")
    X = 4096 + 0.25 * normal(g, 40, 1280)
    gain = torch.ones(1280, device=DEV)
    Q, s, _, Y, mean, rstd = B.ternary_layernorm_quantize(X, gain, None, 0.0, save=True)
    h = X.double()
    want = 1 / h.var(1, correction=0).sqrt()
    # the mean is off by at most (36 + 2) half steps of 4096 2^-24, 0.0093, which adds its square to a variance of 1/16
    assert bool(((rstd.double() - want).abs() <= want * (0.5 * 0.0093 ** 2 * 16 + 1e-4)).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", ROWS + [(1782, 729), (600, 3456), (32, 64), (33, 64), (17, 500), (32, 766), (19, 1022)])
def test_layernorm_backward(R, C, kind):
    say(f"layernorm backward {R}x{C} {kind}")
    dt, g = KINDS[kind], gen("lnb", R, C, kind)
    H, dY, dH = (normal(g, R, C, dtype=dt, scale=x) for x in (2.0, 1e-3, 1e-3))
    gain = 1 + normal(g, C, scale=0.1)
    _, _, _, _, mean, rstd = B.ternary_layernorm_quantize(H, gain, save=True)
    for d, beta in ((dH, True), (None, True), (dH, False)):
        dX, dgain, dbeta = B.ternary_layernorm_backward(dY, H, gain, mean, rstd, dH=d, beta=beta)
        dx, ex, dg, eg, db, eb = gref.layernorm_backward(dY.double(), H.double(), gain.double(), mean.double(),
                                                         rstd.double(), None if d is None else d.double())
        ref.check(dX, dx, ref.rounded(dx, ex, dt), "dX")
        ref.check(dgain, dg, eg, "dgain")
        if beta:
            ref.check(dbeta, db, eb, "dbeta")
        else:
            assert dbeta is None
    # in place, with a workspace of its own and outputs that lie anywhere
    p = Placed(3)
    args = [placed_copy(p, t) for t in (dY, H, gain, mean, rstd, dH)]
    ws = torch.empty(B._queried("ternary_layernorm_backward_workspace", R, C), dtype=torch.uint8, device=DEV)
    got = B.ternary_layernorm_backward(*args, dX=args[5], dgain=p((C,), torch.float32), dbeta=p((C,), torch.float32),
                                       workspace=ws)
    torch.cuda.synchronize()
    p.check()
    for a, b in zip(got, B.ternary_layernorm_backward(dY, H, gain, mean, rstd, dH=dH)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", [(1, 1), (1, 3), (3, 7), (27, 243), (65, 511), (5, 513), (32, 512), (33, 512), (16, 729), (17, 729), (9, 1001), (200, 729),
                                 (130, 3456), (7, 4104), (3, 8191), (4, 8200), (2, 16384), (3, 16401), (2500, 64)])
def test_gated_backward(R, C, kind, act):
    say(f"gated backward {R}x{C} {kind} {act}")
    dt, g = KINDS[kind], gen("gb", R, C, kind, act)
    dY, Z = normal(g, R, C, dtype=dt, scale=1e-3), normal(g, R, 2 * C, dtype=dt, scale=2.0)
    gs, us = 0.03125, 0.75
    if R > 2:
        dY[1] = 0                             # a row whose scale is 0
        Z[2, :C] = torch.linspace(-120, 120, C, device=DEV).to(dt)
    dZ, db, Q, s = B.ternary_gated_backward(dY, Z, gs, us, act=act)
    dz, e, b, eb = gref.gated_backward(dY.double(), Z.double(), act)
    ref.check(dZ, dz, ref.rounded(dz, e, dt), "dZ")
    ref.check(db, b, eb, "dbias")
    k = torch.cat((torch.full((C,), gs, device=DEV), torch.full((C,), us, device=DEV))).double()
    ref.check_int8(Q, s, dz * k, e * k + ref.U * (dz * k).abs(), "rows")
    again = B.ternary_gated_backward(dY, Z, gs, us, act=act, bias=False)
    assert again[1] is None and all(torch.equal(a, b) for a, b in zip(again, (dZ, None, Q, s)) if b is not None)
    p = Placed(1)
    ws = torch.empty(B._queried("ternary_gated_backward_workspace", R, C), dtype=torch.uint8, device=DEV)
    got = B.ternary_gated_backward(placed_copy(p, dY), placed_copy(p, Z), gs, us, act=act, dZ=p((R, 2 * C), dt),
                                   dbias=p((2 * C,), torch.float32), Q=p((R, 2 * C), torch.int8),
                                   scale=p((R,), torch.float32), workspace=ws)
    torch.cuda.synchronize()
    p.check()
    assert all(torch.equal(a, b) for a, b in zip(got, (dZ, db, Q, s)))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("C", [6, 200, 3456, 16400])
def test_gated_backward_values_that_are_not_finite(C, act):
    """A NaN anywhere, an infinity in dY or u: the row's scale shows it, other rows and columns do not change."""
    say(f"gated backward not finite {C} {act}")
    g = gen("gbn", C, act)
    dY, Z = normal(g, 8, C, scale=1e-3), normal(g, 8, 2 * C)
    Z[:, 0] = Z[:, 0].abs() + 0.5             # a gate that no activation closes
    clean = B.ternary_gated_backward(dY, Z, 0.5, 2.0, act=act)
    dYb, Zb = dY.clone(), Z.clone()
    dYb[1, 0], Zb[3, C - 1], Zb[5, 2 * C - 1], Zb[6, C] = INF, NAN, NAN, INF
    dZ, db, Q, s = B.ternary_gated_backward(dYb, Zb, 0.5, 2.0, act=act)
    for r in (1, 3, 5, 6):
        assert not bool(torch.isfinite(s[r])) and bool((Q[r] == 0).all()), r
    assert bool(torch.isnan(dZ[3, 2 * C - 1])) and bool(torch.isnan(dZ[5, C - 1])) and bool(torch.isinf(dZ[6, 0]))
    keep = [0, 2, 4, 7]
    for a, b in ((dZ, clean[0]), (Q, clean[2]), (s, clean[3])):
        assert torch.equal(a[keep], b[keep])
    cols = torch.ones(2 * C, dtype=torch.bool, device=DEV)
    cols[[0, C, C - 1, 2 * C - 1]] = False
    assert torch.equal(db[cols], clean[1][cols])


def test_gated_gates_far_below_zero_are_closed():
    Z = torch.tensor([[-90.0, -300.0, -1e30, -INF, 1.0, 1.0, 1.0, 1.0]], device=DEV)
    dY = torch.full((1, 4), 1e3, device=DEV)
    for act in ("silu", "gelu_tanh"):
        dZ = B.ternary_gated_backward(dY, Z, 1.0, 1.0, act=act, bias=False)[0]
        assert float(dZ.abs().max()) < 1e-30, act


def test_offsets_past_32_bits():
    """2.2e9 elements of Z and dZ: the last rows are those of a small call."""
    R, C = 66000, 16640
    say(f"gated backward {R}x{C}")
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GiB")
    Z = torch.zeros(R, 2 * C, dtype=torch.bfloat16, device=DEV)
    dY = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV)
    g = gen("far rows")
    Z[-3:], dY[-3:] = normal(g, 3, 2 * C, dtype=torch.bfloat16), normal(g, 3, C, dtype=torch.bfloat16)
    dZ, _, Q, s = B.ternary_gated_backward(dY, Z, 1.0, 1.0, bias=False)
    want = B.ternary_gated_backward(dY[-3:].contiguous(), Z[-3:].contiguous(), 1.0, 1.0, bias=False)
    assert torch.equal(dZ[-3:], want[0]) and torch.equal(Q[-3:], want[2]) and torch.equal(s[-3:], want[3])
    assert not bool(dZ[:-3].any())


def test_tensors_of_another_device_are_refused(monkeypatch):
    """A call launches on the current device: tensors of another one are an error before any launch."""
    say("another current device")
    x, q, w = (torch.ones(2, 64, device=DEV, dtype=d) for d in (torch.float32, torch.int8, torch.uint8))
    v, z = torch.ones(64, device=DEV), torch.ones(2, 128, device=DEV)
    r = torch.ones(2, device=DEV)
    calls = (lambda: B.ternary_layernorm_quantize(x, v), lambda: B.ternary_layernorm_backward(x, x, v, r, r),
             lambda: B.ternary_gated_backward(x, z, 1.0, 1.0), lambda: B.ternary_gemm_s8s8_epilogue(q, q, r),
             lambda: B.ternary_gemm_s8_gated(q, w[:, :16].contiguous(), r, 1.0, 1.0))
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: x.device.index + 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
