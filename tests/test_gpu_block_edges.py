"""Infinities and values near the ends of the range in the operators around
the product, at widths that are not whole vectors; few short rows; int8 rows
by IEEE division."""
import numpy
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
from test_gpu_block import DEV, KINDS, gen, normal, say  # noqa: E402

pytestmark = pytest.mark.gpu


def same_kind_of_values(got, want, what):
    """NaN where the formula has NaN, an infinity of its sign where it has one, finite elsewhere."""
    got, want = got.double(), want.double()
    bad = (torch.isnan(got) != torch.isnan(want)) | (torch.isinf(got) != torch.isinf(want)) | (
        torch.isinf(want) & (got.sign() != want.sign()))
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} are of another kind, first at {i}: {float(got[i])} for {float(want[i])}")


# a wave a row; a workgroup a row with one unit a thread and with more; the
# looped kernels.  9 columns from the end hold every place of a row's last two
# vectors, of which the last may overlap the one before.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [9, 243, 509, 1282, 3461, 8197, 16379, 16401])
def test_norm_backward_infinities(C, kind):
    say(f"norm backward infinities {C} {kind}")
    dt, g, n = KINDS[kind], gen(C, kind, 21), 9
    H, dY = normal(g, n + 3, C, dtype=dt), normal(g, n + 3, C, dtype=dt, scale=1e-2)
    H[H.abs() < 0.01] = 0.5                    # no 0 x infinity from a value that a type rounds to 0
    gain = 1 + 0.1 * torch.rand(C, generator=g, device=DEV)
    rstd = (H.double().square().mean(1) + 1e-5).rsqrt().float()
    clean = B.ternary_rmsnorm_backward(dY, H, gain, rstd)
    for i in range(n):
        dY[i, C - 1 - i] = float("inf") if i % 2 else -float("inf")
    dX, dgain = B.ternary_rmsnorm_backward(dY, H, gain, rstd)
    dx, _, dg, _ = ref.norm_backward(dY.double(), H.double(), gain.double(), rstd.double(), None)
    same_kind_of_values(dX, dx, "dX")
    same_kind_of_values(dgain, dg, "dgain")
    assert torch.equal(dX[n:], clean[0][n:]) and torch.equal(dgain[:C - n], clean[1][:C - n])
    H[n, C - 2] = float("inf")                 # its rstd is 0: the product is NaN, and so is the row's sum
    rstd[n] = 0
    dX, dgain = B.ternary_rmsnorm_backward(dY, H, gain, rstd)
    dx, _, dg, _ = ref.norm_backward(dY.double(), H.double(), gain.double(), rstd.double(), None)
    same_kind_of_values(dX, dx, "dX")
    same_kind_of_values(dgain, dg, "dgain")
    assert torch.equal(dX[n + 1:], clean[0][n + 1:])


# relu2's slope 2 z is as large as the value: the product 2 z dy overflows only
# where the formula's does.  A wave a row, a workgroup a row, the looped kernel.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [3, 16, 2051, 16401])
def test_relu2_backward_of_large_gradients(C, kind):
    say(f"relu2 backward of large gradients {C} {kind}")
    dt = KINDS[kind]
    top = 2.0e38                               # more than half the largest float32
    z = torch.tensor([0.0, 0.1, 1e-3, -0.0, -1.0, 0.75, 3.0, 1e-30], device=DEV, dtype=dt)
    dY = torch.full((z.numel(), C), 1.0, device=DEV, dtype=dt)
    dY[:, -1], dY[:, 0] = top, -top
    Z = z[:, None].repeat(1, C)
    dZ, dbias, Q, s = B.ternary_epilogue_backward(dY, Z, act="relu2")
    dz, e, _, _ = ref.epilogue_backward(dY.double(), Z.double(), "relu2")
    over = dz.abs() > 3.4e38                   # 2 z dy for z of 3: past the type
    assert bool((over.any(1) == (z == 3)).all())
    ref.check(torch.where(over, 0, dZ.double()), torch.where(over, 0, dz), ref.rounded(dz, e, dt), "dZ")
    assert torch.equal(dZ[over].double(), torch.where(dz[over] > 0, float("inf"), -float("inf")).double())
    for r in range(z.numel()):
        if bool(over[r].any()):
            assert not bool(torch.isfinite(s[r])) and bool((Q[r] == 0).all())
        else:
            ref.check_int8(Q[r:r + 1], s[r:r + 1], dz[r:r + 1], e[r:r + 1], f"row {r}")


# one workgroup for every row, whose waves take up to two rows each, and the
# first size past it
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [9, 243, 256, 512])
@pytest.mark.parametrize("R", [2, 15, 16, 17, 31, 32, 33])
def test_backward_of_few_short_rows(R, C, kind):
    say(f"backward of few short rows {R}x{C} {kind}")
    dt, g = KINDS[kind], gen(R, C, kind, 23)
    H, dY, Z = normal(g, R, C, dtype=dt), normal(g, R, C, dtype=dt, scale=1e-2), normal(g, R, C, dtype=dt, scale=2.0)
    gain = 1 + normal(g, C, scale=0.1)
    rstd = (H.double().square().mean(1) + 1e-5).rsqrt().float()
    dX, dgain = B.ternary_rmsnorm_backward(dY, H, gain, rstd)
    dx, e, dg, eg = ref.norm_backward(dY.double(), H.double(), gain.double(), rstd.double(), None)
    ref.check(dX, dx, ref.rounded(dx, e, dt), "dX")
    ref.check(dgain, dg, eg, "dgain")
    dZ, dbias, Q, s = B.ternary_epilogue_backward(dY, Z, act="silu")
    dz, e, db, eb = ref.epilogue_backward(dY.double(), Z.double(), "silu")
    ref.check(dZ, dz, ref.rounded(dz, e, dt), "dZ")
    ref.check(dbias, db, eb, "dbias")
    ref.check_int8(Q, s, dz, e, "dZ")


# bfloat16 gradients without an activation often lie on the border between two
# int8 values, where a scale one step off changes them: the scale and the
# quotient are those of IEEE division, on a host
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", [(453, 601), (41, 192), (4079, 1353), (3, 16401)])
def test_int8_rows_are_those_of_ieee_division(R, C, kind):
    say(f"int8 rows by IEEE division {R}x{C} {kind}")
    dY = normal(gen(R, C, kind, 25), R, C, dtype=KINDS[kind], scale=1e-3)
    dZ, _, Q, s = B.ternary_epilogue_backward(dY, dY, act="none")
    y = dY.float().cpu().numpy()
    scale = abs(y).max(1) / numpy.float32(127)
    assert scale.dtype == numpy.float32 and (s.cpu().numpy() == scale).all()
    assert (Q.cpu().numpy() == numpy.clip(numpy.rint(y / scale[:, None]), -127, 127)).all()
    assert torch.equal(dZ, dY)
