"""The variants of the operators around the product that test_gpu_block.py does
not reach: the norm's rows of two to four vectors a lane, which it takes from
1024 rows on; wide float32 rows of the epilogue's backward pass; clipped lists
that are written past the caches, that take more than one launch and whose
partial sums the launches share; elements past 32-bit offsets."""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
import test_gpu_block as block  # noqa: E402
from test_gpu_block import DEV, KINDS, gen, normal, say  # noqa: E402

pytestmark = pytest.mark.gpu

# bfloat16: two vectors a lane to 1024 columns, three to 1536, four to 2048;
# float32: half of that, and the wider of these in a workgroup a row
MANY_ROWS = [(1030, 261), (1024, 512), (1030, 521), (1030, 700), (1024, 768), (1030, 1021), (2051, 1024), (1100, 1280),
             (1030, 1531), (1024, 1536), (1030, 2041), (1025, 2048), (1030, 2049)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", MANY_ROWS)
def test_norm_of_many_rows(R, C, kind):
    block.test_norm(R, C, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C,offset", [(1030, 521, 1), (1100, 1280, 3), (1030, 1531, 5), (1030, 2041, 1), (1030, 261, 1),
                                        (1030, 700, 3), (1030, 1021, 1)])
def test_norm_of_many_rows_misaligned_and_in_place(R, C, kind, offset):
    block.test_norm_misaligned_and_in_place(R, C, kind, offset)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [521, 1021, 1531, 2041])
def test_norm_of_many_rows_that_are_not_finite(C, kind):
    say(f"norm of many rows, not finite {C} {kind}")
    dt, g = KINDS[kind], gen(C, kind, 31)
    X, gain = normal(g, 1030, C, dtype=dt), 1 + normal(g, C, scale=0.1)
    clean = B.ternary_rmsnorm_quantize(X, gain, save=True)
    bad = [5 + 3 * i for i in range(9)]        # one in each place of a row's last two vectors
    for i, r in enumerate(bad):
        X[r, C - 1 - i] = float("nan") if i % 2 else float("inf")
    Q, s, _, Y, rstd = B.ternary_rmsnorm_quantize(X, gain, save=True)
    assert not bool(torch.isfinite(s[bad]).any()) and bool((Q[bad] == 0).all())
    keep = [r for r in range(1030) if r not in bad]
    for a, b in ((Q, clean[0]), (s, clean[1]), (Y, clean[3]), (rstd, clean[4])):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("R,C", [(3, 9001), (2, 12288), (5, 12289)])
def test_epilogue_backward_of_wide_rows(R, C, act, kind):
    block.test_epilogue_backward(R, C, act, kind)


LISTS = {
    "written past the caches": [(16384, 1280), (5,), (3457, 1281)],
    "partial sums shared by launches": [(60000 + 17 * i,) for i in range(150)],
    "shared, and past the caches": [(0,)] + [(130001 + i,) for i in range(200)] + [(3,)],
}


@pytest.mark.parametrize("kind", list(KINDS) + ["mixed"])
@pytest.mark.parametrize("name", LISTS)
def test_clip(name, kind, monkeypatch):
    monkeypatch.setitem(block.LISTS, name, LISTS[name])
    block.test_clip(name, kind)


# ---------------------------------------------------------------------------
# offsets past 2^32 elements: the last rows against the same rows alone
# ---------------------------------------------------------------------------

@pytest.fixture
def room():
    yield
    torch.cuda.empty_cache()


BF = torch.bfloat16


def rows_past_32_bits(C, seed):
    """A matrix of one row repeated, but for the last three."""
    R = (1 << 32) // C + 8
    X = torch.empty((R, C), dtype=BF, device=DEV)
    X[:] = normal(gen(C, seed), 1, C, dtype=BF)
    X[-3:] = normal(gen(C, seed, 1), 3, C, dtype=BF)
    return X


@pytest.mark.parametrize("C", [16384, 40000])
def test_norm_past_32_bits(C, room):
    say(f"norm past 32 bits {C}")
    X, gain = rows_past_32_bits(C, 1), 1 + normal(gen(C), C, scale=0.1)
    few = B.ternary_rmsnorm_quantize(X[-3:].clone(), gain, residual=X[-6:-3].clone(), save=True)
    res = torch.empty_like(X)
    res[:] = X[:1]
    got = B.ternary_rmsnorm_quantize(X, gain, residual=res, save=True, H=res)     # in place
    for a, b in zip(got, few):
        assert torch.equal(a[-3:], b)
    rstd, H = got[4], got[2]
    del got, few
    few = B.ternary_rmsnorm_backward(X[-3:].clone(), H[-3:].clone(), gain, rstd[-3:].clone())
    dX, _ = B.ternary_rmsnorm_backward(X, H, gain, rstd)
    assert torch.equal(dX[-3:], few[0])


@pytest.mark.parametrize("C", [16384, 40000])
def test_epilogue_backward_past_32_bits(C, room):
    say(f"epilogue backward past 32 bits {C}")
    dY, Z = rows_past_32_bits(C, 2), rows_past_32_bits(C, 3)
    dZ, dbias, Q, s = B.ternary_epilogue_backward(dY, Z, act="silu")
    few = B.ternary_epilogue_backward(dY[-3:].clone(), Z[-3:].clone(), act="silu")
    for a, b in ((dZ, few[0]), (Q, few[2]), (s, few[3])):
        assert torch.equal(a[-3:], b)
    # dbias: the repeated row as often as it is there, and the last three
    one, e, _, _ = ref.epilogue_backward(dY[:1].double(), Z[:1].double(), "silu")
    last, el, _, _ = ref.epilogue_backward(dY[-3:].double(), Z[-3:].double(), "silu")
    n = dY.shape[0] - 3
    want = n * one[0] + last.sum(0)
    ref.check(dbias, want, n * e[0] + el.sum(0) + (n + 7) * ref.U * (n * one[0].abs() + last.abs().sum(0)), "dbias")


def test_product_epilogue_past_32_bits(room):
    say("product epilogue past 32 bits: many rows")
    N, K = 16384, 64
    M = (1 << 32) // N + 8
    A = torch.empty((M, K), dtype=torch.int8, device=DEV)
    A[:] = torch.randint(-127, 128, (1, K), generator=gen(41), device=DEV, dtype=torch.int8)
    few, Wp, rs, ws, bias, res = block.product_inputs(300, N, K, BF, 41)
    A[-300:] = few
    scale = rs[:1].repeat(M)
    scale[-300:] = rs
    want = B.ternary_gemm_s8_epilogue(few, Wp, rs, ws, bias=bias, act="gelu_tanh", residual=res, save=True)
    Y = torch.zeros((M, N), dtype=BF, device=DEV)
    Y[-300:] = res
    _, Z = B.ternary_gemm_s8_epilogue(A, Wp, scale, ws, bias=bias, act="gelu_tanh", residual=Y, save=True, Y=Y)
    assert torch.equal(Y[-300:], want[0]) and torch.equal(Z[-300:], want[1])
    first = B.ternary_gemm_s8_epilogue(A[:300].clone(), Wp, scale[:300].clone(), ws, bias=bias, act="gelu_tanh")[0]
    assert torch.equal(Y[:300], first) and torch.equal(Y[M // 2:M // 2 + 300], first)


def test_product_epilogue_of_few_rows_past_32_bits(room):
    say("product epilogue past 32 bits: few rows")
    M, K = 32, 64
    N = (1 << 27) + 16
    A, few, rs, ws, bias, res = block.product_inputs(M, 400, K, BF, 42)
    Wp = torch.zeros((N, K // 4), dtype=torch.uint8, device=DEV)
    Wp[-400:] = few
    b, Y = torch.zeros(N, device=DEV), torch.zeros((M, N), dtype=BF, device=DEV)
    b[-400:] = bias
    Y[:, -400:] = res
    want = B.ternary_gemm_s8_epilogue(A, few, rs, ws, bias=bias, act="silu", residual=res, save=True)
    _, Z = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=b, act="silu", residual=Y, save=True, Y=Y)
    assert torch.equal(Y[:, -400:], want[0]) and torch.equal(Z[:, -400:], want[1])
    assert not bool(Y[:, :1000].any()) and not bool(Y[:, -2000:-400].any())


def test_clip_past_32_bits(room):
    say("clip past 32 bits")
    n = (1 << 32) + 20001
    x = torch.zeros(n, dtype=BF, device=DEV)
    x[:3], x[1 << 31], x[(1 << 32) + 5], x[-2:] = 1, -2, 3, 4
    y = torch.full((7,), 2.0, device=DEV)
    total = (3 + 4 + 9 + 32 + 28) ** 0.5
    out, norm = B.ternary_clip_grad_norm([x, y], 1.0)
    assert abs(float(norm) - total) <= 2 * ref.U * total
    f = 1.0 / (total + float(torch.tensor(1e-6)))
    at = [0, 2, 3, 1 << 31, (1 << 32) + 5, n - 3, n - 2, n - 1]
    want = x[at].double() * f
    ref.check(out[0][at], want, ref.rounded(want, 6 * ref.U * want.abs(), BF), "out")
    ref.check(out[1], y.double() * f, 6 * ref.U * y.double() * f, "float32 out")
    assert int((out[0] != 0).sum()) == 7
