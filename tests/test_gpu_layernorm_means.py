"""The layer norm of rows whose mean is far above their deviation, and of rows of
one value: the mean that is taken off is the row's, not its nearest float32."""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
from block_ref import TINY, U, depth  # noqa: E402
from test_gpu_block import DEV, KINDS, gen, normal, say  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = float(torch.tensor(1e-5))

# every plan of the layer norm: a wave a row of one to four units a lane, workgroups
# of one to sixteen waves of one to four, the looped kernel below and above them
SHAPES = [(2, 3), (3, 7), (40, 243), (30, 513), (1100, 1280), (1030, 2000), (40, 1280), (9, 2048), (20, 3456), (1025, 767),
          (7, 6001), (4, 8200), (3, 12289), (2, 16384), (3, 16401), (2, 40000)]


def definition(h, gain, beta, eps):
    """As gated_ref.layernorm, for a mean that is kept in two float32 parts, hi and lo."""
    C = h.shape[1]
    mean = h.sum(1) / C
    d = h - mean[:, None]
    # of the sum: a lane adds up to 16 differences of up to 2 max|d|, takes them to the wave's value in three roundings and
    # meets the other lanes in seven additions, in float32; the rest is in 64 bits
    lost = 27 * U * 2 * d.abs().amax(1) + (depth(C) + 4) * 2.0 ** -53 * h.abs().sum(1) / C
    e_mean = U * mean.abs() + lost + TINY
    # |h - hi| <= |d| + U |mean|, rounded; lo is at most U |mean|, off by U of itself, as is its product with 1 / deviation;
    # their difference is rounded once
    e_d = 2 * U * d.abs() + (4 * U * U * mean.abs() + lost)[:, None] * 1.01
    var = d.square().sum(1) / C
    # sum (h - hi)^2 / C is at most twice the variance; lo^2, taken off it, is at most the variance, and stands for
    # 2 lo sum(h - hi) / C - lo^2 to within 2 |lo| times what the sum lost
    e_var = (2 * d.abs() * e_d + e_d * e_d).sum(1) / C + 2 * (depth(C) + 6) * U * (var + eps) + 2 * var.sqrt() * lost
    rstd = 1 / (var + eps).sqrt()
    x = e_var / (var + eps)
    rel = 0.5 * x * (1 + x) + 4 * U
    y = d * rstd[:, None] * gain
    e = (g := (rstd[:, None] * gain).abs()) * e_d * (1 + rel[:, None]) + y.abs() * (rel[:, None] + 3 * U)
    assert g.shape == e.shape
    y = y + beta
    return mean, e_mean, rstd, rel, y, e + U * y.abs() + TINY


@pytest.mark.parametrize("mean,dev", [(4096.0, 0.03), (1000.0, 0.01), (-3e4, 2.0), (0.1, 1e-6)])
@pytest.mark.parametrize("R,C", SHAPES)
def test_means_far_above_the_deviation(R, C, mean, dev):
    say(f"layernorm about {mean} by {dev}: {R}x{C}")
    g = gen("means", R, C, mean)
    X, res = mean + dev * normal(g, R, C), dev * normal(g, R, C)
    X[:, 0] = mean + dev                      # two values at least, in every row
    X[:, 1] = mean - dev
    res[:, :2] = 0
    gain, beta = 1 + normal(g, C, scale=0.1), normal(g, C, scale=0.1)
    for residual, eps in ((None, 0.0), (res, 0.0), (None, EPS)):
        Q, s, H, Y, mu, rstd = B.ternary_layernorm_quantize(X, gain, beta, eps, residual=residual, save=True)
        m, em, r, rel, y, e = definition(H.double(), gain.double(), beta.double(), eps)
        ref.check(mu, m, em, "mean")
        ref.check(rstd, r, rel * r, "rstd")
        ref.check(Y, y, e, "Y")
        ref.check_int8(Q, s, y, e, "layernorm")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", SHAPES)
def test_rows_of_one_value(R, C, kind):
    """Their variance is 0: y is beta, and without an eps 1 / deviation is inf and y NaN, as the formula has it."""
    say(f"layernorm of rows of one value: {R}x{C} {kind}")
    g = gen("one value", R, C)
    v = normal(g, R, dtype=KINDS[kind], scale=100.0)
    v[0] = 1e30
    X = v[:, None].expand(R, C).contiguous()
    gain, beta = 1 + normal(g, C, scale=0.1), normal(g, C)
    want = torch.tensor(EPS).sqrt().reciprocal().item()
    for residual in (None, torch.zeros_like(X)):
        Q, s, _, Y, mean, rstd = B.ternary_layernorm_quantize(X, gain, beta, EPS, residual=residual, save=True)
        assert torch.equal(mean, v.float())
        assert bool(((rstd - want).abs() <= 4 * U * want).all())
        assert torch.equal(Y, beta.to(Y.dtype).expand(R, C))
        Q, s, _, Y, mean, rstd = B.ternary_layernorm_quantize(X, gain, beta, 0.0, residual=residual, save=True)
        assert torch.equal(mean, v.float()) and bool((rstd == float("inf")).all())
        assert bool(torch.isnan(Y).all()) and bool(torch.isnan(s).all()) and not bool(Q.any())
