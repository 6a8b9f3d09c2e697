"""Backward passes of rows so wide that their column sums have more groups of
columns than a launch has workgroups for."""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
from test_gpu_block import DEV, say  # noqa: E402

pytestmark = pytest.mark.gpu
WIDE = (1 << 27) + 5      # 32 threads a column of the sums: 2^32 of them


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def pattern(n, seed, dtype=torch.float32):
    """Values whose neighbours, and whose distant columns, differ."""
    k = torch.arange(n, device=DEV)
    return (((k * 2654435761 + seed) >> 7) % 4093 - 2046).to(torch.float32).mul_(2.0 ** -10).to(dtype).view(1, n)


def test_gated_biases():
    say("gated backward of 2^26 columns a half")
    room(40)
    C = WIDE // 2
    dY, Z = pattern(C, 1), pattern(2 * C, 2)
    dZ, db, Q, s = B.ternary_gated_backward(dY, Z, 0.5, 0.25, act="relu")
    assert torch.equal(db, dZ[0])             # one row: the sums are its values
    assert torch.equal(dZ[0, C:], dY[0] * Z[0, :C].clamp_min(0))


def test_layernorm_gradients():
    say("layer norm backward of 2^26 columns")
    room(40)
    C = WIDE // 2 + 1
    dY, H, gain = pattern(C, 1), pattern(C, 2), pattern(C, 3)[0].abs()
    mean, rstd = torch.tensor([0.25], device=DEV), torch.tensor([2.0], device=DEV)
    _, dgain, dbeta = B.ternary_layernorm_backward(dY, H, gain, mean, rstd)
    assert torch.equal(dbeta, dY[0]) and torch.equal(dgain, dY[0] * ((H[0] - 0.25) * 2))


def test_rmsnorm_gradient():
    say("RMS norm backward of 2^27 columns")
    room(40)
    dY, H, gain = pattern(WIDE, 1), pattern(WIDE, 2), pattern(WIDE, 3)[0].abs()
    _, dgain = B.ternary_rmsnorm_backward(dY, H, gain, torch.tensor([2.0], device=DEV))
    assert torch.equal(dgain, dY[0] * (H[0] * 2))


def test_epilogue_bias():
    """bfloat16, and more columns than the partial sums' launch has threads for."""
    say("epilogue backward of 2^28 columns")
    room(40)
    C = (1 << 28) + 300
    dY, Z = pattern(C, 1, torch.bfloat16), pattern(C, 2, torch.bfloat16)
    dZ, db, Q, s = B.ternary_epilogue_backward(dY, Z, act="relu")
    assert torch.equal(db, dZ[0].float()) and torch.equal(dZ, torch.where(Z > 0, dY, torch.zeros_like(dY)))
