"""The product's epilogue in every kernel that its dispatch can choose: each
tile of the tiled kernel with aligned and unaligned loads, whole and ragged,
and each column width of the few-row kernel, beside the shapes of
test_gpu_block.py.  (test_epilogue_plan.py asks the plan whether any choice is
left out.)"""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
from test_gpu_block import KINDS, Placed, product_inputs, say  # noqa: E402

pytestmark = pytest.mark.gpu

# 128 x 144 tiles, 256 x 128 tiles and 64 x 64 tiles, each whole and ragged
# with K % 16 == 0 (vector loads), then with rows of 4-byte pieces
TILED = [(8192, 2304, 80), (8191, 2301, 80), (8191, 2301, 68), (4096, 4096, 80), (4095, 4093, 80), (4096, 4096, 68),
         (4095, 4093, 336), (4095, 4091, 148), (640, 704, 80), (1990, 2000, 144), (500, 1777, 404)]
# the kernel of mid-size outputs with its last columns mostly past the output, and five tiles a CU
RING = [(16384, 243, 256), (4101, 4224, 128)]
FEW_ROWS = [(1, 4100, 128), (7, 8200, 128), (12, 4100, 64), (16, 8207, 192), (20, 4100, 128), (32, 4099, 1024)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", TILED + RING + FEW_ROWS)
def test_product_epilogue_in_every_kernel(M, N, K, kind):
    pl = B.epilogue_plan(M, N, K)
    say(f"product epilogue {M}x{N}x{K} {kind}: kernel {pl.kernel}, tile {pl.tile_rows}x{pl.tile_cols}, fast {pl.fast_path}")
    dt = KINDS[kind]
    A, Wp, rs, ws, bias, res = product_inputs(M, N, K, dt, kind, 11)
    p = Placed(8)
    for act, b, r, save in (("relu2", bias, res, True), ("none", None, None, False), ("gelu_tanh", bias, None, True),
                            ("silu", None, res, False)):
        z, ez, y, ey = ref.product(A, Wp, rs, float(torch.tensor(ws)), b, act, r)
        Y, Z = B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=b, act=act, residual=r, out_dtype=dt, save=save,
                                          Y=p((M, N), dt), Z=p((M, N), dt) if save else None)
        torch.cuda.synchronize()
        p.check()
        p.made.clear()
        ref.check(Y, y, ref.rounded(y, ey, dt), f"{act}: Y")
        if save:
            ref.check(Z, z, ref.rounded(z, ez, dt), f"{act}: Z")
        if r is not None:                     # into the residual stream itself
            Yi = r.clone()
            B.ternary_gemm_s8_epilogue(A, Wp, rs, ws, bias=b, act=act, residual=Yi, out_dtype=dt, Y=Yi)
            assert torch.equal(Yi, Y), act
