"""Which kernel the product with its epilogue takes, by the host-only plan query."""
import ctypes

import pytest

from shapes import TILES
from ternary_weight_int8_amd import binding as B


def test_refusals():
    pl = B.TgemmPlan()
    q = B.lib().ternary_gemm_epilogue_plan
    assert q(4, 8, 16, 256, 256, 8, None) == B.ERR_NULL
    p = ctypes.byref(pl)
    for M, N, K in ((0, 8, 16), (4, 0, 16), (4, 8, 0)):
        assert q(M, N, K, 256, 256, 8, p) == B.ERR_DIM
    assert q(4, 8, 18, 256, 256, 8, p) == B.ERR_PACK
    assert q(4, 8, 1 << 24, 256, 256, 8, p) == B.ERR_BOUND
    for cus, xcds in ((0, 8), (256, 0), (100, 8)):
        assert q(4, 8, 16, 256, cus, xcds, p) == B.ERR_DIM


def test_kernel_choice():
    k = lambda *s, **kw: B.epilogue_plan(*s, **kw).kernel  # noqa: E731
    tile = lambda *s, **kw: (B.epilogue_plan(*s, **kw).tile_rows, B.epilogue_plan(*s, **kw).tile_cols)  # noqa: E731
    assert k(1, 3456, 1280) == k(32, 64, 64) == B.KERNEL_SKINNY
    assert k(33, 3456, 1280) == k(32, 64, 80) == B.KERNEL_TILED
    assert k(16384, 3456, 1280) == B.KERNEL_STREAM                 # 768 tiles of 512 x 144
    assert k(16384, 1280, 3456) == B.KERNEL_RING                   # 288 of them: a second round for 32
    assert k(4096, 1280, 3456) == B.KERNEL_RING
    assert k(4096, 1280, 3456, align=8) == k(4096, 1280, 3452) == B.KERNEL_TILED
    assert k(1000, 1000, 1024) == B.KERNEL_TILED                   # 64 tiles of 128 x 128
    assert k(2000, 2048, 2048) == B.KERNEL_RING                    # 256
    assert k(4096, 4096, 4096) == B.KERNEL_TILED                   # 512 tiles of 256 x 128
    assert tile(2000, 2000, 2000) == (64, 64)                      # at most one 128 x 144 tile a CU
    assert tile(8192, 2304, 1020) == (128, 144)
    assert tile(4096, 4096, 1020) == (256, 128)
    # without an epilogue none takes the ring kernel, and the forward's own plan stands
    assert B.plan("fwd", 4096, 1280, 3456).kernel == B.KERNEL_TILED


@pytest.mark.parametrize("M,N,K", [(1, 17, 64), (4096, 1280, 3456), (3001, 1250, 1088), (16384, 1280, 128),
                                   (15001, 2301, 128), (8191, 2301, 68), (2000, 2000, 2000)])
@pytest.mark.parametrize("cus,xcds", [(256, 8), (64, 2)])
def test_every_output_tile_covered_once(M, N, K, cus, xcds):
    pl = B.epilogue_plan(M, N, K, cus=cus, xcds=xcds)
    seen = [t for wg in range(pl.workgroups) for it in range(pl.tiles_per_workgroup)
            if (t := B.tile_of(pl, wg, it)) is not None]
    want = {(r, c) for r in range(0, M, pl.tile_rows) for c in range(0, N, pl.tile_cols)}
    assert len(seen) == len(want) == pl.tiles and set(seen) == want
    assert pl.lds_bytes <= 160 * 1024 and pl.threads_per_workgroup in (256, 512)
    if pl.kernel == B.KERNEL_TILED:
        assert (pl.tile_rows, pl.tile_cols) in TILES


def gpu_shapes():
    """(M, N, K, alignment of the operands) of every product that the GPU tests of the epilogue run."""
    pytest.importorskip("torch")
    import test_gpu_block as block
    import test_gpu_epilogue_kernels as kernels

    def of(f):
        return next(m.args[1] for m in f.pytestmark if m.name == "parametrize" and m.args[0].startswith("M,N,K"))

    shapes = [(*s, 256) for s in block.PRODUCTS + kernels.TILED + kernels.RING + kernels.FEW_ROWS + of(block.test_product_epilogue_large)]
    for M, N, K, offset in of(block.test_product_epilogue_misaligned):
        shapes += [(M, N, K, 256), (M, N, K, offset & -offset)]
    return shapes


def test_gpu_tests_reach_every_choice():
    seen, ragged = set(), set()
    for M, N, K, align in gpu_shapes():
        pl = B.epilogue_plan(M, N, K, align=align)
        choice = (pl.kernel, pl.tile_rows, pl.tile_cols, M > 8 if pl.kernel == B.KERNEL_SKINNY else pl.fast_path)
        seen.add(choice)
        ragged.add((*choice, M % pl.tile_rows != 0 or N % pl.tile_cols != 0))
    want = {(B.KERNEL_TILED, *t, fast) for t in TILES for fast in (0, 1)}
    want |= {(B.KERNEL_SKINNY, 16, c, al) for c in (16, 32, 64) for al in (False, True)}
    want |= {(B.KERNEL_SKINNY, 32, c, True) for c in (16, 32, 64)}
    want |= {(B.KERNEL_STREAM, 512, 144, 1), (B.KERNEL_RING, 128, 128, 1)}
    assert seen == want, (want - seen, seen - want)
    # the tiles' guarded and unguarded ends
    for c in want:
        if c[0] != B.KERNEL_SKINNY and c[3]:
            assert (*c, True) in ragged and (*c, False) in ragged, c


# 256 x 128 tiles of the tiled kernel that fill a CU's last round beat the ring
# kernel's 128 x 128 ones over many steps, at every size where they do and not at one
@pytest.mark.parametrize("K", [64, 512, 576, 1024, 4096])
@pytest.mark.parametrize("M,N,a_cu", [
    (2000, 2048, 1), (4096, 1536, 2), (4096, 2048, 2), (4096, 2176, 3), (2816, 4096, 3), (6144, 2048, 3), (4096, 3200, 4),
    (4096, 3584, 4), (4096, 3968, 4), (4096, 4096, 4), (4095, 4095, 4), (8192, 1920, 4), (4096, 4224, 5), (4096, 4352, 5),
    (50000, 288, 5), (65000, 288, 6), (100000, 144, 7)])
def test_ring_kernel_by_the_tiles_of_a_cu(M, N, a_cu, K):
    assert -(-(-(-M // 128) * -(-N // 128)) // 256) == a_cu
    assert B.plan("fwd", M, N, K).kernel != B.KERNEL_STREAM
    assert (B.epilogue_plan(M, N, K).kernel == B.KERNEL_RING) == (a_cu in (1, 2, 3, 5) or (a_cu == 4 and K <= 512))


def test_ring_kernel_where_the_stream_kernel_would_idle():
    for tiles, ring in ((288, True), (352, True), (384, False), (448, False), (512, False), (544, True), (608, False)):
        N = 144 * tiles // 32                                    # 16384 rows: 32 of 512
        assert B.plan("fwd", 16384, N, 1024).kernel == B.KERNEL_STREAM and B.plan("fwd", 16384, N, 1024).tiles == tiles
        assert (B.epilogue_plan(16384, N, 1024).kernel == B.KERNEL_RING) == ring, tiles
