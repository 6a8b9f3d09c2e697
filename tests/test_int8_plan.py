"""Which kernel and tile the gated product and the product with int8 weights take,
by the host-only plan queries, held to recorded times of every tile."""
import ctypes
import math
import os

import pytest

from ternary_weight_int8_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILES = [(256, 192), (256, 128), (128, 192), (128, 128), (64, 128), (64, 64)]
KIND = {"f32": B.OUT_F32, "bf16": B.OUT_BF16}


def tile(pl):
    return pl.tile_rows, pl.tile_cols


def test_refusals():
    pl = B.TgemmPlan()
    p = ctypes.byref(pl)
    s8s8 = lambda M=100, N=8, K=16, al=256, act=0, kind=B.OUT_F32, cus=256, xcds=8, out=p: (  # noqa: E731
        B.lib().ternary_gemm_s8s8_plan(M, N, K, al, act, 0, 0, kind, cus, xcds, out))
    gated = lambda M=100, N=8, K=16, al=256, act=0, kind=B.OUT_F32, cus=256, xcds=8, out=p: (  # noqa: E731
        B.lib().ternary_gemm_s8_gated_plan(M, N, K, al, act, 0, kind, cus, xcds, out))
    for q in (s8s8, gated):
        assert q() == B.OK and q(out=None) == B.ERR_NULL
        assert q(M=0) == q(N=0) == q(K=0) == q(N=(1 << 27) + 1) == q(cus=0) == q(xcds=0) == q(cus=100) == B.ERR_DIM
        assert q(act=5) == q(act=-1) == B.ERR_VALUE and q(kind=0) == q(kind=3) == B.ERR_KIND
    assert gated(K=18) == B.ERR_PACK and gated(K=16777220) == B.ERR_BOUND and s8s8(K=131072) == B.ERR_BOUND


def test_kernels():
    assert B.s8s8_plan(32, 3456, 1280).kernel == B.s8s8_plan(64, 1280, 1280).kernel == B.KERNEL_INT8_FEW
    assert B.s8s8_plan(33, 4096, 4096).kernel == B.s8s8_plan(65, 1280, 1280).kernel == B.KERNEL_INT8
    assert B.s8s8_plan(33, 4096, 4096, align=8).kernel == B.s8s8_plan(64, 4096, 4095).kernel == B.KERNEL_INT8_FEW
    assert B.gated_plan(128, 16384, 1280).kernel == B.gated_plan(192, 8192, 1280).kernel == B.KERNEL_SKINNY
    assert B.gated_plan(129, 16384, 1280).kernel == B.gated_plan(193, 64, 64).kernel == B.KERNEL_INT8
    assert B.gated_plan(1, 64, 68).kernel == B.gated_plan(1, 64, 64, align=8).kernel == B.KERNEL_INT8
    assert B.s8s8_plan(65, 8, 16).fast_path == 1 and B.s8s8_plan(65, 8, 17).fast_path == B.s8s8_plan(65, 8, 16, align=4).fast_path == 0


@pytest.mark.parametrize("M,N,K", [(65, 31, 16), (65, 1280, 320), (65, 3456, 1280), (128, 1280, 1280), (200, 1280, 320),
                                   (200, 1280, 1280), (300, 1280, 1280), (512, 1280, 1280), (873, 232, 80)])
@pytest.mark.parametrize("residual,save", [(True, True), (True, False), (False, True)])
def test_few_tiles_are_small_ones(M, N, K, residual, save):
    """Where 64 x 64 tiles leave CUs idle, larger ones leave more: float32 with residual and Z, 200x1280x1280 takes 7.4 us
    in them, 9.1 in 64 x 128 and 12.3 in 128 x 128."""
    assert math.ceil(M / 64) * math.ceil(N / 64) <= 256
    for kind in KIND.values():
        for act in ("none", "silu"):
            assert tile(B.s8s8_plan(M, N, K, act=act, residual=residual, save=save, kind=kind)) == (64, 64)


def recorded():
    rows = []
    with open(os.path.join(ROOT, "profiles", "int8_tiles.md")) as f:
        for line in f:
            w = line.split()
            if len(w) == 14 and w[0] in ("s8s8", "gated") and w[1].isdigit():
                rows.append((w[0], *map(int, w[1:4]), w[4], w[5], *map(int, w[6:8]), [float(x) for x in w[8:]]))
    return rows


def test_the_rule_on_recorded_times():
    rows, loss = recorded(), []
    assert len(rows) == 578
    for op, M, N, K, kind, act, res, save, us in rows:
        if op == "s8s8":
            pl = B.s8s8_plan(M, N, K, act=act, residual=bool(res), save=bool(save), kind=KIND[kind])
        else:
            pl = B.gated_plan(M, N, K, act=act, save=bool(save), kind=KIND[kind])
        assert pl.kernel == B.KERNEL_INT8
        loss.append(us[TILES.index(tile(pl))] / min(us))
    assert sum(x > 1.02 for x in loss) <= 62 and sum(x > 1.1 for x in loss) <= 7 and max(loss) < 1.2
    assert math.exp(sum(map(math.log, loss)) / len(loss)) < 1.0065


@pytest.mark.parametrize("M,N,K", [(1, 17, 64), (40, 300, 128), (65, 31, 16), (700, 1000, 1285), (1782, 1280, 3456),
                                   (4100, 2050, 80), (16384, 3456, 1280)])
@pytest.mark.parametrize("cus,xcds", [(256, 8), (64, 2)])
@pytest.mark.parametrize("op", ["s8s8", "gated"])
def test_every_output_tile_covered_once(op, M, N, K, cus, xcds):
    if op == "gated":
        K -= K % 4
    pl = (B.s8s8_plan if op == "s8s8" else B.gated_plan)(M, N, K, cus=cus, xcds=xcds)
    seen = [t for wg in range(pl.workgroups) for it in range(pl.tiles_per_workgroup)
            if (t := B.tile_of(pl, wg, it)) is not None]
    want = {(r, c) for r in range(0, M, pl.tile_rows) for c in range(0, pl.out_cols, pl.tile_cols)}
    assert pl.out_cols == (N if op == "s8s8" else 2 * N)
    assert len(seen) == len(want) == pl.tiles and set(seen) == want
    assert pl.lds_bytes <= 160 * 1024 and pl.threads_per_workgroup in (256, 512, 1024)


STAGES = {(256, 192): 2, (256, 128): 3, (128, 192): 3, (128, 128): 4, (64, 128): 3, (64, 64): 4}


def plans_of(op, M, N, K):
    """(plan, kind, sigmoid, save, residual) of the calls that the GPU tests make at a size."""
    for kind in KIND.values():
        for act in ("relu", "silu"):
            for save in (False, True):
                for res in (False, True) if op == "s8s8" else (False,):
                    pl = (B.s8s8_plan(M, N, K, act=act, residual=res, save=save, kind=kind) if op == "s8s8" else
                          B.gated_plan(M, N, K, act=act, save=save, kind=kind))
                    yield pl, kind, act == "silu", save, res


@pytest.mark.parametrize("op", ["s8s8", "gated"])
def test_gpu_tests_reach_every_kernel(op):
    """Each of the six tiles in each form, with more than one tile a workgroup, tiles inside the output and past its
    last row and column, a last step that is not whole, steps up to a tile's stages and more; every few-row kernel."""
    pytest.importorskip("torch")
    import test_gpu_int8_kernels as gpu
    tiles, deep, few = set(), set(), set()
    for M, N, K in (gpu.INT8_TILES + gpu.INT8_FEW if op == "s8s8" else gpu.GATED_TILES + gpu.GATED_FEW):
        for pl, *form in plans_of(op, M, N, K):
            t = tile(pl)
            if pl.kernel != B.KERNEL_INT8:
                few.add((*t, pl.threads_per_workgroup, M > 8 if op == "gated" else None, form[1]))
                continue
            whole = M // t[0] >= 2 and pl.out_cols // t[1] >= 2
            if whole and pl.tiles_per_workgroup >= 2 and M % t[0] and pl.out_cols % t[1] and K % 128:
                tiles.add((*t, *form))
                deep.add((*t, form[0], -(-K // 128) > STAGES[t]))
    assert tiles == {(*t, k, s, z, r) for t in TILES for k in KIND.values() for s in (False, True) for z in (False, True)
                     for r in ((False, True) if op == "s8s8" else (False,))}
    assert {(*t, k, True) for t in TILES for k in KIND.values()} <= deep
    if op == "s8s8":
        want = {(r, c, w) for r in (16, 32) for c, w in ((16, 512), (16, 1024), (32, 512), (64, 512))}
        assert few == {(*x, None, s) for x in want for s in (False, True)}
    else:
        want = {(16, c, al) for c in (16, 32, 64) for al in (False, True)} | {(32, c, True) for c in (16, 32, 64)}
        assert few == {(r, c, 512, al, s) for r, c, al in want for s in (False, True)}
