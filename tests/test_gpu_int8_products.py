"""GPU parity of the gated ternary product and of the product with int8 weights
with their definitions in 64 bits, at the sizes, contractions, alignments and
rows where they can go wrong."""
import pytest

from ternary_weight_int8_amd import binding as B

torch = pytest.importorskip("torch")
import block_ref as ref  # noqa: E402
import gated_ref as gref  # noqa: E402
from test_gpu_block import ACTS, DEV, KINDS, Placed, gen, normal, placed_copy, say  # noqa: E402

pytestmark = pytest.mark.gpu


def int8(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def packed(g, n, k):
    return torch.randint(0, 256, (n, k // 4), generator=g, device=DEV, dtype=torch.uint8)


# (M, N, K): one element; rows around the kernels' limits; contractions that are
# no whole chunk, step or super-step; ragged tiles of each size; many tiles
SIZES = [(1, 1, 4), (1, 5, 8), (3, 17, 60), (1, 729, 244), (2, 100, 256), (8, 33, 320), (9, 130, 1280), (17, 64, 2048),
         (27, 3456, 1280), (31, 65, 2112), (33, 70, 128), (64, 129, 576), (65, 31, 16), (65, 64, 64), (66, 200, 68),
         (100, 300, 1000), (129, 257, 400), (200, 1280, 320), (700, 1000, 192), (1782, 729, 244), (1000, 2000, 260),
         (2049, 1025, 144), (4100, 2050, 80), (5000, 3000, 272)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated(M, N, K, kind):
    dt, g = KINDS[kind], gen("gated", M, N, K, kind)
    for i, act in enumerate(ACTS):
        say(f"gated {M}x{N}x{K} {kind} {act}")
        A, W, rs = int8(g, M, K), packed(g, 2 * N, K), 0.01 + torch.rand(M, generator=g, device=DEV)
        gs, us, bias = 0.7 / K ** 0.5 / 40, 0.02, normal(g, 2 * N) if i % 2 else None
        Y, Z = B.ternary_gemm_s8_gated(A, W, rs, gs, us, bias=bias, act=act, out_dtype=dt, save=i != 2)
        f = lambda v: float(torch.tensor(v))  # noqa: E731  (the call takes a float32)
        z, ez, y, ey = gref.gated_product(A, W, rs, f(gs), f(us), bias, act)
        ref.check(Y, y, ref.rounded(y, ey, dt), "Y")
        if i != 2:
            ref.check(Z, z, ref.rounded(z, ez, dt), "Z")
        else:
            assert Z is None
            assert torch.equal(B.ternary_gemm_s8_gated(A, W, rs, gs, us, bias=bias, act=act, out_dtype=dt, save=True)[0], Y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", SIZES + [(1, 16384, 1283), (5, 9000, 515), (40, 8200, 100), (1, 3, 1), (2, 2, 15), (70, 40, 1),
                                           (300, 500, 131), (1500, 700, 1285)])
def test_int8_weights(M, N, K, kind):
    dt, g = KINDS[kind], gen("s8s8", M, N, K, kind)
    for i, act in enumerate(ACTS):
        say(f"s8s8 {M}x{N}x{K} {kind} {act}")
        A, W, rs = int8(g, M, K), int8(g, N, K), 0.01 + torch.rand(M, generator=g, device=DEV)
        cs = (0.5 + torch.rand(N, generator=g, device=DEV)) / (5000 * K ** 0.5) if i != 3 else None
        if cs is None:
            rs = rs / (5000 * K ** 0.5)
        bias, res = normal(g, N) if i % 2 else None, normal(g, M, N, dtype=dt) if i in (0, 3) else None
        save = i != 1
        Y, Z = B.ternary_gemm_s8s8_epilogue(A, W, rs, cs, bias=bias, act=act, residual=res, out_dtype=dt, save=save)
        z, ez, y, ey = gref.int8_product(A, W, rs, cs, bias, act, res)
        ref.check(Y, y, ref.rounded(y, ey, dt), "Y")
        if save:
            ref.check(Z, z, ref.rounded(z, ez, dt), "Z")
        else:
            assert Z is None
        if res is not None:                   # the residual in place
            r = res.clone()
            got, _ = B.ternary_gemm_s8s8_epilogue(A, W, rs, cs, bias=bias, act=act, residual=r, out_dtype=dt, Y=r)
            assert got is r and torch.equal(r, Y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K,offset", [(1, 729, 244, 1), (27, 130, 256, 4), (64, 100, 512, 1), (65, 100, 512, 1),
                                          (300, 333, 320, 16), (300, 333, 100, 3), (1000, 1030, 64, 8)])
def test_placed_anywhere(M, N, K, offset, kind):
    say(f"products at offset {offset}: {M}x{N}x{K} {kind}")
    dt, g = KINDS[kind], gen("placed", M, N, K, kind)
    A, W, W8, rs = int8(g, M, K), packed(g, 2 * N, K), int8(g, N, K), torch.rand(M, generator=g, device=DEV)
    cs, b, b2, res = torch.rand(N, generator=g, device=DEV), normal(g, N), normal(g, 2 * N), normal(g, M, N, dtype=dt)
    p = Placed(offset)
    Ap, Wp, W8p, rsp, csp, bp, b2p, rp = (placed_copy(p, t) for t in (A, W, W8, rs, cs, b, b2, res))
    want = B.ternary_gemm_s8_gated(A, W, rs, 1e-3, 2e-3, bias=b2, out_dtype=dt, save=True)
    got = B.ternary_gemm_s8_gated(Ap, Wp, rsp, 1e-3, 2e-3, bias=b2p, out_dtype=dt, save=True, Y=p((M, N), dt),
                                  Z=p((M, 2 * N), dt))
    want8 = B.ternary_gemm_s8s8_epilogue(A, W8, rs, cs, bias=b, residual=res, out_dtype=dt, save=True)
    got8 = B.ternary_gemm_s8s8_epilogue(Ap, W8p, rsp, csp, bias=bp, residual=rp, out_dtype=dt, save=True, Y=p((M, N), dt),
                                        Z=p((M, N), dt))
    torch.cuda.synchronize()
    p.check()
    assert all(torch.equal(a, b) for a, b in zip(got + got8, want + want8))


@pytest.mark.parametrize("M", [5, 64, 65, 600])
def test_rows_do_not_depend_on_the_batch(M):
    """The sums are whole numbers and every kernel rounds alike: a row of any batch is the row of a batch of one."""
    say(f"rows of a batch of {M}")
    g = gen("rows", M)
    A, W, W8, rs = int8(g, M, 512), packed(g, 600, 512), int8(g, 300, 512), torch.rand(M, generator=g, device=DEV) * 1e-3
    cs, b = torch.rand(300, generator=g, device=DEV), normal(g, 300)
    Y, _ = B.ternary_gemm_s8_gated(A, W, rs, 0.5, 0.25, act="gelu_tanh", out_dtype=torch.float32)
    Y8, _ = B.ternary_gemm_s8s8_epilogue(A, W8, rs, cs, bias=b, act="silu", out_dtype=torch.float32)
    for r in {0, M // 2, M - 1}:
        a, s = A[r:r + 1].contiguous(), rs[r:r + 1].contiguous()
        assert torch.equal(B.ternary_gemm_s8_gated(a, W, s, 0.5, 0.25, act="gelu_tanh", out_dtype=torch.float32)[0][0], Y[r])
        assert torch.equal(B.ternary_gemm_s8s8_epilogue(a, W8, s, cs, bias=b, act="silu", out_dtype=torch.float32)[0][0], Y8[r])


@pytest.mark.parametrize("M", [3, 100])
def test_longest_contraction_is_exact(M):
    """131071 products of -128 and -128: one short of the sums that int32 cannot hold."""
    say(f"longest contraction, {M} rows")
    K = 131071
    A = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    W = torch.full((5, K), -128, dtype=torch.int8, device=DEV)
    Y, _ = B.ternary_gemm_s8s8_epilogue(A, W, torch.ones(M, device=DEV), out_dtype=torch.float32)
    assert bool((Y == float(torch.tensor(K * 16384, dtype=torch.float32))).all())


def test_offsets_past_32_bits():
    """Inputs and outputs of more than 2^32 bytes: the last rows are those of a small call."""
    say("offsets past 32 bits")
    g = gen("far product")
    M, N, K = 70000, 17000, 80
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    A, W, W8 = int8(g, M, K), packed(g, 2 * N, K), int8(g, N, K)
    rs, cs = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    last, ls = A[-70:].contiguous(), rs[-70:].contiguous()
    Y, Z = B.ternary_gemm_s8_gated(A, W, rs, 1e-3, 1e-3, out_dtype=torch.float32, save=True)
    y, z = B.ternary_gemm_s8_gated(last, W, ls, 1e-3, 1e-3, out_dtype=torch.float32, save=True)
    assert torch.equal(Y[-70:], y) and torch.equal(Z[-70:], z)
    del Y, Z
    Y, _ = B.ternary_gemm_s8s8_epilogue(A, W8, rs, cs, out_dtype=torch.float32)
    assert torch.equal(Y[-70:], B.ternary_gemm_s8s8_epilogue(last, W8, ls, cs, out_dtype=torch.float32)[0])
    del Y, A, W8
    A, W8 = int8(g, 90, 48000), int8(g, 100000, 48000)    # 4.8 GB of weights
    rs, cs = rs[:90].contiguous(), torch.rand(100000, generator=g, device=DEV)
    Y, _ = B.ternary_gemm_s8s8_epilogue(A, W8, rs, cs, out_dtype=torch.float32)
    few, _ = B.ternary_gemm_s8s8_epilogue(A[:3].contiguous(), W8, rs[:3].contiguous(), cs, out_dtype=torch.float32)
    w, c = W8[-70:].contiguous(), cs[-70:].contiguous()
    assert torch.equal(Y[:, -70:], B.ternary_gemm_s8s8_epilogue(A, w, rs, c, out_dtype=torch.float32)[0])
    assert torch.equal(few, Y[:3])


def test_very_many_rows_and_columns():
    """More rows to lay out than a launch has workgroups for: 2^27 of the gated weights, then 2^27 + 5 of A."""
    say("very many rows and columns")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    g, N = gen("many"), 1 << 26
    A, W, rs = int8(g, 1, 4), packed(g, 2 * N, 4), torch.ones(1, device=DEV)
    Y, _ = B.ternary_gemm_s8_gated(A, W, rs, 0.5, 0.25, act="none", out_dtype=torch.float32)
    acc = torch.zeros(2 * N, dtype=torch.int32, device=DEV)
    for k in range(4):
        c = (W[:, 0] >> (2 * k)) & 3
        acc += ((c & 1).int() - (c >> 1).int()) * int(A[0, k])
    assert torch.equal(Y[0], (acc[:N].float() * 0.5) * (acc[N:].float() * 0.25))
    del Y, W, acc
    M = (1 << 27) + 5
    A, W, rs = int8(g, M, 17), int8(g, 3, 17), torch.rand(M, generator=g, device=DEV)
    Y, _ = B.ternary_gemm_s8s8_epilogue(A, W, rs, out_dtype=torch.float32)
    for n in range(3):
        acc = torch.zeros(M, dtype=torch.int32, device=DEV)
        for k in range(17):
            acc += A[:, k].int() * int(W[n, k])
        assert torch.equal(Y[:, n], acc.float() * rs)


def test_longest_gated_contraction():
    """16777212 products a sum: a tile's rows lie up to 2^32 bytes apart, and the last of the sums is as large as it can be."""
    say("longest gated contraction")
    M, N, K, part = 300, 2, 16777212, 1 << 18
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    g = gen("long gated")
    A, W, rs = int8(g, M, K), packed(g, 2 * N, K), torch.ones(M, device=DEV)
    A[M - 1], W[0] = 127, 0x55                        # the gate's first row: every weight 1
    _, Z = B.ternary_gemm_s8_gated(A, W, rs, 1.0, 1.0, act="none", out_dtype=torch.float32, save=True)
    want = torch.zeros(M, 2 * N, dtype=torch.float64, device=DEV)
    for b in range(0, K // 4, part):
        codes = torch.stack([(W[:, b:b + part] >> (2 * k)) & 3 for k in range(4)], dim=2).flatten(1)
        w = (codes & 1).double() - (codes >> 1).double()
        want += A[:, 4 * b:4 * (b + part)].double() @ w.t().contiguous()
    assert want[M - 1, 0] == 127 * K
    assert torch.equal(Z, want.float())               # whole numbers: exact in 64 bits, rounded once
