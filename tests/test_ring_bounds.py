"""CPU model of the addresses that tgemm_ring (the epilogue's forward on
mid-size outputs) computes for its direct-to-LDS loads, which have no range
check: against the buffers' sizes for every shape that the GPU tests run on
it, and its LDS destinations against their stages.  Its waits by count are
checked too, by following the operations of a wave in issue order.

The offsets, restated: A load i of wave w, lane l: tile row r = 16 (kALoads w +
i) + l / 4, row min(m0 + r, M - 1), byte 16 ((l % 4) ^ ((r >> 1) % 4), plus 64 s
in step s; packed load i: dword d = 64 (first_unit(w) + i) + l, row min(n0 + d / 4,
N - 1), byte 4 (d % 4) plus 16 s.
"""
import numpy as np
import pytest

BM, BN, WM, WN, D = 128, 128, 4, 2, 4
NW, BK = WM * WN, 64
A_STAGE, A_LOADS = BM * BK, BM * BK // 1024 // NW
UNITS = BN // 16
Q, R = divmod(UNITS, NW)
WD_STAGE, WP_STAGE, PS = BN * BK, UNITS * 256, D - 1
SHAPES = [(4096, 1280, 64), (7700, 2400, 192), (8191, 2305, 128), (3001, 1250, 1088), (2048, 2048, 320), (16384, 243, 256),
          (4096, 1280, 3456)]


def units_of(w):
    return Q + (1 if w >= NW - R else 0)


def first_unit(w):
    return Q * w + (w - (NW - R) if w > NW - R else 0)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_load_addresses_stay_in_their_buffers(M, N, K):
    lane, kb, nk = np.arange(64), K // 4, K // BK
    tiles_c = -(-N // BN)
    for pos in range(tiles_c * -(-M // BM)):
        m0, n0 = pos // tiles_c * BM, pos % tiles_c * BN
        for w in range(NW):
            for i in range(A_LOADS):
                r = 16 * (A_LOADS * w + i) + (lane >> 2)
                off = np.minimum(m0 + r, M - 1) * K + 16 * ((lane & 3) ^ ((r >> 1) & 3))
                assert off.min() >= 0 and off.max() + 64 * (nk - 1) + 16 <= M * K
            for i in range(units_of(w)):
                d = 64 * (first_unit(w) + i) + lane
                off = np.minimum(n0 + (d >> 2), N - 1) * kb + 4 * (d & 3)
                assert off.min() >= 0 and off.max() + 16 * (nk - 1) + 4 <= N * kb


def test_lds_destinations_stay_in_their_stages():
    off_wd = D * A_STAGE
    off_wp = off_wd + 3 * WD_STAGE
    assert off_wp + PS * WP_STAGE <= 80 * 1024
    rows, units = set(), set()
    for w in range(NW):
        for i in range(A_LOADS):
            a = w * A_LOADS * 1024 + 1024 * i + 16 * np.arange(64)
            assert a.max() + 16 <= A_STAGE
            rows |= set(a.tolist())
        for i in range(units_of(w)):
            u = first_unit(w) + i
            units.add(u)
            d = 64 * u + np.arange(64)
            assert 256 * u + 4 * 63 + 4 <= WP_STAGE and (d >> 2).max() < BN     # loaded, and decoded rows of 64 bytes
    assert len(rows) * 16 == A_STAGE and units == set(range(UNITS))


@pytest.mark.parametrize("nk", [1, 2, 3, 4, 5, 20])
@pytest.mark.parametrize("w", range(NW))
def test_waits_cover_what_is_read(nk, w):
    # operations of one wave in issue order: ("W" | "A", step, stage); a wait
    # for at most n leaves the last n in flight
    ops, batch = [], A_LOADS + Q
    wait_mid, wait_end = A_LOADS + (D - 2) * batch, (D - 2) * batch

    def issue(step, stage_w, stage_a):
        ops.extend([("W", step, stage_w)] * units_of(w) + [("A", step, stage_a)] * A_LOADS)

    def landed(n, kind, step):
        return all(o[:2] != (kind, step) for o in ops[len(ops) - n:] if n) if n else True

    for s in range(D - 1):
        issue(s, s, s)
    n = A_LOADS + (D - 3) * batch
    assert landed(n, "W", 0) and landed(n, "W", 1)
    issue(D - 1, 0, D - 1)
    assert landed(wait_end, "A", 0) and landed(wait_end, "A", 1)
    holds_w = {(D - 1) % PS: D - 1, **{s: s for s in range(1, D - 1)}}
    q0, pl, pd = 0, 1 % PS, 2 % PS
    for g in range(nk):
        assert holds_w[pl] <= g + 1          # overwritten once it is decoded
        issue(g + D, pl, q0)
        holds_w[pl] = g + D
        assert landed(wait_mid, "W", g + 2) and holds_w[pd] == g + 2
        assert landed(wait_end, "A", g + 2)
        q0, pl, pd = (q0 + 1) % D, (pl + 1) % PS, (pd + 1) % PS
