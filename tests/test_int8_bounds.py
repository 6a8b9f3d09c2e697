"""A CPU model of the tiled int8 kernel's loads straight into LDS, its fragment
reads and its waits: every load stays inside the rows that it may read, every
stage is filled once and read where it was filled, and a wave waits for what it
reads.  The statements that the model restates are held to the source."""
import os
import re

import numpy as np
import pytest

from ternary_weight_int8_amd.build import PKG

SRC = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(os.path.join(PKG, "csrc", "int8.hip")).read()))
CFGS = [tuple(map(int, m.split(","))) for m in re.findall(r"typedef mm::Cfg<([\d, ]+)> T\d+x\d+;", SRC)]


class Model:
    def __init__(self, cfg):
        self.BM, self.BN, self.WM, self.WN, self.KS, self.D, self.PERCU = cfg
        self.NW = self.WM * self.WN
        self.U, self.CH = self.KS // 64, self.KS // 16
        self.RPL = 64 // self.CH
        self.a_stage, self.stage = self.BM * self.KS, (self.BM + self.BN) * self.KS
        self.a_loads, self.w_loads = self.a_stage // 1024 // self.NW, self.BN * self.KS // 1024 // self.NW
        self.batch = self.a_loads + self.w_loads
        self.wait = (self.D - 2) * self.batch

    def swizzle(self, r, c):
        return c ^ ((r >> 1) & (self.CH - 1))

    def rows(self, loads):
        """[wave][load][lane] -> (row of the operand's tile, chunk that the lane fetches)"""
        w, i, l = np.ogrid[:self.NW, :loads, :64]
        r = self.RPL * (loads * w + i) + l // self.CH
        return r, self.swizzle(r, l % self.CH) + 0 * r

    def offsets(self, loads, have, K, last, tail):
        """Byte offsets from the tile's first row, `have` rows of the operand being left."""
        r, c = self.rows(loads)
        off = np.minimum(r, have - 1).astype(np.int64) * K + 16 * c
        if last:
            off = np.where(c >= tail, off - 16 * (c - (tail - 1)), off)
        return off


@pytest.mark.parametrize("cfg", CFGS)
def test_stages_are_filled_once_and_read_where_they_were_filled(cfg):
    m = Model(cfg)
    assert m.a_loads * 1024 * m.NW == m.a_stage and m.w_loads * 1024 * m.NW == m.BN * m.KS
    for loads, base, size in ((m.a_loads, 0, m.a_stage), (m.w_loads, m.a_stage, m.BN * m.KS)):
        r, c = m.rows(loads)
        w, i, l = np.ogrid[:m.NW, :loads, :64]
        at = base + 1024 * (loads * w + i) + 16 * l      # where the load puts the lane's 16 bytes
        assert np.array_equal(np.sort(at.ravel()), np.arange(base, base + size, 16))
        # a fragment read of row r, chunk c finds what the loads put there
        assert np.array_equal(at, base + r * m.KS + 16 * m.swizzle(r, c))
        # 16 rows at one chunk, and 8 of them, in different 16-byte groups of the 64 banks
        rr = np.arange(16)
        for chunk in range(m.CH):
            g = (rr * m.KS + 16 * m.swizzle(rr, chunk)) // 16 % 16
            assert len(set(g.tolist())) == 16


@pytest.mark.parametrize("cfg", CFGS)
@pytest.mark.parametrize("R,N,K", [(65, 31, 16), (65, 64, 64), (129, 257, 400), (700, 1000, 192), (2049, 1025, 144), (300, 40, 2080),
                                   (256, 4, 16777216), (16384, 3456, 1280)])
def test_loads_stay_inside_their_operands(cfg, R, N, K):
    m = Model(cfg)
    nk = -(-K // m.KS)
    tail = (K - (nk - 1) * m.KS) // 16
    assert 1 <= tail <= m.CH
    for rows, block, loads in ((R, m.BM, m.a_loads), (N, m.BN, m.w_loads)):
        for t in {0, (rows - 1) // block}:
            have = min(rows - t * block, block)
            for s in {0, nk - 1}:
                off = m.offsets(loads, have, K, s == nk - 1, tail)
                assert off.min() >= 0 and off.max() < 2 ** 32      # the loads' 32-bit offsets
                end = t * block * K + m.KS * s + off + 16
                assert end.max() <= rows * K
                # and a chunk that counts is the one of its row at its place
                r, c = m.rows(loads)
                counts = (m.KS * s + 16 * c < K) & (r < have)
                assert np.array_equal((m.KS * s + off)[counts], (r * K + m.KS * s + 16 * c)[counts])


@pytest.mark.parametrize("cfg", CFGS)
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 9, 10])
def test_waits_and_reuse(cfg, steps):
    """One wave's operations in order, over two tiles: at the barrier of step g the loads of step g + 1 have landed, and a
    stage is loaded again only after the barrier that every wave passes with its reads of it done."""
    m = Model(cfg)
    ops = []                       # (what, step) in issue order
    for s in range(m.D):
        ops += [("load", s)] * m.batch
    stores, after = 24, 0
    for g in range(2 * steps):
        allowed = m.wait + after
        landed = ops[:len(ops) - allowed] if allowed else ops
        assert landed.count(("load", g + 1)) == m.batch, (g, allowed)
        assert landed.count(("load", g)) == m.batch
        after = 0
        if g % steps == 0:
            ops += [("aux", g // steps)]
        # stage g % D: step g's fragments have all been read; the loads of step g + D take it
        ops += [("load", g + m.D)] * m.batch
        if g % steps == steps - 1:
            if steps >= m.D:       # else the kernel waits for everything
                seen = ops[:len(ops) - m.batch]              # what the last barrier could see
                seen = seen[:len(seen) - m.wait] if m.wait else seen
                assert ("aux", g // steps) in seen
            ops += [("store", g)] * stores
            after = stores


@pytest.mark.parametrize("text,times", [
    ("const int lrow = lane / C::CH, lslot = lane % C::CH;", 1),
    ("const int r = C::RPL * (C::kALoads * wave + i) + lrow;", 1),
    ("const int r = C::RPL * (C::kWLoads * wave + i) + lrow;", 1),
    ("offA[i] = (uint32_t)(r < mr ? r : mr) * (uint32_t)a.K + 16 * (uint32_t)(lslot ^ ((r >> 1) & (C::CH - 1)));", 1),
    ("offW[i] = (uint32_t)(r < nr ? r : nr) * (uint32_t)a.K + 16 * (uint32_t)(lslot ^ ((r >> 1) & (C::CH - 1)));", 1),
    ("if (c >= a.tail) offA[i] -= 16 * (uint32_t)(c - (a.tail - 1));", 1),
    ("if (c >= a.tail) offW[i] -= 16 * (uint32_t)(c - (a.tail - 1));", 1),
    ("return r * KS + 16 * (c ^ ((r >> 1) & (CH - 1)));", 1),
    ("ab = a.A + m0 * a.K; wb = a.W + n0 * a.K;", 1),
    ("lbase + st * C::kStage + 1024 * (C::kALoads * wave + i)", 1),
    ("lbase + st * C::kStage + C::kAStage + 1024 * (C::kWLoads * wave + i - C::kALoads)", 1),
    ("static constexpr int kWait = (D - 2) * kBatch;", 1),
    ("wait_barrier<(D - 1) * C::kBatch>();", 1),
    ("if (u == U - 1 && i == 0) { if (after == 2) wait_barrier<C::kWait + kStoresZ>(); else if (after) wait_barrier<C::kWait + kStores>(); "
     "else wait_barrier<C::kWait>(); after = 0; if (s == 0) load_aux(it); }", 1),
    ("if (a.nk < D) wait_barrier<0>();", 1),
    ("load(x, st, s_ld);", 1)])
def test_statements_are_the_models(text, times):
    assert SRC.count(text) == times


def test_configurations():
    assert len(CFGS) == 6
    for cfg in CFGS:
        m = Model(cfg)
        aux = 256 * (m.BM // 64 + 2 * (m.BN // 64))
        assert (m.D * m.stage + aux) * m.PERCU <= 160 * 1024 and m.KS == 128
