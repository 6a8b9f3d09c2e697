"""The CPU model of the ring kernel (test_ring_bounds.py) against the kernel's
own constants and statements, and on every shape that the GPU tests run on it."""
import re

import pytest

import test_ring_bounds as model
from ternary_weight_int8_amd import binding as B
from ternary_weight_int8_amd.build import SRC
from test_epilogue_plan import gpu_shapes

TEXT = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(SRC).read()))
CFG = TEXT[TEXT.index("namespace rg {"):TEXT.index("template <class C, int E, bool BF>")]
KERNEL = TEXT[TEXT.index("void tgemm_ring(SArgs a) {"):TEXT.index("namespace sk {")]


def constants():
    """The kernel's configuration, its expressions evaluated in order."""
    c = dict(zip(("BM", "BN", "WM", "WN", "D"), map(int, re.search(r"typedef rg::Cfg<([\d, ]+)> Ring;", TEXT).group(1).split(","))))
    assert "constexpr int LP = BK;" in TEXT
    c["LP"] = int(re.search(r"constexpr int BK = (\d+);", TEXT).group(1))
    for names in re.findall(r"static constexpr int ([^;{]*);", CFG):
        for name, value in re.findall(r"(\w+) = ((?:[^,(]|\([^)]*\))+)", names):
            value = re.sub(r"\((\w+) \? 1 : 0\)", r"(1 if \1 else 0)", value).replace("/", "//")
            if name not in c:
                c[name] = eval(value, {}, c)
    return c


def test_configuration_is_the_models():
    c = constants()
    m = {"BM": model.BM, "BN": model.BN, "WM": model.WM, "WN": model.WN, "D": model.D, "LP": model.BK, "NW": model.NW,
         "kAStage": model.A_STAGE, "kALoads": model.A_LOADS, "kUnits": model.UNITS, "kUnitQ": model.Q, "kUnitR": model.R,
         "kWdStage": model.WD_STAGE, "kWpStage": model.WP_STAGE, "PS": model.PS, "kOffWd": model.D * model.A_STAGE,
         "kBatch": model.A_LOADS + model.Q, "kWaitEnd": (model.D - 2) * (model.A_LOADS + model.Q),
         "kWaitMid": model.A_LOADS + (model.D - 2) * (model.A_LOADS + model.Q)}
    assert {k: c[k] for k in m} == m
    pl = B.epilogue_plan(4096, 1280, 3456)
    assert pl.kernel == B.KERNEL_RING and (pl.tile_rows, pl.tile_cols) == (model.BM, model.BN)
    assert pl.threads_per_workgroup == 64 * model.NW and pl.lds_bytes == c["kLds"] <= 80 * 1024


# what the model restates: a statement that changes has to be changed there too
@pytest.mark.parametrize("text", [
    "return kUnitQ + (w >= NW - kUnitR ? 1 : 0);",
    "return kUnitQ * w + (w > NW - kUnitR ? w - (NW - kUnitR) : 0);"])
def test_units_are_the_models(text):
    assert text in CFG


@pytest.mark.parametrize("text,times", [
    # addresses
    ("const int r = 16 * (C::kALoads * wave + i) + (lane >> 2);", 1),
    ("const int32_t m = m0 + r < a.R ? m0 + r : a.R - 1;", 1),
    ("offA[i] = (uint32_t)(m * a.ldq + 16 * ((lane & 3) ^ ((r >> 1) & 3)));", 1),
    ("const int d = 64 * (C::first_unit(wave) + (i < C::units_of(wave) ? i : 0)) + lane;", 1),
    ("const int32_t n = n0 + (d >> 2) < a.Cc ? n0 + (d >> 2) : a.Cc - 1;", 1),
    ("offW[i] = (uint32_t)(n * a.kb + 4 * (d & 3));", 1),
    ("dma16(lbase + st * C::kAStage + wave * (C::kALoads * 1024) + 1024 * i, offA[i], a.Q + 64 * s);", 1),
    ("const uint32_t lw = lbase + C::kOffWp + ps * C::kWpStage + 256 * C::first_unit(wave);", 1),
    ("if (i < C::units_of(wave)) dma4(lw + 256 * i, offW[i], a.Wp + 16 * s);", 1),
    ("auto last = [&](int32_t s) { return s < a.nk ? s : a.nk - 1; };", 1),
    # order of the operations, stages and waits
    ("for (int s = 0; s < D - 1; ++s) { load_w(s, last(s));", 1),
    ("wait_vm<C::kALoads + (D - 3) * C::kBatch>(); { uint32_t x0[C::kWpLoads], x1[C::kWpLoads]; decode_read(x0, 0); decode_read(x1, 1);", 1),
    ("load_w(0, last(D - 1));", 1),
    ("load_a(D - 1, i, last(D - 1)); wait_barrier<C::kWaitEnd>();", 1),
    ("int q0 = 0, w0 = 0, pl = 1 % C::PS, pd = 2 % C::PS;", 1),
    ("const int32_t sl = last(g + D);", 1),
    ("if (jj == 0) load_w(pl, sl);", 1),
    ("if (jj >= 1 && jj <= C::kALoads) load_a(q0, jj - 1, sl);", 1),
    ("wait_vm<C::kWaitMid>(); decode_read(x, pd);", 1),
    ("wait_barrier<C::kWaitEnd>();", 3),
    ("q0 = q1; w0 = w1; pl = pl + 1 == C::PS ? 0 : pl + 1; pd = pd + 1 == C::PS ? 0 : pd + 1;", 1)])
def test_statements_are_the_models(text, times):
    assert KERNEL.count(text) == times


def test_load_addresses_of_every_gpu_shape():
    shapes = {s[:3] for s in gpu_shapes() if B.epilogue_plan(*s[:3], align=s[3]).kernel == B.KERNEL_RING}
    assert (8191, 2305, 64) in shapes and (4096, 1280, 3456) in shapes
    for s in sorted(shapes):
        model.test_load_addresses_stay_in_their_buffers(*s)
