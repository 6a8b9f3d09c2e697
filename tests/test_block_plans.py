"""How the row operators split their work, as far as a host without a GPU sees it."""
import pytest

from ternary_weight_int8_amd import binding as B


@pytest.mark.parametrize("query", ["ternary_rmsnorm_backward_workspace", "ternary_epilogue_backward_workspace"])
def test_few_short_rows_need_no_workspace(query):
    bytes_of = lambda R, C: B._queried(query, R, C)  # noqa: E731
    for C in (4, 243, 256):                   # at most one vector a lane of a wave, in either type
        for R in (1, 27, 32):
            assert bytes_of(R, C) == (0 if C >= 8 else 4 * R * C), (R, C)    # bf16 rows of 4 take the looped kernels
        for R in (33, 64, 200):
            assert bytes_of(R, C) > 0, (R, C)
    assert bytes_of(32, 260) > 0 and bytes_of(1, 16384) == 0
