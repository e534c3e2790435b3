"""What the block operators launch at the ends of their ranges (CPU only, see
test_blocks_plans.py, whose recording library this uses)."""
import pytest

from test_blocks_plans import (APART, FP8, LAYER, NORM_COLUMNS, PAIR, PAD, SLOPE, TOP, Biases, Kind, Kind8,
                               Pairs, Rows, Scales, Weight, Weights, lib, pair_of, rows)  # noqa: F401


@pytest.mark.parametrize("m,n", [(1, 1), (16, 16), (17, 64), (32, 9000), (33, 64), (200, 200)])
@pytest.mark.parametrize("out", [0, 2])
def test_ends_of_splits_stay_within_32_bits(lib, m, n, out):
    """The kernels hold summed indices in 32 bits: also the end of the last split, which
    is rounded up to whole steps."""
    one = Scales(1 << 20, 1, 1, 1)
    for k in [TOP - d for d in (0, 1, 64, 127, 128, 4000, 4095, 4096, 8000, 9000)]:
        need = lib.pgemm_linear_fp8_workspace(m, n, k)
        for give in (0, need):
            assert lib.pgemm_linear_fp8(Kind8(0, 0, out, 0), m, n, k, rows(k + 16), one, rows(k + 16), one, None,
                                        Rows(None, 1), Rows(None, 1), rows(n), (1 << 20) if give else None,
                                        give, None) == 0
            got = lib.launched()
            assert len(got) == 1 and got[0].what == FP8 and got[0].partial <= give
            if got[0].splits > 1:
                assert got[0].k_split % 128 == 0
                assert (got[0].splits - 1) * got[0].k_split < k <= got[0].splits * got[0].k_split < 1 << 31
        lib.type_size(2)
        need = lib.pgemm_gated_linear_workspace(2, m, n, k)
        assert lib.pgemm_gated_linear(Kind(2, 2, 0), m, n, k, rows(k + 16), pair_of(k, n), Biases(None, None),
                                      Pairs(Rows(None, 1), Rows(None, 1)), rows(n), 1 << 20, need, None) == 0
        for x in lib.launched():
            if x.what == PAIR and x.splits > 1:
                assert (x.splits - 1) * x.k_split < k <= x.splits * x.k_split < 1 << 31
