"""What the block operators launch at the ends of their ranges (CPU only, see
test_blocks_plans.py, whose recording library this uses)."""
import pytest

from test_blocks_plans import (FP8, NORM_COLUMNS, PAIR, SLOPE, TOP, Biases, Kind, Kind8, Pairs, Rows,
                               Scales, Weight, Weights, lib, pair_of, rows)  # noqa: F401


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


@pytest.mark.parametrize("n", [1, 63, 500, 8192, 100000, 1 << 19, 1 << 20, (1 << 28) + 1])
@pytest.mark.parametrize("dtype", [0, 2])
def test_bias_gradients_add_few_rows_one_after_the_other(lib, dtype, n):
    """However wide the rows: a thread of the gated gradients adds at most 1024 (and what
    the chunks' rounding adds), as one of the norm's gradients does; a launch takes the chunks."""
    size = 4 if dtype == 0 else 2
    lib.type_size(size)
    kind = Kind(dtype, 0, 0)
    half = -(-n // (128 // size)) * (128 // size)
    tpr = 1
    while tpr < 64 and tpr * 8 < half:
        tpr *= 2
    for m in (1, 7, 1000, 40000, 1 << 20, (1 << 24) + 3, TOP):
        if 3 * m * n * size > 288e9:             # (dY and Z do not fit a card)
            continue
        need = lib.pgemm_gated_linear_backward_workspace(kind, m, n, 8)
        assert lib.pgemm_gated_linear_backward(
            kind, m, n, 8, rows(n), Pairs(rows(n), rows(n)), Rows(None, 1), pair_of(8, n), Rows(None, 1),
            Weights(Weight(None, 1, 0, 0), Weight(None, 1, 0, 0)), Biases(1 << 20, 1 << 20), 1 << 20, need,
            None) == 0
        slope, sums = lib.launched()
        assert slope.what == SLOPE and sums.what == NORM_COLUMNS
        chunks = slope.count
        assert 1 <= chunks <= 65535 and slope.partial <= need - -(-m * 2 * half * size // 256) * 256
        assert -(-(-(-m // chunks)) // (256 // tpr)) <= 1025, (m, chunks)


# layers/launch.hpp's kernels for 16 and 32 rows, and their forms of twice the width
FEW, WIDE = {16: 3, 32: 4}, {16: 5, 32: 6}


@pytest.mark.parametrize("m", [1, 16, 17, 32])
def test_kernels_of_few_rows(lib, m):
    """Which sizes take the wide kernels, split or not: the sizes of the GPU tests."""
    top, none, one = 16 if m <= 16 else 32, Pairs(Rows(None, 1), Rows(None, 1)), Scales(1 << 20, 1, 1, 1)

    def gated(n, k, order, dtype):
        lib.type_size(4 if dtype == 0 else 2)
        need = lib.pgemm_gated_linear_workspace(dtype, m, n, k)
        assert lib.pgemm_gated_linear(Kind(dtype, dtype, 4), m, n, k, rows(k), pair_of(k, n, order),
                                      Biases(None, None), none, rows(n), 1 << 20, need, None) == 0
        return lib.launched()

    def fp8(n, k, out, split):
        need = lib.pgemm_linear_fp8_workspace(m, n, k) if split else 0
        assert lib.pgemm_linear_fp8(Kind8(0, 0, out, 0), m, n, k, rows(k), one, rows(k), one, None, Rows(None, 1),
                                    Rows(None, 1), rows(n), (1 << 20) if need else None, need, None) == 0
        return lib.launched()

    for n, k in ((8161, 1001), (8200, 1032), (8191, 72)):
        for order in (0, 1):
            for dtype in (0, 1, 2):
                got = gated(n, k, order, dtype)
                assert [x.what for x in got] == [PAIR] and got[0].kernel == WIDE[top] and got[0].splits == 1
        for out in (0, 1, 2):
            got = fp8(n, k, out, True)
            assert len(got) == 1 and got[0].kernel == WIDE[top] and got[0].splits == 1
    assert gated(8160, 72, 1, 2)[0].kernel == FEW[top]
    for n in (1, 16, 40, 72, 129):
        for k in (4096, 4224, 8320, 8337, 11000, 16512, 16517, 30848, 31000):
            for out in (0, 2):
                got = fp8(n, k, out, True)
                assert got[0].kernel == FEW[top] and got[0].splits == -(-k // got[0].k_split) > 1
                got = fp8(n, k, out, False)
                assert got[0].kernel == FEW[top] and got[0].splits == 1


def test_8_bit_products_of_odd_rows_with_fp32_results(lib):
    """Through registers and with fp32 results the small tiles are the faster ones."""
    one = Scales(1 << 20, 1, 1, 1)
    for m, n, k in ((2000, 2048, 4095), (4096, 4096, 4095), (8191, 8192, 4095)):
        for ld, out, want in ((k, 0, 2), (k + 1, 0, 1), (k, 2, 1)):
            need = lib.pgemm_linear_fp8_workspace(m, n, k)
            assert lib.pgemm_linear_fp8(Kind8(0, 0, out, 0), m, n, ld if ld % 16 == 0 else k, rows(ld), one, rows(ld),
                                        one, None, Rows(None, 1), Rows(None, 1), rows(n), 1 << 20, need, None) == 0
            got = lib.launched()
            assert got[0].kernel == want and got[0].partial <= need, (m, n, k, ld, out)
