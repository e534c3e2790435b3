"""What the layer operators' entry points launch (CPU only: the host code is built
with launches that only record themselves)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LAYERS = os.path.join(ROOT, "precision_gemm_02_amd", "layers")

pg = pytest.importorskip("precision_gemm_02_amd", reason="libpgemm.so not built")
from precision_gemm_02_amd import layer_ops as lo  # noqa: E402

FAKE = 1 << 20          # 16-byte aligned placeholder address, never dereferenced
BIG = 1 << 62           # workspace bytes
F32, F16, BF16 = 0, 1, 2
KERNELS = ("tile256", "tile128", "tile64", "few16", "few32", "few16wide", "few32wide")
DENSE, ROWS, SUMS = 0, 1, 2

DRIVER = r"""
#include "layers_api.hip"

using namespace pgemm::layers;

struct Launch {
  long long what, mode, kernel, x, y, threads;
};
static Launch log_[64];
static int count_;
static hipError_t note(Launch l) {
  if (count_ < 64) log_[count_] = l;
  ++count_;
  return hipSuccess;
}
static hipError_t prod(const ProdArgs& a, int, int, int mode, int kernel, int, hipStream_t) {
  const ProdGrid g = prod_grid(a, mode, kernel);
  return note({0, mode, kernel, g.x, g.y, prod_threads(kernel)});
}
static hipError_t slope(const SlopeArgs& a, int groups, hipStream_t) {
  return note({1, groups, a.chunks, a.n, a.rows, 0});
}
static hipError_t column_sum(const float*, void*, int n, int groups, int chunks, int, hipStream_t) {
  return note({2, groups, chunks, n, 0, 0});
}
static hipError_t combine(const CombineArgs& a, hipStream_t) { return note({3, a.m, a.n, 0, 0, 0}); }
static hipError_t combine_back(const CombineBackArgs& a, hipStream_t) {
  return note({4, a.m, a.n, 0, 0, 0});
}
static hipError_t route(const RouteArgs& a, hipStream_t) { return note({5, a.m, a.experts, 0, 0, 0}); }
static hipError_t route_back(const RouteBackArgs& a, hipStream_t) {
  return note({6, a.m, a.experts, 0, 0, 0});
}
static const TypeOps kOps = {&prod, &slope, &column_sum, &combine, &combine_back, &route, &route_back};
namespace pgemm {
namespace layers {
const TypeOps& ops_f32() { return kOps; }
const TypeOps& ops_f16() { return kOps; }
const TypeOps& ops_bf16() { return kOps; }
}  // namespace layers
}  // namespace pgemm

extern "C" int launches(Launch* to) {
  const int n = count_;
  for (int i = 0; i < n && i < 64; ++i) to[i] = log_[i];
  count_ = 0;
  return n;
}
"""


class Launch(ctypes.Structure):
    _fields_ = [(x, ctypes.c_longlong) for x in ("what", "mode", "kernel", "x", "y", "threads")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    hipcc = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc is not available")
    at = tmp_path_factory.mktemp("plans")
    (at / "driver.hip").write_text(DRIVER)
    proc = subprocess.run(
        [hipcc, "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic",
         "-I" + LAYERS, "-I" + os.path.join(ROOT, "include"), str(at / "driver.hip"), "-o",
         str(at / "plans.so")], capture_output=True, text=True)
    assert proc.returncode == 0, proc.stderr[-3000:]
    L = ctypes.CDLL(str(at / "plans.so"))
    for name in pg.LAYER_EXPORTS:
        fn, own = getattr(L, name), getattr(pg.library(), name)
        fn.argtypes, fn.restype = own.argtypes, own.restype

    def launched():
        to = (Launch * 64)()
        return to[:L.launches(to)]
    L.launched = launched
    return L


def rows(ld, data=FAKE):
    return lo._Rows(data, ld)


def weight(k, n, experts=1, data=FAKE):
    return lo._Weight(data, n, 0, k * n if experts > 1 else 0)


def expert_linear(L, dtype, R, n, k, E):
    plan = lo._Plan(E, FAKE, None, R)
    st = L.pgemm_expert_linear(lo._Kind(dtype, dtype, 0), R, n, k, plan, rows(k), weight(k, n, E),
                               None, rows(n, None), rows(n), None)
    return st, L.launched()


def expert_backward(L, dtype, R, n, k, E, act=0):
    plan = lo._Plan(E, FAKE, None, R)
    st = L.pgemm_expert_linear_backward(
        lo._Kind(dtype, dtype, act), R, n, k, plan, rows(n), rows(n), rows(k), weight(k, n, E),
        rows(k), weight(k, n, E), FAKE, FAKE, BIG, None)
    return st, L.launched()


def linear(L, dtype, m, n, k):
    st = L.pgemm_linear(lo._Kind(dtype, dtype, 0), m, n, k, rows(k), weight(k, n), None,
                        rows(n, None), rows(n, None), rows(n), None, 0, None)
    return st, L.launched()


# dtype, experts, n, k, rows: thousands of tiles over hundreds of experts
MANY = [(BF16, 384, 7168, 2048, 16384), (BF16, 384, 4096, 7168, 24576), (BF16, 512, 4096, 1024, 24576),
        (BF16, 1024, 2048, 1024, 65536), (F32, 256, 7168, 1024, 24576), (F32, 256, 4096, 1024, 65536),
        (F16, 1024, 16384, 1024, 2048), (F16, 1024, 4096, 4096, 262144)]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_many_experts_are_one_launch(lib, case):
    """A launch takes what it has workgroups for: a tile for each of an expert's
    64 to 256 rows, whatever the number of experts."""
    dtype, E, n, k, R = case
    st, got = expert_linear(lib, dtype, R, n, k, E)
    assert st == 0 and len(got) == 1 and got[0].mode == ROWS
    p = got[0]
    shape = {"tile256": 256, "tile128": 128, "tile64": 64}.get(KERNELS[p.kernel])
    if shape:
        assert p.x == (-(-R // shape) + min(E, R)) * -(-n // shape)
    else:
        wide = 64 if KERNELS[p.kernel].endswith("wide") else 16
        assert p.x == -(-n // wide) * min(E, R)
    assert p.y == 1 and p.x * p.threads < 1 << 32
    # the gradients: the same product the other way, and a sum per expert
    st, got = expert_backward(lib, dtype, R, k, n, E, act=4)
    assert st == 0 and [x.what for x in got] == [1, 2, 0, 0]
    assert [x.mode for x in got[2:]] == [ROWS, SUMS]
    assert all(x.x * x.threads < 1 << 32 for x in got[2:])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_products_of_too_many_tiles_are_refused(lib, dtype):
    """Beyond 2^32 threads there is no launch: refused before anything runs."""
    st, got = linear(lib, dtype, 1 << 30, 1 << 20, 64)
    assert st == -2 and got == []
    st, got = expert_linear(lib, dtype, 1 << 30, 1 << 20, 64, 16)
    assert st == -2 and got == []
    # dX of 2^30 rows and 2^20 columns; dZ and the bias gradient alone would fit
    st, got = expert_backward(lib, dtype, 1 << 30, 64, 1 << 20, 16)
    assert st == -2 and got == []
    st = lib.pgemm_linear_backward(
        lo._Kind(dtype, dtype, 4), 1 << 30, 64, 1 << 20, rows(64), rows(64), rows(1 << 20),
        weight(1 << 20, 64), rows(1 << 20), weight(1 << 20, 64), FAKE, FAKE, BIG, None)
    assert st == -2 and lib.launched() == []


def test_large_products_take_larger_tiles(lib):
    """Where the tiles of a small class are too many for a launch, a larger one
    takes the product: 2^36 results in 16 bits."""
    for m, n, k in ((1 << 24, 1 << 12, 8), (1 << 30, 64, 8), (1 << 20, 1 << 16, 1)):
        st, got = linear(lib, BF16, m, n, k)
        assert st == 0 and got[0].x * got[0].threads < 1 << 32


def test_few_rows_of_a_long_weight(lib):
    for n in (16, 4096, 1 << 20, 1 << 28, 1 << 29):
        st, got = linear(lib, BF16, 1, n, 8)
        assert st == 0 and got[0].x * got[0].threads < 1 << 32, n


@pytest.mark.parametrize("over", [1, 2, 4095])
def test_sizes_that_32_bits_do_not_step_past_are_refused(lib, over):
    """The kernels' indices go up to a few tiles beyond a size."""
    top = (1 << 31) - 4096
    big, kind, none = top + over, lo._Kind(BF16, BF16, 0), rows(1, None)
    w = lo._Weight(FAKE, 1 << 31, 0, 1 << 62)
    plan = lo._Plan(4, FAKE, FAKE, 8)
    for pos in (2, 3, 4):
        for size, want in ((big, -pos), (top, 0)):
            sizes = [16, 16, 16]
            sizes[pos - 2] = size
            r = rows(1 << 31)
            assert lib.pgemm_linear(kind, *sizes, r, w, None, none, none, r, None, 0, None) == want
            assert len(lib.launched()) == (want == 0)
            assert lib.pgemm_linear_backward(kind, *sizes, r, r, r, w, r, w, FAKE, FAKE, BIG,
                                             None) == want
            assert (len(lib.launched()) > 0) == (want == 0)
            if pos != 2 and want == 0:
                sizes[pos - 2] = 1 << 28       # (more columns are too many tiles for a launch)
            assert lib.pgemm_expert_linear(kind, *sizes, plan, r, w, None, none, r, None) == want
            assert len(lib.launched()) == (want == 0)
            assert lib.pgemm_expert_linear_backward(kind, *sizes, plan, r, r, r, w, r, w, FAKE, FAKE,
                                                    BIG, None) == want
            assert (len(lib.launched()) > 0) == (want == 0)
    r = rows(1 << 31)
    assert lib.pgemm_combine(BF16, 8, big, 2, 16, r, FAKE, FAKE, none, r, None) == -3
    assert lib.pgemm_combine(BF16, 8, top, 2, 16, r, FAKE, FAKE, none, r, None) == 0
    assert lib.pgemm_combine_backward(BF16, 8, big, 2, 16, r, r, FAKE, FAKE, r, FAKE, None) == -3
    assert lib.pgemm_combine_backward(BF16, 8, top, 2, 16, r, r, FAKE, FAKE, r, FAKE, None) == 0
    assert len(lib.launched()) == 2
