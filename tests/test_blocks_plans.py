"""What the block operators' entry points launch, over random sizes, orders, strides and
workspaces (CPU only: the host code is built with launches that only record themselves,
and once more under AddressSanitizer and UndefinedBehaviorSanitizer)."""
import ctypes
import glob
import os
import random
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "precision_gemm_02_amd")

DRIVER = r"""
#include "blocks_api.hip"

using namespace pgemm::blocks;
using namespace pgemm::layers;

struct Launch {
  long long what, kernel, whole, M, N, K, splits, k_split, threads, partial, count, step;
};
enum { kNorm, kNormBack, kNormSums, kNormColumns, kQuantize, kFp8, kPair, kApartBoth, kSlope, kLayer, kPad };
static Launch log_[64];
static int count_;
static hipError_t note(Launch l) {
  if (count_ < 64) log_[count_] = l;
  ++count_;
  return hipSuccess;
}
static Launch product(int what, const ProdArgs& a, int kernel, bool whole, int count, int step) {
  const long long x = (long long)a.tiles_m * a.tiles_n * (what == kApartBoth ? count : 1);
  return {what, kernel, whole, a.M, a.N, a.K, a.splits, a.k_split,
          x * (a.splits > 1 ? a.splits : 1) * prod_threads(kernel),
          a.splits > 1 ? (long long)a.splits * a.M * a.N * 4 * count : 0, count, step};
}
static hipError_t norm(const NormArgs& a, hipStream_t) { return note({kNorm, 0, 0, a.m, a.n}); }
static hipError_t norm_back(const NormBackArgs& a, hipStream_t) {
  return note({kNormBack, 0, a.partial != nullptr, a.m, a.n, a.groups});
}
static hipError_t norm_sums(const NormBackArgs& a, hipStream_t) {
  return note({kNormSums, 0, 0, a.m, a.n, a.groups});
}
static hipError_t norm_columns(const NormColumnArgs& a, hipStream_t) {
  return note({kNormColumns, 0, 0, 0, a.n, a.groups, 0, 0, 0, (long long)a.groups * 2 * a.n * 4});
}
static int size_;   // of the call's type (the launches do not carry it)
static hipError_t pair(const PairArgs& a, int, int pair, int kernel, int loading, bool whole, hipStream_t) {
  if (whole && loading != kDirect) return hipErrorInvalidValue;
  return note(product(kPair, a.p, kernel, whole, pair == kColumns ? 2 : 1, 128 / size_));
}
static hipError_t apart(const PairArgs& a, int kernel, hipStream_t) {
  return note(product(kApartBoth, a.p, kernel, true, a.count, 128 / size_));
}
static hipError_t slope(const GateSlopeArgs& a, bool, hipStream_t) {
  return note({kSlope, 0, 0, a.rows, a.n, a.half, 0, 0, 0,
               a.partial ? (long long)a.chunks * 2 * a.n * 4 : 0, a.chunks});
}
static hipError_t layer(const ProdArgs& a, int, int, int mode, int kernel, int, hipStream_t) {
  (void)mode;
  return note(product(kLayer, a, kernel, false, 1, 128 / size_));
}
static hipError_t prod8(const Prod8Args& a, int, int kernel, int loading, hipStream_t) {
  return note(product(kFp8, a.p, kernel, loading == kWhole, 1, 128));
}
static hipError_t no_sum(const float*, void*, int, int, int, int, hipStream_t) { return hipErrorInvalidValue; }
static const TypeOps kLayers = {&layer, nullptr, &no_sum, nullptr, nullptr, nullptr, nullptr};
static const NormOps kNorms = {&norm, &norm_back, &norm_sums, &norm_columns};
static hipError_t pad(const PadRowsArgs& a, int count, hipStream_t) {
  Launch l{kPad};
  for (int i = 0; i < count; ++i) {
    if (a.of[i].ldt < a.of[i].cols || a.of[i].ldt % 8) return hipErrorInvalidValue;
    l.M = (long long)(uintptr_t)a.of[i].to + a.of[i].rows * a.of[i].ldt * size_;    // the copies' end
  }
  return note(l);
}
static const GateOps kGates = {&pair, &apart, &slope, &pad};
namespace pgemm {
namespace layers {
const TypeOps& ops_f32() { return kLayers; }
const TypeOps& ops_f16() { return kLayers; }
const TypeOps& ops_bf16() { return kLayers; }
}  // namespace layers
namespace blocks {
const NormOps& norm_ops(int) { return kNorms; }
hipError_t quantize_op(const QuantizeArgs& a, int, int, bool outer, hipStream_t) {
  return note({kQuantize, 0, outer, a.r, a.c, a.blocks});
}
hipError_t prod8_e4m3(const Prod8Args& a, int w, int k, int l, hipStream_t s) { return prod8(a, w, k, l, s); }
hipError_t prod8_e5m2(const Prod8Args& a, int w, int k, int l, hipStream_t s) { return prod8(a, w, k, l, s); }
hipError_t prod8_e4m3_wide(const Prod8Args& a, int w, int k, int l, hipStream_t s) {
  return prod8(a, w, k, l, s);
}
hipError_t prod8_e5m2_wide(const Prod8Args& a, int w, int k, int l, hipStream_t s) {
  return prod8(a, w, k, l, s);
}
const GateOps& gate_ops_f32() { return kGates; }
const GateOps& gate_ops_f16() { return kGates; }
const GateOps& gate_ops_bf16() { return kGates; }
}  // namespace blocks
}  // namespace pgemm

extern "C" int launches(Launch* to) {
  const int n = count_;
  for (int i = 0; i < n && i < 64; ++i) to[i] = log_[i];
  count_ = 0;
  return n;
}
extern "C" void type_size(int size) { size_ = size; }
"""

(NORM, NORM_BACK, NORM_SUMS, NORM_COLUMNS, QUANTIZE, FP8, PAIR, APART, SLOPE, LAYER, PAD) = range(11)
TOP = (1 << 31) - 4096
i, f, p, q, z = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_size_t


def struct(**fields):
    return type("S", (ctypes.Structure,), {"_fields_": list(fields.items())})


Launch = struct(**{n: q for n in ("what", "kernel", "whole", "M", "N", "K", "splits", "k_split", "threads",
                                  "partial", "count", "step")})
Rows, Weight = struct(data=p, ld=q), struct(data=p, ld=q, order=i, stride=q)
Kind, Kind8 = struct(dtype=i, out=i, act=i), struct(x=i, w=i, out=i, act=i)
Scales = struct(data=p, row=q, block=q, rows=i)
Weights, Pairs, Biases = struct(g=Weight, u=Weight), struct(g=Rows, u=Rows), struct(g=p, u=p)


def load(so):
    L = ctypes.CDLL(so)
    types = dict(
        pgemm_layer_norm=[i, i, i, Rows, p, p, f, p, p, Rows, p],
        pgemm_layer_norm_backward=[Kind, i, i, Rows, Rows, p, p, p, Rows, Rows, p, p, p, z, p],
        pgemm_quantize=[i, i, i, i, Weight, Rows, Scales, p],
        pgemm_linear_fp8=[Kind8, i, i, i, Rows, Scales, Rows, Scales, p, Rows, Rows, Rows, p, z, p],
        pgemm_gated_linear=[Kind, i, i, i, Rows, Weights, Biases, Pairs, Rows, p, z, p],
        pgemm_gated_linear_backward=[Kind, i, i, i, Rows, Pairs, Rows, Weights, Rows, Weights, Biases, p, z,
                                     p])
    sizes = dict(pgemm_layer_norm_backward_workspace=[i, i], pgemm_linear_fp8_workspace=[i, i, i],
                 pgemm_gated_linear_workspace=[i] * 4,
                 pgemm_gated_linear_backward_workspace=[Kind, i, i, i])
    for name, args in types.items():
        getattr(L, name).argtypes = args
    for name, args in sizes.items():
        getattr(L, name).argtypes, getattr(L, name).restype = args, z

    def launched():
        to = (Launch * 64)()
        return to[:L.launches(to)]
    L.launched = launched
    return L


def sound(got, bytes_):
    """No launch that the hardware does not take, no split without work, each but the last of
    whole steps, and no partial sum behind the workspace."""
    for x in got:
        assert x.partial <= bytes_, (x.what, x.partial, bytes_)
        if x.what in (FP8, PAIR, APART, LAYER):
            assert 0 <= x.kernel <= 6 and 0 < x.threads < 1 << 32, (x.what, x.kernel, x.threads)
            assert x.splits >= 1
            if x.splits > 1:
                assert x.k_split % x.step == 0
                assert (x.splits - 1) * x.k_split < x.K <= x.splits * x.k_split
        if x.what == SLOPE:
            assert x.K >= x.N and 1 <= x.count <= max(1, x.M)


def drive(L, seed, times):
    """Random calls; returns how many were taken."""
    rng = random.Random(seed)

    def size():
        return rng.randint(0, rng.choice((0, 1, 40, 300, 5000, 100000, (1 << 31) - 1)))

    def at():
        return 0 if rng.random() < 0.03 else (1 << 20) + rng.choice((0, 0, 0, 0, 4, 8, 16))

    def rows(cols, maybe=False):
        return Rows(None if maybe and rng.random() < 0.5 else at(),
                    max(1, cols) + rng.choice((0, 0, 1, 2, 8, 1 << 33)))

    def weights(k, n):
        order, pad = rng.randint(0, 1), rng.choice((0, 0, 1, 2, 8, 1 << 33))
        ld = max(1, k if order else n) + pad
        return Weights(*[Weight(at(), ld, order, 0) for _ in range(2)])

    def scales(r, c, either=True):
        by = rng.choice((1, 128)) if either else 1
        blocks = max(1, -(-c // 128))
        return Scales(at() & ~3, blocks + rng.choice((0, 3)), 1, by)

    taken = 0
    for _ in range(times):
        d = rng.randint(0, 2)
        es = 4 if d == 0 else 2
        L.type_size(es)
        kind = Kind(d, rng.choice((0, d)), 0)
        m, n, k = size(), size(), size()
        st = [L.pgemm_layer_norm(d, m, n, rows(n), at(), at(), 1e-5, at() & ~3, at() & ~3, rows(n), None)]
        sound(L.launched(), 0)
        need = L.pgemm_layer_norm_backward_workspace(m, n) if 0 <= m <= TOP and 0 <= n <= TOP else 0
        st.append(L.pgemm_layer_norm_backward(
            kind, m, n, rows(n), rows(n), at() & ~3, at() & ~3, at(), rows(n, True), rows(n, True), at() & ~3,
            at() & ~3, 1 << 20, max(0, need - (rng.random() < 0.1)), None))
        got = L.launched()
        sound(got, need)
        for x in got:
            if x.what in (NORM_SUMS, NORM_COLUMNS):
                assert x.K * 2 * x.N * 4 <= need
        t = rng.randint(0, 1)
        st.append(L.pgemm_quantize(d, t, m, n, weights(m, n).g, rows(n), scales(m, n), None))
        L.launched()
        kind.act = rng.randint(0, 4)
        out = rng.randint(0, 2)
        need = L.pgemm_linear_fp8_workspace(m, n, k)
        give = rng.choice((0, need, need // 2))
        st.append(L.pgemm_linear_fp8(Kind8(t, rng.randint(0, 1), out, kind.act), m, n, k, rows(k),
                                     scales(m, k, False), rows(k), scales(n, k), at() & ~3, rows(n, True),
                                     rows(n, True), rows(n), (1 << 20) if give else None, give, None))
        sound(L.launched(), give)
        need = L.pgemm_gated_linear_workspace(d, m, n, k)
        give = rng.choice((0, need, need // 2))
        st.append(L.pgemm_gated_linear(kind, m, n, k, rows(k), weights(k, n), Biases(at() & ~3, None),
                                       Pairs(rows(n, True), rows(n, True)), rows(n),
                                       (1 << 20) if give else None, give, None))
        sound(L.launched(), give)
        need = L.pgemm_gated_linear_backward_workspace(kind, m, n, k)
        dW = weights(k, n)
        if rng.random() < 0.3:
            dW.u = Weight(rng.choice((None, at())), max(1, k, n) + 1, rng.randint(0, 1), 0)
        st.append(L.pgemm_gated_linear_backward(
            kind, m, n, k, rows(n), Pairs(rows(n), rows(n)), rows(k), weights(k, n), rows(k, True), dW,
            Biases(at() & ~3, at() & ~3), 1 << 20, max(0, need - (rng.random() < 0.1)), None))
        got = L.launched()
        half = -(-n // (128 // es)) * (128 // es)
        sound(got, need - -(-m * 2 * half * es // 256) * 256)
        if st[-1] == 0 and got and n > 0:
            if got[0].what == PAD:            # copies behind the rest, inside the workspace
                assert m >= 64 and got.pop(0).M <= (1 << 20) + need
            assert got[0].what == SLOPE and got[0].K == half
        assert all(-15 <= s <= 0 for s in st), st
        taken += sum(s == 0 for s in st)
    return taken


def compiler():
    hipcc = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc is not available")
    return hipcc


def build(at, *flags):
    (at / "driver.hip").write_text(DRIVER)
    so = str(at / "plans.so")
    proc = subprocess.run(
        [compiler(), "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic",
         "-I" + os.path.join(PACKAGE, "blocks"), "-I" + os.path.join(ROOT, "include"), *flags,
         str(at / "driver.hip"), "-o", so], capture_output=True, text=True)
    assert proc.returncode == 0, proc.stderr[-3000:]
    return so


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return load(build(tmp_path_factory.mktemp("plans")))


def test_random_calls_launch_what_fits(lib):
    assert drive(lib, 5, 4000) > 4000


def test_random_calls_under_sanitizers(tmp_path):
    runtimes = glob.glob("/opt/rocm/lib/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    compiler()
    if not runtimes:
        pytest.skip("the address-sanitizer runtime is not available")
    so = build(tmp_path, "-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
               "-Xarch_host", "-fno-sanitize-recover=all", "-shared-libsan")
    code = ("import sys; sys.path.insert(0, %r); import test_blocks_plans as t; "
            "assert t.drive(t.load(%r), 6, 4000) > 4000; print('ok')" % (os.path.dirname(__file__), so))
    proc = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                          env={**os.environ, "LD_PRELOAD": runtimes[0],
                               "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1",
                               "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"})
    assert proc.returncode == 0 and proc.stdout.strip().endswith("ok"), (proc.stdout[-3000:],
                                                                         proc.stderr[-3000:])


def rows(ld, data=1 << 20):
    return Rows(data, ld)


def pair_of(k, n, order=1, data=1 << 20):
    return Weights(*[Weight(data, k if order else n, order, 0) for _ in range(2)])


@pytest.mark.parametrize("order", [0, 1])
def test_aligned_operands_take_the_whole_tile_kernels(lib, order):
    """Sizes of any remainder of the steps, where rows are whole chunks of 16 bytes."""
    lib.type_size(2)
    none = Pairs(Rows(None, 1), Rows(None, 1))
    for m, n, k in ((1000, 1000, 72), (70, 4096, 4104), (333, 264, 1000)):
        kind = Kind(2, 2, 4)
        assert lib.pgemm_gated_linear(kind, m, n, k, rows(k), pair_of(k, n, order), Biases(None, None), none,
                                      rows(n), None, 0, None) == 0
        got = lib.launched()
        assert len(got) == 1 and got[0].whole
        need = lib.pgemm_gated_linear_backward_workspace(kind, m, n, k)
        assert lib.pgemm_gated_linear_backward(
            kind, m, n, k, rows(n), Pairs(rows(n), rows(n)), rows(k), pair_of(k, n, order), rows(k),
            pair_of(k, n, order), Biases(1 << 20, 1 << 20), 1 << 20, need, None) == 0
        got = lib.launched()
        assert [x.what for x in got] == [SLOPE, NORM_COLUMNS, PAIR, APART] and got[2].whole
    # rows that are not whole chunks are copied first, where there are enough
    m, n, k = 555, 265, 1001
    need = lib.pgemm_gated_linear_backward_workspace(kind, m, n, k)
    assert lib.pgemm_gated_linear_backward(
        kind, m, n, k, rows(n), Pairs(rows(n), rows(n)), rows(k), pair_of(k, n, order), rows(k),
        pair_of(k, n, order), Biases(None, None), 1 << 20, need, None) == 0
    got = lib.launched()
    assert [x.what for x in got] == [PAD, SLOPE, PAIR, APART] and got[2].whole
    # rows too far apart for a tile's 32-bit offsets, and unaligned ones
    for ld in (1 << 24, 4097):
        assert lib.pgemm_gated_linear(Kind(2, 2, 0), 300, 512, 4096, rows(ld), pair_of(4096, 512),
                                      Biases(None, None), none, rows(512), None, 0, None) == 0
        assert not lib.launched()[0].whole


def test_products_of_too_many_tiles_are_refused(lib):
    """Beyond 2^32 threads there is no launch: refused before anything runs."""
    lib.type_size(2)
    none = Pairs(Rows(None, 1), Rows(None, 1))
    m, n = 1 << 30, 1 << 20
    assert lib.pgemm_gated_linear(Kind(2, 2, 0), m, n, 64, rows(64), pair_of(64, n), Biases(None, None), none,
                                  rows(n), None, 0, None) == -2
    one = Scales(1 << 20, 1, 1, 1)
    assert lib.pgemm_linear_fp8(Kind8(0, 0, 2, 0), m, n, 64, rows(64), one, rows(64), one, None,
                                Rows(None, 1), Rows(None, 1), rows(n), None, 0, None) == -2
    for k, n in ((1 << 20, 64), (1 << 24, 1 << 26)):     # dX, then dW
        need = lib.pgemm_gated_linear_backward_workspace(Kind(2, 2, 0), m, n, k)
        assert lib.pgemm_gated_linear_backward(
            Kind(2, 2, 0), m, n, k, rows(n), Pairs(rows(n), rows(n)), rows(k), pair_of(k, n), rows(k),
            pair_of(k, n), Biases(None, None), 1 << 20, need, None) == -2
    assert lib.launched() == []


def test_forward_copies_only_with_their_workspace(lib):
    """Odd rows are copied into whole chunks where the workspace has the room; with less
    they go through registers."""
    lib.type_size(2)
    none, kind = Pairs(Rows(None, 1), Rows(None, 1)), Kind(2, 2, 4)
    for m, n, k, order, copied in ((130, 129, 64, 0, True), (130, 136, 65, 0, True), (127, 129, 64, 0, False),
                                   (130, 136, 65, 1, False), (1000, 2047, 2047, 1, True)):
        need = lib.pgemm_gated_linear_workspace(2, m, n, k)
        for give, first in ((need, PAD if copied else PAIR), (need - 1, PAIR), (0, PAIR)):
            assert lib.pgemm_gated_linear(
                kind, m, n, k, rows(k), pair_of(k, n, order), Biases(None, None), none, rows(n),
                (1 << 20) if give > 0 else None, max(0, give), None) == 0
            got = lib.launched()
            assert got[0].what == first, (m, n, k, order, give)
            if first == PAD:
                assert got[0].M <= (1 << 20) + need and got[1].whole
                assert got[1].partial <= got[0].M - (1 << 20)
    # an X that no copy makes whole (its address): the weights are not copied for nothing
    need = lib.pgemm_gated_linear_workspace(2, 300, 129, 64)
    assert lib.pgemm_gated_linear(kind, 300, 129, 64, rows(64, (1 << 20) + 2), pair_of(64, 129, 0),
                                  Biases(None, None), none, rows(129), 1 << 20, need, None) == 0
    assert [x.what for x in lib.launched()] == [PAIR]
