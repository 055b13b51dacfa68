"""What the feed-forward operators' C calls launch, without a GPU: a stand-in
for the HIP runtime's launch functions notes every launch (and refuses what the
runtime refuses: 2^32 threads or more along an axis, 2^16 workgroups or more
along y), so that the largest sizes that a call accepts can be looked at, and
what follows a launch that fails."""
import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "uniform_grid_fp4_amd", "libufp4.so")
F32, BF16 = 0, 1
OK, HIP = 0, -5

RUNTIME = r"""
#include <cstddef>
#include <cstdint>
struct dim3 { uint32_t x, y, z; };
static dim3 grid_, block_;
static size_t lds_;
static void *stream_;
static int last_, failing_ = -1;
static int64_t launches_, threads_;
extern "C" {
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void *st) {
  grid_ = g; block_ = b; lds_ = lds; stream_ = st;
  return 0;
}
int __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *lds, void **st) {
  *g = grid_; *b = block_; *lds = lds_; *st = stream_;
  return 0;
}
int hipFuncSetAttribute(const void *, int, int value) { return value <= 160 * 1024 ? 0 : 1; }
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipLaunchKernel(const void *, dim3 g, dim3 b, void **, size_t lds, void *) {
  const uint64_t x = (uint64_t)g.x * b.x, y = (uint64_t)g.y * b.y, z = (uint64_t)g.z * b.z;
  const uint64_t most = x > y ? (x > z ? x : z) : (y > z ? y : z);
  if ((int64_t)most > threads_) threads_ = (int64_t)most;
  const bool bad = !x || !y || !z || most >> 32 || g.y >> 16 || g.z >> 16 ||
                   b.x * b.y * b.z > 1024 || lds > 160 * 1024 || launches_ == failing_;
  ++launches_;
  return bad ? last_ = 9 : 0;
}
int hipGetLastError(void) { const int e = last_; last_ = 0; return e; }
void watch(int failing) { failing_ = failing; launches_ = threads_ = last_ = 0; }
int64_t launches(void) { return launches_; }
int64_t threads(void) { return threads_; }
}
"""

# Runs in a process of its own: the stand-in is loaded first and for everyone.
DRIVER = r"""
import ctypes, json, sys
W = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
L = ctypes.CDLL(sys.argv[2])
W.launches.restype = W.threads.restype = ctypes.c_int64
I, Q, F, D, P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p
A, MUCH = P(0x10000), ctypes.c_size_t((1 << 63) - 1)          # never dereferenced
none = P(None)

class Rows(ctypes.Structure):
    _fields_ = [("q", P), ("scale", P), ("rows", Q), ("k", Q)]

class Quantized(ctypes.Structure):
    _fields_ = [("codes", P), ("scales", P), ("rows", Q), ("k", Q), ("kpad", Q), ("grid", I),
                ("rht", I), ("mask", ctypes.c_uint32), ("reserved", I)]

def call(op, a):
    t, c, k, e, dt = (a.get(n) for n in ("t", "c", "k", "e", "dt"))
    if op == "norm":
        return L.ufp4_layernorm(A, Q(c), A, Q(c), A, A, I(dt), I(dt), Q(t), Q(c), F(1e-6), A, A, A,
                                A, none)
    if op == "norm_bwd":
        return L.ufp4_layernorm_bwd(A, Q(c), A, Q(c), A, A, A, A, Q(c), I(dt), I(dt), Q(t), Q(c),
                                    A, A, A, A, MUCH, none)
    if op == "dropout":
        return L.ufp4_dropout(A, Q(c), A, Q(c), I(dt), Q(t), Q(c), D(0.1), Q(1), Q(2), none, A,
                              none)
    if op == "gated_bwd":
        return L.ufp4_gated_bwd(A, Q(c), A, Q(2 * c), I(1), I(dt), Q(t), Q(c), A, none)
    if op == "quantize":
        return L.ufp4_int8_quantize(A, Q(c), I(dt), Q(t), Q(c), A, A, none)
    off = A if e > 1 else none
    if op == "gated":
        x = Quantized(0x10000, 0x10000, t, k, (k + 15) // 16 * 16)
        w = Quantized(0x10000, 0x10000, 2 * c * e, k, (k + 15) // 16 * 16)
        return L.ufp4_gated_gemm(ctypes.byref(x), ctypes.byref(w), I(1), I(e), off, I(dt), A,
                                 Q(c), A, Q(2 * c), none)
    w = Rows(0x10000, 0x10000, e * c * (2 if a["act"] else 1), k)
    if op == "linear":
        return L.ufp4_int8_linear(A, Q(k), I(dt), Q(t), Q(k), ctypes.byref(w), none, I(a["act"]),
                                  I(e), off, I(dt), A, Q(c), A, MUCH, none)
    x = Rows(0x10000, 0x10000, t, k)
    return L.ufp4_int8_gemm(ctypes.byref(x), ctypes.byref(w), none, I(a["act"]), I(e), off, I(dt),
                            A, Q(c), none)

out = []
for op, a, failing in json.loads(sys.stdin.read()):
    W.watch(failing)
    status = call(op, a)
    out.append((status, W.launches(), W.threads()))
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """(status, launches, most threads along an axis) of each (call, sizes,
    number of the launch that fails, or -1)."""
    gxx = shutil.which("g++")
    assert gxx, "g++ builds the stand-in"
    at = tmp_path_factory.mktemp("launches")
    (at / "runtime.cpp").write_text(RUNTIME)
    (at / "driver.py").write_text(DRIVER)
    subprocess.run([gxx, "-shared", "-fPIC", "-O1", str(at / "runtime.cpp"), "-o",
                    str(at / "libruntime.so")], check=True)

    def go(calls):
        p = subprocess.run([sys.executable, str(at / "driver.py"), str(at / "libruntime.so"), LIB],
                           input=json.dumps(calls), capture_output=True, text=True, timeout=300)
        assert p.returncode == 0, p.stderr[-2000:]
        return json.loads(p.stdout)

    return go


# Each call at sizes that it accepts, up to the largest.
CALLS = [(op, dict(t=t, c=c, dt=dt)) for dt in (F32, BF16)
         for op in ("norm", "norm_bwd", "dropout", "quantize")
         for t, c in ((1, 1), (1 << 40, 16), (1 << 40, 1), (1 << 32, 2048), (1 << 31, 8192),
                      (1 << 20, 1 << 24))]
CALLS += [("gated_bwd", dict(t=t, c=c, dt=dt)) for dt in (F32, BF16)
          for t, c in ((1, 1), (1 << 40, 8), (1 << 32, 2048), (1 << 20, 1 << 23))]
CALLS += [("gated", dict(t=t, c=c, k=k, e=e, dt=dt)) for dt in (F32, BF16)
          for t, c, k, e in ((1, 1, 1, 1), (1, 1, 16, 1024), (8192, 8192, 2048, 1),
                             (1 << 36, 4096, 64, 1), (1 << 36, 100, 65536, 1024))]
CALLS += [(op, dict(t=t, c=c, k=k, e=e, dt=dt, act=act)) for dt in (F32, BF16) for act in (0, 2)
          for op in ("gemm", "linear")
          for t, c, k, e in ((1, 1, 1, 1), (1, 1, 16, 1024), (64, 1 << 23, 64, 1),
                             (128, 2048, 6144, 32), (1000, 565, 1411, 1), (8192, 8192, 2048, 1),
                             (1 << 32, 512, 64, 1), (1 << 26, 1 << 18, 128, 1),
                             (1 << 27, 131071, 131071, 1024))]


def test_every_launch_is_one_that_the_runtime_takes(run):
    for (op, sizes), (status, launches, threads) in zip(CALLS, run([(*c, -1) for c in CALLS])):
        assert status == OK and launches > 0 and threads < 1 << 32, (op, sizes, status, threads)


MANY = [("norm_bwd", dict(t=300, c=2048, dt=BF16)), ("norm_bwd", dict(t=300, c=40000, dt=F32)),
        ("norm_bwd", dict(t=0, c=64, dt=F32)), ("dropout", dict(t=1 << 22, c=8192, dt=BF16)),
        ("linear", dict(t=40, c=64, k=64, e=1, dt=BF16, act=0)),
        ("linear", dict(t=4000, c=640, k=64, e=1, dt=BF16, act=1)),
        ("gemm", dict(t=1 << 32, c=64, k=64, e=1, dt=BF16, act=0))]


@pytest.mark.parametrize("op,sizes", MANY)
def test_a_launch_that_fails_ends_the_call(run, op, sizes):
    """Whatever the call would have launched after it works on what was not
    written, or overwrites what a second try needs."""
    (status, launches, _), = run([(op, sizes, -1)])
    assert status == OK and launches > 1
    for i, (status, done, _) in enumerate(run([(op, sizes, i) for i in range(launches)])):
        assert (status, done) == (HIP, i + 1), i
