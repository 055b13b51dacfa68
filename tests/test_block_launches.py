"""What the block operators' C calls launch, without a GPU: a stand-in for the
HIP runtime's launch functions notes every launch (and refuses what the runtime
refuses: 2^32 threads or more along an axis), so that the largest sizes that a
call accepts can be looked at, and what follows a launch that fails."""
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
int hipLaunchKernel(const void *, dim3 g, dim3 b, void **, size_t, void *) {
  const uint64_t x = (uint64_t)g.x * b.x, y = (uint64_t)g.y * b.y, z = (uint64_t)g.z * b.z;
  const uint64_t most = x > y ? (x > z ? x : z) : (y > z ? y : z);
  if ((int64_t)most > threads_) threads_ = (int64_t)most;
  const bool bad = !x || !y || !z || most >> 32 || b.x * b.y * b.z > 1024 ||
                   launches_ == failing_;
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
L.ufp4_rmsnorm_bwd_workspace_size.restype = ctypes.c_size_t
L.ufp4_moe_route_workspace_size.restype = ctypes.c_size_t
I, Q, F, D, P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p
A, MUCH = P(0x10000), ctypes.c_size_t((1 << 63) - 1)          # never dereferenced
none = P(None)

class Grad(ctypes.Structure):
    _fields_ = [("data", P), ("out", P), ("n", Q), ("dtype", I), ("out_dtype", I)]

r = (ctypes.c_void_p * 8)(*[0x10000] * 8)

def call(op, a):
    t, e, k, c, dt = (a.get(n) for n in ("t", "e", "k", "c", "dt"))
    if op == "norm":
        return L.ufp4_rmsnorm(A, Q(c), A, Q(c), A, I(dt), I(dt), Q(t), Q(c), F(1e-6), A, A, A, A,
                              A, none)
    if op == "norm_bwd":
        return L.ufp4_rmsnorm_bwd(A, Q(c), A, Q(c), A, A, A, Q(c), I(dt), I(dt), Q(t), Q(c), A, A,
                                  A, MUCH, none)
    if op == "route":
        return L.ufp4_moe_route(A, Q(e), I(dt), A, Q(t), I(e), I(k), I(1), r, A, MUCH, none)
    if op == "route_bwd":
        return L.ufp4_moe_route_bwd(A, Q(e), I(dt), Q(t), I(e), I(k), I(1), r, A, A, A, none)
    if op == "dispatch":
        return L.ufp4_moe_dispatch(A, Q(c), A, I(dt), Q(t), I(k), Q(c), A, none)
    if op == "dispatch_bwd":
        return L.ufp4_moe_dispatch_bwd(A, A, I(dt), Q(t), I(k), Q(c), A, none)
    if op == "combine":
        return L.ufp4_moe_combine(A, A, A, A, Q(c), I(dt), Q(t), I(k), Q(c), A, none)
    if op == "combine_bwd":
        return L.ufp4_moe_combine_bwd(A, Q(c), A, A, A, I(dt), Q(t), I(k), Q(c), A, A, none)
    g = (Grad * t)(*[Grad(0x10000, 0x20000, c, dt, dt)] * t)
    if op == "grad_norm":
        return L.ufp4_grad_norm(g, Q(t), A, MUCH, A, none)
    return L.ufp4_grad_clip(g, Q(t), A, D(1.0), D(0.0), none)

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
CALLS = [("route", dict(t=t, e=e, k=k, dt=dt)) for dt in (F32, BF16)
         for t, e, k in ((1, 64, 6), (65, 64, 6), (65536, 256, 8), ((1 << 28) - 64, 8, 2),
                         (1 << 28, 8, 2), ((1 << 31) - 1, 1, 1), ((1 << 31) - 1, 256, 1),
                         ((1 << 31) - 1, 1024, 1), ((1 << 27) - 1, 1024, 16))]
CALLS += [("route_bwd", dict(t=t, e=e, k=1, dt=dt)) for dt in (F32, BF16)
          for t, e in ((1, 1), (40000, 24), ((1 << 31) - 1, 256), ((1 << 31) - 1, 1024))]
CALLS += [(op, dict(t=t, k=k, c=c, dt=dt)) for dt in (F32, BF16)
          for op in ("dispatch", "dispatch_bwd", "combine", "combine_bwd")
          for t, k, c in ((1, 1, 1), (16, 8, 6144), ((1 << 31) - 1, 1, 1),
                          ((1 << 27) - 1, 16, 2048), (1 << 20, 4, 1 << 24))]
CALLS += [(op, dict(t=t, c=c, dt=dt)) for dt in (F32, BF16) for op in ("norm", "norm_bwd")
          for t, c in ((1, 1), (1 << 40, 16), (1 << 40, 1), (1 << 32, 2048), (1 << 31, 8192),
                       (1 << 20, 1 << 24))]
CALLS += [(op, dict(t=t, c=c, dt=dt)) for dt in (F32, BF16) for op in ("grad_norm", "grad_clip")
          for t, c in ((1, 1), (432, 9216), (5, 1 << 44))]


def test_every_launch_is_one_that_the_runtime_takes(run):
    for (op, sizes), (status, launches, threads) in zip(CALLS, run([(*c, -1) for c in CALLS])):
        assert status == OK and launches > 0 and threads < 1 << 32, (op, sizes, status, threads)


@pytest.mark.parametrize("sizes,launches", [(dict(t=1, e=64, k=6, dt=F32), 1),
                                            (dict(t=65536, e=256, k=8, dt=BF16), 3),
                                            (dict(t=1 << 29, e=8, k=2, dt=BF16), 9)])
def test_router_ends_with_the_first_launch_that_fails(run, sizes, launches):
    """The later launches would index by what the failed one did not write."""
    got = run([("route", sizes, i) for i in (-1, *range(launches))])
    assert got[0][:2] == [OK, launches]
    for i, (status, done, _) in enumerate(got[1:]):
        assert (status, done) == (HIP, i + 1)


MANY = [("route", dict(t=70, e=16, k=2, dt=F32)),
        ("norm_bwd", dict(t=300, c=2048, dt=BF16)), ("norm_bwd", dict(t=300, c=40000, dt=F32)),
        ("norm_bwd", dict(t=0, c=64, dt=F32)), ("grad_norm", dict(t=300, c=1 << 20, dt=F32)),
        ("grad_clip", dict(t=300, c=1 << 20, dt=BF16))]


@pytest.mark.parametrize("op,sizes", MANY)
def test_a_launch_that_fails_ends_the_call(run, op, sizes):
    """Whatever the call would have launched after it works on what was not
    written, or overwrites what a second try needs."""
    (status, launches, _), = run([(op, sizes, -1)])
    assert status == OK and launches > 1
    for i, (status, done, _) in enumerate(run([(op, sizes, i) for i in range(launches)])):
        assert (status, done) == (HIP, i + 1), i
