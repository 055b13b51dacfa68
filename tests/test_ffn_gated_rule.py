"""Which of its two kernels the gated product launches, without a GPU: the
stand-in for the runtime's launch functions of test_ffn_launches.py tells them
apart by their dynamic LDS, which only the kernel of 128 x 64 tiles has.  The GPU
tests of that kernel's values name their sizes; here every one of them is held to
the kernel that it is there for."""
import json
import subprocess
import sys

import pytest

from test_ffn_launches import DRIVER, LIB, RUNTIME
from test_gpu_ffn_gated_tiles import DENSE, GROUPED, LONGEST, ROWS_OF_A_TILE, SEAM

MORE = 'extern "C" int64_t dynamic_lds(void) { return (int64_t)lds_; }\n'


@pytest.fixture(scope="module")
def dynamic_lds(tmp_path_factory):
    at = tmp_path_factory.mktemp("rule")
    (at / "runtime.cpp").write_text(RUNTIME + MORE)
    (at / "driver.py").write_text(
        DRIVER.replace("W.threads.restype", "W.dynamic_lds.restype = W.threads.restype")
        .replace("W.threads()))", "W.dynamic_lds()))"))
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", str(at / "runtime.cpp"), "-o",
                    str(at / "libruntime.so")], check=True)

    def go(sizes):
        calls = [("gated", dict(t=t, k=k, c=f, e=e, dt=1), -1) for t, k, f, e in sizes]
        p = subprocess.run([sys.executable, str(at / "driver.py"), str(at / "libruntime.so"), LIB],
                           input=json.dumps(calls), capture_output=True, text=True, timeout=300)
        assert p.returncode == 0, p.stderr[-2000:]
        out = json.loads(p.stdout)
        assert all(status == 0 and launches == 1 for status, launches, _ in out)
        return [lds for _, _, lds in out]

    return go


def test_sizes_of_the_large_tiles(dynamic_lds):
    sizes = [(t, k, f, 1) for t, k, f in [*DENSE, LONGEST, SEAM[1]]]
    sizes += [(sum(counts), k, f, len(counts)) for counts, k, f in GROUPED]
    for at, lds in zip(sizes, dynamic_lds(sizes)):
        assert lds > 0, at


def test_sizes_of_the_few_tiles(dynamic_lds):
    assert dynamic_lds([(*SEAM[0], 1), (ROWS_OF_A_TILE, 2048, 64, 1)]) == [0, 0]
