"""How many kernels ufp4_int8_linear launches, without a GPU (the stand-in of
test_ffn_launches.py): few rows in one, but where each of many workgroups would
quantize them again and a workspace is there."""
import json
import subprocess
import sys

import pytest

from test_ffn_launches import DRIVER, LIB, RUNTIME
from uniform_grid_fp4_amd import ffn as F


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    at = tmp_path_factory.mktemp("linear")
    (at / "runtime.cpp").write_text(RUNTIME)
    given = "Q(c), P(a['ws']), ctypes.c_size_t(a['size']), none)"
    assert DRIVER.count("Q(c), A, MUCH, none)") == 1
    (at / "driver.py").write_text(DRIVER.replace("Q(c), A, MUCH, none)", given))
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", str(at / "runtime.cpp"), "-o",
                    str(at / "libruntime.so")], check=True)

    def go(t, k, c, act=0, ws=0x10000, size=1 << 40, e=1):
        call = ("linear", dict(t=t, k=k, c=c, act=act, ws=ws, size=size, e=e, dt=1), -1)
        p = subprocess.run([sys.executable, str(at / "driver.py"), str(at / "libruntime.so"), LIB],
                           input=json.dumps([call]), capture_output=True, text=True, timeout=300)
        assert p.returncode == 0, p.stderr[-2000:]
        (status, n, _), = json.loads(p.stdout)
        return n if status == 0 else status

    return go


@pytest.mark.parametrize("act", [0, 2])
def test_few_rows(launches, act):
    most = F.INT8_FEW_COLUMNS
    for t, k in ((1, 2048), (2, 8192), (16, 1024), (16, 3)):
        assert launches(t, k, 2048, act) == launches(t, k, most, act) == 1
        assert launches(t, k, most + 1, act) == launches(t, k, 65536, act) == 2
        # without a workspace, or with less than it takes
        need = F.ufp4_int8_linear_workspace_size(t, k, True)
        assert F.ufp4_int8_linear_workspace_size(t, k) == 0
        assert launches(t, k, 65536, act, ws=0, size=0) == launches(t, k, 65536, act, ws=0) == 1
        assert launches(t, k, 65536, act, size=need - 1) == 1
        assert launches(t, k, 65536, act, size=need) == 2


def test_the_fewest_elements(launches):
    assert F.INT8_FEW_ELEMENTS == 16 * 128
    assert launches(15, 128, 65536) == launches(1, 1920, 65536) == 1
    assert launches(1, 1921, 65536) == 2


def test_more_rows(launches):
    need = F.ufp4_int8_linear_workspace_size(17, 64)
    assert need > 0 and launches(17, 64, 2048, size=need) == 2
    assert launches(17, 64, 2048, size=need - 1) == launches(17, 64, 65536, ws=0) == -1
    assert launches(8, 64, 2048, e=2) == 2
