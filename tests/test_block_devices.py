"""What the operators around a mixing layer keep per device, and the launches they make, without a
GPU: the library's host code linked with a stand-in for the runtime (fake_devices.cpp)."""
import ctypes
import os
import re
import subprocess

import pytest

from gated_delta_rule_41_gb300 import block
from gated_delta_rule_41_gb300 import build as kbuild
from gated_delta_rule_41_gb300.block import KdaAddNormDims, KdaGatedNormDims, KdaScanDims

FAKE = 1 << 20                          # never dereferenced: nothing runs
HERE = os.path.dirname(os.path.abspath(__file__))


class Launch(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint),
                ("smem", ctypes.c_ulonglong)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    kbuild.build()
    src, out = os.path.join(HERE, "fake_devices.cpp"), str(tmp_path_factory.mktemp("fake") / "fake.so")
    with open(src) as f:
        wraps = re.findall(r"__wrap_(\w+)\(", f.read())
    objs = [os.path.join(kbuild.BUILD, f) for f in os.listdir(kbuild.BUILD) if f.endswith(".o")]
    subprocess.run([kbuild._nvcc(), *kbuild.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-o", out, src,
                    *objs, *(x for w in wraps for x in ("-Xlinker", f"--wrap={w}"))], check=True)
    lib = ctypes.CDLL(out)
    real = block._lib()
    for name in ("kda_gated_scan_fwd", "kda_gated_scan_bwd", "kda_gated_norm_fwd", "kda_gated_norm_bwd",
                 "kda_add_norm_fwd", "kda_add_norm_bwd", "kda_gated_norm_workspace_bytes",
                 "kda_add_norm_workspace_bytes", "kda_pack8", "kda_unpack8"):
        f = getattr(lib, name)
        f.argtypes, f.restype = getattr(real, name).argtypes, getattr(real, name).restype
    return lib


@pytest.fixture(autouse=True)
def _fresh(lib):
    lib.fake_reset()
    lib.fake_use(0)


def launched(lib):
    out = (Launch * 16)()
    return list(out[:lib.fake_launches(out, 16)])


def add_calls(lib, D, t, res):
    d = KdaAddNormDims(5000, D, t, res, 0, 1e-5, 1.0, D, D)
    return (lambda: lib.kda_add_norm_fwd(d, FAKE, FAKE, None, FAKE, FAKE, FAKE, None),
            lambda: lib.kda_add_norm_bwd(d, *([FAKE] * 11), 1 << 40, None))


def gated_calls(lib, D, t):
    d = KdaGatedNormDims(5000, 1, D, t, 0, 0, 1e-5, D, D)
    return (lambda: lib.kda_gated_norm_fwd(d, FAKE, FAKE, FAKE, FAKE, None, None, None, None, None),
            lambda: lib.kda_gated_norm_bwd(d, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40,
                                           None))


def scan_calls(lib, C, t):
    d = KdaScanDims(2, 500, C, t, 0, 500 * C, C, 500 * C, C)
    return (lambda: lib.kda_gated_scan_fwd(d, None, 0, FAKE, FAKE, None, FAKE, None, None, None),
            lambda: lib.kda_gated_scan_bwd(d, None, 0, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, None, None))


CALLS = ([("add", add_calls, (D, t, r)) for D in (64, 256, 300, 512, 1000, 1001, 2048, 4096, 8192, 16384)
          for t, r in ((1, 1), (0, 0), (1, 0))]
         + [("gated", gated_calls, (D, t)) for D in (128, 1001, 2048, 16384) for t in (1, 0)]
         + [("scan", scan_calls, (C, t)) for C in (64, 1000, 1001) for t in (1, 0)])


@pytest.mark.parametrize("calls,args", [c[1:] for c in CALLS], ids=[f"{n}-{a}" for n, _, a in CALLS])
def test_both_devices(lib, calls, args):
    """A kernel's shared memory is allowed on each device by itself, whichever comes first."""
    for call in calls(lib, *args):
        for dev in (0, 1, 0):
            lib.fake_reset()
            lib.fake_use(dev)
            assert call() == 0
            got = launched(lib)
            assert got and all(x.device == dev for x in got)


def test_a_failed_attribute_is_reported_and_not_kept(lib):
    """The call that meets it says so; the next one tries again."""
    # a width whose kernels no other test asks for: they have set nothing yet
    d = KdaAddNormDims(5000, 32, 0, 0, 0, 1e-5, 1.0, 32, 32)

    def call():
        return lib.kda_add_norm_bwd(d, *([FAKE] * 11), 1 << 40, None)

    lib.fake_fail_attributes(1)
    assert call() == 6 and not launched(lib)
    assert call() == 0 and max(x.smem for x in launched(lib)) > 48 * 1024


@pytest.mark.parametrize("D", [(1 << 31) - 31, (1 << 31) - 1, (1 << 31) - 32, 1])
def test_rows_of_almost_2_31(lib, D):
    """Blocks of a row are counted without an overflow of 32 bits."""
    for t in (1, 0):
        for at in (FAKE, FAKE + 4):           # at 4 bytes past a 16-byte boundary: element by element
            lib.fake_reset()
            assert lib.kda_pack8(at, t, 1, D, D, FAKE, FAKE, None) == 0
            assert lib.kda_unpack8(FAKE, FAKE, 1, D, at, t, None) == 0
            assert len(launched(lib)) == 2
            if D > 1 and D % 32:
                # as many CTAs as walk over rows of this size
                assert [x.grid[0] for x in launched(lib)] == [8 * 152] * 2


def test_a_failure_of_the_scan_is_not_the_next_calls_error(lib):
    """An attribute or a launch that fails is said by the call that meets it, and by no other."""
    d = KdaScanDims(1, 300, 24, 1, 1, 300 * 24, 24, 300 * 24, 24)       # tied: asked for by no other test
    for call in (lambda: lib.kda_gated_scan_fwd(d, None, 0, FAKE, FAKE, None, FAKE, None, None, None),
                 lambda: lib.kda_gated_scan_bwd(d, None, 0, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, None,
                                                None)):
        for fail in (lib.fake_fail_attributes, lib.fake_fail_launches):
            lib.fake_reset()
            fail(1)
            assert call() == 6 and not launched(lib)
            assert lib.kda_unpack8(FAKE, FAKE, 4, 64, FAKE, 1, None) == 0
        assert call() == 0 and len(launched(lib)) == 2
