"""The order of the launches and waits that ob_adamw's host side makes, and
the powers it forms, without a GPU: ob_adamw.hip built with g++ over a HIP
runtime that only writes down what was called."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "communication_compressed_distributed_02_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def oa():
    if not os.path.exists(os.path.join(PKG, "libob_adam.so")):
        pytest.skip("libob_adam.so not built")
    from communication_compressed_distributed_02_amd import ob_adamw
    return ob_adamw


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    if not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("no HIP headers")
    so = str(tmp_path_factory.mktemp("shim") / "libhost.so")
    subprocess.check_call(
        ["g++", "-std=c++17", "-O1", "-g", "-Wall", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
         "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-static-libubsan",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"),
         "-isystem", os.path.join(ROCM, "include"),
         os.path.join(ROOT, "tests", "c_abi", "adamw_host_shim.cpp"), "-o", so])
    L = ctypes.CDLL(so)
    L.shim_calls.restype = ctypes.c_char_p
    return L


class Handle:
    """A handle over addresses that nothing follows."""

    def __init__(self, shim, oa, sizes, with_params=False, **kw):
        self.L, cfg = shim, oa.make_config(len(sizes), **kw)
        _, _, need = oa.ob_adamw_layout(cfg, sizes)
        params = (ctypes.c_void_p * len(sizes))(*[(1 << 24) * (i + 1) for i in range(len(sizes))])
        self.h = ctypes.c_void_p(0)
        shim.shim_forget()
        st = shim.ob_adamw_init(ctypes.byref(cfg), (ctypes.c_int64 * len(sizes))(*sizes), None,
                                ctypes.c_void_p(1 << 40), ctypes.c_uint64(need),
                                params if with_params else None, None, ctypes.byref(self.h))
        assert st == 0
        self.made = shim.shim_calls().decode()

    def __enter__(self):
        return self

    def __exit__(self, *_):
        assert self.L.ob_adamw_destroy(self.h) == 0


@pytest.mark.parametrize("sizes", [[1], [5000, 0, 300], [9] * 500, [1 << 28]])
def test_init_has_read_the_parameters_when_it_returns(shim, oa, sizes):
    """The wait comes after the last kernel that reads the parameters or writes
    the workspace, so a caller may write either at once, on any stream."""
    with Handle(shim, oa, sizes, True, param_dtype=oa.OB_ADAMW_BF16, master=True) as h:
        assert "m" in h.made and "u" in h.made and h.made.endswith("w")
        assert max(h.made.rfind(c) for c in "mfut") < h.made.index("w")


def power(beta, steps):
    """beta^steps by as many products in double precision, stopping where a
    product changes nothing."""
    p = 1.0
    for _ in range(steps):
        q = p * beta
        if q == p:
            break
        p = q
    return p


def test_steps_are_set_without_walking_over_powers_that_no_longer_change(shim, oa):
    """A power of a beta above a half ends among the smallest denormals, not at
    zero.  The slowest beta here is there after some 750 000 products, a few
    milliseconds; the 2^31 - 1 that are allowed take seconds to minutes."""
    import time
    f32 = [ctypes.c_float(b).value for b in (0.0, 0.25, 0.5, 0.6, 0.9, 0.98, 0.999)]
    last = (1 << 31) - 1
    for b1, b2 in zip(f32, f32[1:] + f32[:1]):
        with Handle(shim, oa, [100], beta1=b1, beta2=b2) as h:
            got = (ctypes.c_double * 2)()
            for steps in (0, 1, 7, 7000, 800000, last):
                t = time.monotonic()
                assert shim.ob_adamw_set_steps(h.h, ctypes.c_int64(steps)) == 0
                assert time.monotonic() - t < 0.5
                shim.shim_powers(got)
                assert tuple(got) == (power(b1, steps), power(b2, steps)), (b1, b2, steps)
            assert 0.0 < power(0.9, last) < 1e-322
