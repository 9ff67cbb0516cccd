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
