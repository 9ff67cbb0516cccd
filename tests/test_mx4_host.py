"""ob_mx4 without a GPU: the library exports what include/ob_mx4.h declares,
layouts, workspaces, and every refusal that comes before the first launch."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mx4_common as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ob_mx4.h")
LIB = os.path.join(ROOT, "communication_compressed_distributed_02_amd", "libob_adam.so")


@pytest.fixture(scope="module")
def mx():
    if not os.path.exists(LIB):
        pytest.skip("libob_adam.so not built")
    from communication_compressed_distributed_02_amd import ob_mx4
    return ob_mx4


def test_library_exports_every_declared_symbol(mx):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ob_mx4_\w+)\s*\(", src)))
    out = subprocess.check_output(["nm", "-D", "--defined-only", LIB], text=True)
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert names == sorted(mx.EXPORTED) and set(names) <= exported


def test_layout(mx):
    for rows, cols in ((0, 0), (1, 0), (3, 1), (1, 128), (2, 129), (5, 512), (5, 513), (1, 1 << 33),
                       (1 << 28, 3), (1, 1 << 35)):
        assert mx.ob_mx4_layout(rows, cols) == ref.widths(cols)
    for rows, cols in ((-1, 1), (1, -1), (1, (1 << 35) + 1), ((1 << 28) + 1, 1), (1 << 20, (1 << 15) + 1),
                       ((1 << 63) - 1, (1 << 63) - 1)):
        refused(mx, lambda: mx.ob_mx4_layout(rows, cols), "SHAPE")


def refused(mx, call, kind):
    from communication_compressed_distributed_02_amd import ob_adam
    with pytest.raises(ob_adam.ObAdamError) as e:
        call()
    assert e.value.status == getattr(ob_adam, "OB_ERR_" + kind)


def place(i):
    """An address that nothing follows, apart from the others."""
    return (i + 1) << 40


def quantize_args(mx, **kw):
    a = mx.ob_mx4_quantize_args()
    a.x, a.rows, a.cols, a.stride = place(0), 8, 100, 100
    a.codes, a.scales = place(1), place(2)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_quantize_refusals(mx):
    both = dict(codes_t=place(3), scales_t=place(4))
    for kw in (dict(dtype=2), dict(stochastic=2), dict(stride=-1), dict(stride=1 << 60), dict(codes=None),
               dict(scales=None), dict(codes=None, scales=None), dict(codes_t=place(3)),
               dict(scales_t=place(3)), dict(x=None), dict(x=place(0) + 2), dict(x=place(0) + 1, dtype=1),
               dict(codes=place(1) + 8), dict(scales=place(2) + 4), dict(both, codes_t=place(3) + 1),
               dict(both, scales_t=place(3) + 1), dict(residual=place(5) + 2),
               dict(both, residual=place(5)), dict(seed_device=place(6) + 4),
               # overlaps
               dict(codes=place(0)), dict(scales=place(0) + 16), dict(scales=place(1)),
               dict(codes=place(0) + 7 * 400 + 384), dict(residual=place(0)),
               dict(residual=place(1) - 4 * 799), dict(both, codes_t=place(1) + 8 * 64 - 16),
               dict(both, scales_t=place(2)), dict(seed_device=place(1) + 8)):
        refused(mx, lambda: mx.ob_mx4_quantize(quantize_args(mx, **kw), None), "ARG")
    for kw in (dict(rows=-1), dict(cols=-1), dict(rows=(1 << 28) + 1, cols=1), dict(cols=1 << 33),
               dict(both, rows=1, cols=(1 << 28) + 1)):
        refused(mx, lambda: mx.ob_mx4_quantize(quantize_args(mx, **kw), None), "SHAPE")
    with pytest.raises(ctypes.ArgumentError):
        mx._lib.ob_mx4_quantize(1, None)
    assert mx._lib.ob_mx4_quantize(None, None) != 0
    # nothing to do: no pointer is needed
    for kw in (dict(rows=0), dict(cols=0)):
        mx.ob_mx4_quantize(quantize_args(mx, x=None, codes=None, scales=None, **kw), None)


def test_average_refusals(mx):
    def call(codes=(place(0), place(1)), scales=(place(2), place(3)), rows=8, cols=100, dtype=0,
             out=place(4), stride=100):
        mx.ob_mx4_average(codes, scales, rows, cols, dtype, out, stride, None)

    for kw in (dict(dtype=2), dict(stride=99), dict(stride=1 << 60), dict(out=None), dict(out=place(4) + 2),
               dict(out=place(4) + 1, dtype=1), dict(codes=(place(0), None)),
               dict(scales=(place(2) + 8, place(3))), dict(codes=(place(0), place(1) + 1)),
               dict(out=place(1)), dict(out=place(3) + 8 * 16 - 4), dict(out=place(0) - 4 * 799)):
        refused(mx, lambda: call(**kw), "ARG")
    for kw in (dict(rows=-1), dict(cols=1 << 36, stride=1 << 36), dict(codes=(), scales=()),
               dict(codes=(place(0),) * 65, scales=(place(2),) * 65)):
        refused(mx, lambda: call(**kw), "SHAPE")
    call(rows=0, out=None)
    call(cols=0, out=None, stride=0)


def matmul_args(mx, **kw):
    a = mx.ob_mx4_matmul_args()
    a.m, a.n, a.k = 40, 50, 300
    a.a_codes, a.a_scales, a.b_codes, a.b_scales = (place(i) for i in range(4))
    a.out, a.out_stride = place(4), 50
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_matmul_refusals(mx):
    raw = dict(a_codes=None, a_scales=None, a=place(5), a_stride=300)
    for kw in (dict(out_dtype=2), dict(accumulate=2), dict(raw, a_dtype=2), dict(raw, a_stride=-1),
               dict(raw, a=None), dict(raw, a=place(5) + 2), dict(a=place(5)), dict(a_codes=None),
               dict(a_scales=None), dict(b_codes=None), dict(b_scales=None), dict(out=None),
               dict(out=place(4) + 2), dict(out=place(4) + 1, out_dtype=1), dict(out_stride=49),
               dict(a_codes=place(0) + 8), dict(a_scales=place(1) + 8), dict(b_codes=place(2) + 8),
               dict(b_scales=place(3) + 8), dict(out=place(0)), dict(out=place(3) + 796),
               dict(raw, out=place(5))):
        refused(mx, lambda: mx.ob_mx4_matmul(matmul_args(mx, **kw), None), "ARG")
    for kw in (dict(m=-1), dict(n=-1), dict(k=-1), dict(k=(1 << 24) + 1), dict(m=(1 << 28) + 1),
               dict(n=(1 << 28) + 1), dict(m=1 << 20, n=1 << 20, out_stride=1 << 20)):
        refused(mx, lambda: mx.ob_mx4_matmul(matmul_args(mx, **kw), None), "SHAPE")
        refused(mx, lambda: mx.ob_mx4_matmul_workspace(matmul_args(mx, **kw)), "SHAPE")
    for kw in (dict(m=0), dict(n=0, out_stride=0)):
        mx.ob_mx4_matmul(matmul_args(mx, **kw), None)
    # nothing to add
    mx.ob_mx4_matmul(matmul_args(mx, k=0, accumulate=1, a_codes=None, a_scales=None, b_codes=None,
                                 b_scales=None), None)


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("shim") / "libmx4plan.so")
    subprocess.check_call(
        ["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC",
         "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-static-libubsan",
         "-I", os.path.join(ROOT, "include"),
         "-I", os.path.join(ROOT, "communication_compressed_distributed_02_amd", "csrc"),
         os.path.join(ROOT, "tests", "c_abi", "mx4_plan_shim.cpp"), "-o", so])
    L = ctypes.CDLL(so)
    L.shim_narrow_lds.restype = ctypes.c_int64
    return L


def test_products_are_planned_within_their_limits(mx, shim):
    """Every plan covers the sum once, gives the kernels what they assume and
    takes a workspace of the parts' size."""
    r = np.random.default_rng(1)
    sizes = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 1600, 4096,
             6400, 16384, 1 << 20, 1 << 24]
    cases = [tuple(r.choice(sizes, 3)) for _ in range(3000)] + [(1 << 28, 1, 1), (1, 1 << 28, 1),
                                                               (1, 1, 1 << 24), (64, 64, 1 << 24)]
    for m, n, k in cases:
        m, n, k = int(m), int(n), int(k)
        for raw in (False, True):
            kw = dict(a_codes=None, a_scales=None, a=place(5), a_stride=k) if raw else {}
            a = matmul_args(mx, m=m, n=n, k=k, out_stride=n, **kw)
            out = (ctypes.c_int64 * 8)()
            st = shim.shim_plan(ctypes.byref(a), out)
            pad = [128 * -(-v // 128) for v in (m, n, k)]
            if max(m, n) * pad[2] > 1 << 35 or m * pad[1] > 1 << 35 or n * pad[0] > 1 << 35:
                assert st != 0
                continue
            assert st == 0
            empty, quantize, shape, splits, per, a_scales, parts, ws = out
            lds = shim.shim_narrow_lds(ctypes.c_int64(m), ctypes.c_int64(k))
            assert not empty and (shape != 0 or m <= 64)
            assert quantize == (raw and (shape != 0 or m * ref.widths(k)[0] * 2 > 24 * 1024))
            if raw and not quantize:
                assert lds <= 32 * 1024
                units = -(-k // 128)  # rows of codes, 16 bytes apart, and their scales
                assert lds >= m * (units * 64 + 16 + (units + 1) // 2 * 8)
            if quantize:
                codes, scales = ref.widths(k)
                assert a_scales % 256 == 0 and a_scales >= m * codes
                assert parts % 256 == 0 and parts >= a_scales + m * scales
            else:
                assert parts == 0
            # what a launch counts stays below 2^32 threads
            if shape == 0:
                assert -(-n // 16) * 512 < 1 << 32
            else:
                edge, threads = (256, 512) if shape == 2 else (128, 256)
                assert shape != 3 or (splits * -(-m // 128) * -(-n // 128) <= 256 and per >= 16)
                assert -(-m // edge) * -(-n // edge) * threads < 1 << 32
                assert splits == 1 or m * -(-n // 4) < 1 << 32
            if shape:
                units = -(-k // 256)
                assert splits >= 1 and per >= 1 and (splits - 1) * per < units <= splits * per
                assert splits == 1 or per % 2 == 0
                assert splits <= 65535
                assert ws == parts + (splits * m * (-(-n // 4) * 4) * 4 if splits > 1 else 0)
            else:
                assert ws == parts
    # a workspace that is missing, misaligned, short or overlapped
    big = dict(m=300, n=300, k=4096, out_stride=300, a_codes=None, a_scales=None, a=place(5),
               a_stride=4096)
    need = mx.ob_mx4_matmul_workspace(matmul_args(mx, **big))
    assert need > 300 * 2048
    for kw in (dict(workspace=None, ws_bytes=need), dict(workspace=place(6) + 16, ws_bytes=need),
               dict(workspace=place(6), ws_bytes=need - 1)):
        refused(mx, lambda: mx.ob_mx4_matmul(matmul_args(mx, **big, **kw), None), "WORKSPACE")
    for where in (place(4), place(5) - 256, place(2)):
        refused(mx, lambda: mx.ob_mx4_matmul(
            matmul_args(mx, **big, workspace=where, ws_bytes=need), None), "ARG")


def test_tensors_off_the_gpu_are_refused(mx):
    x = torch.ones(4, 64)
    for call in (lambda: mx.quantize(x), lambda: mx.quantize_both(x), lambda: mx.linear(x, x),
                 lambda: mx.matmul(x, None), lambda: mx.MX4.empty(4, 64, "cpu"),
                 lambda: mx.average(())):
        with pytest.raises(ValueError):
            call()


def test_the_definition_itself():
    """The numpy form that the GPU tests compare with, on values done by hand."""
    c = np.zeros((1, 32), dtype=np.float32)
    c[0, :8] = [6.0, -5.0, 2.5, 0.25, 0.26, 3.5, 1.75, -0.0]
    codes, scales = ref.quantize(c)
    assert scales[0, 0] == 127 and (scales[0, 1:] == 0).all()
    assert ref.values(codes, scales, 32)[0, :8].tolist() == [6, -4, 2, 0, 0.5, 4, 2, 0]
    assert codes[0, 3] >> 4 == 8  # the zero keeps its sign
    c[0, 0] = 6.9
    assert ref.quantize(c)[1][0, 0] == 127 and ref.quantized(c)[0, 0] == 6
    assert ref.quantize(c, 1)[1][0, 0] == 128
    c[0, 0] = 7.0
    assert ref.quantize(c)[1][0, 0] == 128 and ref.quantized(c)[0, 0] == 8
