"""The layer and gradient-set operators' refusals and workspace sizes, without
a GPU: through the C symbols with addresses that are never followed, through
the binding with host tensors, and the host code under sanitizers."""

import ctypes
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT

from sparsified_gradient_compression_amd import dgc

OK, EINVAL, ECAP = dgc.DGC_OK, dgc.DGC_EINVAL, dgc.DGC_ECAPACITY
CSRC = os.path.join(ROOT, "sparsified_gradient_compression_amd", "csrc")
A = 1 << 20  # an aligned address

# the argument blocks of include/dgc.h, field by field
LINEAR, LINEAR_BACKWARD = "=5q" + "Qq" * 2 + "Q" + "Qq" * 3, "=6q" + "Qq" * 6 + "Q"
FFN, FFN_BACKWARD = "=5q" + "Qq" * 6, "=6q" + "Qq" * 9


def call(name, fmt, values, ws, size):
    return getattr(dgc.lib(), name)(struct.pack(fmt, *values), ws, size, None)


def linear(ws=A, size=1 << 40, **kw):
    v = dict(type=1, act=0, m=4, n=8, k=16, x=A, ldx=16, w=A, ldw=16, bias=0, residual=0, ldr=0, y=A, ldy=8, pre=0, ldpre=0)
    v.update(kw)
    return call("dgc_linear", LINEAR, v.values(), ws, size)


def linear_backward(ws=A, size=1 << 40, **kw):
    v = dict(type=1, grad_type=1, act=0, m=4, n=8, k=16, dy=A, lddy=8, x=A, ldx=16, w=A, ldw=16, pre=0, ldpre=0,
             dx=A, lddx=16, dw=A, lddw=16, dbias=0)
    v.update(kw)
    return call("dgc_linear_backward", LINEAR_BACKWARD, v.values(), ws, size)


def ffn(ws=A, size=1 << 40, **kw):
    v = dict(type=1, act=2, m=4, d=16, f=8, x=A, ldx=16, w_gate=A, ldw_gate=16, w_up=A, ldw_up=16, h=A, ldh=8,
             gate=0, ldgate=0, up=0, ldup=0)
    v.update(kw)
    return call("dgc_gated_ffn", FFN, v.values(), ws, size)


def ffn_backward(ws=A, size=1 << 40, **kw):
    v = dict(type=1, grad_type=1, act=2, m=4, d=16, f=8, dh=A, lddh=8, x=A, ldx=16, w_gate=A, ldw_gate=16, w_up=A,
             ldw_up=16, gate=A, ldgate=8, up=A, ldup=8, dx=A, lddx=16, dw_gate=A, lddw_gate=16, dw_up=A, lddw_up=16)
    v.update(kw)
    return call("dgc_gated_ffn_backward", FFN_BACKWARD, v.values(), ws, size)


COMMON = [dict(type=0), dict(type=3), dict(act=-1), dict(act=5), dict(m=-1), dict(m=1 << 41), dict(x=0), dict(x=A + 1),
          dict(ldx=15), dict(ldx=1 << 60)]


@pytest.mark.parametrize("fn,bad", [
    (linear, COMMON + [dict(w=0), dict(ldw=15), dict(y=0), dict(ldy=7), dict(bias=A + 1), dict(residual=A, ldr=7),
                       dict(pre=A, ldpre=7), dict(n=-1), dict(k=-5), dict(y=A + 1), dict(m=1 << 40, ldx=1 << 39)]),
    (linear_backward, COMMON + [dict(dy=0), dict(lddy=7), dict(w=0), dict(act=1, pre=0), dict(act=1, pre=A, ldpre=7),
                                dict(grad_type=2), dict(grad_type=0), dict(grad_type=3, dw=A + 2), dict(lddx=15),
                                dict(grad_type=3, dbias=A + 2), dict(lddw=15), dict(ws=A + 8), dict(ws=None)]),
    (ffn, COMMON + [dict(w_gate=0), dict(w_up=0), dict(ldw_up=15), dict(h=0), dict(ldh=7), dict(gate=A, ldgate=7),
                    dict(up=A, ldup=7), dict(d=-1), dict(f=-1)]),
    (ffn_backward, COMMON + [dict(dh=0), dict(gate=0), dict(up=0), dict(ldgate=7), dict(dw_up=0), dict(dw_gate=0),
                             dict(grad_type=2), dict(lddx=15), dict(lddw_up=15), dict(w_gate=0), dict(ws=A + 8),
                             dict(ws=None), dict(grad_type=3, dw_gate=A + 2)])])
def test_bad_arguments_are_refused_before_any_launch(fn, bad):
    for kw in bad:
        assert fn(**kw) == EINVAL, kw


def test_null_argument_blocks_and_small_workspaces():
    L = dgc.lib()
    for name in ("dgc_linear", "dgc_linear_backward", "dgc_gated_ffn", "dgc_gated_ffn_backward"):
        assert getattr(L, name)(None, A, 1 << 40, None) == EINVAL
    assert linear_backward(size=dgc.dgc_linear_workspace_bytes(4, 8, 16, True) - 1) == ECAP
    assert ffn_backward(size=dgc.dgc_gated_ffn_workspace_bytes(4, 16, 8, True) - 1) == ECAP
    big = dict(m=64, n=64, k=8192, ldx=8192, ldw=8192, ldy=64)
    need = dgc.dgc_linear_workspace_bytes(64, 64, 8192)
    assert need > 0 and linear(size=need - 1, **big) == ECAP and linear(ws=None, **big) == EINVAL


def test_empty_calls_launch_nothing():
    """Without rows or columns there is nothing to do, and no pointer is needed."""
    assert linear(m=0, x=0, y=0) == OK and linear(n=0, w=0, y=0, ldy=0) == OK
    assert ffn(m=0, x=0, h=0) == OK
    assert linear_backward(m=0, n=0, k=0, dbias=0) == OK
    assert ffn_backward(dx=0, dw_gate=0, dw_up=0) == OK


def test_workspace_sizes():
    out = ctypes.c_size_t(7)
    L = dgc.lib()
    for fn in (L.dgc_linear_workspace_bytes, L.dgc_gated_ffn_workspace_bytes):
        assert fn(1, 1, 1, 0, None) == EINVAL
        assert fn(-1, 1, 1, 0, ctypes.byref(out)) == EINVAL
        assert fn(1 << 41, 1, 1, 0, ctypes.byref(out)) == EINVAL
        assert fn(1 << 40, 1 << 13, 1, 0, ctypes.byref(out)) == EINVAL
        for sizes in ((0, 0, 0), (1, 1, 1), (8192, 8192, 8192), (3, 8192, 65), (1, 1 << 30, 1 << 20)):
            for back in (0, 1):
                assert fn(*sizes, back, ctypes.byref(out)) == OK
                # never more than a few times what the call itself reads and writes, and a fixed part
                m, n, k = sizes
                assert out.value <= 32 * (m * n + m * k + n * k) + (1 << 28), (sizes, back)
    with pytest.raises(dgc.DGCError):
        dgc.linear_workspace(-1, 2, 3, device="cpu")


def gradset_call(fn, *args):
    return getattr(dgc.lib(), fn)(*args)


def test_gradset_refusals():
    out = ctypes.c_size_t(0)
    n, t = np.array([5, 0, 7], np.int64), np.array([1, 2, 3], np.int32)

    def size(T=3, n=n, t=t, o=ctypes.byref(out)):
        return gradset_call("dgc_gradset_bytes", T, None if n is None else n.ctypes.data,
                            None if t is None else t.ctypes.data, o)

    assert size() == OK and out.value > 0
    assert size(T=0) == EINVAL and size(n=None) == EINVAL and size(t=None) == EINVAL and size(o=None) == EINVAL
    assert size(n=np.array([5, -1, 7], np.int64)) == EINVAL
    assert size(n=np.array([5, 1 << 60, 7], np.int64)) == EINVAL
    assert size(t=np.array([1, 2, 4], np.int32)) == EINVAL
    h = ctypes.c_void_p()
    init = lambda ws, have, o=ctypes.byref(h): gradset_call(  # noqa: E731
        "dgc_gradset_init", o, 3, n.ctypes.data, t.ctypes.data, ws, have, None)
    assert init(A, out.value, None) == EINVAL and init(None, out.value) == EINVAL
    assert init(A + 8, out.value) == EINVAL and init(A, out.value - 1) == ECAP and not h.value
    for fn in ("dgc_gradset_clip", "dgc_gradset_pack"):
        assert gradset_call(fn, None, A, A, 0.5, 0, 1.0, None, None, None) == EINVAL
    assert gradset_call("dgc_gradset_norm", None, A, 0, 1.0, A, None) == EINVAL
    dgc.lib().dgc_gradset_destroy(None)


def test_binding_refuses_before_it_calls():
    """Host tensors are never handed to the library; shapes, types and strides are checked first."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    x, w = z(4, 16), z(8, 16)
    cases = [lambda: dgc.linear(x, w, out=z(4, 8)), lambda: dgc.linear(x, z(8, 15)), lambda: dgc.linear(z(16), w),
             lambda: dgc.linear(z(4, 16, dtype=torch.float32), w), lambda: dgc.linear(x, w, act="tanh", out=z(4, 8)),
             lambda: dgc.linear_backward(z(4, 8), x, w, act="silu"),
             lambda: dgc.linear_backward(z(4, 8), x, w, dw=z(8, 16, dtype=torch.float16)),
             lambda: dgc.gated_ffn(x, w, w, out=z(4, 8)), lambda: dgc.gated_ffn(x, w, w, act="swish", out=z(4, 8)),
             lambda: dgc.gated_ffn_backward(z(4, 8), x, w, w, z(4, 8), z(4, 8), dw_gate=w)]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError):
            case()
            pytest.fail(str(i))
    with pytest.raises(ValueError):
        dgc.GradSet([(4,)], [torch.float64], device="cpu")
    with pytest.raises(ValueError):
        dgc.GradSet([(4,)], [], device="cpu")


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_host_code_under_asan_ubsan(tmp_path):
    exe = tmp_path / "layers_host_check"
    sanitize = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    sources = [os.path.join(CSRC, f) for f in ("dgc_layers.hip", "dgc_gradset.hip", "layers_bf16.hip", "layers_fp16.hip")]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops"] + sanitize + ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    sources.append(os.path.join(ROOT, "tests", "layers_host_check.cpp"))
    objects = [str(tmp_path / (os.path.basename(s) + ".o")) for s in sources]
    jobs = [subprocess.Popen(["hipcc"] + flags + ["-c", s, "-o", o], stderr=subprocess.PIPE, text=True)
            for s, o in zip(sources, objects)]
    for j in jobs:
        err = j.communicate()[1]
        assert j.returncode == 0, err[-3000:]
    r = subprocess.run(["hipcc", "--offload-arch=gfx950"] + sanitize + objects + ["-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, (r.stdout[-1000:], r.stderr[-3000:])
    assert "host check: ok" in r.stdout


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    """Kernels are launched on the current device: tensors of another are not handed to it."""
    class Elsewhere:
        is_cuda = True

        @staticmethod
        def get_device():
            return 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for stream in (None, 0):
        with pytest.raises(ValueError, match="device 1, the current device is 0"):
            dgc._stream_on(Elsewhere(), stream)
