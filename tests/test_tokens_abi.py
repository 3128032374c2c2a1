"""The token operators' refusals and workspace sizes, without a GPU: through the C
symbols with addresses that are never followed, through the binding with host
tensors, and the host code under sanitizers."""

import ctypes
import os
import shutil
import struct
import subprocess

import pytest
import torch

from conftest import ROOT

from sparsified_gradient_compression_amd import dgc

OK, EINVAL, ECAP = dgc.DGC_OK, dgc.DGC_EINVAL, dgc.DGC_ECAPACITY
CSRC = os.path.join(ROOT, "sparsified_gradient_compression_amd", "csrc")
A = 1 << 20  # an aligned address
NAN, INF = float("nan"), float("inf")

# the argument blocks of include/dgc.h, field by field
NORM, NORM_BACKWARD = "=4qd" + "Qq" + "QQ" + "Qq" + "QQ", "=5q" + "Qq" * 2 + "QQQ" + "Qq" * 2 + "QQ"
DROPOUT = "=3qdQQQ" + "Qq" * 3
EMBEDDING, EMBEDDING_BACKWARD = "=5qQ" + "Qq" + "d" + "Qq", "=7q" + "Qq" + "Qd" + "Qq"
RECURRENCE, RECURRENCE_BACKWARD = "=5qQ" + "Qq" * 5, "=5qQ" + "Qq" * 9


def call(name, fmt, values, *more):
    return getattr(dgc.lib(), name)(struct.pack(fmt, *values), *more, None)


def norm(**kw):
    v = dict(type=1, weight_type=1, m=4, d=16, eps=1e-5, x=A, ldx=16, weight=A, bias=A, y=A, ldy=16, mean=A, rstd=A)
    v.update(kw)
    return call("dgc_layer_norm", NORM, v.values())


def norm_backward(ws=A, size=1 << 40, **kw):
    v = dict(type=1, weight_type=1, grad_type=1, m=4, d=16, dy=A, lddy=16, x=A, ldx=16, mean=A, rstd=A, weight=A,
             residual=A, ldr=16, dx=A, lddx=16, dweight=A, dbias=A)
    v.update(kw)
    return call("dgc_layer_norm_backward", NORM_BACKWARD, v.values(), ws, size)


def dropout(**kw):
    v = dict(type=1, m=4, d=16, p=0.5, seed=1, offset=2, step=0, x=A, ldx=16, residual=A, ldr=16, y=A, ldy=16)
    v.update(kw)
    return call("dgc_dropout", DROPOUT, v.values())


def embedding(**kw):
    v = dict(type=1, index_type=5, m=4, vocab=9, d=16, ids=A, table=A, ldt=16, scale=1.0, y=A, ldy=16)
    v.update(kw)
    return call("dgc_embedding", EMBEDDING, v.values())


def embedding_backward(ws=A, size=1 << 40, **kw):
    v = dict(type=1, grad_type=3, index_type=5, m=4, vocab=9, d=16, accumulate=0, dy=A, lddy=16, ids=A, scale=1.0,
             dtable=A, lddt=16)
    v.update(kw)
    return call("dgc_embedding_backward", EMBEDDING_BACKWARD, v.values(), ws, size)


def recurrence(ws=A, size=1 << 40, **kw):
    v = dict(type=1, index_type=4, m=6, d=16, batch=2, offsets=0, gate=A, ldg=16, x=A, ldx=16, h0=A, ldh0=16, h=A, ldh=16,
             state=A, lds=16)
    v.update(kw)
    return call("dgc_recurrence", RECURRENCE, v.values(), ws, size)


def recurrence_backward(ws=A, size=1 << 40, **kw):
    v = dict(type=1, index_type=4, m=6, d=16, batch=2, offsets=0, dh=A, lddh=16, gate=A, ldg=16, x=A, ldx=16, h=A, ldh=16,
             h0=A, ldh0=16, dstate=A, ldds=16, dgate=A, lddg=16, dx=A, lddx=16, dh0=A, lddh0=16)
    v.update(kw)
    return call("dgc_recurrence_backward", RECURRENCE_BACKWARD, v.values(), ws, size)


COMMON = [dict(type=0), dict(type=4), dict(m=-1), dict(m=1 << 31), dict(d=-1), dict(d=1 << 31), dict(ws=A + 8), dict(ws=None)]
PLAIN = [kw for kw in COMMON if "ws" not in kw]
X = [dict(x=0), dict(x=A + 1), dict(type=3, x=A + 2), dict(ldx=15), dict(ldx=1 << 60)]
WEIGHTS = [dict(weight_type=2), dict(weight_type=0), dict(weight_type=3, weight=A + 2), dict(weight=A + 1)]


@pytest.mark.parametrize("fn,bad", [
    (norm, PLAIN + X + WEIGHTS + [dict(eps=NAN), dict(eps=-1.0), dict(eps=INF), dict(y=0), dict(ldy=15), dict(bias=A + 1),
                                  dict(mean=A + 2), dict(rstd=A + 2)]),
    (norm_backward, COMMON + X + WEIGHTS + [dict(grad_type=2), dict(grad_type=0), dict(dy=0), dict(lddy=15), dict(mean=0),
                                            dict(rstd=0), dict(mean=A + 2), dict(ldr=15), dict(lddx=15),
                                            dict(grad_type=3, dweight=A + 2), dict(dbias=A + 1),
                                            dict(m=(1 << 31) - 1, d=(1 << 31) - 1, ldx=1 << 31)]),
    (dropout, PLAIN + X + [dict(p=NAN), dict(p=-0.1), dict(p=1.1), dict(step=A + 4), dict(ldr=15), dict(y=0), dict(ldy=15)]),
    (embedding, PLAIN + [dict(index_type=1), dict(vocab=-1), dict(vocab=1 << 31), dict(ids=0), dict(ids=A + 4),
                         dict(index_type=4, ids=A + 2), dict(table=0), dict(ldt=15), dict(scale=NAN), dict(scale=INF),
                         dict(y=0), dict(ldy=15)]),
    (embedding_backward, COMMON + [dict(grad_type=2), dict(index_type=0), dict(vocab=-1), dict(accumulate=2),
                                   dict(accumulate=-1), dict(dy=0), dict(lddy=15), dict(ids=A + 4), dict(scale=NAN),
                                   dict(dtable=0), dict(dtable=A + 2), dict(lddt=15)]),
    (recurrence, COMMON + X + [dict(batch=-1), dict(batch=1 << 31), dict(batch=4), dict(batch=0), dict(gate=0), dict(ldg=15),
                               dict(offsets=A, index_type=3), dict(offsets=A + 2), dict(offsets=A + 4, index_type=5),
                               dict(h0=A + 2), dict(ldh0=15), dict(h=0), dict(ldh=15), dict(state=A + 2), dict(lds=15)]),
    (recurrence_backward, COMMON + X + [dict(batch=4), dict(dh=0), dict(lddh=15), dict(gate=0), dict(ldg=15), dict(h=0),
                                        dict(ldh=15), dict(h0=A + 2), dict(ldds=15), dict(dgate=A + 1), dict(lddg=15),
                                        dict(lddx=15), dict(dh0=A + 1), dict(lddh0=15), dict(offsets=A, index_type=0)])])
def test_bad_arguments_are_refused_before_any_launch(fn, bad):
    for kw in bad:
        assert fn(**kw) == EINVAL, kw


def test_null_argument_blocks_and_small_workspaces():
    L = dgc.lib()
    for name in ("dgc_layer_norm", "dgc_dropout", "dgc_embedding"):
        assert getattr(L, name)(None, None) == EINVAL
    for name in ("dgc_layer_norm_backward", "dgc_embedding_backward", "dgc_recurrence", "dgc_recurrence_backward"):
        assert getattr(L, name)(None, A, 1 << 40, None) == EINVAL
    assert norm_backward(size=dgc.dgc_layer_norm_workspace_bytes(4, 16, True) - 1) == ECAP
    assert embedding_backward(size=dgc.dgc_embedding_workspace_bytes(4, 9, 16) - 1) == ECAP
    assert recurrence(size=dgc.dgc_recurrence_workspace_bytes(6, 16, 2) - 1) == ECAP
    assert recurrence_backward(size=dgc.dgc_recurrence_workspace_bytes(6, 16, 2, True) - 1) == ECAP


def test_empty_calls_launch_nothing():
    """Without rows or columns there is nothing to do, and no pointer is needed."""
    assert norm(m=0, x=0, y=0) == OK and norm(d=0, x=0, y=0, weight=0, bias=0, ldx=0, ldy=0) == OK
    assert norm_backward(d=0, dy=0, x=0, mean=0, rstd=0, dx=0, dweight=0, dbias=0, ws=None) == OK
    assert dropout(m=0, x=0, y=0) == OK and dropout(d=0, x=0, y=0, ldx=0, ldy=0, ldr=0) == OK
    assert embedding(m=0, ids=0, y=0) == OK and embedding(d=0, table=0, y=0, ldt=0, ldy=0) == OK
    assert embedding_backward(vocab=0, dtable=0) == OK
    assert embedding_backward(m=0, dy=0, ids=0, accumulate=1, ws=None) == OK
    assert embedding_backward(d=0, dy=0, dtable=0, ws=None) == OK
    assert recurrence(m=0, batch=0, gate=0, x=0, h=0, ws=None) == OK
    assert recurrence(d=0, gate=0, x=0, h=0, ldg=0, ldx=0, ldh=0, ldh0=0, lds=0, ws=None) == OK
    assert recurrence_backward(m=0, batch=0, dh=0, gate=0, x=0, h=0, ws=None) == OK


def test_workspace_sizes():
    out = ctypes.c_size_t(7)
    L = dgc.lib()
    b = ctypes.byref(out)
    for fn, sizes in ((L.dgc_layer_norm_workspace_bytes, (5, 7)), (L.dgc_embedding_workspace_bytes, (5, 7, 9)),
                      (L.dgc_recurrence_workspace_bytes, (5, 7, 1))):
        assert fn(*sizes, 1, None) == EINVAL and fn(*sizes, 1, b) == OK and out.value > 0
        for i in range(len(sizes)):
            for bad in (-1, 1 << 31):
                assert fn(*(bad if j == i else s for j, s in enumerate(sizes)), 1, b) == EINVAL
            assert fn(*(0 if j == i else s for j, s in enumerate(sizes)), 1, b) == OK
        assert fn(*((1 << 31) - 1,) * len(sizes), 1, b) == EINVAL
    for m, d in ((1, 1), (16384, 4096), (1 << 20, 64), (3, 1 << 20)):
        # never more than a few times what the call itself reads and writes in 16 bits, and a fixed part
        assert dgc.dgc_layer_norm_workspace_bytes(m, d) == 0
        assert dgc.dgc_layer_norm_workspace_bytes(m, d, True) <= 8 * m * d + 256
        assert dgc.dgc_embedding_workspace_bytes(m, 1000, d, False) == 0
        assert dgc.dgc_embedding_workspace_bytes(m, 1000, d) <= 2 * m * d + 32 * m + 16 * d + (1 << 14)
        for back in (False, True):
            assert dgc.dgc_recurrence_workspace_bytes(m, d, 1, back) <= 2 * m * d + 4 * m + (1 << 16) + 64 * d
    with pytest.raises(dgc.DGCError):
        dgc.layer_norm_workspace(-1, 2, True, device="cpu")
    with pytest.raises(dgc.DGCError):
        dgc.embedding_workspace(1, -2, 2, device="cpu")
    with pytest.raises(dgc.DGCError):
        dgc.recurrence_workspace(1, 2, -1, device="cpu")


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def test_binding_refuses_before_it_calls():
    """Host tensors are never handed to the library; shapes, types and strides are checked first."""
    x, f, ids = z(4, 16), torch.float32, z(4, dtype=torch.int64)
    cases = [lambda: dgc.layer_norm(x), lambda: dgc.layer_norm(z(4, 16, dtype=torch.float64)), lambda: dgc.layer_norm(z(16)),
             lambda: dgc.layer_norm(x, z(16), z(16, dtype=f)), lambda: dgc.layer_norm(x, z(16, dtype=torch.float16)),
             lambda: dgc.layer_norm(x, z(15)), lambda: dgc.layer_norm(x, out=z(16, 4).t()), lambda: dgc.layer_norm(x, eps="a"),
             lambda: dgc.layer_norm_backward(x, x, z(4), z(4, dtype=f)), lambda: dgc.layer_norm_backward(x, x, None, None),
             lambda: dgc.layer_norm_backward(z(4), z(4), z(4, dtype=f), z(4, dtype=f)),
             lambda: dgc.dropout(x, 0.5, 1), lambda: dgc.dropout(x, 0.5, -1), lambda: dgc.dropout(x, 0.5, 1 << 64),
             lambda: dgc.dropout(x, 0.5, 1, 1.5), lambda: dgc.dropout(x, 0.5, 1, step=z(1, dtype=torch.int32)),
             lambda: dgc.dropout(x, 0.5, 1, step=z(2, dtype=torch.int64)), lambda: dgc.dropout(x, None, 1),
             lambda: dgc.embedding(ids, x), lambda: dgc.embedding(ids.float(), x), lambda: dgc.embedding(z(2, 2, dtype=torch.int64), x),
             lambda: dgc.embedding(ids, z(16)), lambda: dgc.embedding_backward(x, ids, z(9, 15)),
             lambda: dgc.embedding_backward(x, ids[:3], z(9, 16)), lambda: dgc.embedding_backward(x, ids, z(9, 16, dtype=torch.float16)),
             lambda: dgc.embedding_backward(x, ids, z(16)),
             lambda: dgc.recurrence(x, x), lambda: dgc.recurrence(x, z(4, 15)), lambda: dgc.recurrence(x, x, batch=2, offsets=ids),
             lambda: dgc.recurrence(x, x, offsets=ids.float()), lambda: dgc.recurrence(x, x, z(2, 16), batch=2),
             lambda: dgc.recurrence(x, x, z(2, 16, dtype=f), batch=4), lambda: dgc.recurrence(z(4), z(4)),
             lambda: dgc.recurrence_backward(x, x, x, z(4, 8)), lambda: dgc.recurrence_backward(x, x, x, x, dh0=z(1, 16)),
             lambda: dgc.recurrence_backward(x, x, x, x, offsets=z(0, dtype=torch.int32))]
    for i, case in enumerate(cases):
        with pytest.raises(ValueError):
            case()
            pytest.fail(str(i))


def calls(device, grad):
    """Each call with one of its tensors requiring a gradient if `grad`, and what it writes."""
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=device)  # noqa: E731
    f = torch.float32
    x = new(4, 16).requires_grad_(grad)
    y, dx, w, dw, db = new(4, 16), new(4, 16), new(16), new(16), new(16)
    mean, rstd, ids = new(4, dtype=f), new(4, dtype=f), new(4, dtype=torch.int64)
    state, dh0, dt = new(2, 16, dtype=f), new(2, 16, dtype=f), new(9, 16)
    return [(lambda: dgc.layer_norm(x, w, out=y, mean=mean, rstd=rstd), [y, mean, rstd]),
            (lambda: dgc.layer_norm_backward(y, x, mean, rstd, w, None, dx, dw, db), [dx, dw, db]),
            (lambda: dgc.dropout(x, 0.5, 1, out=y), [y]), (lambda: dgc.dropout_backward(x, 0.5, 1, dx=dx), [dx]),
            (lambda: dgc.embedding(ids, x, out=y), [y]), (lambda: dgc.embedding_backward(x, ids, dt), [dt]),
            (lambda: dgc.recurrence(y, x, batch=2, out=dx, state=state), [dx, state]),
            (lambda: dgc.recurrence_backward(y, y, x, y, batch=2, dgate=dx, dh0=dh0), [dx, dh0])]


def test_tensors_that_require_a_gradient_are_refused():
    for i, (call_, _) in enumerate(calls("cpu", True)):
        with pytest.raises(ValueError, match="torch.no_grad"):
            call_()
            pytest.fail(str(i))
        with torch.no_grad(), pytest.raises(ValueError, match="on the device of x"):  # only the device is wrong
            call_()


@pytest.mark.gpu
def test_outputs_know_that_they_were_written():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with torch.no_grad():
        for i, (call_, outs) in enumerate(calls("cuda", True)):
            before = [t._version for t in outs]
            call_()
            assert all(t._version > b for t, b in zip(outs, before)), i
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_values_that_only_the_library_can_refuse():
    """Nothing is launched: outputs stay as they were."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.ones(6, 16, device="cuda")
    y, dt, ids = torch.full_like(x, 7), torch.full_like(x, 7), torch.zeros(6, dtype=torch.int64, device="cuda")
    for call_ in (lambda: dgc.layer_norm(x, eps=-1.0, out=y), lambda: dgc.dropout(x, 1.5, 1, out=y),
                  lambda: dgc.dropout(x, float("nan"), 1, out=y), lambda: dgc.embedding(ids, x, float("inf"), out=y),
                  lambda: dgc.embedding_backward(x, ids, dt, float("nan")), lambda: dgc.recurrence(x, x, batch=4, out=y),
                  lambda: dgc.recurrence(x, x, batch=-1, out=y),
                  lambda: dgc.recurrence(x, x, out=y, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                  lambda: dgc.layer_norm_backward(x, x, x[0, :6].contiguous(), x[0, :6].contiguous(), dx=y, dbias=dt[0],
                                                  workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
                  lambda: dgc.embedding_backward(x, ids, dt, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dgc.DGCError):
            call_()
    torch.cuda.synchronize()
    assert bool((y == 7).all()) and bool((dt == 7).all())


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_host_code_under_asan_ubsan(tmp_path):
    exe = tmp_path / "tokens_host_check"
    sanitize = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    sources = [os.path.join(CSRC, f) for f in ("dgc_norm.hip", "dgc_dropout.hip", "dgc_embedding.hip", "dgc_recurrence.hip")]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-ffp-contract=off", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops"] + sanitize + ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    sources.append(os.path.join(ROOT, "tests", "tokens_host_check.cpp"))
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
