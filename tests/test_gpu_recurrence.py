"""The gated recurrence and its gradients on the GPU against their formulas in
64 bits, row by row: sequences of no row, one and many, even and ragged, rows
behind the last one, states, odd widths, strides, types, gates that hold
everything or nothing, offsets that are no row numbers, streams and graphs."""

import itertools

import pytest
import torch

import token_reference as R
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc
from test_gpu_layers import Maker

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    return torch


def ends(lengths, first=0):
    return list(itertools.accumulate([first] + list(lengths)))


def gates(mk, m, d, dtype, kind="mixed"):
    z = mk.normal(m, d, dtype, 2.0)
    if kind == "mixed":  # memories of a few to thousands of steps
        z.add_(torch.linspace(-1.0, 7.0, d, device="cuda"))
    elif kind == "hold":
        z.fill_(30.0)
    elif kind == "drop":
        z.fill_(-200.0 if dtype != FP16 else -60.0)
    return z


def halves(mk, m, d, dtype, kind):
    """gate and x side by side in one matrix."""
    both = mk.normal(m, 2 * d, dtype)
    both[:, :d] = gates(mk, m, d, dtype, kind)
    return both[:, :d], both[:, d:]


class Case:
    def __init__(self, lengths, d, dtype, ragged=True, state=True, tail=0, first=0, fused=False, pad=0, shift=0, kind="mixed",
                 itype=I32, seed=1):
        self.mk = Maker(seed, pad, shift)
        self.dtype, self.d, self.at, self.n = dtype, d, ends(lengths, first), len(lengths)
        self.m = self.at[-1] + tail
        mk, m = self.mk, self.m
        self.gate, self.x = halves(mk, m, d, dtype, kind) if fused else (gates(mk, m, d, dtype, kind), mk.normal(m, d, dtype))
        self.h0 = mk.normal(self.n, d, FP32) if state else None
        self.rows = {"offsets": torch.tensor(self.at, dtype=itype, device="cuda")} if ragged else {"batch": self.n}
        self.inside = torch.zeros(m, dtype=torch.bool, device="cuda")
        self.inside[first:self.at[-1]] = True
        self.state = state

    def forward(self, **kw):
        h = self.mk.empty(self.m, self.d, self.dtype)
        state = self.mk.empty(self.n, self.d, FP32) if self.state else None
        dgc.recurrence(self.gate, self.x, self.h0, out=h, state=state, **self.rows, **kw)
        torch.cuda.synchronize()
        return h, state

    def check_forward(self, **kw):
        h, state = self.forward(**kw)
        want, e, last, elast = R.recurrence(self.gate, self.x, self.h0, self.at)
        R.check("h", h[self.inside], want[self.inside], e[self.inside], self.dtype)
        assert bool(torch.isnan(h[~self.inside]).all())
        if state is not None:
            R.check("state", state, last, elast, FP32)
        self.mk.untouched()
        return h

    def backward_inputs(self):
        mk = self.mk
        h = R.recurrence(self.gate, self.x, self.h0, self.at)[0].to(self.dtype)
        return mk.normal(self.m, self.d, self.dtype), h, mk.normal(self.n, self.d, FP32) if self.state else None

    def check_backward(self, which=("dgate", "dx", "dh0"), **kw):
        mk, m, d = self.mk, self.m, self.d
        dh, h, dstate = self.backward_inputs()
        got = {"dgate": mk.empty(m, d, self.dtype), "dx": mk.empty(m, d, self.dtype), "dh0": mk.empty(self.n, d, FP32)}
        dgc.recurrence_backward(dh, self.gate, self.x, h, self.h0, dstate, **self.rows, **{k: got[k] for k in which}, **kw)
        torch.cuda.synchronize()
        want = R.recurrence_backward(dh, self.gate, self.x, h, self.h0, dstate, self.at)
        for name in which:
            on = slice(None) if name == "dh0" else self.inside
            R.check(name, got[name][on], want[name][0][on], want[name][1][on], FP32 if name == "dh0" else self.dtype)
            if name != "dh0":
                assert bool(torch.isnan(got[name][~self.inside]).all())
        mk.untouched()


RAGGED = [[], [0], [1], [0, 0, 3, 0], [5], [1] * 40, [7, 0, 1, 33], [16, 16, 15, 17], [63, 64, 65, 1], [127, 0, 129, 255, 257],
          [300, 1, 1, 700], [1024, 1023, 1], [2000], [3, 4500, 2], [0] * 300 + [5] * 300]
WIDTHS = [1, 7, 64, 100, 129, 520]


@pytest.mark.parametrize("lengths", RAGGED, ids=lambda v: f"{len(v)}x{max(v, default=0)}")
def test_ragged(lengths):
    for i, d in enumerate(WIDTHS):
        dtype = (BF16, FP16, FP32)[i % 3]
        say(f"ragged {len(lengths)} of up to {max(lengths, default=0)}, width {d} {dtype}")
        for tail, first, itype in ((0, 0, I32), (9, 5, I64)):
            c = Case(lengths, d, dtype, tail=tail, first=first, state=i % 2 == 0, itype=itype)
            c.check_forward()
            c.check_backward()


@pytest.mark.parametrize("batch,length,d", [(1, 0, 5), (3, 0, 5), (1, 1, 1), (32, 1, 1280), (7, 1, 129), (5, 2, 64), (64, 3, 2056),
                                            (4, 16, 1000), (2, 64, 40), (3, 100, 264), (2, 513, 72), (1, 5000, 8),
                                            (6, 700, 200), (1, 2049, 1152), (300, 17, 64), (2, 1500, 4096)])
def test_even(batch, length, d):
    for i, dtype in enumerate((BF16, FP16, FP32)):
        say(f"even {batch} x {length} x {d} {dtype}")
        c = Case([length] * batch, d, dtype, ragged=False, state=i != 1, fused=i == 0)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (13, 3), (0, 1), (64, 4)])
def test_strides_and_alignment(pad, shift):
    for lengths, d in (([3, 0, 50], 72), ([400, 300], 131)):
        for dtype in (BF16, FP16, FP32):
            c = Case(lengths, d, dtype, pad=pad, shift=shift, tail=2)
            c.check_forward()
            c.check_backward()
    Case([90] * 4, 65, FP16, ragged=False, fused=True, pad=pad, shift=shift).check_forward()


@pytest.mark.parametrize("kind", ("hold", "drop"))
def test_gates_that_hold_everything_or_nothing(kind):
    for dtype in (BF16, FP16, FP32):
        c = Case([1, 700, 0, 40], 72, dtype, kind=kind)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("which", (("dgate",), ("dx",), ("dh0",), ()))
def test_some_of_the_gradients(which):
    Case([5, 800, 0], 100, BF16).check_backward(which)
    Case([400] * 3, 100, BF16, ragged=False).check_backward(which)


@pytest.mark.parametrize("lengths,ragged", [([1] * 50, False), ([5, 0, 3000, 1], True), ([700] * 3, False)])
def test_states_in_place(lengths, ragged):
    """state may be h0, and dh0 may be dstate."""
    c = Case(lengths, 136, BF16, ragged=ragged)
    h, state = c.forward()
    s = c.h0.contiguous()
    again = torch.empty_like(h)
    dgc.recurrence(c.gate, c.x, s, out=again, state=s, **c.rows)
    assert torch.equal(s, state) and torch.equal(again[c.inside], h[c.inside])
    dh, h, dstate = c.backward_inputs()
    want = [torch.zeros_like(h), torch.zeros_like(h), torch.empty_like(s)]
    dgc.recurrence_backward(dh, c.gate, c.x, h, c.h0, dstate, **c.rows, dgate=want[0], dx=want[1], dh0=want[2])
    got = [torch.zeros_like(h), torch.zeros_like(h), dstate.contiguous()]
    dgc.recurrence_backward(dh, c.gate, c.x, h, c.h0, got[2], **c.rows, dgate=got[0], dx=got[1], dh0=got[2])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_sequence_in_steps_is_the_sequence():
    """Chunks of a sequence handed on by the states, down to single rows, as while answering."""
    d, m = 200, 70
    mk = Maker(6)
    gate, x = gates(mk, m, d, FP32), mk.normal(m, d, FP32)
    whole = dgc.recurrence(gate, x)
    state, parts = torch.zeros(1, d, device="cuda"), []
    for at, n in ((0, 40), (40, 1), (41, 1), (42, 28)):
        parts.append(dgc.recurrence(gate[at:at + n], x[at:at + n], state, state=state))
    _, e, last, elast = R.recurrence(gate, x, None, [0, m])
    assert bool(((torch.cat(parts) - whole).double().abs() <= 2 * e).all())
    R.check("state", state, last, elast, FP32)


def test_sequences_do_not_touch_each_other():
    """Infinities and NaN, in the rows or a state, stay in their sequence; earlier rows of it are as they were."""
    lengths = [50, 600, 0, 300, 40]
    c = Case(lengths, 72, BF16, tail=3)
    h, state = c.forward()
    dh, hin, dstate = c.backward_inputs()
    clean = [torch.zeros_like(h), torch.zeros_like(h), torch.empty_like(dstate)]
    dgc.recurrence_backward(dh, c.gate, c.x, hin, c.h0, dstate, **c.rows, dgate=clean[0], dx=clean[1], dh0=clean[2])
    for bad in (float("inf"), float("nan")):
        c.x[250], c.h0[3, :] = bad, bad
        c.gate[-1], c.x[-1] = bad, bad  # behind the last sequence
        h2, state2 = c.forward()
        keep = torch.ones(c.m, dtype=torch.bool, device="cuda")
        keep[250:650], keep[650:950], keep[990:] = False, False, False
        assert torch.equal(h2[keep], h[keep]) and torch.equal(state2[[0, 2, 4]], state[[0, 2, 4]])
        assert not bool(torch.isfinite(h2[250]).any()) and not bool(torch.isfinite(h2[650]).any())
        dh2 = dh.clone()
        dh2[400], dh2[-1] = bad, bad
        got = [torch.zeros_like(h), torch.zeros_like(h), torch.empty_like(dstate)]
        x, h0 = Case(lengths, 72, BF16, tail=3).x, Case(lengths, 72, BF16, tail=3).h0
        dgc.recurrence_backward(dh2, c.gate, x, hin, h0, dstate, **c.rows, dgate=got[0], dx=got[1], dh0=got[2])
        keep = torch.ones(c.m, dtype=torch.bool, device="cuda")
        keep[50:401] = False
        assert all(torch.equal(p[keep], q[keep]) for p, q in zip(got[:2], clean[:2]))
        assert torch.equal(got[2][[0, 2, 3, 4]], clean[2][[0, 2, 3, 4]])
        assert not bool(torch.isfinite(got[1][400]).any())


@pytest.mark.parametrize("itype", (I32, I64))
@pytest.mark.parametrize("offsets", ([-5, 10, 10 ** 9], [50, 20, 70], [0, 100, 40], [200, 300, 400], [-3, -2, -1]))
def test_offsets_that_are_no_row_numbers_stay_inside(offsets, itype):
    """Whatever they are, nothing outside of the matrices is touched, and rows of no sequence stay."""
    mk = Maker(7, pad=3)
    m, d = 100, 40
    gate, x, h = gates(mk, m, d, BF16), mk.normal(m, d, BF16), mk.empty(m, d, BF16)
    state, dh0, dgate, dx = mk.empty(2, d, FP32), mk.empty(2, d, FP32), mk.empty(m, d, BF16), mk.empty(m, d, BF16)
    at = torch.tensor(offsets, dtype=itype, device="cuda")
    dgc.recurrence(gate, x, out=h, state=state, offsets=at)
    dgc.recurrence_backward(x, gate, x, x, offsets=at, dgate=dgate, dx=dx, dh0=dh0)
    torch.cuda.synchronize()
    mk.untouched()
    inside = torch.zeros(m, dtype=torch.bool)
    for b in range(2):
        lo, hi = (min(max(v, 0), m) for v in offsets[b:b + 2])
        inside[lo:hi] = True
    assert bool(torch.isnan(h[~inside]).all()) and bool(torch.isnan(dx[~inside]).all())


def test_gradients_against_differences():
    lengths, d = [30, 0, 200], 24
    c = Case(lengths, d, FP32)
    dh, h, dstate = c.backward_inputs()
    got = [torch.empty_like(h), torch.empty_like(h), torch.empty_like(dstate)]
    dgc.recurrence_backward(dh, c.gate, c.x, h, c.h0, dstate, **c.rows, dgate=got[0], dx=got[1], dh0=got[2])
    point = [t.double() for t in (c.gate, c.x, c.h0)]

    def loss(gate, x, h0):
        h, _, state, _ = R.recurrence(gate, x, h0, c.at)
        return (h * dh.double()).sum() + (state * dstate.double()).sum()

    for i in range(3):
        way = torch.randn(point[i].shape, device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = list(point), list(point)
        up[i], down[i] = point[i] + step * way, point[i] - step * way
        slope = float((loss(*up) - loss(*down)) / (2 * step))
        value = float((got[i].double() * way).sum())
        # the difference is off by step^2 of third derivatives and 2^-53 |loss| / step; h and the gradients by roundings
        scale = float((got[i].double().abs() * way.abs()).sum())
        assert abs(value - slope) < 1e-4 * scale, (i, value, slope)


@pytest.mark.parametrize("lengths,ragged", [([400, 0, 3000, 7], True), ([900] * 3, False), ([1] * 40, False)])
def test_the_same_bits_every_run_streams_and_graphs(lengths, ragged):
    c = Case(lengths, 264, BF16, ragged=ragged)
    dh, hin, dstate = c.backward_inputs()
    m, d, n = c.m, c.d, c.n
    out, state = torch.zeros(m, d, dtype=BF16, device="cuda"), torch.empty(n, d, device="cuda")
    grads = [torch.zeros_like(out), torch.zeros_like(out), torch.empty_like(state)]
    space = dgc.recurrence_workspace(m, d, n), dgc.recurrence_workspace(m, d, n, backward=True)

    def call(stream=None, own=False):
        dgc.recurrence(c.gate, c.x, c.h0, out=out, state=state, stream=stream, workspace=space[0] if own else None, **c.rows)
        dgc.recurrence_backward(dh, c.gate, c.x, hin, c.h0, dstate, dgate=grads[0], dx=grads[1], dh0=grads[2],
                                stream=stream, workspace=space[1] if own else None, **c.rows)

    def values():
        torch.cuda.synchronize()
        return [t.clone() for t in [out, state] + grads]

    call()
    want = values()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        for t in [out, state] + grads:
            t.fill_(0.0)
        for w in space:
            w.fill_(255)
        torch.cuda.synchronize()
        call(stream, own=True)
        assert all(torch.equal(p, q) for p, q in zip(values(), want)), stream
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call(own=True)
    for i in range(4):
        c.x.mul_(0.5 + 0.25 * i)
        graphs[i % 2].replay()
        got = values()
        call()
        assert all(torch.equal(p, q) for p, q in zip(got, values())), i


def test_rows_far_apart():
    d, ld = 40, (1 << 31) + 8
    buf = torch.empty(2 * ld + d, dtype=BF16, device="cuda")
    x = buf.as_strided((3, d), (ld, 1))
    x.copy_(torch.randn(3, d, device="cuda"))
    near = x.contiguous()
    want = dgc.recurrence(near, near)
    assert torch.equal(dgc.recurrence(x, x), want)
    dwant, got = [torch.empty_like(near) for _ in range(2)], [torch.empty_like(near) for _ in range(2)]
    dgc.recurrence_backward(near, near, near, want, dgate=dwant[0], dx=dwant[1])
    dgc.recurrence_backward(x, x, x, want, dgate=got[0], dx=got[1])
    assert all(torch.equal(p, q) for p, q in zip(got, dwant))
