"""Token operators where their kernels go another way: recurrences that the last
cache does not hold, with rows that begin at cache lines and rows that do not;
many sequences to a workgroup's chunk; more sequences than offsets are kept
nearby; tables of more rows than tokens name, by few and by many tokens; norms of
several long rows to a workgroup."""

import pytest
import torch

import test_gpu_norm
from gpu_harness import say
from sparsified_gradient_compression_amd import dgc
from test_gpu_embedding import run_backward
from test_gpu_recurrence import Case

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dgc.lib()
    return torch


@pytest.mark.parametrize("d", (4096, 4097, 4104))
@pytest.mark.parametrize("lengths,ragged", [([9001, 0, 8000], True), ([8500, 8500], False), ([50] * 340, False)],
                         ids=("ragged", "two", "many"))
def test_recurrences_beyond_the_caches(lengths, ragged, d):
    say(f"recurrence {len(lengths)} of {max(lengths)} x {d}, ragged {ragged}")
    c = Case(lengths, d, BF16, ragged=ragged, tail=4 if ragged else 0)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("batch,length,d", [(200, 24, 136), (64, 128, 520), (500, 9, 129), (40, 136, 1001), (1000, 16, 72),
                                            (3, 8, 1001), (70, 8, 65),
                                            (30, 6, 200), (30, 7, 200)])
def test_many_sequences_of_equal_length(batch, length, d):
    for i, dtype in enumerate((BF16, FP16, FP32)):
        say(f"even {batch} x {length} x {d} {dtype}")
        c = Case([length] * batch, d, dtype, ragged=False, state=i != 1)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("lengths", ([2] * 3000 + [0] * 50, list(range(9, 90)), [12] * 300 + [4000] + [9] * 200),
                         ids=("3050", "81", "501"))
def test_many_ragged_sequences(lengths):
    for d, dtype, itype in ((136, BF16, I32), (65, FP16, I64), (1001, FP32, I32)):
        say(f"ragged {len(lengths)} x {d} {dtype}")
        c = Case(lengths, d, dtype, tail=3, first=2, itype=itype)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("lengths,ragged", [([24] * 200, False), ([130] * 40, False), ([12] * 300 + [3000, 9], True)],
                         ids=("24", "130", "ragged"))
@pytest.mark.parametrize("d", (136, 1001))
def test_states_of_many_sequences_in_place(lengths, ragged, d):
    c = Case(lengths, d, BF16, ragged=ragged)
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


@pytest.mark.parametrize("m", (1, 4096, 4097, 9000))
@pytest.mark.parametrize("vocab,d", [(150000, 40), (200001, 1), (9001, 2100), (70000, 513), (1, 64), (3, 40000)])
def test_rows_that_no_token_names(m, vocab, d):
    if m * d > 1 << 25:
        m = (1 << 25) // d
    for dtype, kind, itype, wide, pad, shift in ((BF16, "zipf", I64, True, 0, 0), (FP16, "stray", I32, False, 5, 3),
                                                 (FP32, "one", I32, True, 1, 1)):
        say(f"embedding_backward {m} {vocab} {d} {dtype} {kind}")
        run_backward(m, vocab, d, dtype, kind, itype, 2.0, wide, False, pad, shift)


@pytest.mark.parametrize("m,d", [(2100, 4099), (2100, 5120), (1100, 5121), (2100, 6144), (1100, 6145), (1100, 8193), (1100, 9001),
                                 (1100, 12288), (1100, 12289), (1100, 16384)])
def test_norms_of_many_long_rows(m, d):
    for dtype, kind, wide, residual in ((BF16, "own", True, True), (FP16, "wide", False, False), (FP32, "own", True, True)):
        say(f"layer_norm {m} {d} {dtype} {kind}")
        test_gpu_norm.run_forward(m, d, dtype, kind)
        test_gpu_norm.run_backward(m, d, dtype, kind, wide, residual)
