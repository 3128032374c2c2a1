"""ctypes binding of libdgc (include/dgc.h): the same entry points, with
torch tensors marshalled to device pointers.  No computation happens here;
every step of the compressor runs in the HIP kernels of libdgc.so, and the
binding refuses to run without that library.
"""

from __future__ import annotations

import ctypes
import os
from fractions import Fraction
from typing import List, Optional, Sequence, Tuple

import numpy as np

from . import build as _build

DGC_OK = 0
DGC_EINVAL = -1
DGC_ECAPACITY = -2
DGC_EHIP = -3
DGC_ECORRUPT = -4
DGC_OPT_SELECT_PATH = 1
DGC_OPT_KERNEL_TIMING = 2
DGC_OPT_DECODE_PATH = 3
DGC_OPT_SELECT_GRID = 4
DGC_OPT_ENCODE_PATH = 5
DGC_TIMER_FUSED = 0
DGC_TIMER_COMPRESS = 1
DGC_TIMER_ENCODE = 2
DGC_TIMER_DECODE = 3
DGC_MAX_BIN = 1024
DGC_BF16 = 1
DGC_FP16 = 2
DGC_FP32 = 3
DGC_ACT_NONE = 0
DGC_ACT_RELU = 1
DGC_ACT_SILU = 2
DGC_ACT_GELU = 3
DGC_ACT_GELU_TANH = 4
DGC_DZ_ROUNDED = 256
DGC_BACKWARD_ROUNDED = 2
DGC_NORM_L2 = 0
DGC_NORM_MAX = 1

_lib = None


class DGCError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {dgc_error_string(code)} ({code})")


def lib_path() -> str:
    """The library this binding loads: the in-tree build, always."""
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libdgc.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m sparsified_gradient_compression_amd.build`")
    L = ctypes.CDLL(path)
    P = ctypes.c_void_p
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    L.dgc_k_for_density.argtypes = [i64, i64, i64]
    L.dgc_k_for_density.restype = i64
    L.dgc_workspace_bytes.argtypes = [i32, P, P, ctypes.POINTER(ctypes.c_size_t)]
    L.dgc_workspace_bytes.restype = ctypes.c_int
    L.dgc_init_state.argtypes = [ctypes.POINTER(P), i32, P, P, ctypes.c_float,
                                 P, P, P, ctypes.c_size_t, P]
    L.dgc_init_state.restype = ctypes.c_int
    L.dgc_compress.argtypes = [P, P, P, ctypes.c_double, P, P, P, P, P]
    L.dgc_compress.restype = ctypes.c_int
    L.dgc_compress_binlocal.argtypes = [P, P, P, P, ctypes.c_double, P, P, P, P,
                                        P, P, P]
    L.dgc_compress_binlocal.restype = ctypes.c_int
    L.dgc_compress_sampled.argtypes = [P, P, P, P, ctypes.c_double, P, P, P, P,
                                       P, P, P]
    L.dgc_compress_sampled.restype = ctypes.c_int
    L.dgc_compress_hier.argtypes = [P, P, P, ctypes.c_double, P, P, P, P, P, P]
    L.dgc_compress_hier.restype = ctypes.c_int
    L.dgc_compress_shared.argtypes = [P, P, P, P, ctypes.c_double, P, P, P, P]
    L.dgc_compress_shared.restype = ctypes.c_int
    L.dgc_shared_sum.argtypes = [P, i32, P, P, P, P, P, P]
    L.dgc_shared_sum.restype = ctypes.c_int
    L.dgc_encode_counts.argtypes = [P, P, P, P, P, P, P, P, P]
    L.dgc_encode_counts.restype = ctypes.c_int
    L.dgc_stream_capacity.argtypes = [P, P]
    L.dgc_stream_capacity.restype = ctypes.c_int
    L.dgc_encode.argtypes = [P, P, P, P, P, P, P, P]
    L.dgc_encode.restype = ctypes.c_int
    L.dgc_decode_accumulate.argtypes = [P, i32, P, P, P, P, P]
    L.dgc_decode_accumulate.restype = ctypes.c_int
    L.dgc_decode_sum.argtypes = [P, i32, P, P, P, P, P]
    L.dgc_decode_sum.restype = ctypes.c_int
    L.dgc_get_status.argtypes = [P]
    L.dgc_get_status.restype = ctypes.c_int
    L.dgc_get_path_counts.argtypes = [P, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.dgc_get_path_counts.restype = ctypes.c_int
    L.dgc_get_select_info.argtypes = [P, P]
    L.dgc_get_select_info.restype = ctypes.c_int
    L.dgc_set_fused_event.argtypes = [P, P]
    L.dgc_set_fused_event.restype = ctypes.c_int
    L.dgc_set_option.argtypes = [P, i32, i64]
    L.dgc_set_option.restype = ctypes.c_int
    L.dgc_get_kernel_time.argtypes = [P, i32, ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(i64)]
    L.dgc_get_kernel_time.restype = ctypes.c_int
    L.dgc_destroy_state.argtypes = [P]
    L.dgc_destroy_state.restype = None
    size = ctypes.c_size_t
    for name in ("dgc_linear", "dgc_gated_ffn"):
        f = getattr(L, name + "_workspace_bytes")
        f.argtypes = [i64, i64, i64, i32, ctypes.POINTER(size)]
        f.restype = ctypes.c_int
        for call in (name, name + "_backward"):  # an argument block, workspace, its bytes, stream
            getattr(L, call).argtypes = [P, P, size, P]
            getattr(L, call).restype = ctypes.c_int
    L.dgc_gradset_bytes.argtypes = [i32, P, P, ctypes.POINTER(size)]
    L.dgc_gradset_bytes.restype = ctypes.c_int
    L.dgc_gradset_init.argtypes = [ctypes.POINTER(P), i32, P, P, P, size, P]
    L.dgc_gradset_init.restype = ctypes.c_int
    L.dgc_gradset_norm.argtypes = [P, P, i32, ctypes.c_double, P, P]
    L.dgc_gradset_norm.restype = ctypes.c_int
    for name in ("dgc_gradset_clip", "dgc_gradset_pack"):
        getattr(L, name).argtypes = [P, P, P, ctypes.c_double, i32, ctypes.c_double, P, P, P]
        getattr(L, name).restype = ctypes.c_int
    L.dgc_gradset_destroy.argtypes = [P]
    L.dgc_gradset_destroy.restype = None
    L.dgc_error_string.argtypes = [ctypes.c_int]
    L.dgc_error_string.restype = ctypes.c_char_p
    _lib = L
    return L


# ---------------------------------------------------------------- marshalling

def _i64(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64))


def _hp(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dp(t) -> Optional[int]:
    """Device pointer of a torch tensor (None passes NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str):
    if rc != DGC_OK:
        raise DGCError(rc, what)


# ---------------------------------------------------------------- entry points

def dgc_error_string(code: int) -> str:
    return lib().dgc_error_string(int(code)).decode()


def dgc_workspace_bytes(sizes: Sequence[int], k_max: Sequence[int]) -> int:
    s, km = _i64(sizes), _i64(k_max)
    out = ctypes.c_size_t(0)
    _check(lib().dgc_workspace_bytes(len(s), _hp(s), _hp(km), ctypes.byref(out)),
           "dgc_workspace_bytes")
    return int(out.value)


def dgc_init_state(sizes, k_max, momentum: float, u, v, workspace,
                   stream=None) -> ctypes.c_void_p:
    s, km = _i64(sizes), _i64(k_max)
    st = ctypes.c_void_p()
    _check(lib().dgc_init_state(ctypes.byref(st), len(s), _hp(s), _hp(km),
                                float(momentum), _dp(u), _dp(v), _dp(workspace),
                                workspace.numel() * workspace.element_size(),
                                _stream(stream)),
           "dgc_init_state")
    return st


def dgc_compress(st, g, k, clip: float, out_idx, out_val, out_norm=None,
                 out_scale=None, stream=None):
    kk = _i64(k)
    _check(lib().dgc_compress(st, _dp(g), _hp(kk), float(clip), _dp(out_idx),
                              _dp(out_val), _dp(out_norm), _dp(out_scale),
                              _stream(stream)),
           "dgc_compress")


def dgc_compress_binlocal(st, g, bin_len, cap, clip: float, out_idx, out_val,
                          out_count, out_total=None, out_norm=None,
                          out_scale=None, stream=None):
    bl, cc = _i64(bin_len), _i64(cap)
    _check(lib().dgc_compress_binlocal(st, _dp(g), _hp(bl), _hp(cc), float(clip),
                                       _dp(out_idx), _dp(out_val), _dp(out_count),
                                       _dp(out_total), _dp(out_norm),
                                       _dp(out_scale), _stream(stream)),
           "dgc_compress_binlocal")


def dgc_compress_hier(st, g, k, clip: float, out_idx, out_val, out_count,
                      out_norm=None, out_scale=None, stream=None):
    kk = _i64(k)
    _check(lib().dgc_compress_hier(st, _dp(g), _hp(kk), float(clip), _dp(out_idx),
                                   _dp(out_val), _dp(out_count), _dp(out_norm),
                                   _dp(out_scale), _stream(stream)),
           "dgc_compress_hier")


def dgc_compress_sampled(st, g, k, cap, clip: float, out_idx, out_val, out_count,
                         out_total=None, out_norm=None, out_scale=None, stream=None):
    kk, cc = _i64(k), _i64(cap)
    _check(lib().dgc_compress_sampled(st, _dp(g), _hp(kk), _hp(cc), float(clip),
                                      _dp(out_idx), _dp(out_val), _dp(out_count),
                                      _dp(out_total), _dp(out_norm), _dp(out_scale),
                                      _stream(stream)),
           "dgc_compress_sampled")


def dgc_compress_shared(st, g, k, shared_idx, clip: float, out_val, out_norm=None,
                        out_scale=None, stream=None):
    kk = _i64(k)
    _check(lib().dgc_compress_shared(st, _dp(g), _hp(kk), _dp(shared_idx), float(clip),
                                     _dp(out_val), _dp(out_norm), _dp(out_scale),
                                     _stream(stream)),
           "dgc_compress_shared")


def dgc_shared_sum(st, vals: Sequence, k, shared_idx, out_sum, dense=None, stream=None):
    kk = _i64(k)
    W = len(vals)
    Arr = ctypes.c_void_p * max(W, 1)
    vv = Arr(*[_dp(x) for x in vals])
    _check(lib().dgc_shared_sum(st, W, ctypes.cast(vv, ctypes.c_void_p), _hp(kk),
                                _dp(shared_idx), _dp(out_sum), _dp(dense),
                                _stream(stream)),
           "dgc_shared_sum")


def dgc_stream_capacity(st, n_tensors: int) -> np.ndarray:
    out = np.zeros(n_tensors + 1, np.int64)
    _check(lib().dgc_stream_capacity(st, _hp(out)), "dgc_stream_capacity")
    return out


def dgc_encode(st, k, idx, val, runs, vals, entries, stream=None):
    kk = _i64(k)
    _check(lib().dgc_encode(st, _hp(kk), _dp(idx), _dp(val), _dp(runs), _dp(vals),
                            _dp(entries), _stream(stream)),
           "dgc_encode")


def dgc_encode_counts(st, cap, count, idx, val, runs, vals, entries, stream=None):
    cc = _i64(cap)
    _check(lib().dgc_encode_counts(st, _hp(cc), _dp(count), _dp(idx), _dp(val),
                                   _dp(runs), _dp(vals), _dp(entries),
                                   _stream(stream)),
           "dgc_encode_counts")


def _decode(fn: str, st, runs: Sequence, vals: Sequence, entries: Sequence, dense,
            stream=None):
    W = len(runs)
    assert len(vals) == W and len(entries) == W
    Arr = ctypes.c_void_p * max(W, 1)
    r = Arr(*[_dp(x) for x in runs])
    vv = Arr(*[_dp(x) for x in vals])
    e = Arr(*[_dp(x) for x in entries])
    _check(getattr(lib(), fn)(st, W, ctypes.cast(r, ctypes.c_void_p),
                              ctypes.cast(vv, ctypes.c_void_p),
                              ctypes.cast(e, ctypes.c_void_p), _dp(dense),
                              _stream(stream)), fn)


def dgc_decode_accumulate(st, runs: Sequence, vals: Sequence, entries: Sequence,
                          dense, stream=None):
    _decode("dgc_decode_accumulate", st, runs, vals, entries, dense, stream)


def dgc_decode_sum(st, runs: Sequence, vals: Sequence, entries: Sequence, dense,
                   stream=None):
    _decode("dgc_decode_sum", st, runs, vals, entries, dense, stream)


def dgc_get_status(st) -> int:
    return int(lib().dgc_get_status(st))


def dgc_get_path_counts(st) -> Tuple[int, int]:
    nw, nd = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(lib().dgc_get_path_counts(st, ctypes.byref(nw), ctypes.byref(nd)),
           "dgc_get_path_counts")
    return int(nw.value), int(nd.value)


def dgc_get_select_info(st, n_tensors: int) -> np.ndarray:
    """[n_tensors, 6] int64: path, window key, candidates, overflow, T, r."""
    out = np.zeros((n_tensors, 6), np.int64)
    _check(lib().dgc_get_select_info(st, _hp(out)), "dgc_get_select_info")
    return out


def dgc_set_fused_event(st, event):
    """event: a torch.cuda.Event (created here if needed), an int handle,
    or None to turn the hook off."""
    handle = None
    if event is not None:
        if isinstance(event, int):
            handle = event
        else:
            if not event.cuda_event:
                event.record()  # torch creates the HIP event lazily
            handle = event.cuda_event
    _check(lib().dgc_set_fused_event(st, handle), "dgc_set_fused_event")


def dgc_set_option(st, option: int, value: int):
    _check(lib().dgc_set_option(st, int(option), int(value)), "dgc_set_option")


def dgc_get_kernel_time(st, timer: int) -> Tuple[float, int]:
    ms, cnt = ctypes.c_double(0.0), ctypes.c_int64(0)
    _check(lib().dgc_get_kernel_time(st, int(timer), ctypes.byref(ms),
                                     ctypes.byref(cnt)),
           "dgc_get_kernel_time")
    return float(ms.value), int(cnt.value)


def dgc_destroy_state(st):
    lib().dgc_destroy_state(st)


def _density_fraction(density) -> Tuple[int, int]:
    """(num, den) of an exact density: a Fraction, an int, or a (num, den)
    pair.  Binary floating point is refused: 1 / 1000 is not 1/1000."""
    if isinstance(density, tuple) and len(density) == 2:
        num, den = density
        if not all(isinstance(x, (int, np.integer)) and not isinstance(x, bool)
                   for x in (num, den)):
            raise TypeError("density (num, den) must be integers")
        return int(num), int(den)
    if isinstance(density, (float, np.floating)):
        raise TypeError("density must be exact (Fraction or (num, den)), not a "
                        f"float: {density!r} is not an exact fraction in binary")
    if isinstance(density, (Fraction, int, np.integer)) and not isinstance(density, bool):
        d = Fraction(density)
        return d.numerator, d.denominator
    raise TypeError(f"density must be a Fraction, an int or (num, den), not "
                    f"{type(density).__name__}")


def dgc_k_for_density(n: int, num: int, den: int) -> int:
    k = int(lib().dgc_k_for_density(int(n), int(num), int(den)))
    if k < 0:
        raise DGCError(k, "dgc_k_for_density")
    return k


def k_for_density(n: int, density) -> int:
    """Entries a tensor of n elements sends at an exact density (warm-up
    schedule), computed by the library's dgc_k_for_density."""
    num, den = _density_fraction(density)
    return dgc_k_for_density(n, num, den)


class Learner:
    """One learner's device state for a tensor layout: u, v, workspace and
    output buffers, as torch tensors on the current device."""

    def __init__(self, sizes: Sequence[int], k_max: Sequence[int],
                 momentum: float = 0.9, device="cuda", stream=None):
        import torch
        self.sizes = [int(s) for s in sizes]
        self.k_max = [int(x) for x in k_max]
        self.T = len(self.sizes)
        self.n = int(sum(self.sizes))
        dev = torch.device(device)
        self.u = torch.empty(max(self.n, 1), dtype=torch.float32, device=dev)
        self.v = torch.empty(max(self.n, 1), dtype=torch.float32, device=dev)
        ws = dgc_workspace_bytes(self.sizes, self.k_max)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        self.state = dgc_init_state(self.sizes, self.k_max, momentum, self.u,
                                    self.v, self.workspace, stream)
        K = max(int(sum(self.k_max)), 1)
        self.idx = torch.empty(K, dtype=torch.int32, device=dev)
        self.val = torch.empty(K, dtype=torch.float32, device=dev)
        self.norm = torch.empty(1, dtype=torch.float64, device=dev)
        self.scale = torch.empty(1, dtype=torch.float32, device=dev)
        self.cap = dgc_stream_capacity(self.state, self.T)
        C = max(int(self.cap[-1]), 1)
        self.runs = torch.empty(C, dtype=torch.int16, device=dev)
        self.vals = torch.empty(C, dtype=torch.float32, device=dev)
        self.entries = torch.empty(self.T, dtype=torch.int64, device=dev)
        self.count = torch.empty(self.T, dtype=torch.int64, device=dev)
        self.total = torch.empty(self.T, dtype=torch.int64, device=dev)

    def _check_grad(self, g):
        """The kernels read n floats from g: refuse a shorter or differently
        typed gradient here, before any launch."""
        import torch
        if g.dtype != torch.float32 or g.numel() < self.n:
            raise ValueError(f"gradient must be float32 with at least {self.n} elements "
                             f"(got {g.dtype}, {g.numel()})")

    def compress(self, g, k: Sequence[int], clip: float, stream=None):
        """One step; returns (idx, val) views holding sum(k) entries."""
        self._check_grad(g)
        K = int(sum(int(x) for x in k))
        dgc_compress(self.state, g, k, clip, self.idx, self.val, self.norm,
                     self.scale, stream)
        return self.idx[:K], self.val[:K]

    def compress_binlocal(self, g, bin_len: Sequence[int], cap: Sequence[int],
                          clip: float, stream=None):
        """One step with the bin-local selector.  Returns (idx, val, count,
        total): idx/val hold sum(cap) slots, tensor t's count[t] delivered
        entries first in its cap[t] slots; total[t] = salient entries."""
        self._check_grad(g)
        C = int(sum(int(x) for x in cap))
        dgc_compress_binlocal(self.state, g, bin_len, cap, clip, self.idx,
                              self.val, self.count, self.total, self.norm,
                              self.scale, stream)
        return self.idx[:C], self.val[:C], self.count, self.total

    def compress_sampled(self, g, k: Sequence[int], cap: Sequence[int], clip: float,
                         stream=None):
        """One step with the sampled threshold (about k[t] entries per
        tensor).  Returns (idx, val, count, total) as compress_binlocal."""
        self._check_grad(g)
        C = int(sum(int(x) for x in cap))
        dgc_compress_sampled(self.state, g, k, cap, clip, self.idx, self.val,
                             self.count, self.total, self.norm, self.scale, stream)
        return self.idx[:C], self.val[:C], self.count, self.total

    def compress_hier(self, g, k: Sequence[int], clip: float, stream=None):
        """One step with hierarchical thresholding (at most k[t] entries per
        tensor).  Returns (idx, val, count): idx/val hold sum(k) slots,
        tensor t's count[t] sent entries first in its k[t] slots."""
        self._check_grad(g)
        K = int(sum(int(x) for x in k))
        dgc_compress_hier(self.state, g, k, clip, self.idx, self.val, self.count,
                          self.norm, self.scale, stream)
        return self.idx[:K], self.val[:K], self.count

    def compress_shared(self, g, k: Sequence[int], shared_idx, clip: float, stream=None):
        """One step at another learner's index set (shared_idx: that
        learner's idx, sum(k) entries).  Returns the val view (sum(k))."""
        self._check_grad(g)
        K = int(sum(int(x) for x in k))
        dgc_compress_shared(self.state, g, k, shared_idx, clip, self.val, self.norm,
                            self.scale, stream)
        return self.val[:K]

    def encode_counts(self, cap: Sequence[int], stream=None):
        """Encode what compress_binlocal delivered (counts on the device)."""
        dgc_encode_counts(self.state, cap, self.count, self.idx, self.val,
                          self.runs, self.vals, self.entries, stream)
        return self.runs, self.vals, self.entries

    def encode(self, k: Sequence[int], stream=None):
        dgc_encode(self.state, k, self.idx, self.val, self.runs, self.vals,
                   self.entries, stream)
        return self.runs, self.vals, self.entries

    def set_option(self, option: int, value: int):
        dgc_set_option(self.state, option, value)

    def set_fused_event(self, event):
        dgc_set_fused_event(self.state, event)

    def status(self) -> int:
        return dgc_get_status(self.state)

    def path_counts(self) -> Tuple[int, int]:
        return dgc_get_path_counts(self.state)

    def select_info(self) -> np.ndarray:
        return dgc_get_select_info(self.state, self.T)

    def kernel_time(self, timer: int) -> Tuple[float, int]:
        return dgc_get_kernel_time(self.state, timer)

    def close(self):
        if self.state is not None:
            dgc_destroy_state(self.state)
            self.state = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def decode_accumulate(layout_learner: Learner, streams: List[Tuple], dense,
                      stream=None):
    """dense += the decoded streams [(runs, vals, entries), ...] in order."""
    dgc_decode_accumulate(layout_learner.state, [s[0] for s in streams],
                          [s[1] for s in streams], [s[2] for s in streams],
                          dense, stream)


def decode_sum(layout_learner: Learner, streams: List[Tuple], dense, stream=None):
    """dense = the decoded streams [(runs, vals, entries), ...] summed in order
    from +0.0 (every element of dense is written)."""
    dgc_decode_sum(layout_learner.state, [s[0] for s in streams],
                   [s[1] for s in streams], [s[2] for s in streams], dense, stream)


def shared_sum(layout_learner: Learner, vals: Sequence, k: Sequence[int], shared_idx,
               out_sum, dense=None, stream=None):
    """out_sum = the learners' value vectors summed in learner order from +0.0;
    dense (optional) = out_sum scattered at shared_idx, +0.0 elsewhere."""
    dgc_shared_sum(layout_learner.state, vals, k, shared_idx, out_sum, dense, stream)


# ----------------------------------------------------- layers and gradient sets

ACTIVATIONS = {"none": DGC_ACT_NONE, "relu": DGC_ACT_RELU, "silu": DGC_ACT_SILU, "gelu": DGC_ACT_GELU,
               "gelu_tanh": DGC_ACT_GELU_TANH}
NORMS = {"l2": DGC_NORM_L2, "max": DGC_NORM_MAX}

_types = {}


def _type_codes():
    """torch dtype -> DGC_* element type."""
    if not _types:
        import torch
        _types.update({torch.bfloat16: DGC_BF16, torch.float16: DGC_FP16, torch.float32: DGC_FP32})
    return _types


def _act(act: str, rounded: bool = False) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
    return code | DGC_DZ_ROUNDED if rounded else code


_native = None


def _torch_calls():
    """The module that checks torch tensors and calls libdgc (csrc/binding.cpp).  Raises if it has not been built."""
    global _native
    if _native is None:
        import importlib.util

        import torch  # noqa: F401  (its libraries, which the module needs)
        lib()
        if not os.path.exists(_build.BINDING):
            raise RuntimeError(f"{_build.BINDING} is missing: build it with "
                               "`python -m sparsified_gradient_compression_amd.build`")
        spec = importlib.util.spec_from_file_location("_dgc_torch", _build.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


def _stream_on(x, stream) -> int:
    """The handle of `stream`, or of the current stream of x's device, which has to be the current one: kernels go there."""
    import torch
    if not x.is_cuda:
        return 0  # refused by the call itself
    device = x.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on device {device}, the current device is {torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _torch_stream(stream):
    """`stream` as torch's object, if it is a handle."""
    import torch
    return torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream


def _empty(shape, dtype, device, stream):
    """Memory for work on `stream` (None: the current one), of that stream's own pool: what the current stream's
    pool hands out may be a block that work on the current stream still uses."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream)):
        return torch.empty(shape, dtype=dtype, device=device)


def _fresh(size: int, x, stream):
    """A workspace of `size` bytes for one call."""
    import torch
    return _empty(size, torch.uint8, x.device, stream if x.is_cuda else None)


def _new(x, shape, dtype, stream):
    """An output for the caller, who will use it on the current stream too."""
    import torch
    if stream is None or not x.is_cuda:
        return _empty(shape, dtype, x.device, None)
    t = _empty(shape, dtype, x.device, stream)
    t.record_stream(torch.cuda.current_stream())
    return t


def _workspace(fn: str, m: int, n: int, k: int, backward: bool, rounded: bool) -> int:
    out = ctypes.c_size_t(0)
    kind = DGC_BACKWARD_ROUNDED if backward and rounded else int(bool(backward))
    _check(getattr(lib(), fn)(m, n, k, kind, ctypes.byref(out)), fn)
    return int(out.value)


def dgc_linear_workspace_bytes(m: int, n: int, k: int, backward: bool = False, rounded: bool = False) -> int:
    return _workspace("dgc_linear_workspace_bytes", m, n, k, backward, rounded)


def dgc_gated_ffn_workspace_bytes(m: int, d: int, f: int, backward: bool = False, rounded: bool = False) -> int:
    return _workspace("dgc_gated_ffn_workspace_bytes", m, d, f, backward, rounded)


def linear_workspace(m: int, n: int, k: int, backward: bool = False, device="cuda", rounded: bool = False):
    """A workspace for linear (or linear_backward; `rounded`: with rounded=True alone) of these sizes."""
    import torch
    return torch.empty(dgc_linear_workspace_bytes(m, n, k, backward, rounded), dtype=torch.uint8, device=device)


def gated_ffn_workspace(m: int, d: int, f: int, backward: bool = False, device="cuda", rounded: bool = False):
    """A workspace for gated_ffn (or gated_ffn_backward; `rounded`: with rounded=True alone) of these sizes."""
    import torch
    return torch.empty(dgc_gated_ffn_workspace_bytes(m, d, f, backward, rounded), dtype=torch.uint8, device=device)


def linear(x, w, bias=None, residual=None, act: str = "none", out=None, pre=None, workspace=None, stream=None):
    """act(x w^T + bias) + residual for x [m, k] and w [n, k] (bfloat16 or float16, contiguous columns).

    No call here records a gradient: tensors that require one are refused outside of torch.no_grad().
    `out` and `pre` are written if given; `pre` receives x w^T + bias for linear_backward.  `out` may be
    `residual`.  `workspace` is what linear_workspace(m, n, k) gives; without one the call allocates it."""
    if out is None:
        out = _new(x, (x.shape[0], w.shape[0]), x.dtype, stream)
    if workspace is None:
        workspace = _fresh(dgc_linear_workspace_bytes(x.shape[0], w.shape[0], x.shape[-1]), x, stream)
    _check(_torch_calls().linear(_act(act), x, w, bias, residual, out, pre, workspace, _stream_on(x, stream)),
           "dgc_linear")
    return out


def linear_backward(dy, x, w, pre=None, act: str = "none", dx=None, dw=None, dbias=None, workspace=None,
                    stream=None, rounded: bool = False):
    """Gradients of linear for the incoming dy [m, n]: with dz = dy * act'(pre), writes each given one of
    dx [m, k] = dz w, dw [n, k] = dz^T x and dbias [n] = the column sums of dz.  dw and dbias are of x's
    type or float32 (the same for both): views of a learner's flat gradient.  Returns (dx, dw, dbias).

    The matrix units take 16-bit operands: behind an activation dz goes to them as the sum of two numbers of
    x's type (three for a bfloat16 x and a float32 dw), so that the gradients are off by little more than
    their own rounding.  `rounded`: as one number, in half the time, with 1.4 times that error, also in a
    float32 dw."""
    if workspace is None:
        workspace = _fresh(dgc_linear_workspace_bytes(x.shape[0], w.shape[0], x.shape[-1], True, rounded), x, stream)
    _check(_torch_calls().linear_backward(_act(act, rounded), dy, x, w, pre, dx, dw, dbias, workspace, _stream_on(x, stream)),
           "dgc_linear_backward")
    return dx, dw, dbias


def gated_ffn(x, w_gate, w_up, act: str = "silu", out=None, gate=None, up=None, workspace=None, stream=None):
    """act(x w_gate^T) * (x w_up^T) for x [m, d] and weights [f, d].  `gate` and `up` receive the two
    products for gated_ffn_backward.  `workspace`: gated_ffn_workspace(m, d, f)."""
    if out is None:
        out = _new(x, (x.shape[0], w_gate.shape[0]), x.dtype, stream)
    if workspace is None:
        workspace = _fresh(dgc_gated_ffn_workspace_bytes(x.shape[0], x.shape[-1], w_gate.shape[0]), x, stream)
    _check(_torch_calls().gated_ffn(_act(act), x, w_gate, w_up, out, gate, up, workspace, _stream_on(x, stream)),
           "dgc_gated_ffn")
    return out


def gated_ffn_backward(dh, x, w_gate, w_up, gate, up, act: str = "silu", dx=None, dw_gate=None, dw_up=None,
                       workspace=None, stream=None, rounded: bool = False):
    """Gradients of gated_ffn for the incoming dh [m, f] and the saved gate and up: writes dx [m, d] if
    given, and dw_gate and dw_up [f, d] (together; x's type or float32).  Returns (dx, dw_gate, dw_up).

    `rounded`: as for linear_backward, of dh * up * act'(gate) and dh * act(gate)."""
    if workspace is None:
        workspace = _fresh(dgc_gated_ffn_workspace_bytes(x.shape[0], x.shape[-1], w_gate.shape[0], True, rounded), x,
                           stream)
    _check(_torch_calls().gated_ffn_backward(_act(act, rounded), dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up, workspace,
                                             _stream_on(x, stream)), "dgc_gated_ffn_backward")
    return dx, dw_gate, dw_up


def dgc_gradset_bytes(sizes: Sequence[int], types: Sequence[int]) -> int:
    s, t = _i64(sizes), np.ascontiguousarray(np.asarray(types, np.int32))
    out = ctypes.c_size_t(0)
    _check(lib().dgc_gradset_bytes(len(s), _hp(s), _hp(t), ctypes.byref(out)), "dgc_gradset_bytes")
    return int(out.value)


class GradSet:
    """The gradients of a model's parameters, by their shapes and dtypes (bfloat16, float16 or float32):
    their norm, and the clipped gradients in their own types or packed into a learner's flat layout.

    `total` (float64) and `scale` (float32) hold the last call's norm and factor on the device."""

    def __init__(self, shapes: Sequence, dtypes: Sequence, device="cuda", stream=None):
        import torch
        self.set = None
        if len(shapes) != len(dtypes):
            raise ValueError("one dtype per shape")
        self.sizes = [int(np.prod(s, dtype=np.int64)) for s in shapes]
        self.dtypes = list(dtypes)
        codes = [_type_codes().get(d) for d in self.dtypes]
        if None in codes:
            raise ValueError("gradients must be bfloat16, float16 or float32")
        self.n = sum(self.sizes)
        self.workspace = _empty(dgc_gradset_bytes(self.sizes, codes), torch.uint8, device, stream)
        self.device = self.workspace.get_device()
        self.total = _empty(1, torch.float64, device, stream)
        self.scale = _empty(1, torch.float32, device, stream)
        self._own_stream = _stream(stream) if self.workspace.is_cuda else None  # whose pool these come from
        handle, s = ctypes.c_void_p(), _i64(self.sizes)
        t = np.ascontiguousarray(np.asarray(codes, np.int32))
        self._layout = s.tobytes(), t.tobytes(), self.device
        _check(lib().dgc_gradset_init(ctypes.byref(handle), len(s), _hp(s), _hp(t), self.workspace.data_ptr(),
                                      self.workspace.numel(), _stream(stream)), "dgc_gradset_init")
        self.set = handle

    def _on(self, stream) -> int:
        """The handle of `stream`.  The set's own tensors are not reused before work on it is done."""
        handle = _stream_on(self.total, stream)
        if handle != self._own_stream:
            for t in (self.workspace, self.total, self.scale):
                t.record_stream(_torch_stream(handle))
        return handle

    @staticmethod
    def _norm(norm: str) -> int:
        code = NORMS.get(norm)
        if code is None:
            raise ValueError(f"unknown norm {norm!r}: one of {', '.join(NORMS)}")
        return code

    def norm(self, grads: Sequence, norm: str = "l2", unscale: float = 1.0, stream=None):
        """unscale * the norm over all gradients, as a float64 tensor of one element."""
        _check(_torch_calls().set_norm(self.set.value, *self._layout, grads, self._norm(norm), unscale, self.total,
                                       self._on(stream)), "dgc_gradset_norm")
        return self.total

    def clip(self, grads: Sequence, clip: float, out: Optional[Sequence] = None, norm: str = "l2",
             unscale: float = 1.0, stream=None):
        """out[t] = grads[t] * scale (in place without `out`), scale = unscale * min(1, clip / norm), for
        clip > 0.  Returns the norm."""
        _check(_torch_calls().set_clip(self.set.value, *self._layout, grads, out, clip, self._norm(norm), unscale,
                                       self.total, self.scale, self._on(stream)), "dgc_gradset_clip")
        return self.total

    def pack(self, grads: Sequence, flat, clip: float, norm: str = "l2", unscale: float = 1.0, stream=None):
        """The clipped gradients in float32, end to end in `flat`: what Learner.compress takes (with its own
        clip 0).  Returns the norm."""
        _check(_torch_calls().set_pack(self.set.value, *self._layout, grads, flat, clip, self._norm(norm), unscale,
                                       self.total, self.scale, self._on(stream)), "dgc_gradset_pack")
        return self.total

    def close(self):
        if self.set is not None:
            lib().dgc_gradset_destroy(self.set)
            self.set = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
