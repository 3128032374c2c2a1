// dgc_gradset.hip -- the norm over many gradient tensors, and the clipped
// gradients in their own types or end to end in binary32.  See include/dgc.h
// for the contract of every function.
//
// Two passes: one reads every gradient and leaves a binary64 partial norm per
// workgroup; the other, once all partials are there, adds them up in each of
// its workgroups, reads every gradient again and writes it scaled.  The
// factor needs the whole norm, so the second read cannot be saved, and both
// passes are bound by memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>
#include <vector>

#include "dgc.h"
#include "launch_grid.hpp"

namespace {

constexpr int kThreads = 256;             // of a norm workgroup
constexpr int kScaleThreads = 128;        // of a scaling one: 16 bytes of output each, or twice that
constexpr int64_t kPiece = 1024;          // elements; a tensor starts a new pair of pieces
constexpr int64_t kPair = 2 * kPiece;
constexpr int64_t kOwner = 64;            // pairs per entry of the group table
constexpr int kGroup = 240;               // tensors per norm launch: their pointers are arguments
constexpr int64_t kMostBlocks = 2048;     // of a norm launch: 8 workgroups per compute unit
constexpr int64_t kMostUnit = 64;         // pairs that a norm workgroup takes at a time, at most
constexpr int64_t kLarge = 256ll << 20;   // bytes: what the last cache holds
constexpr size_t kPad = 256;

size_t round_up(size_t x) { return (x + kPad - 1) / kPad * kPad; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Pointers {
    const void* grad[kGroup];
    void* out[kGroup];
};

// A tensor that has elements.
struct Tensor {
    int64_t pair0, pair1;  // its pairs of pieces
    int64_t size;
    int64_t offset;  // elements before it
    const void* grad;  // this call's addresses, left by the norm pass
    void* out;
    int32_t type;
    int32_t index;  // among the tensors with elements
};

// One norm launch's tensors: t0 .. t0 + count - 1 of those with elements.
struct Span {
    int32_t t0, count, blocks, unit;
    int32_t part0;  // its first partial
    int64_t pair0, pairs, units;
};

// A set's workspace.
struct Tables {
    Tensor* tensors;
    Tensor* owner;  // entry i: the tensor of pair 64 i, a copy
    int32_t count;  // tensors
    double* part;
    float* scale;           // the factor, for the second pass of a large set
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Words of 8 and 16 bytes at any address that an element of 2 or 4 bytes can
// have: the hardware splits what is not aligned.
#define DGC_GLOBAL __attribute__((address_space(1)))

template <int A>
struct Words;
template <>
struct Words<2> {
    typedef u32x2 two __attribute__((aligned(2), may_alias));
    typedef u32x4 four __attribute__((aligned(2), may_alias));
};
template <>
struct Words<4> {
    typedef u32x2 two __attribute__((aligned(4), may_alias));
    typedef u32x4 four __attribute__((aligned(4), may_alias));
};

// L (4 or 8) consecutive elements, at any address their type can have.
// STREAM: past the caches (a billion bf16 gradients' norm: 312 us, not 360).
template <int L, bool STREAM, class T>
__device__ __forceinline__ void load_row(const T* p, float* v) {
    constexpr int kBytes = L * int(sizeof(T));
    T t[L];
    if constexpr (kBytes == 8) {
        typedef typename Words<sizeof(T)>::two V;
        const DGC_GLOBAL V* q = (const DGC_GLOBAL V*)(p);
        *reinterpret_cast<V*>(t) = STREAM ? __builtin_nontemporal_load(q) : *q;
    } else {
        typedef typename Words<sizeof(T)>::four V;
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
            const DGC_GLOBAL V* q = (const DGC_GLOBAL V*)(p) + i;
            reinterpret_cast<V*>(t)[i] = STREAM ? __builtin_nontemporal_load(q) : *q;
        }
    }
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] = float(t[i]);
}

template <int L, bool STREAM, class T>
__device__ __forceinline__ void store_row(T* p, const float* v) {
    typedef typename Words<sizeof(T)>::four V;
    T t[L];
#pragma unroll
    for (int i = 0; i < L; ++i) t[i] = T(v[i]);
#pragma unroll
    for (int i = 0; i < L * int(sizeof(T)) / 16; ++i) {
        const u32x4 w = reinterpret_cast<const V*>(t)[i];
        DGC_GLOBAL V* q = (DGC_GLOBAL V*)(p) + i;
        if constexpr (STREAM)
            __builtin_nontemporal_store(w, q);
        else
            *q = w;
    }
}

// Sum of squares (binary64), or the largest magnitude; a NaN stays.
__device__ __forceinline__ void take(bool most, float g, double& s) {
    if (most) {
        const double a = fabs(double(g));
        s = a > s || a != a ? a : s;
    } else {
        s = fma(double(g), double(g), s);
    }
}
__device__ __forceinline__ double join(bool most, double a, double b) {
    return most ? (b > a || b != b ? b : a) : a + b;
}

// Over the workgroup, in a fixed order; every thread gets the result.
template <int THREADS>
__device__ __forceinline__ double join_block(bool most, double s, double* lds) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s = join(most, s, __shfl_xor(s, d));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = lds[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) s = join(most, s, lds[w]);
    return s;
}

constexpr int kBatch = 4;  // steps whose loads are under way together

template <bool STREAM, class T>
__device__ __forceinline__ void norm_range(const T* p, int64_t at, int64_t end, bool most,
                                           double& s) {
    constexpr int64_t kStep = kThreads * 8;
    int64_t i = at + threadIdx.x * 8;
    for (; i + (kBatch - 1) * kStep + 8 <= end; i += kBatch * kStep) {
        float v[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) load_row<8, STREAM>(p + i + b * kStep, v[b]);
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) take(most, v[b][e], s);
    }
    for (; i + 8 <= end; i += kStep) {
        float v[8];
        load_row<8, STREAM>(p + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) take(most, v[e], s);
    }
    if (i < end)
        for (int e = 0; i + e < end; ++e) take(most, float(p[i + e]), s);
}

// A binary64 partial norm per workgroup.  Workgroups take units in turn.
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void k_set_norm(Pointers g, Span sp, Tables tb, int most) {
    __shared__ double lds[kThreads / 64];
    // the second pass finds the tensors here
    if (blockIdx.x == 0)
        for (int t = threadIdx.x; t < sp.count; t += kThreads) {
            tb.tensors[sp.t0 + t].grad = g.grad[t];
            tb.tensors[sp.t0 + t].out = g.out[t];
        }
    double s = 0.0;
    for (int64_t u = blockIdx.x; u < sp.units; u += sp.blocks) {
        int64_t c = sp.pair0 + u * sp.unit;
        const int64_t stop = sp.pair0 + sp.pairs;
        const int64_t c1 = c + sp.unit < stop ? c + sp.unit : stop;
        for (int t = tb.owner[c / kOwner].index; c < c1; ++t) {
            // (not the addresses: those are being written)
            const int64_t size = tb.tensors[t].size, base = tb.tensors[t].pair0;
            const int64_t all = tb.tensors[t].pair1, to = all < c1 ? all : c1;
            if (to <= c) continue;
            const int64_t at = (c - base) * kPair;
            const int64_t end = (to - base) * kPair < size ? (to - base) * kPair : size;
            const void* p = g.grad[t - sp.t0];
            switch (tb.tensors[t].type) {
                case DGC_BF16:
                    norm_range<STREAM>(static_cast<const __bf16*>(p), at, end, most, s);
                    break;
                case DGC_FP16:
                    norm_range<STREAM>(static_cast<const _Float16*>(p), at, end, most, s);
                    break;
                default: norm_range<STREAM>(static_cast<const float*>(p), at, end, most, s);
            }
            // entries of the group table whose pair lies in here
            if (threadIdx.x == 0)
                for (int64_t o = (c + kOwner - 1) / kOwner; o * kOwner < to; ++o) {
                    tb.owner[o].grad = p;
                    tb.owner[o].out = g.out[t - sp.t0];
                }
            c = to;
        }
    }
    s = join_block<kThreads>(most, s, lds);
    if (threadIdx.x == 0) tb.part[sp.part0 + blockIdx.x] = s;
}

// The norm from all partials.
template <int THREADS>
__device__ __forceinline__ double whole_norm(const double* part, int count, int most,
                                             double unscale, double* lds) {
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += THREADS) s = join(most, s, part[i]);
    s = join_block<THREADS>(most, s, lds);
    return (most ? s : sqrt(s)) * unscale;
}

__device__ __forceinline__ float factor(double norm, double clip, double unscale) {
    const double r = clip > 0.0 && norm > clip ? clip / norm : 1.0;
    return float(r * unscale);
}

// What the second pass needs beside the tensors.
struct Scaling {
    int parts, most, pieces;  // pieces: a workgroup each
    double clip, unscale;
    double* out_norm;
    float* out_scale;
    float* flat;
};

// One workgroup: the norm, and the factor of a large set.
__global__ __launch_bounds__(kThreads) void k_set_total(Tables tb, Scaling k) {
    __shared__ double lds[kThreads / 64];
    const double norm = whole_norm<kThreads>(tb.part, k.parts, k.most, k.unscale, lds);
    if (threadIdx.x != 0) return;
    const float f = factor(norm, k.clip, k.unscale);
    if (k.out_norm) *k.out_norm = norm;
    if (k.out_scale) *k.out_scale = f;
    *tb.scale = f;
}

// The piece [at, at + kPiece) of a tensor, as far as it goes: a wave takes L
// elements a lane, side by side, STEPS times.  The loads are under way while
// `f` finds the factor out.
template <bool STREAM, int L, class T, class O, class F>
__device__ __forceinline__ void scale_piece(const T* p, O* o, int64_t at, int64_t n, F f) {
    constexpr int kSteps = kPiece / (kScaleThreads * L), kStep = 64 * L;
    const int first = (threadIdx.x >> 6) * kSteps * kStep + (threadIdx.x & 63) * L;
    p += at + first;
    o += at + first;
    if (n - at >= kPiece) {
        float v[kSteps][L];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) load_row<L, STREAM>(p + j * kStep, v[j]);
        const float s = f();
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
#pragma unroll
            for (int e = 0; e < L; ++e) v[j][e] *= s;
            store_row<L, STREAM>(o + j * kStep, v[j]);
        }
    } else {
        const float s = f();
        const int left = int(n - at) - first;
        for (int i = 0; i < kSteps * kStep && i < left; i += kStep) {
            if (i + L <= left) {
                float v[L];
                load_row<L, STREAM>(p + i, v);
#pragma unroll
                for (int e = 0; e < L; ++e) v[e] *= s;
                store_row<L, STREAM>(o + i, v);
            } else {
                for (int e = i; e < left; ++e) o[e] = O(float(p[e]) * s);
            }
        }
    }
}

// A workgroup per piece, and no loop: a wave never waits for its own stores
// before its next loads, and what is under way lies close together (a billion
// bf16 into binary32, a plain conversion: 970-1060 us so, 1130-1280 us with
// workgroups that loop over pieces, however they take them; two waves per
// workgroup and 2 KB of output per wave lose least to the look-up).
//   FLAT: into flat at the tensor's offset; else into the tensor's own
//   output.  FEW: a set of few pieces and partials, whose workgroups add the
//   partials up by themselves and save a launch.
template <bool FLAT, bool STREAM, bool FEW>
__global__ __launch_bounds__(kScaleThreads) void k_set_scale(Tables tb, Scaling k) {
    __shared__ double lds[kThreads / 64];
    const int64_t piece = dgc::block_number(), pair = piece / 2;
    if (piece >= k.pieces) return;
    Tensor x = tb.owner[pair / kOwner];
    if (pair >= x.pair1) {
        // a later tensor, one of the at most 64 that start behind the entry's
        // pair: every lane looks at one, all for one load's latency
        const int mine = x.index + 1 + int(threadIdx.x & 63);
        const int64_t start = tb.tensors[mine < tb.count ? mine : x.index].pair0;
        const int later = __builtin_popcountll(__ballot(mine < tb.count && start <= pair));
        x = tb.tensors[__builtin_amdgcn_readfirstlane(x.index + later)];
    }
    const int64_t at = (pair - x.pair0) * kPair + piece % 2 * kPiece;
    const float known = FEW ? 0.0f : *tb.scale;
    const auto f = [&]() -> float {
        if constexpr (!FEW) return known;
        const double norm = whole_norm<kScaleThreads>(tb.part, k.parts, k.most, k.unscale, lds);
        const float s = factor(norm, k.clip, k.unscale);
        if (piece == 0 && threadIdx.x == 0) {
            if (k.out_norm) *k.out_norm = norm;
            if (k.out_scale) *k.out_scale = s;
        }
        return s;
    };
    const auto one = [&](const auto* p) {
        typedef std::remove_const_t<std::remove_pointer_t<decltype(p)>> T;
        if constexpr (FLAT)
            scale_piece<STREAM, 4>(p, k.flat + x.offset, at, x.size, f);
        else
            scale_piece<STREAM, 16 / sizeof(T)>(p, static_cast<T*>(x.out), at, x.size, f);
    };
    switch (x.type) {
        case DGC_BF16: one(static_cast<const __bf16*>(x.grad)); break;
        case DGC_FP16: one(static_cast<const _Float16*>(x.grad)); break;
        default: one(static_cast<const float*>(x.grad));
    }
}

}  // namespace

struct dgc_gradset {
    std::vector<int64_t> size;
    std::vector<int32_t> type;
    std::vector<int32_t> filled;  // the tensors that have elements
    std::vector<Span> spans;
    int32_t parts = 0;  // partial norms of all spans
    int64_t elements = 0, bytes = 0, pairs = 0;
    size_t at_owner = 0, at_part = 0, at_scale = 0, total = 0;
    Tables tables{};
};

namespace {

int plan_set(int32_t T, const int64_t* sizes, const int32_t* types, dgc_gradset& s) {
    if (T <= 0 || !sizes || !types) return DGC_EINVAL;
    for (int32_t t = 0; t < T; ++t) {
        if (sizes[t] < 0 || sizes[t] > (int64_t(1) << 40) ||
            (types[t] != DGC_BF16 && types[t] != DGC_FP16 && types[t] != DGC_FP32))
            return DGC_EINVAL;
        s.elements += sizes[t];
        s.bytes += sizes[t] * (types[t] == DGC_FP32 ? 4 : 2);
        s.pairs += cdiv(sizes[t], kPair);
        // a workgroup per piece
        if (2 * s.pairs > 0x7FFFFFFF) return DGC_EINVAL;
    }
    s.size.assign(sizes, sizes + T);
    s.type.assign(types, types + T);
    for (int32_t t = 0; t < T; ++t)
        if (sizes[t] > 0) s.filled.push_back(t);
    const int32_t filled = int32_t(s.filled.size());
    int64_t pair0 = 0;
    for (int32_t t0 = 0; t0 < std::max(filled, 1); t0 += kGroup) {
        Span sp{};
        sp.t0 = t0;
        sp.count = std::min(kGroup, filled - t0);
        sp.pair0 = pair0;
        for (int32_t t = t0; t < t0 + sp.count; ++t) sp.pairs += cdiv(sizes[s.filled[t]], kPair);
        pair0 += sp.pairs;
        // one round of workgroups, or units that hide their tensors' look-up;
        // by fours where there are enough: loads go out four at a time
        const int64_t unit = std::min(cdiv(sp.pairs, kMostBlocks), kMostUnit);
        sp.unit = int32_t(unit < 3 ? std::max<int64_t>(unit, 1) : (unit + 3) / 4 * 4);
        sp.units = cdiv(sp.pairs, sp.unit);
        sp.blocks = int32_t(std::max<int64_t>(1, std::min(sp.units, kMostBlocks)));
        sp.part0 = s.parts;
        s.parts += sp.blocks;
        s.spans.push_back(sp);
    }
    s.at_owner = round_up(size_t(filled) * sizeof(Tensor));
    s.at_part = s.at_owner + round_up(size_t(cdiv(s.pairs, kOwner)) * sizeof(Tensor));
    s.at_scale = s.at_part + round_up(size_t(s.parts) * 8);
    s.total = s.at_scale + kPad;
    return DGC_OK;
}

bool pointers_ok(const dgc_gradset* s, const void* const* p) {
    if (!p) return false;
    for (size_t t = 0; t < s->size.size(); ++t)
        if (s->size[t] > 0 &&
            (!p[t] || reinterpret_cast<uintptr_t>(p[t]) % (s->type[t] == DGC_FP32 ? 4 : 2) != 0))
            return false;
    return true;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The norm pass.  Gradients that the last cache cannot hold go past it.
int norm_pass(const dgc_gradset* s, const void* const* grads, void* const* outs, int most,
              hipStream_t stream) {
    const auto kernel = s->bytes > kLarge ? k_set_norm<true> : k_set_norm<false>;
    for (const Span& sp : s->spans) {
        Pointers g{};
        for (int32_t i = 0; i < sp.count; ++i) {
            const int32_t t = s->filled[size_t(sp.t0 + i)];
            g.grad[i] = grads[t];
            if (outs) g.out[i] = outs[t];
        }
        kernel<<<dim3(unsigned(sp.blocks)), kThreads, 0, stream>>>(g, sp, s->tables, most);
        if (hipGetLastError() != hipSuccess) return DGC_EHIP;
    }
    return DGC_OK;
}

template <bool FLAT>
int scale_pass(const dgc_gradset* s, const void* const* grads, void* const* outs,
               const Scaling& k, hipStream_t stream) {
    if (!s || (k.most != DGC_NORM_L2 && k.most != DGC_NORM_MAX) || !std::isfinite(k.unscale) ||
        k.unscale <= 0.0 || std::isnan(k.clip) || !pointers_ok(s, grads) ||
        !aligned(k.out_norm, 8) || !aligned(k.out_scale, 4))
        return DGC_EINVAL;
    if (FLAT ? (!k.flat && s->elements > 0) || !aligned(k.flat, 4) : !pointers_ok(s, outs))
        return DGC_EINVAL;
    const int rc = norm_pass(s, grads, outs, k.most, stream);
    if (rc != DGC_OK) return rc;
    Scaling l = k;
    l.parts = s->parts;
    // one round of workgroups and a few partials each: no launch in between
    const int64_t blocks = 2 * s->pairs;
    l.pieces = int(blocks);
    const bool few = blocks > 0 && blocks <= 2 * kMostBlocks && s->parts <= 2 * kThreads;
    if (!few) k_set_total<<<1, kThreads, 0, stream>>>(s->tables, l);
    const bool large = s->bytes + (FLAT ? 4 * s->elements : s->bytes) > kLarge;
    if (blocks > 0) {
        const auto kernel = few ? k_set_scale<FLAT, false, true>
                                : large ? k_set_scale<FLAT, true, false> : k_set_scale<FLAT, false, false>;
        kernel<<<dgc::grid_of(blocks, kScaleThreads), kScaleThreads, 0, stream>>>(s->tables, l);
    }
    return hipGetLastError() == hipSuccess ? DGC_OK : DGC_EHIP;
}

}  // namespace

extern "C" {

int dgc_gradset_bytes(int32_t n_tensors, const int64_t* sizes, const int32_t* types,
                      size_t* bytes) {
    if (!bytes) return DGC_EINVAL;
    try {
        dgc_gradset s;
        const int rc = plan_set(n_tensors, sizes, types, s);
        if (rc == DGC_OK) *bytes = s.total;
        return rc;
    } catch (const std::bad_alloc&) {
        return DGC_ECAPACITY;
    }
}

int dgc_gradset_init(dgc_gradset** out, int32_t n_tensors, const int64_t* sizes,
                     const int32_t* types, void* workspace, size_t workspace_bytes,
                     hipStream_t stream) {
    if (!out) return DGC_EINVAL;
    *out = nullptr;
    dgc_gradset* s = nullptr;
    try {
        s = new dgc_gradset;
        int rc = plan_set(n_tensors, sizes, types, *s);
        if (rc == DGC_OK &&
            (!workspace || reinterpret_cast<uintptr_t>(workspace) % kPad != 0))
            rc = DGC_EINVAL;
        if (rc == DGC_OK && workspace_bytes < s->total) rc = DGC_ECAPACITY;
        if (rc == DGC_OK) {
            std::vector<char> host(s->at_part);
            Tensor* const first = reinterpret_cast<Tensor*>(host.data());
            Tensor* tensors = first;
            Tensor* owner = reinterpret_cast<Tensor*>(host.data() + s->at_owner);
            int64_t pairs = 0, elements = 0;
            for (int32_t t = 0; t < n_tensors; ++t) {
                if (sizes[t] == 0) continue;
                const int64_t own = cdiv(sizes[t], kPair);
                const Tensor x{pairs,   pairs + own, sizes[t], elements,
                               nullptr, nullptr,     types[t], int32_t(tensors - first)};
                *tensors++ = x;
                for (int64_t o = cdiv(pairs, kOwner); o * kOwner < pairs + own; ++o) owner[o] = x;
                elements += sizes[t];
                pairs += own;
            }
            char* ws = static_cast<char*>(workspace);
            s->tables.tensors = reinterpret_cast<Tensor*>(ws);
            s->tables.owner = reinterpret_cast<Tensor*>(ws + s->at_owner);
            s->tables.count = int32_t(s->filled.size());
            s->tables.part = reinterpret_cast<double*>(ws + s->at_part);
            s->tables.scale = reinterpret_cast<float*>(ws + s->at_scale);
            if (hipMemcpyAsync(workspace, host.data(), host.size(), hipMemcpyHostToDevice,
                               stream) != hipSuccess ||
                hipStreamSynchronize(stream) != hipSuccess)
                rc = DGC_EHIP;
        }
        if (rc != DGC_OK) {
            delete s;
            return rc;
        }
    } catch (const std::bad_alloc&) {
        delete s;
        return DGC_ECAPACITY;
    }
    *out = s;
    return DGC_OK;
}

int dgc_gradset_norm(const dgc_gradset* s, const void* const* grads, int32_t norm,
                     double unscale, double* out_norm, hipStream_t stream) {
    if (!s || (norm != DGC_NORM_L2 && norm != DGC_NORM_MAX) || !std::isfinite(unscale) ||
        unscale <= 0.0 || !out_norm || reinterpret_cast<uintptr_t>(out_norm) % 8 != 0 ||
        !pointers_ok(s, grads))
        return DGC_EINVAL;
    const int rc = norm_pass(s, grads, nullptr, norm, stream);
    if (rc != DGC_OK) return rc;
    k_set_total<<<1, kThreads, 0, stream>>>(
        s->tables, Scaling{s->parts, norm, 0, 0.0, unscale, out_norm, nullptr, nullptr});
    return hipGetLastError() == hipSuccess ? DGC_OK : DGC_EHIP;
}

int dgc_gradset_clip(const dgc_gradset* s, const void* const* grads, void* const* outs,
                     double clip, int32_t norm, double unscale, double* out_norm,
                     float* out_scale, hipStream_t stream) {
    return scale_pass<false>(s, grads, outs,
                             Scaling{0, norm, 0, clip, unscale, out_norm, out_scale, nullptr}, stream);
}

int dgc_gradset_pack(const dgc_gradset* s, const void* const* grads, float* flat, double clip,
                     int32_t norm, double unscale, double* out_norm, float* out_scale,
                     hipStream_t stream) {
    return scale_pass<true>(s, grads, nullptr,
                            Scaling{0, norm, 0, clip, unscale, out_norm, out_scale, flat}, stream);
}

void dgc_gradset_destroy(dgc_gradset* s) { delete s; }

}  // extern "C"
