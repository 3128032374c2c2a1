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
#include <vector>

#include "dgc.h"

namespace {

constexpr int kThreads = 256;
constexpr int kLane = 8;                      // elements per thread and step
constexpr int64_t kChunk = kThreads * kLane;  // elements per workgroup and step
constexpr int kGroup = 480;                   // tensors per launch: pointers travel as arguments
constexpr int64_t kMostBlocks = 2048;         // per launch: 8 workgroups per compute unit
constexpr size_t kPad = 256;

size_t round_up(size_t x) { return (x + kPad - 1) / kPad * kPad; }

struct Pointers {
    const void* p[kGroup];
};

// One launch's tensors: t0 .. t0 + count - 1, its workgroups' chunks.
struct Span {
    int32_t t0, count, blocks;
    int32_t part0;  // its first partial
    int64_t chunks;
};

struct Tables {
    const int64_t* chunk0;  // chunks before tensor t within its span
    const int64_t* size;
    const int64_t* offset;  // elements before tensor t
    const int32_t* type;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int A>
struct __attribute__((packed, aligned(A), may_alias)) Bytes16 {
    u32x4 v;
};

__device__ __forceinline__ void load8(const __bf16* p, float* v) {
    const u32x4 t = reinterpret_cast<const Bytes16<2>*>(p)->v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(t[i] << 16);
        v[2 * i + 1] = __uint_as_float(t[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const _Float16* p, float* v) {
    _Float16 t[8];
    *reinterpret_cast<Bytes16<2>*>(t) = *reinterpret_cast<const Bytes16<2>*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = float(t[i]);
}
__device__ __forceinline__ void load8(const float* p, float* v) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<Bytes16<4>*>(v + 4 * i) =
            reinterpret_cast<const Bytes16<4>*>(p)[i];
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float* v) {
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = T(v[i]);
    constexpr int kPieces = int(sizeof(T)) / 2;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        reinterpret_cast<Bytes16<sizeof(T)>*>(p)[i] =
            reinterpret_cast<const Bytes16<sizeof(T)>*>(t)[i];
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
__device__ __forceinline__ double join_block(bool most, double s, double* lds) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s = join(most, s, __shfl_xor(s, d));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = lds[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) s = join(most, s, lds[w]);
    return s;
}

// The tensor of the span that holds chunk c: the last t with chunk0[t] <= c
// among those that have chunks.
__device__ __forceinline__ int find(const Tables& tb, const Span& sp, int64_t c) {
    int lo = 0, hi = sp.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tb.chunk0[sp.t0 + mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int64_t chunk_of(const Span& sp, int64_t block) {
    return block * sp.chunks / sp.blocks;
}

template <class T>
__device__ __forceinline__ void norm_range(const T* p, int64_t at, int64_t end, bool most,
                                           double& s) {
    int64_t i = at + threadIdx.x * kLane;
#pragma unroll 4
    for (; i + kLane <= end; i += kChunk) {
        float v[kLane];
        load8(p + i, v);
#pragma unroll
        for (int e = 0; e < kLane; ++e) take(most, v[e], s);
    }
    if (i < end)
        for (int e = 0; i + e < end; ++e) take(most, float(p[i + e]), s);
}

__global__ __launch_bounds__(kThreads) void k_set_norm(Pointers g, Span sp, Tables tb, int most,
                                                       const void** table, double* part) {
    __shared__ double lds[kThreads / 64];
    // the second pass finds the gradients here
    if (blockIdx.x == 0)
        for (int t = threadIdx.x; t < sp.count; t += kThreads) table[sp.t0 + t] = g.p[t];
    int64_t c = chunk_of(sp, blockIdx.x);
    const int64_t c1 = chunk_of(sp, blockIdx.x + 1);
    double s = 0.0;
    int t = c < c1 ? find(tb, sp, c) : 0;
    while (c < c1) {
        const int64_t base = tb.chunk0[sp.t0 + t], n = tb.size[sp.t0 + t];
        const int64_t own = (n + kChunk - 1) / kChunk;
        const int64_t stop = base + own < c1 ? base + own : c1;
        if (stop > c) {
            const int64_t at = (c - base) * kChunk;
            const int64_t end = (stop - base) * kChunk < n ? (stop - base) * kChunk : n;
            switch (tb.type[sp.t0 + t]) {
                case DGC_BF16:
                    norm_range(static_cast<const __bf16*>(g.p[t]), at, end, most, s);
                    break;
                case DGC_FP16:
                    norm_range(static_cast<const _Float16*>(g.p[t]), at, end, most, s);
                    break;
                default: norm_range(static_cast<const float*>(g.p[t]), at, end, most, s);
            }
            c = stop;
        }
        ++t;
    }
    s = join_block(most, s, lds);
    if (threadIdx.x == 0) part[sp.part0 + blockIdx.x] = s;
}

// The norm and the factor from all partials.
__device__ __forceinline__ double whole_norm(const double* part, int count, int most,
                                             double unscale, double* lds) {
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) s = join(most, s, part[i]);
    s = join_block(most, s, lds);
    return (most ? s : sqrt(s)) * unscale;
}

__device__ __forceinline__ float factor(double norm, double clip, double unscale) {
    const double r = clip > 0.0 && norm > clip ? clip / norm : 1.0;
    return float(r * unscale);
}

__global__ __launch_bounds__(kThreads) void k_set_total(const double* part, int count, int most,
                                                        double unscale, double* out_norm) {
    __shared__ double lds[kThreads / 64];
    const double norm = whole_norm(part, count, most, unscale, lds);
    if (threadIdx.x == 0) *out_norm = norm;
}

template <class T, class O>
__device__ __forceinline__ void scale_range(const T* p, O* o, int64_t at, int64_t end, float f) {
    int64_t i = at + threadIdx.x * kLane;
#pragma unroll 4
    for (; i + kLane <= end; i += kChunk) {
        float v[kLane];
        load8(p + i, v);
#pragma unroll
        for (int e = 0; e < kLane; ++e) v[e] *= f;
        store8(o + i, v);
    }
    if (i < end)
        for (int e = 0; i + e < end; ++e) o[i + e] = O(float(p[i + e]) * f);
}

// FLAT: into flat at the tensor's offset; else into the tensor's own output.
template <bool FLAT>
__global__ __launch_bounds__(kThreads) void k_set_scale(Pointers out, Span sp, Tables tb,
                                                        int most, const void* const* table,
                                                        const double* part, int parts,
                                                        double clip, double unscale,
                                                        float* flat, double* out_norm,
                                                        float* out_scale) {
    __shared__ double lds[kThreads / 64];
    const double norm = whole_norm(part, parts, most, unscale, lds);
    const float f = factor(norm, clip, unscale);
    if (blockIdx.x == 0 && sp.t0 == 0 && threadIdx.x == 0) {
        if (out_norm) *out_norm = norm;
        if (out_scale) *out_scale = f;
    }
    int64_t c = chunk_of(sp, blockIdx.x);
    const int64_t c1 = chunk_of(sp, blockIdx.x + 1);
    int t = c < c1 ? find(tb, sp, c) : 0;
    while (c < c1) {
        const int64_t base = tb.chunk0[sp.t0 + t], n = tb.size[sp.t0 + t];
        const int64_t own = (n + kChunk - 1) / kChunk;
        const int64_t stop = base + own < c1 ? base + own : c1;
        if (stop > c) {
            const int64_t at = (c - base) * kChunk;
            const int64_t end = (stop - base) * kChunk < n ? (stop - base) * kChunk : n;
            const void* g = table[sp.t0 + t];
            float* fo = FLAT ? flat + tb.offset[sp.t0 + t] : nullptr;
            void* o = FLAT ? nullptr : const_cast<void*>(out.p[t]);
            switch (tb.type[sp.t0 + t]) {
                case DGC_BF16:
                    if (FLAT)
                        scale_range(static_cast<const __bf16*>(g), fo, at, end, f);
                    else
                        scale_range(static_cast<const __bf16*>(g), static_cast<__bf16*>(o), at,
                                    end, f);
                    break;
                case DGC_FP16:
                    if (FLAT)
                        scale_range(static_cast<const _Float16*>(g), fo, at, end, f);
                    else
                        scale_range(static_cast<const _Float16*>(g), static_cast<_Float16*>(o),
                                    at, end, f);
                    break;
                default:
                    scale_range(static_cast<const float*>(g), FLAT ? fo : static_cast<float*>(o),
                                at, end, f);
            }
            c = stop;
        }
        ++t;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

struct dgc_gradset {
    std::vector<int64_t> size;
    std::vector<int32_t> type;
    std::vector<Span> spans;
    int32_t parts = 0;  // partial norms of all spans
    size_t at_table = 0, at_part = 0, total = 0;
    char* ws = nullptr;
    Tables tables{};
};

namespace {

int plan_set(int32_t T, const int64_t* sizes, const int32_t* types, dgc_gradset& s,
             std::vector<int64_t>& chunk0, std::vector<int64_t>& offset) {
    if (T <= 0 || !sizes || !types) return DGC_EINVAL;
    int64_t n = 0;
    for (int32_t t = 0; t < T; ++t) {
        if (sizes[t] < 0 || sizes[t] > (int64_t(1) << 44) ||
            (types[t] != DGC_BF16 && types[t] != DGC_FP16 && types[t] != DGC_FP32))
            return DGC_EINVAL;
        offset.push_back(n);
        n += sizes[t];
        if (n > (int64_t(1) << 50)) return DGC_EINVAL;
    }
    s.size.assign(sizes, sizes + T);
    s.type.assign(types, types + T);
    for (int32_t t0 = 0; t0 < T; t0 += kGroup) {
        Span sp{};
        sp.t0 = t0;
        sp.count = std::min(kGroup, T - t0);
        for (int32_t t = t0; t < t0 + sp.count; ++t) {
            chunk0.push_back(sp.chunks);
            sp.chunks += cdiv(sizes[t], kChunk);
        }
        sp.blocks = int32_t(std::max<int64_t>(1, std::min(sp.chunks, kMostBlocks)));
        sp.part0 = s.parts;
        s.parts += sp.blocks;
        s.spans.push_back(sp);
    }
    const size_t T8 = size_t(T) * 8;
    s.at_table = round_up(3 * T8 + size_t(T) * 4);
    s.at_part = s.at_table + round_up(T8);
    s.total = s.at_part + round_up(size_t(s.parts) * 8);
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

int norm_pass(const dgc_gradset* s, const void* const* grads, int most, hipStream_t stream) {
    for (const Span& sp : s->spans) {
        Pointers g;
        std::memcpy(g.p, grads + sp.t0, size_t(sp.count) * sizeof(void*));
        k_set_norm<<<dim3(unsigned(sp.blocks)), kThreads, 0, stream>>>(
            g, sp, s->tables, most, reinterpret_cast<const void**>(s->ws + s->at_table),
            reinterpret_cast<double*>(s->ws + s->at_part));
        if (hipGetLastError() != hipSuccess) return DGC_EHIP;
    }
    return DGC_OK;
}

int scale_pass(const dgc_gradset* s, const void* const* grads, void* const* outs, float* flat,
               double clip, int32_t norm, double unscale, double* out_norm, float* out_scale,
               hipStream_t stream) {
    if (!s || (norm != DGC_NORM_L2 && norm != DGC_NORM_MAX) || !std::isfinite(unscale) ||
        unscale <= 0.0 || std::isnan(clip) || !pointers_ok(s, grads) ||
        reinterpret_cast<uintptr_t>(out_norm) % 8 != 0 ||
        reinterpret_cast<uintptr_t>(out_scale) % 4 != 0)
        return DGC_EINVAL;
    if (outs ? !pointers_ok(s, outs) : reinterpret_cast<uintptr_t>(flat) % 4 != 0)
        return DGC_EINVAL;
    const int rc = norm_pass(s, grads, norm, stream);
    if (rc != DGC_OK) return rc;
    const void* const* table = reinterpret_cast<const void* const*>(s->ws + s->at_table);
    const double* part = reinterpret_cast<const double*>(s->ws + s->at_part);
    for (const Span& sp : s->spans) {
        Pointers o;
        if (outs) {
            std::memcpy(o.p, outs + sp.t0, size_t(sp.count) * sizeof(void*));
            k_set_scale<false><<<dim3(unsigned(sp.blocks)), kThreads, 0, stream>>>(
                o, sp, s->tables, norm, table, part, s->parts, clip, unscale, nullptr, out_norm,
                out_scale);
        } else {
            k_set_scale<true><<<dim3(unsigned(sp.blocks)), kThreads, 0, stream>>>(
                o, sp, s->tables, norm, table, part, s->parts, clip, unscale, flat, out_norm,
                out_scale);
        }
        if (hipGetLastError() != hipSuccess) return DGC_EHIP;
    }
    return DGC_OK;
}

}  // namespace

extern "C" {

int dgc_gradset_bytes(int32_t n_tensors, const int64_t* sizes, const int32_t* types,
                      size_t* bytes) {
    if (!bytes) return DGC_EINVAL;
    try {
        dgc_gradset s;
        std::vector<int64_t> chunk0, offset;
        const int rc = plan_set(n_tensors, sizes, types, s, chunk0, offset);
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
        std::vector<int64_t> chunk0, offset;
        int rc = plan_set(n_tensors, sizes, types, *s, chunk0, offset);
        if (rc == DGC_OK &&
            (!workspace || reinterpret_cast<uintptr_t>(workspace) % kPad != 0))
            rc = DGC_EINVAL;
        if (rc == DGC_OK && workspace_bytes < s->total) rc = DGC_ECAPACITY;
        if (rc == DGC_OK) {
            const size_t T8 = size_t(n_tensors) * 8;
            std::vector<char> host(3 * T8 + size_t(n_tensors) * 4);
            std::memcpy(host.data(), chunk0.data(), T8);
            std::memcpy(host.data() + T8, sizes, T8);
            std::memcpy(host.data() + 2 * T8, offset.data(), T8);
            std::memcpy(host.data() + 3 * T8, types, size_t(n_tensors) * 4);
            s->ws = static_cast<char*>(workspace);
            s->tables.chunk0 = reinterpret_cast<const int64_t*>(s->ws);
            s->tables.size = reinterpret_cast<const int64_t*>(s->ws + T8);
            s->tables.offset = reinterpret_cast<const int64_t*>(s->ws + 2 * T8);
            s->tables.type = reinterpret_cast<const int32_t*>(s->ws + 3 * T8);
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
    const int rc = norm_pass(s, grads, norm, stream);
    if (rc != DGC_OK) return rc;
    k_set_total<<<1, kThreads, 0, stream>>>(reinterpret_cast<const double*>(s->ws + s->at_part),
                                            s->parts, norm, unscale, out_norm);
    return hipGetLastError() == hipSuccess ? DGC_OK : DGC_EHIP;
}

int dgc_gradset_clip(const dgc_gradset* s, const void* const* grads, void* const* outs,
                     double clip, int32_t norm, double unscale, double* out_norm,
                     float* out_scale, hipStream_t stream) {
    if (!outs) return DGC_EINVAL;
    return scale_pass(s, grads, outs, nullptr, clip, norm, unscale, out_norm, out_scale, stream);
}

int dgc_gradset_pack(const dgc_gradset* s, const void* const* grads, float* flat, double clip,
                     int32_t norm, double unscale, double* out_norm, float* out_scale,
                     hipStream_t stream) {
    if (!flat) return DGC_EINVAL;
    return scale_pass(s, grads, nullptr, flat, clip, norm, unscale, out_norm, out_scale, stream);
}

void dgc_gradset_destroy(dgc_gradset* s) { delete s; }

}  // extern "C"
