// dgc_norm.hip -- layer norm and its gradients.  See include/dgc.h for the
// contract of every function.
#include <algorithm>

#include "tokens.hpp"

using namespace dgc::tokens;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostBlocks = 1 << 20;  // of a launch: workgroups take what is left in turn
constexpr int64_t kMostParts = 512;       // stripes of rows whose column sums are joined
constexpr int64_t kPartRows = 16;         // rows of a stripe, at least
constexpr int kColumns = 512;             // of a workgroup of the column sums: 64 lanes, 8 each

struct Forward {
    int64_t m, d;
    float eps;
    const void* x;
    int64_t ldx;
    const void* weight;
    const void* bias;
    int wide;  // weight and bias in binary32
    void* y;
    int64_t ldy;
    float* mean;
    float* rstd;
};

struct Backward {
    int64_t m, d;
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const float* mean;
    const float* rstd;
    const void* weight;
    int wide;
    const void* residual;
    int64_t ldr;
    void* dx;
    int64_t lddx;
    void* dweight;
    void* dbias;
    int wide_grad;
    float* part;  // [parts][2][d]: the stripes' column sums
    int64_t parts;
};

// A workgroup per row, which is read three times: rows of any length.  Sums in
// binary64: a thread's share of a long row has many terms.
template <class T>
__global__ __launch_bounds__(kThreads) void k_norm_long(Forward a) {
    __shared__ double lds[2][kThreads / 64];
    for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x) {
        const T* const x = static_cast<const T*>(a.x) + r * a.ldx;
        T* const y = static_cast<T*>(a.y) + r * a.ldy;
        float v[kRow], w[kRow], b[kRow];
        double s = 0.0;
        for (int64_t c = threadIdx.x * kRow; c < a.d; c += kThreads * kRow) {
            load8(x + c, valid_of(a.d, c), v);
#pragma unroll
            for (int i = 0; i < kRow; ++i) s += double(v[i]);
        }
        const float mean = float(sum_block<kThreads>(s, lds[0]) / double(a.d));
        s = 0.0;
        for (int64_t c = threadIdx.x * kRow; c < a.d; c += kThreads * kRow) {
            const int valid = valid_of(a.d, c);
            load8(x + c, valid, v);
#pragma unroll
            for (int i = 0; i < kRow; ++i)
                if (i < valid) s += double((v[i] - mean) * (v[i] - mean));
        }
        const float var = float(sum_block<kThreads>(s, lds[1]) / double(a.d));
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        for (int64_t c = threadIdx.x * kRow; c < a.d; c += kThreads * kRow) {
            const int valid = valid_of(a.d, c);
            load8(x + c, valid, v);
#pragma unroll
            for (int i = 0; i < kRow; ++i) v[i] = (v[i] - mean) * rstd;
            if (a.weight) {
                load8_either<T>(a.weight, c, a.wide, valid, w);
#pragma unroll
                for (int i = 0; i < kRow; ++i) v[i] *= w[i];
            }
            if (a.bias) {
                load8_either<T>(a.bias, c, a.wide, valid, b);
#pragma unroll
                for (int i = 0; i < kRow; ++i) v[i] += b[i];
            }
            store8(y + c, valid, v);
        }
    }
}

// g = dy * weight and n = (x - mean) * rstd of 8 columns.
template <class T>
__device__ __forceinline__ void pair8(const Backward& a, int64_t r, int64_t c, int valid, float mean, float rstd,
                                      float* g, float* n) {
    float w[kRow];
    load8(static_cast<const T*>(a.dy) + r * a.lddy + c, valid, g);
    load8(static_cast<const T*>(a.x) + r * a.ldx + c, valid, n);
#pragma unroll
    for (int i = 0; i < kRow; ++i) n[i] = (n[i] - mean) * rstd;
    if (a.weight) {
        load8_either<T>(a.weight, c, a.wide, valid, w);
#pragma unroll
        for (int i = 0; i < kRow; ++i) g[i] *= w[i];
    }
}

// dx of rows of any length: a workgroup per row, which is read twice.
template <class T>
__global__ __launch_bounds__(kThreads) void k_norm_back_long(Backward a) {
    __shared__ double lds[2][kThreads / 64];
    for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float g[kRow], n[kRow], res[kRow];
        double sg = 0.0, sgn = 0.0;
        for (int64_t c = threadIdx.x * kRow; c < a.d; c += kThreads * kRow) {
            const int valid = valid_of(a.d, c);
            pair8<T>(a, r, c, valid, mean, rstd, g, n);
#pragma unroll
            for (int i = 0; i < kRow; ++i)
                if (i < valid) {
                    sg += double(g[i]);
                    sgn += double(g[i] * n[i]);
                }
        }
        const float mg = float(sum_block<kThreads>(sg, lds[0]) / double(a.d));
        const float mgn = float(sum_block<kThreads>(sgn, lds[1]) / double(a.d));
        for (int64_t c = threadIdx.x * kRow; c < a.d; c += kThreads * kRow) {
            const int valid = valid_of(a.d, c);
            pair8<T>(a, r, c, valid, mean, rstd, g, n);
            if (a.residual) load8(static_cast<const T*>(a.residual) + r * a.ldr + c, valid, res);
#pragma unroll
            for (int i = 0; i < kRow; ++i) {
                g[i] = rstd * (g[i] - mg - n[i] * mgn);
                if (a.residual) g[i] += res[i];
            }
            store8(static_cast<T*>(a.dx) + r * a.lddx + c, valid, g);
        }
    }
}

// Column sums of dy n and dy over a stripe of rows: 64 lanes of 8 columns by 4
// rows at a time.
template <class T>
__global__ __launch_bounds__(kThreads) void k_norm_columns(Backward a) {
    __shared__ float lds[3][64][2 * kRow + 1];
    const int lane = threadIdx.x & 63, y = threadIdx.x >> 6;
    const int64_t c = int64_t(blockIdx.x) * kColumns + lane * kRow;
    const int valid = valid_of(a.d, c);
    float sw[kRow] = {}, sb[kRow] = {};
    if (valid > 0)
        for (int64_t r = int64_t(blockIdx.y) * 4 + y; r < a.m; r += a.parts * 4) {
            float dy[kRow], x[kRow];
            load8(static_cast<const T*>(a.dy) + r * a.lddy + c, valid, dy);
            load8(static_cast<const T*>(a.x) + r * a.ldx + c, valid, x);
            const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
            for (int i = 0; i < kRow; ++i) {
                sw[i] += dy[i] * ((x[i] - mean) * rstd);
                sb[i] += dy[i];
            }
        }
    if (y > 0)
#pragma unroll
        for (int i = 0; i < kRow; ++i) {
            lds[y - 1][lane][i] = sw[i];
            lds[y - 1][lane][kRow + i] = sb[i];
        }
    __syncthreads();
    if (y > 0) return;
    float* const part = a.part + int64_t(blockIdx.y) * 2 * a.d;
#pragma unroll
    for (int i = 0; i < kRow; ++i) {
        for (int k = 0; k < 3; ++k) {
            sw[i] += lds[k][lane][i];
            sb[i] += lds[k][lane][kRow + i];
        }
        if (i < valid) {
            part[c + i] = sw[i];
            part[a.d + c + i] = sb[i];
        }
    }
}

// The stripes' sums joined: a workgroup per 64 columns, a wave per 16th of the
// stripes.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_join(Backward a) {
    __shared__ double lds[16][64];
    const int lane = threadIdx.x & 63, y = threadIdx.x >> 6;
    for (int64_t first = int64_t(blockIdx.x) * 64; first < 2 * a.d; first += int64_t(gridDim.x) * 64) {
        const int64_t c = first + lane;  // of dweight's columns, then dbias's
        double s = 0.0;
        if (c < 2 * a.d)
            for (int64_t p = y; p < a.parts; p += 16) s += double(a.part[p * 2 * a.d + c]);
        __syncthreads();
        lds[y][lane] = s;
        __syncthreads();
        void* const out = c < a.d ? a.dweight : a.dbias;
        if (y > 0 || c >= 2 * a.d || !out) continue;
        for (int k = 1; k < 16; ++k) s += lds[k][lane];
        const int64_t at = c < a.d ? c : c - a.d;
        if (a.wide_grad)
            static_cast<float*>(out)[at] = float(s);
        else
            static_cast<T*>(out)[at] = T(float(s));
    }
}

int64_t parts_of(int64_t m) { return std::min(kMostParts, std::max<int64_t>(cdiv(m, kPartRows), 1)); }

size_t back_bytes(int64_t m, int64_t d) { return d == 0 ? 0 : round_up(size_t(parts_of(m)) * 2 * size_t(d) * 4); }

dim3 rows_grid(int64_t m) { return dim3(unsigned(std::min(m, kMostBlocks))); }

}  // namespace

extern "C" {

int dgc_layer_norm_workspace_bytes(int64_t m, int64_t d, int32_t backward, size_t* bytes) {
    if (!bytes || !side_ok(m) || !side_ok(d) || (d > 0 && m > kMostArea / d)) return DGC_EINVAL;
    *bytes = backward ? back_bytes(m, d) : 0;
    return DGC_OK;
}

int dgc_layer_norm(const dgc_layer_norm_args* a, hipStream_t stream) {
    if (!a || !type_ok(a->type) || !side_ok(a->m) || !side_ok(a->d) || !std::isfinite(a->eps) || a->eps < 0.0 ||
        (a->weight_type != a->type && a->weight_type != DGC_FP32))
        return DGC_EINVAL;
    const int64_t m = a->m, d = a->d;
    const int size = size_of(a->type), wsize = size_of(a->weight_type);
    if (!mat_ok(a->x, a->ldx, m, d, size) || !mat_ok(a->y, a->ldy, m, d, size) ||
        !optional_vec_ok(a->weight, d, wsize) || !optional_vec_ok(a->bias, d, wsize) ||
        !optional_vec_ok(a->mean, m, 4) || !optional_vec_ok(a->rstd, m, 4))
        return DGC_EINVAL;
    if (m == 0 || d == 0) return DGC_OK;
    const Forward f{m, d, float(a->eps), a->x, a->ldx, a->weight, a->bias, a->weight_type == DGC_FP32,
                    a->y, a->ldy, a->mean, a->rstd};
    return with_type(a->type, [&](auto t) {
        k_norm_long<decltype(t)><<<rows_grid(m), kThreads, 0, stream>>>(f);
        return launched();
    });
}

int dgc_layer_norm_backward(const dgc_layer_norm_backward_args* a, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    if (!a || !type_ok(a->type) || !side_ok(a->m) || !side_ok(a->d) ||
        (a->weight_type != a->type && a->weight_type != DGC_FP32) ||
        (a->grad_type != a->type && a->grad_type != DGC_FP32))
        return DGC_EINVAL;
    const int64_t m = a->m, d = a->d;
    const int size = size_of(a->type), gsize = size_of(a->grad_type);
    if (!mat_ok(a->dy, a->lddy, m, d, size) || !mat_ok(a->x, a->ldx, m, d, size) ||
        (d > 0 && (!vec_ok(a->mean, m, 4) || !vec_ok(a->rstd, m, 4))) ||
        !optional_vec_ok(a->weight, d, size_of(a->weight_type)) || !optional_ok(a->residual, a->ldr, m, d, size) ||
        !optional_ok(a->dx, a->lddx, m, d, size) || !optional_vec_ok(a->dweight, d, gsize) ||
        !optional_vec_ok(a->dbias, d, gsize) || (d > 0 && m > kMostArea / d))
        return DGC_EINVAL;
    const bool sums = a->dweight || a->dbias;
    const int rc = space_ok(workspace, workspace_bytes, sums ? back_bytes(m, d) : 0);
    if (rc != DGC_OK) return rc;
    if (d == 0) return DGC_OK;
    const Backward b{m, d, a->dy, a->lddy, a->x, a->ldx, a->mean, a->rstd, a->weight, a->weight_type == DGC_FP32,
                     a->residual, a->ldr, a->dx, a->lddx, a->dweight, a->dbias, a->grad_type == DGC_FP32,
                     static_cast<float*>(workspace), parts_of(m)};
    return with_type(a->type, [&](auto t) {
        typedef decltype(t) T;
        // (before dx, which may be dy itself)
        if (sums) {
            k_norm_columns<T><<<dim3(unsigned(cdiv(d, kColumns)), unsigned(b.parts)), kThreads, 0, stream>>>(b);
            k_norm_join<T><<<dim3(unsigned(std::min(cdiv(2 * d, 64), kMostBlocks))), 1024, 0, stream>>>(b);
        }
        if (a->dx && m > 0) k_norm_back_long<T><<<rows_grid(m), kThreads, 0, stream>>>(b);
        return launched();
    });
}

}  // extern "C"
