// layers_tile.hpp -- matrix products of 16-bit operands with 32-bit sums, and
// what finishes an output element.
//
// All products of the layer operators are sums over k of a(m, k) * b(n, k).
// An operand is either stored with k contiguous (rows of a layer's input or
// weight) or with m (n) contiguous (every operand of a weight gradient, and
// the weight of an input gradient).  Both go through LDS tiles of 64 steps
// of k in the order they have in memory; the second kind is turned on the way
// to the registers by the transposing LDS read of gfx950, so no operand is
// ever rewritten in memory.
#pragma once

#include <hip/hip_runtime.h>

#include "launch_grid.hpp"
#include "layers.hpp"

namespace dgc {
namespace layers {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Sixteen bytes at any even address: the hardware splits what is not aligned.
struct __attribute__((packed, aligned(2), may_alias)) Bytes16 {
    u32x4 v;
};

#define DGC_LDS __attribute__((address_space(3)))

template <class T>
struct Arith;
template <>
struct Arith<__bf16> {
    typedef bf16x8 v8;
    static __device__ __forceinline__ f32x4 mma(v8 x, v8 y, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
    }
};
template <>
struct Arith<_Float16> {
    typedef fp16x8 v8;
    static __device__ __forceinline__ f32x4 mma(v8 x, v8 y, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
    }
};

constexpr int kStep = 64;  // k per LDS tile

// ------------------------------------------------------------ activations

// All are z times a share of it that lies between 0 and 1: 1 / (1 + exp(-q))
// or the normal distribution's integral.  The hardware's exp2 and reciprocal
// are off by a step or two of binary32, far less than a step of the 16-bit
// types; a finish takes a dozen instructions per element instead of the fifty
// of the correctly rounded functions.

__device__ __forceinline__ float sigmoid(float q) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(q * -1.44269504f));
}

// The integral of the normal density up to z, and exp(-z^2 / 2).  The tail
// beyond |z| is exp(-x^2) times a slow function of x = |z| / sqrt(2), here a
// polynomial of 1 / (1 + c x) without a constant: all seven numbers by a
// minimax fit of the relative error for x up to 14, weighted 30 times higher
// up to x = 1 than from 2.5 on.  Off by 6e-7 of 1, and by 3e-5 of the tail
// itself, so that gelu's small values far below 0 keep a 16-bit type's
// precision.
__device__ __forceinline__ float normal_share(float z, float& e) {
    const float x = fabsf(z) * 0.70710678f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.42687309f * x);
    e = __builtin_amdgcn_exp2f(x * x * -1.44269504f);
    const float p =
        t * (0.12072082f + t * (0.11535566f + t * (0.14152817f + t * (-0.011156623f +
             t * (0.21107882f + t * -0.077527322f)))));
    const float tail = p * e;
    return z < 0.0f ? tail : 1.0f - tail;
}

// gelu_tanh: (1 + tanh(q)) / 2 = sigmoid(2 q)
__device__ __forceinline__ float tanh_twice(float z) {
    return 1.59576912f * (z + 0.044715f * z * z * z);
}

__device__ __forceinline__ float act_value(int act, float z) {
    float e;
    switch (act) {
        case DGC_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
        case DGC_ACT_SILU: return z * sigmoid(z);
        case DGC_ACT_GELU: return z * normal_share(z, e);
        case DGC_ACT_GELU_TANH: return z * sigmoid(tanh_twice(z));
        default: return z;
    }
}

// act(z) and act'(z) from shared parts.
__device__ __forceinline__ void act_pair(int act, float z, float& value, float& slope) {
    switch (act) {
        case DGC_ACT_RELU:
            value = z > 0.0f ? z : (z != z ? z : 0.0f);
            slope = z > 0.0f ? 1.0f : 0.0f;
            break;
        case DGC_ACT_SILU: {
            const float p = sigmoid(z);
            value = z * p;
            slope = p * (1.0f + z * (1.0f - p));
            break;
        }
        case DGC_ACT_GELU: {
            float e;
            const float p = normal_share(z, e);
            value = z * p;
            slope = p + z * 0.39894228f * e;
            break;
        }
        case DGC_ACT_GELU_TANH: {
            const float p = sigmoid(tanh_twice(z));
            value = z * p;
            // bounded, so that a 0 before it makes it 0 for the largest z too
            const float square = fminf(z * z, 1e30f);
            slope = p + value * (1.0f - p) * 1.59576912f * (1.0f + 0.134145f * square);
            break;
        }
        default: value = z; slope = 1.0f;
    }
}

// ----------------------------------------------------- rows of few elements

// C consecutive elements of a row, of which the first `valid` exist.
// ONCE: past the caches, for what is not read again soon.
template <class T, int C, bool ONCE = false>
__device__ __forceinline__ void load_row(const T* p, int valid, float* v) {
    if (valid >= C) {
        T t[C];
        if constexpr (C % 8 == 0) {
            typedef u32x4 V __attribute__((aligned(2), may_alias));
#pragma unroll
            for (int i = 0; i < C / 8; ++i) {
                const V* q = reinterpret_cast<const V*>(p + 8 * i);
                const u32x4 w = ONCE ? __builtin_nontemporal_load(q) : *q;
                __builtin_memcpy(t + 8 * i, &w, 16);
            }
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            typedef u32x2 V __attribute__((aligned(2), may_alias));
            static_assert(C == 4, "rows of 4 or of eights");
            const V* q = reinterpret_cast<const V*>(p);
            const u32x2 w = ONCE ? __builtin_nontemporal_load(q) : *q;
            __builtin_memcpy(t, &w, 8);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = float(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = i < valid ? float(p[i]) : 0.0f;
    }
}

template <class T, int C>
__device__ __forceinline__ void store_row(T* p, int valid, const float* v) {
    if (valid >= C) {
        T t[C];
#pragma unroll
        for (int i = 0; i < C; ++i) t[i] = T(v[i]);  // to nearest, ties to even: the one rounding
        if constexpr (C % 8 == 0) {
#pragma unroll
            for (int i = 0; i < C / 8; ++i)
                *reinterpret_cast<Bytes16*>(p + 8 * i) =
                    *reinterpret_cast<const Bytes16*>(t + 8 * i);
        } else {
            struct __attribute__((packed, aligned(2), may_alias)) B { uint64_t v; };
            *reinterpret_cast<B*>(p) = *reinterpret_cast<const B*>(t);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < valid) p[i] = T(v[i]);
    }
}

template <int C>
__device__ __forceinline__ void store_wide(float* p, int valid, const float* v) {
    struct __attribute__((packed, aligned(4), may_alias)) B { f32x4 v; };
    if (valid >= C) {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
            B b;
            b.v = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            *reinterpret_cast<B*>(p + 4 * i) = b;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < valid) p[i] = v[i];
    }
}

// Finish C consecutive elements (m, n..n+C-1) of output `z` of a product, of
// which `valid` exist.  v holds the 32-bit sums, v2 the second product's
// (kPair); bias and residual are used if the finish has them.
template <class T, bool PAIR, int C>
__device__ __forceinline__ void finish_row(const Finish& f, int z, int64_t m, int64_t n,
                                           int valid, float* v, float* v2, const float* bias,
                                           const float* residual) {
    if constexpr (PAIR) {
        if (f.pre[0]) store_row<T, C>(static_cast<T*>(f.pre[0]) + m * f.ldp[0] + n, valid, v);
        if (f.pre[1]) store_row<T, C>(static_cast<T*>(f.pre[1]) + m * f.ldp[1] + n, valid, v2);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = act_value(f.act, v[i]) * v2[i];
        store_row<T, C>(static_cast<T*>(f.out[0]) + m * f.ldo + n, valid, v);
    } else if (f.wide) {
        store_wide<C>(static_cast<float*>(f.out[z]) + m * (z ? f.ldo2 : f.ldo) + n, valid, v);
    } else {
        if (f.bias) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += bias[i];
        }
        if (f.pre[0]) store_row<T, C>(static_cast<T*>(f.pre[0]) + m * f.ldp[0] + n, valid, v);
        if (f.act != DGC_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = act_value(f.act, v[i]);
        }
        if (f.residual) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += residual[i];
        }
        store_row<T, C>(static_cast<T*>(f.out[z]) + m * (z ? f.ldo2 : f.ldo) + n, valid, v);
    }
}

// The same with the bias and residual read here.
template <class T, bool PAIR, int C>
__device__ __forceinline__ void finish_one(const Finish& f, int z, int64_t m, int64_t n,
                                           int64_t N, float* v, float* v2) {
    const int valid = N - n < C ? int(N - n) : C;
    if (valid <= 0) return;
    float bias[C], residual[C];
    if (!PAIR && f.bias) load_row<T, C>(static_cast<const T*>(f.bias) + n, valid, bias);
    if (!PAIR && f.residual)
        load_row<T, C>(static_cast<const T*>(f.residual) + m * f.ldr + n, valid, residual);
    finish_row<T, PAIR, C>(f, z, m, n, valid, v, v2, bias, residual);
}

// ------------------------------------------------------------- LDS layouts
//
// One wave reads 16-byte pieces (8 steps of k) of 16 rows at once, so rows
// 128 bytes apart would all meet in the same banks: the piece index is
// XORed with three bits that differ between those rows.
//   k contiguous:   [R rows][64], piece c of row r at c ^ key(r)
//   m/n contiguous: [64 rows of k][R], 32-byte block b of row k at
//                   b ^ key(k): the transposing read takes 4 rows x 32
//                   bytes per 16 lanes, 16 rows of k per instruction

// Rows of the n side are dealt to the matrix instructions so that a lane ends
// up with 4 * NT consecutive columns of its row: wide stores, whole lines.
template <int NT>
__device__ __forceinline__ int n_row(int i, int j) {
    return (i >> 2) * (4 * NT) + j * 4 + (i & 3);
}

template <int NT, bool NSIDE>
__device__ __forceinline__ int row_key(int r) {
    if constexpr (NSIDE) {
        constexpr int shift = NT == 4 ? 4 : NT == 2 ? 3 : 2;
        return (r & 3) | (((r >> shift) & 1) << 2);
    } else {
        return r & 7;
    }
}

template <int R>
__device__ __forceinline__ int k_key(int k) {
    return ((k & 3) | (((k >> 3) & 3) << 2)) & (R / 16 - 1);
}

// Element offset of 16-byte piece `piece` of row (TR: step of k) `row`.
template <int R, int NT, bool TR, bool NSIDE>
__device__ __forceinline__ int piece_at(int row, int piece) {
    if constexpr (TR)
        return row * R + ((((piece >> 1) ^ k_key<R>(row)) << 1) | (piece & 1)) * 8;
    else
        return row * kStep + (piece ^ row_key<NT, NSIDE>(row)) * 8;
}

// Where a lane's fragments lie in a region, and their reads.
template <class T, bool TR, int NT, bool NSIDE, int R>
struct Frags {
    typedef typename Arith<T>::v8 v8;
    int frag[TR ? NT : 2];

    // base: the wave's first row (column) in the region
    __device__ __forceinline__ void init(int lane, int base) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (TR) {
            const int kk = g * 8 + (i >> 2);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                frag[j] = kk * R + ((((base >> 4) + j) ^ k_key<R>(kk)) << 4) + (i & 3) * 4;
        } else {
            const int fr = base + (NSIDE ? n_row<NT>(i, 0) : i);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                frag[s] = fr * kStep + (((s * 4 + g) ^ row_key<NT, NSIDE>(fr)) << 3);
        }
    }

    // Fragment j, steps 32 s .. 32 s + 31, of a region.
    __device__ __forceinline__ v8 get(const T* lds, int j, int s) const {
        if constexpr (TR) {
            union { s16x4 h[2]; v8 v; } u;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (DGC_LDS s16x4*)(const_cast<T*>(lds + frag[j] + s * 32 * R + h * 4 * R)));
            return u.v;
        } else {
            return *reinterpret_cast<const v8*>(lds + frag[s] + j * (NSIDE ? 4 : 16) * kStep);
        }
    }
};

// --------------------------------------------------------------- the tiles

// One product's tiles.
struct TileArgs {
    const void* a[2];
    const void* b[2];
    int64_t lda[2], ldb[2];
    int64_t M, N, K;
    int64_t mt, nt;        // tiles over m and n
    int64_t per;           // steps of 64 per workgroup along the long axis
    int32_t splits, parts, outs;  // outs: outputs of kDw, else 1
    int32_t pieces;        // of a, `low` elements apart
    uint32_t inverse;      // 2^31 / pieces, rounded up
    int32_t fold;          // rows of dz in two pieces (Product), or 0
    int64_t low;
    float* part;           // the splits' sums, or null
    Finish fin;
};

// How many rows a has (kDw: columns).
template <int FORM>
__device__ __forceinline__ int64_t a_rows(const TileArgs& A) {
    return FORM == kDx && A.fold ? 2 * A.fold : A.M;
}

// How many steps of 64 a sum takes.  SPLIT: of an `a` in pieces (kDx, kDw).
template <int FORM, bool SPLIT, class I>
__device__ __forceinline__ I all_steps(const TileArgs& A, I ksteps) {
    return ksteps * (SPLIT ? A.pieces : 1) * (FORM == kDx ? A.parts : 1);
}

// Step t of a sum: which of kDx's terms, which piece of a, and the first k.  The
// pieces of one step of k follow each other, so that the second finds the other
// operand in the die's L2.  (A template: the arithmetic costs 5% of 8192 x 8192 x
// 4096, where a is whole; a branch among the loads cost 25%.)
struct StepAt {
    int term;
    int64_t piece, k0;  // piece: elements into a
};

template <int FORM, bool SPLIT, class I>
__device__ __forceinline__ StepAt step_at(const TileArgs& A, I t, I ksteps) {
    const I all = SPLIT ? ksteps * A.pieces : ksteps;
    const int term = FORM == kDx && t >= all ? 1 : 0;
    const I u = t - term * all;
    if constexpr (!SPLIT) return {term, 0, int64_t(u) * kStep};
    // u / pieces without a branch: exact below 2^30 steps
    const I k = I((uint64_t(u) * 2 * A.inverse) >> 32);
    const int piece = int(u - k * A.pieces);
    return {term, (piece > 0 ? A.low : 0) + (piece > 1 ? A.low : 0), int64_t(k) * kStep};
}

// Where workgroup `id` of a product works.  Workgroups go to the 8 dies in
// turn, each with an L2 of its own: die x takes the x-th eighth of the splits,
// outputs and tiles, and walks the tiles in bands of 8 rows, so that what runs
// there at once shares operands.
struct Spot {
    int split, z;
    int64_t tm, tn;
};

// A product's workgroups.
template <int FORM>
__device__ __forceinline__ int64_t all_blocks(const TileArgs& A) {
    return A.mt * A.nt * (FORM == kDw ? A.outs : 1) * A.splits;
}

template <int FORM>
__device__ __forceinline__ Spot spot(const TileArgs& A, int id) {
    const int mt = int(A.mt), nt = int(A.nt), tiles = mt * nt;
    const int outs = FORM == kDw ? A.outs : 1, all = tiles * outs * A.splits;
    const int x = id % 8, rem = all % 8;
    int t = x * (all / 8) + (x < rem ? x : rem) + id / 8;
    Spot s;
    s.split = t / (tiles * outs);
    t -= s.split * tiles * outs;
    s.z = FORM == kDw ? t / tiles : 0;
    t -= s.z * tiles;
    constexpr int kBand = 8;
    const int band = t / (kBand * nt), in = t - band * kBand * nt;
    const int high = mt - band * kBand < kBand ? mt - band * kBand : kBand;
    s.tm = band * kBand + in % high;
    s.tn = in / high;
    return s;
}

// A workgroup's outputs leave through LDS: rows of COLS columns in binary32
// (kPair: the first product's columns, then the second's), so that the lanes
// that finish a row hold 8 consecutive columns each and store whole lines, in
// one short loop.  Columns lie in fours, XORed with the row: lanes that write
// a matrix tile hold the same columns of 16 rows.
__device__ __forceinline__ int out_at(int r, int col4) { return (col4 ^ ((r & 7) << 1)) * 4; }

// Finishes rows 0 .. ROWS - 1, outputs m0 + row, n0 + column.
//   at(r): where row r lies; groups: so many sums of every output, `stride`
//   floats apart, are added in that order
template <class T, int FORM, int ROWS, int COLS, int THREADS, class At>
__device__ __forceinline__ void put_rows(const TileArgs& A, int split, int z, int64_t m0,
                                         int64_t n0, int groups, int stride, At at) {
    constexpr bool PAIR = FORM == kPair;
    constexpr int kCols = PAIR ? COLS / 2 : COLS;
    constexpr int kLanes = kCols / 8, kStepRows = THREADS / kLanes;
    constexpr int kSteps = (ROWS + kStepRows - 1) / kStepRows;
    constexpr int kAhead = kSteps < 4 ? kSteps : 4;  // rows whose loads are under way together
    const int c = threadIdx.x % kLanes;
    const int64_t n = n0 + c * 8;
    const int valid = A.N - n < 8 ? int(A.N - n) : 8;
    if (valid <= 0) return;
    const Finish& f = A.fin;
    float bias[8];
    if (!PAIR && f.bias) load_row<T, 8>(static_cast<const T*>(f.bias) + n, valid, bias);
    const int rows = A.M - m0 < ROWS ? int(A.M - m0) : ROWS;
    const int fold = FORM == kDx ? A.fold : 0;
    constexpr bool BACK = FORM == kDx || FORM == kDw;
    const float unscale = BACK && f.unscale ? *f.unscale : 1.0f;
    const auto sum = [&](int r, int col4) {
        const float* p = at(r) + out_at(r, col4);
        f32x4 t = *reinterpret_cast<const f32x4*>(p);
        for (int w = 1; w < groups; ++w) t += *reinterpret_cast<const f32x4*>(p + w * stride);
        return t;
    };
#pragma unroll 1
    for (int first = threadIdx.x / kLanes; first < rows; first += kAhead * kStepRows) {
        float residual[kAhead][8];
        if (!PAIR && f.residual) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (first + u * kStepRows < rows)
                    load_row<T, 8>(static_cast<const T*>(f.residual) +
                                       (m0 + first + u * kStepRows) * f.ldr + n, valid,
                                   residual[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = first + u * kStepRows;
            if (r >= rows) break;
            float v[8], v2[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x4 t = sum(r, 2 * c + q), t2 = {0, 0, 0, 0};
                if (PAIR) t2 = sum(r, 2 * c + q + COLS / 8);
                if (fold) t += sum(r + fold, 2 * c + q);
                *reinterpret_cast<f32x4*>(v + 4 * q) = t;
                *reinterpret_cast<f32x4*>(v2 + 4 * q) = t2;
            }
            const int64_t m = m0 + r;
            if (A.part) {
                const int planes = PAIR ? 2 : A.outs;
                float* o = A.part + (((int64_t(split) * planes + z) * A.M + m) * A.N + n);
                store_wide<8>(o, valid, v);
                if (PAIR) store_wide<8>(o + A.M * A.N, valid, v2);
            } else {
                if (BACK) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= unscale;
                }
                finish_row<T, PAIR, 8>(f, z, m, n, valid, v, v2, bias, residual[u]);
            }
        }
    }
}

// Columns that a lane holds of matrix tile j of the NT from column `col` on
// (dealt by n_row<NT>; TR: side by side), into row r of that LDS.
template <int NT, bool TR>
__device__ __forceinline__ void put_tile(float* row, int r, int col, int j, int lane, f32x4 v) {
    const int g = lane >> 4;
    const int c4 = col / 4 + (TR ? j * 4 + g : g * NT + j);
    *reinterpret_cast<f32x4*>(row + out_at(r, c4)) = v;
}

// The sums of all splits, added in their order, then finished.  One thread
// per 4 columns of a row.
template <class T, bool PAIR>
__global__ __launch_bounds__(64) void k_join(TileArgs A) {
    const int64_t groups = (A.N + 3) / 4, z_count = A.outs;
    int64_t id = block_number() * 64 + threadIdx.x;
    if (id >= groups * A.M * z_count) return;
    const int z = int(id / (groups * A.M));
    id -= z * groups * A.M;
    const int64_t m = id / groups, n = (id - m * groups) * 4;
    const int valid = A.N - n < 4 ? int(A.N - n) : 4;
    const int planes = PAIR ? 2 : int(A.outs);
    const int64_t plane = A.M * A.N;
    float v[4] = {0, 0, 0, 0}, v2[4] = {0, 0, 0, 0};
    struct __attribute__((packed, aligned(4), may_alias)) B { f32x4 v; };
    constexpr int P = PAIR ? 2 : 1;
    for (int s0 = 0; s0 < A.splits; s0 += 8) {  // 8 splits' loads are under way together
        f32x4 t[8][P];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            if (s0 + s >= A.splits) break;
            const float* p = A.part + (int64_t(s0 + s) * planes + z) * plane + m * A.N + n;
#pragma unroll
            for (int w = 0; w < P; ++w, p += plane) {
                if (valid == 4)
                    t[s][w] = reinterpret_cast<const B*>(p)->v;
                else
                    for (int e = 0; e < 4; ++e) t[s][w][e] = e < valid ? p[e] : 0.0f;
            }
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            if (s0 + s >= A.splits) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] += t[s][0][e];
                v2[e] += t[s][P - 1][e];
            }
        }
    }
    if (!PAIR && A.fin.unscale) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= *A.fin.unscale;
    }
    finish_one<T, PAIR, 4>(A.fin, z, m, n, A.N, v, v2);
}

}  // namespace layers
}  // namespace dgc
