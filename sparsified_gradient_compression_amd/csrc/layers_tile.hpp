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

__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case DGC_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
        case DGC_ACT_SILU: return z / (1.0f + expf(-z));
        case DGC_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
        case DGC_ACT_GELU_TANH:
            return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
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
            const float s = 1.0f / (1.0f + expf(-z));
            value = z * s;
            slope = s * (1.0f + z * (1.0f - s));
            break;
        }
        case DGC_ACT_GELU: {
            const float c = 0.5f * (1.0f + erff(z * 0.70710678f));
            value = z * c;
            slope = c + z * 0.39894228f * expf(-0.5f * z * z);
            break;
        }
        case DGC_ACT_GELU_TANH: {
            const float t = tanhf(0.79788456f * (z + 0.044715f * z * z * z));
            value = 0.5f * z * (1.0f + t);
            slope = 0.5f * (1.0f + t) +
                    0.5f * z * (1.0f - t * t) * 0.79788456f * (1.0f + 0.134145f * z * z);
            break;
        }
        default: value = z; slope = 1.0f;
    }
}

// ----------------------------------------------------- rows of few elements

// C consecutive elements of a row, of which the first `valid` exist.
template <class T, int C>
__device__ __forceinline__ void load_row(const T* p, int valid, float* v) {
    if (valid >= C) {
        T t[C];
        if constexpr (C % 8 == 0) {
#pragma unroll
            for (int i = 0; i < C / 8; ++i)
                *reinterpret_cast<Bytes16*>(t + 8 * i) =
                    *reinterpret_cast<const Bytes16*>(p + 8 * i);
        } else {
            struct __attribute__((packed, aligned(2), may_alias)) B { uint64_t v; };
            static_assert(C == 4, "rows of 4 or of eights");
            *reinterpret_cast<B*>(t) = *reinterpret_cast<const B*>(p);
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

// Finish C consecutive elements (m, n..n+C-1) of output `z` of a product.
// v holds the 32-bit sums, v2 the second product's (kPair).
template <class T, bool PAIR, int C>
__device__ __forceinline__ void finish_row(const Finish& f, int z, int64_t m, int64_t n,
                                           int64_t N, float* v, float* v2) {
    const int valid = N - n < C ? int(N - n) : C;
    if (valid <= 0) return;
    if constexpr (PAIR) {
        if (f.pre[0]) store_row<T, C>(static_cast<T*>(f.pre[0]) + m * f.ldp[0] + n, valid, v);
        if (f.pre[1]) store_row<T, C>(static_cast<T*>(f.pre[1]) + m * f.ldp[1] + n, valid, v2);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = act_value(f.act, v[i]) * v2[i];
        store_row<T, C>(static_cast<T*>(f.out[0]) + m * f.ldo + n, valid, v);
    } else if (f.wide) {
        store_wide<C>(static_cast<float*>(f.out[z]) + m * (z ? f.ldo2 : f.ldo) + n, valid, v);
    } else {
        float t[C];
        if (f.bias) {
            load_row<T, C>(static_cast<const T*>(f.bias) + n, valid, t);
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += t[i];
        }
        if (f.pre[0]) store_row<T, C>(static_cast<T*>(f.pre[0]) + m * f.ldp[0] + n, valid, v);
        if (f.act != DGC_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = act_value(f.act, v[i]);
        }
        if (f.residual) {
            load_row<T, C>(static_cast<const T*>(f.residual) + m * f.ldr + n, valid, t);
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += t[i];
        }
        store_row<T, C>(static_cast<T*>(f.out[z]) + m * (z ? f.ldo2 : f.ldo) + n, valid, v);
    }
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

// Element offset of the 16-byte piece with index c of a tile's load.
//   TR false: row c / 8, piece c % 8;  TR true: k c / (R/8), piece c % (R/8)
template <int R, int NT, bool TR, bool NSIDE>
__device__ __forceinline__ int piece_at(int row, int piece) {
    if constexpr (TR)
        return row * R + ((((piece >> 1) ^ k_key<R>(row)) << 1) | (piece & 1)) * 8;
    else
        return row * kStep + (piece ^ row_key<NT, NSIDE>(row)) * 8;
}

// Eight elements of row `row` from column `col` of a matrix with `rows` rows
// and `cols` columns; what lies outside reads as zero.
template <class T>
__device__ __forceinline__ u32x4 guarded(const T* p, int64_t ld, int64_t row, int64_t col,
                                         int64_t rows, int64_t cols) {
    u32x4 r = {0, 0, 0, 0};
    if (row >= rows || col >= cols) return r;
    const T* q = p + row * ld + col;
    if (col + 8 <= cols) return reinterpret_cast<const Bytes16*>(q)->v;
    uint16_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        t[i] = col + i < cols ? reinterpret_cast<const uint16_t*>(q)[i] : uint16_t(0);
    __builtin_memcpy(&r, t, 16);
    return r;
}

// --------------------------------------------------------------- the tiles

struct TileArgs {
    const void* a[2];
    const void* b[2];
    int64_t lda[2], ldb[2];
    int64_t M, N, K;
    int64_t mt, nt;        // tiles over m and n
    int64_t per;           // steps of 64 per workgroup along the long axis
    int32_t splits, parts, outs;  // outs: outputs of kDw, else 1
    float* part;           // the splits' sums, or null
    Finish fin;
};

// Where workgroup `id` works.  Workgroups go to the 8 dies in turn, each
// with an L2 of its own: die x takes the x-th eighth of the tiles, and walks
// them in bands of 8 rows, so that what runs there at once shares operands.
__device__ __forceinline__ void place(int64_t id, int64_t mt, int64_t nt, int64_t& tm,
                                      int64_t& tn) {
    const int64_t total = mt * nt, per = total / 8, rem = total % 8;
    const int64_t x = id % 8, i = id / 8;
    const int64_t t = x * per + (x < rem ? x : rem) + i;
    constexpr int64_t kBand = 8;
    const int64_t band = t / (kBand * nt), in = t - band * kBand * nt;
    const int64_t high = mt - band * kBand < kBand ? mt - band * kBand : kBand;
    tm = band * kBand + in % high;
    tn = in / high;
}

// Fragment reads of one wave from a tile in LDS.
template <class T, int R, int NT, bool TR, bool NSIDE>
struct Frag {
    typedef typename Arith<T>::v8 v8;
    // tile j of 16 rows (or columns) from `base`, k from 32 * s
    static __device__ __forceinline__ v8 get(const T* lds, int base, int j, int s, int lane) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (TR) {
            const int k = s * 32 + g * 8 + (i >> 2);
            const int blk = (base >> 4) + j;
            union { s16x4 h[2]; v8 v; } u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const T* p = lds + (k + 4 * h) * R + ((blk ^ k_key<R>(k + 4 * h)) << 4) +
                             (i & 3) * 4;
                u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (DGC_LDS s16x4*)(const_cast<T*>(p)));
            }
            return u.v;
        } else {
            const int r = base + (NSIDE ? n_row<NT>(i, j) : j * 16 + i);
            return *reinterpret_cast<const v8*>(
                lds + r * kStep + (((s * 4 + g) ^ row_key<NT, NSIDE>(r)) << 3));
        }
    }
};

// A wave's outputs leave through its own LDS (MT * 16 rows of NTW * 16
// columns in binary32, NTW = 2 or 4): what finishes an element is then one
// short loop whose lanes hold 8 consecutive columns each, instead of the
// whole of it unrolled over every register.
//   columns of the first and the second half of the wave's start at n0, n1
//   (kPair: of the first and the second product, the same ones)
//   groups: so many waves hold sums of the same outputs, `stride` floats
//   apart, to be added in that order; each finishes its share of the rows
template <class T, int FORM, int MT, int NTW>
__device__ __forceinline__ void put_wave(const TileArgs& A, int split, int z, int64_t m0,
                                         int64_t n0, int64_t n1, int lane, const float* lds,
                                         int group, int groups, int stride) {
    constexpr bool PAIR = FORM == kPair;
    constexpr int W = NTW * 16;                     // columns in LDS
    constexpr int kLanes = PAIR ? W / 16 : W / 8;   // lanes per row
    constexpr int kRows = 64 / kLanes;
    const int c = lane % kLanes;
    const int64_t n = c * 8 < W / 2 ? n0 + c * 8 : n1 + c * 8 - W / 2;
#pragma unroll 1
    for (int r = group * kRows + lane / kLanes; r < MT * 16; r += kRows * groups) {
        const int64_t m = m0 + r;
        if (m >= A.M) break;
        float v[8], v2[8];
        const int key = (r & (W / 8 - 1)) << 1;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float* p = lds + r * W + ((2 * c + q) ^ key) * 4;
            const float* p2 = lds + r * W + ((2 * c + q + W / 8) ^ key) * 4;
            f32x4 t = *reinterpret_cast<const f32x4*>(p), t2 = {0, 0, 0, 0};
            if (PAIR) t2 = *reinterpret_cast<const f32x4*>(p2);
            for (int w = 1; w < groups; ++w) {
                t += *reinterpret_cast<const f32x4*>(p + w * stride);
                if (PAIR) t2 += *reinterpret_cast<const f32x4*>(p2 + w * stride);
            }
            *reinterpret_cast<f32x4*>(v + 4 * q) = t;
            *reinterpret_cast<f32x4*>(v2 + 4 * q) = t2;
        }
        const int valid = A.N - n < 8 ? int(A.N - n) : 8;
        if (valid <= 0) continue;
        if (A.part) {
            const int planes = PAIR ? 2 : A.outs;
            float* o = A.part + (((int64_t(split) * planes + z) * A.M + m) * A.N + n);
            store_wide<8>(o, valid, v);
            if (PAIR) store_wide<8>(o + A.M * A.N, valid, v2);
        } else {
            finish_row<T, PAIR, 8>(A.fin, z, m, n, A.N, v, v2);
        }
    }
}

// Matrix tile j (of NT that share their columns by n_row<NT>, or TR: that lie
// side by side) of rows 16 mt, at column `col`, into that LDS.
template <int NTW, int NT, bool TR>
__device__ __forceinline__ void put_tile(float* lds, int mt, int col, int j, int lane, f32x4 v) {
    constexpr int W = NTW * 16;
    const int r = mt * 16 + (lane & 15), g = lane >> 4;
    const int c4 = col / 4 + (TR ? j * 4 + g : g * NT + j);
    *reinterpret_cast<f32x4*>(lds + r * W + (c4 ^ ((r & (W / 8 - 1)) << 1)) * 4) = v;
}

// BM x BN outputs per workgroup of WM x WN waves.  LDS holds two tiles of
// each side; the next one travels through registers while this one is used.
template <class T, int FORM, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void k_tile(TileArgs A) {
    constexpr bool PAIR = FORM == kPair, ATR = FORM == kDw, BTR = FORM == kDx || FORM == kDw;
    constexpr int kThreads = WM * WN * 64;
    constexpr int MT = BM / WM / 16, NTW = BN / WN / 16;  // 16 x 16 tiles of a wave
    constexpr int NT = PAIR ? NTW / 2 : NTW;              // ... of one product
    constexpr int kPiecesA = BM * 8 / kThreads, kPiecesB = BN * 8 / kThreads;
    typedef typename Arith<T>::v8 v8;
    __shared__ __align__(16) T smem[2 * (BM + BN) * kStep];
    T (&sa)[2][BM * kStep] = *reinterpret_cast<T (*)[2][BM * kStep]>(smem);
    T (&sb)[2][BN * kStep] = *reinterpret_cast<T (*)[2][BN * kStep]>(smem + 2 * BM * kStep);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;

    const int64_t tiles = A.mt * A.nt;
    int64_t id = blockIdx.x;
    const int split = int(id / (tiles * (FORM == kDw ? A.parts : 1)));
    id -= split * (tiles * (FORM == kDw ? A.parts : 1));
    const int z = FORM == kDw ? int(id / tiles) : 0;
    id -= z * tiles;
    int64_t tm, tn;
    place(id, A.mt, A.nt, tm, tn);
    const int64_t m0 = tm * BM, n0 = tn * (PAIR ? BN / 2 : BN);

    const int64_t ksteps = (A.K + kStep - 1) / kStep;
    const int64_t total = ksteps * (FORM == kDx ? A.parts : 1);
    const int64_t first = split * A.per;
    const int64_t last = first + A.per < total ? first + A.per : total;

    u32x4 ra[kPiecesA], rb[kPiecesB];
    auto fetch = [&](int64_t t) {
        const int seg = FORM == kDx && t >= ksteps ? 1 : 0;
        const int64_t k0 = (t - seg * ksteps) * kStep;
        const T* pa = static_cast<const T*>(A.a[FORM == kDw ? z : seg]);
        const int64_t lda = A.lda[FORM == kDw ? z : seg];
#pragma unroll
        for (int i = 0; i < kPiecesA; ++i) {
            const int c = tid + i * kThreads;
            ra[i] = ATR ? guarded(pa, lda, k0 + c / (BM / 8), m0 + c % (BM / 8) * 8, A.K, A.M)
                        : guarded(pa, lda, m0 + c / 8, k0 + c % 8 * 8, A.M, A.K);
        }
#pragma unroll
        for (int i = 0; i < kPiecesB; ++i) {
            const int c = tid + i * kThreads;
            if constexpr (PAIR) {  // rows of the first half are the gate's
                const int r = c / 8, w = r >= BN / 2;
                rb[i] = guarded(static_cast<const T*>(A.b[w]), A.ldb[w], n0 + r - w * (BN / 2),
                                k0 + c % 8 * 8, A.N, A.K);
            } else {
                const T* pb = static_cast<const T*>(A.b[seg]);
                rb[i] = BTR ? guarded(pb, A.ldb[seg], k0 + c / (BN / 8), n0 + c % (BN / 8) * 8,
                                      A.K, A.N)
                            : guarded(pb, A.ldb[seg], n0 + c / 8, k0 + c % 8 * 8, A.N, A.K);
            }
        }
    };
    auto place_lds = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kPiecesA; ++i) {
            const int c = tid + i * kThreads;
            constexpr int kPer = ATR ? BM / 8 : 8;
            *reinterpret_cast<u32x4*>(&sa[buf][piece_at<BM, 4, ATR, false>(c / kPer, c % kPer)]) =
                ra[i];
        }
#pragma unroll
        for (int i = 0; i < kPiecesB; ++i) {
            const int c = tid + i * kThreads;
            constexpr int kPer = BTR ? BN / 8 : 8;
            *reinterpret_cast<u32x4*>(&sb[buf][piece_at<BN, NT, BTR, true>(c / kPer, c % kPer)]) =
                rb[i];
        }
    };

    f32x4 acc[MT][NTW];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NTW; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    if (first < last) {
        fetch(first);
        place_lds(0);
    }
    for (int64_t t = first; t < last; ++t) {
        const int buf = int(t - first) & 1;
        // tile t is in LDS, and nobody reads the other buffer any more
        __syncthreads();
        if (t + 1 < last) fetch(t + 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v8 fb[NTW], fa[MT];
#pragma unroll
            for (int j = 0; j < NTW; ++j) {
                const int base = PAIR ? (j >= NT ? BN / 2 : 0) + wn * NT * 16 : wn * NTW * 16;
                fb[j] = Frag<T, BN, NT, BTR, true>::get(sb[buf], base, PAIR ? j % NT : j, s, lane);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
                fa[i] = Frag<T, BM, 4, ATR, false>::get(sa[buf], wm * MT * 16, i, s, lane);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NTW; ++j) acc[i][j] = Arith<T>::mma(fb[j], fa[i], acc[i][j]);
        }
        if (t + 1 < last) place_lds(buf ^ 1);
    }

    __syncthreads();
    constexpr int kOwn = MT * NTW * 256;  // outputs of a wave
    static_assert(WM * WN * kOwn * 4 <= int(sizeof(sa) + sizeof(sb)), "outputs fit the tiles' LDS");
    float* out = reinterpret_cast<float*>(smem) + wave * kOwn;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NTW; ++j)
            put_tile<NTW, NT, BTR>(out, mt, j / NT * NT * 16, j % NT, lane, acc[mt][j]);
    const int64_t mw = m0 + wm * MT * 16, nw = n0 + wn * NT * 16;
    put_wave<T, FORM, MT, NTW>(A, split, z, mw, nw, PAIR ? nw : nw + NTW * 8, lane, out, 0, 1,
                               0);
}

// The sums of all splits, added in their order, then finished.  One thread
// per 4 columns of a row.
template <class T, bool PAIR>
__global__ __launch_bounds__(256) void k_join(TileArgs A) {
    const int64_t groups = (A.N + 3) / 4, z_count = A.outs;
    int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (id >= groups * A.M * z_count) return;
    const int z = int(id / (groups * A.M));
    id -= z * groups * A.M;
    const int64_t m = id / groups, n = (id - m * groups) * 4;
    const int valid = A.N - n < 4 ? int(A.N - n) : 4;
    const int planes = PAIR ? 2 : int(A.outs);
    const int64_t plane = A.M * A.N;
    float v[4] = {0, 0, 0, 0}, v2[4] = {0, 0, 0, 0};
    struct __attribute__((packed, aligned(4), may_alias)) B { f32x4 v; };
    for (int s = 0; s < A.splits; ++s) {
        const float* p = A.part + (int64_t(s) * planes + z) * plane + m * A.N + n;
#pragma unroll
        for (int w = 0; w < (PAIR ? 2 : 1); ++w, p += plane) {
            float* o = w ? v2 : v;
            if (valid == 4) {
                const f32x4 t = reinterpret_cast<const B*>(p)->v;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += t[e];
            } else {
                for (int e = 0; e < valid; ++e) o[e] += p[e];
            }
        }
    }
    finish_row<T, PAIR, 4>(A.fin, z, m, n, A.N, v, v2);
}

}  // namespace layers
}  // namespace dgc
