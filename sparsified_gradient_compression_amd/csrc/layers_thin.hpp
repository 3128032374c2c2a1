// layers_thin.hpp -- layer outputs of up to 32 rows: bound by reading the
// weight once.
//
// A workgroup takes 16 rows of the weight (16 columns of the output; of both
// weights for a gated block) and all rows of x.  Its eight waves split k; each
// reads its pieces of the weight from memory straight into the registers the
// matrix instruction takes them from, four steps of 64 ahead, and x from the
// caches.  The waves' sums meet in LDS and are finished there, so nothing
// passes through memory and there is one launch.  Any strides and alignment.
// 1 x 4096, k 4096: 8.2 us of the kernel (traced: 7.9 to 8.8), 4.1 TB/s; 3 x
// 8192, k 2048, both weights of a gated block: 12.6 us, 5.3 TB/s.
#pragma once

#include "layers_tile.hpp"

namespace dgc {
namespace layers {

template <class T, bool PAIR, int MT>
__global__ __launch_bounds__(512) void k_thin(TileArgs A) {
    typedef typename Arith<T>::v8 v8;
    constexpr int P = PAIR ? 2 : 1, kWaves = 8, kAhead = 4;
    // [wave][product][row][16 columns], columns in fours XORed with the row
    __shared__ __align__(16) float sums[kWaves][P][MT * 16][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = block_number() * 16;
    // rows that do not exist repeat the last one; their sums are not stored
    const int64_t n = n0 + i < A.N ? n0 + i : A.N - 1;
    const T* w[P];
    const T* x[MT];
#pragma unroll
    for (int p = 0; p < P; ++p) w[p] = static_cast<const T*>(A.b[p]) + n * A.ldb[p] + g * 8;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int64_t m = j * 16 + i < A.M ? j * 16 + i : A.M - 1;
        x[j] = static_cast<const T*>(A.a[0]) + m * A.lda[0] + g * 8;
    }
    f32x4 acc[P][MT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[p][j] = f32x4{0, 0, 0, 0};

    const auto load = [](const T* p) -> v8 {
        const Bytes16 b = *reinterpret_cast<const Bytes16*>(p);
        v8 v;
        __builtin_memcpy(&v, &b, 16);
        return v;
    };
    const int64_t whole = A.K / 64;  // steps of 64; the rest below
    int64_t s = wave;
    for (; s + (kAhead - 1) * kWaves < whole; s += kAhead * kWaves) {
        v8 fw[kAhead][2][P], fx[kAhead][2][MT];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = (s + a * kWaves) * 64 + h * 32;
#pragma unroll
                for (int p = 0; p < P; ++p) fw[a][h][p] = load(w[p] + k);
#pragma unroll
                for (int j = 0; j < MT; ++j) fx[a][h][j] = load(x[j] + k);
            }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[p][j] = Arith<T>::mma(fw[a][h][p], fx[a][h][j], acc[p][j]);
    }
    // what is left of k, zeros beyond its end
    for (; s * 64 < A.K; s += kWaves) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = s * 64 + h * 32;
            const int64_t have = A.K - k - g * 8;
            const auto part = [&](const T* p) -> v8 {
                if (have >= 8) return load(p + k);
                v8 v;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = e < have ? p[k + e] : T(0.0f);
                return v;
            };
            v8 fx[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) fx[j] = part(x[j]);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const v8 fw = part(w[p]);
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[p][j] = Arith<T>::mma(fw, fx[j], acc[p][j]);
            }
        }
    }

    // lane (g, i) holds row i of a tile and columns 4g .. 4g + 3
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            *reinterpret_cast<f32x4*>(&sums[wave][p][j * 16 + i][(g ^ (i & 3)) * 4]) = acc[p][j];
    __syncthreads();
    const int r = threadIdx.x >> 1, c = threadIdx.x & 1;
    if (r >= MT * 16 || r >= A.M) return;
    float v[8], v2[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int at = ((2 * c + q) ^ (r & 3)) * 4;
        f32x4 t[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            t[p] = *reinterpret_cast<const f32x4*>(&sums[0][p][r][at]);
#pragma unroll
            for (int u = 1; u < kWaves; ++u)
                t[p] += *reinterpret_cast<const f32x4*>(&sums[u][p][r][at]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[4 * q + e] = t[0][e];
            v2[4 * q + e] = t[P - 1][e];
        }
    }
    finish_one<T, PAIR, 8>(A.fin, 0, r, n0 + c * 8, A.N, v, v2);
}

}  // namespace layers
}  // namespace dgc
