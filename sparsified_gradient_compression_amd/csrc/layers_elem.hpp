// layers_elem.hpp -- the element-wise passes of the layer gradients: what the
// activation's slope makes of an incoming gradient, and column sums.
//
// The products that follow take 16-bit operands, so dz (da, db) is rounded
// once to the elements' own type here, as the incoming gradient was: a
// relative 2^-9 (bf16) or 2^-12 (fp16) at random per element, no more than
// the rounding of the output that it is summed into.
#pragma once

#include "layers_tile.hpp"

namespace dgc {
namespace layers {

// dz = dy * act'(pre), and the sums of dz's columns over `per` rows each.
// A block covers 512 columns (64 threads, 8 columns each) by `per` rows
// (4 rows of threads).  The column sums use dz before it is rounded.
template <class T>
__global__ __launch_bounds__(256) void k_slope(int64_t M, int64_t N, int64_t per, const T* dy, int64_t lddy,
                                               const T* pre, int64_t ldp, int act, T* dz,
                                               int64_t ldz, float* part) {
    __shared__ float sums[4][512];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t n = int64_t(blockIdx.x) * 512 + tx * 8;
    const int valid = N - n >= 8 ? 8 : N > n ? int(N - n) : 0;
    const int64_t m0 = int64_t(blockIdx.y) * per;
    const int64_t m1 = m0 + per < M ? m0 + per : M;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (valid > 0) {
#pragma unroll 4
        for (int64_t m = m0 + ty; m < m1; m += 4) {
            float d[8], z[8];
            load_row<T, 8>(dy + m * lddy + n, valid, d);
            if (act != DGC_ACT_NONE) {
                load_row<T, 8>(pre + m * ldp + n, valid, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float value, slope;
                    act_pair(act, z[i], value, slope);
                    d[i] *= slope;
                }
            }
            if (dz) store_row<T, 8>(dz + m * ldz + n, 8, d);  // zeros in the padding
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += d[i];
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[ty][tx * 8 + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
        const int64_t at = int64_t(blockIdx.x) * 512 + c;
        if (at < N)
            part[int64_t(blockIdx.y) * N + at] =
                (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
    }
}

// The partial column sums, added in order: 32 columns per block, 8 threads each.
template <class O>
__global__ __launch_bounds__(256) void k_sum_columns(int64_t rows, int64_t N, const float* part,
                                                     O* out) {
    __shared__ float sums[8][32];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t n = int64_t(blockIdx.x) * 32 + tx;
    float s = 0.0f;
    if (n < N)
#pragma unroll 8
        for (int64_t r = ty; r < rows; r += 8) s += part[r * N + n];
    sums[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && n < N) {
        for (int i = 1; i < 8; ++i) s += sums[i][tx];
        out[n] = O(s);
    }
}

// da = dh * up * act'(gate), db = dh * act(gate), rows of `ld` elements.
template <class T>
__global__ __launch_bounds__(256) void k_gate_slope(int64_t M, int64_t F, const T* dh,
                                                    int64_t lddh, const T* gate, int64_t ldg,
                                                    const T* up, int64_t ldu, int act, T* da,
                                                    T* db, int64_t ld) {
    const int64_t groups = (F + 7) / 8;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (id >= groups * M) return;
    const int64_t m = id / groups, n = (id - m * groups) * 8;
    const int valid = F - n >= 8 ? 8 : int(F - n);
    float d[8], a[8], b[8], oa[8], ob[8];
    load_row<T, 8>(dh + m * lddh + n, valid, d);
    load_row<T, 8>(gate + m * ldg + n, valid, a);
    load_row<T, 8>(up + m * ldu + n, valid, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float value, slope;
        act_pair(act, a[i], value, slope);
        oa[i] = d[i] * b[i] * slope;
        ob[i] = d[i] * value;
    }
    store_row<T, 8>(da + m * ld + n, 8, oa);  // zeros in the padding
    store_row<T, 8>(db + m * ld + n, 8, ob);
}

}  // namespace layers
}  // namespace dgc
