// layers_elem.hpp -- the element-wise passes of the layer gradients: what the
// activation's slope makes of an incoming gradient, column sums, and operands
// laid out anew.
//
// The products that follow take 16-bit operands, so dz (da, db) is stored as a
// sum of numbers of the elements' own type, and each of them is multiplied.  Two
// hold it to 2^-16 (bf16) or 2^-22 (fp16) of itself, far less than the rounding
// of a 16-bit output; three hold a bf16 dz to binary32's own precision, for
// weight gradients in binary32.  One number, half a step of 2^-8 or 2^-11, is
// for callers that ask for it: the outputs' error is then 1.4 times their own
// rounding, and the products take half the time.  Up to 32 rows a second number
// costs nothing: it takes places of the same tiles that would be empty.
//
// fp16 has 5 bits of exponent, and dz is a product of up to three numbers: it
// may be 2^16 times larger or smaller than any of them.  A pass before finds
// the largest |dz| of the call; dz is stored times a power of two that brings
// it into [2^14, 2^15), and the products' finish undoes that.  So nothing
// overflows, and what a number below fp16's normal range loses is at most
// 2^-39 of the largest.  bf16 has the range of the binary32 that dz is made in.
// The pass costs a launch and a read: 9 us of 47 for a gated block's gradients
// of 333 rows, 1152 x 3456.
//
// All passes are bound by memory.  A gated block's slopes of 8192 x 12288: 155
// us, 6.5 TB/s, and 259, 5.4 TB/s, in two pieces; a layer's of 1531 x 3840 with
// its column sums: 13 and 20 us, one round of workgroups, most of it the way to
// memory and back.
#pragma once

#include "layers_tile.hpp"

namespace dgc {
namespace layers {

// v as the sum of P numbers of T, all of v's sign and none of them 0 (unless v
// is): each but the last lies below what is left of v in magnitude, also where T
// holds that itself.  So every product with an infinite operand is the infinity
// that v's is; a piece that is 0 or of the other sign would make it NaN.  The sum
// is off by half a step of the last piece, or by two of T's least numbers.  An
// infinite or NaN v is all pieces.
template <class T, int P>
__device__ __forceinline__ void split(float v, float* piece) {
    asm("" : "+v"(v));  // rounded once: T made from the product before it may be another number
#pragma unroll
    for (int p = 0; p < P; ++p) piece[p] = float(T(v));
    if (P == 1 || !(fabsf(v) < __builtin_inff()) || v == 0.0f) return;
    const uint16_t least = __builtin_bit_cast(uint32_t, v) >> 31 << 15 | 1;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        uint16_t h = __builtin_bit_cast(uint16_t, T(v));
        if (p < P - 1 && fabsf(float(T(v))) >= fabsf(v)) --h;  // a step towards 0
        if ((h & 0x7FFF) == 0 || v == 0.0f || h >> 15 != least >> 15) h = least;
        piece[p] = float(__builtin_bit_cast(T, h));
        v -= piece[p];
    }
}

// C values as P pieces, `low` elements apart.  (A template: the registers of
// many pieces would cost one 3% of its rate.)
template <class T, int C, int P>
__device__ __forceinline__ void store_pieces(T* p, int64_t low, const float* v) {
    if constexpr (P == 1) {
        store_row<T, C>(p, C, v);
        return;
    }
    float piece[C][P], row[C];
#pragma unroll
    for (int i = 0; i < C; ++i) split<T, P>(v[i], piece[i]);
#pragma unroll
    for (int q = 0; q < P; ++q) {
#pragma unroll
        for (int i = 0; i < C; ++i) row[i] = piece[i][q];
        store_row<T, C>(p + q * low, C, row);
    }
}

template <class T, int C>
__device__ __forceinline__ void scale_row(float* v, float scale) {
    if constexpr (__is_same(T, _Float16)) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] *= scale;
    }
}

// The largest of 256 threads' values, to all of them.
__device__ __forceinline__ float most_of_block(float v, float* lds) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
}

// The largest finite |dz| (|da|, |db|) of a workgroup's rows, into most[].
// `across` threads (a power of two) lie side by side along a row.
template <class T>
__global__ __launch_bounds__(256) void k_most(SlopeArgs A, int across) {
    __shared__ float lds[4];
    const int tx = threadIdx.x & (across - 1), ty = threadIdx.x / across, rows = 256 / across;
    float most = 0.0f;
    for (int64_t m = int64_t(blockIdx.x) * rows + ty; m < A.M; m += int64_t(gridDim.x) * rows)
        for (int64_t n = tx * 8; n < A.N; n += across * 8) {
            const int valid = A.N - n >= 8 ? 8 : int(A.N - n);
            float d[8], z[8], u[8];
            load_row<T, 8>(static_cast<const T*>(A.dy) + m * A.lddy + n, valid, d);
            load_row<T, 8>(static_cast<const T*>(A.pre) + m * A.ldp + n, valid, z);
            if (A.up) load_row<T, 8>(static_cast<const T*>(A.up) + m * A.ldu + n, valid, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float value, slope;
                act_pair(A.act, z[i], value, slope);
                const float a = fabsf(A.up ? d[i] * u[i] * slope : d[i] * slope);
                const float b = A.up ? fabsf(d[i] * value) : 0.0f;
                // neither an infinity nor a NaN
                if (a < __builtin_inff()) most = fmaxf(most, a);
                if (b < __builtin_inff()) most = fmaxf(most, b);
            }
        }
    most = most_of_block(most, lds);
    if (threadIdx.x == 0) A.most[blockIdx.x] = most;
}

// The power of two that brings the largest |dz| into [2^14, 2^15).
__device__ __forceinline__ float dz_scale(const SlopeArgs& A, float* lds) {
    static_assert(kMostParts == 512, "two per thread");
    float most = threadIdx.x < A.parts ? A.most[threadIdx.x] : 0.0f;
    if (threadIdx.x + 256 < A.parts) most = fmaxf(most, A.most[threadIdx.x + 256]);
    most = most_of_block(most, lds);
    // its exponent, where it is 2^-86 or more; 0 and less: as 2^-86
    const int e = int(__builtin_bit_cast(uint32_t, most) >> 23) - 127;
    const int up = most > 0.0f ? 14 - (e > -86 ? e : -86) : 0;
    if (block_number() == 0 && threadIdx.x == 0)
        *A.unscale = __builtin_bit_cast(float, uint32_t(127 - up) << 23);
    return __builtin_bit_cast(float, uint32_t(127 + up) << 23);
}

// dz = dy * act'(pre) and the sums of dz's columns (before it is rounded) over
// `per` rows each.  A block of 256 threads covers 512 columns (64 threads, 8
// columns each) by `per` rows (4 rows of threads).
template <class T, int P>
__device__ __forceinline__ void slope_block(const SlopeArgs& A, int64_t id, float (*sums)[512],
                                            float scale) {
    const int64_t across = (A.N + 511) / 512;
    const int64_t by = id / across, bx = id - by * across;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t n = bx * 512 + tx * 8;
    const int valid = A.N - n >= 8 ? 8 : A.N > n ? int(A.N - n) : 0;
    const int64_t m0 = by * A.per;
    const int64_t m1 = m0 + A.per < A.M ? m0 + A.per : A.M;
    const T* dy = static_cast<const T*>(A.dy);
    const T* pre = static_cast<const T*>(A.pre);
    T* dz = static_cast<T*>(A.dz);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (valid > 0) {
        for (int64_t m = m0 + ty; m < m1; m += 8) {  // two rows' loads under way
            float d[2][8], z[2][8];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (m + 4 * r < m1) {
                    load_row<T, 8, true>(dy + (m + 4 * r) * A.lddy + n, valid, d[r]);
                    if (A.act != DGC_ACT_NONE)
                        load_row<T, 8, true>(pre + (m + 4 * r) * A.ldp + n, valid, z[r]);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (m + 4 * r < m1) {
                    if (A.act != DGC_ACT_NONE) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float value, slope;
                            act_pair(A.act, z[r][i], value, slope);
                            d[r][i] *= slope;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] += d[r][i];
                    scale_row<T, 8>(d[r], scale);
                    // zeros in the padding
                    if (dz) store_pieces<T, 8, P>(dz + (m + 4 * r) * A.ldz + n, A.low, d[r]);
                }
        }
    }
    if (!A.part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[ty][tx * 8 + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
        const int64_t at = bx * 512 + c;
        if (at < A.N)
            A.part[by * A.N + at] = (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
    }
}

// The partial column sums, added in order: 32 columns per workgroup.
template <class T, int THREADS>
__device__ __forceinline__ void sum_columns(const Sums& A, int64_t id, float* lds) {
    constexpr int kRows = THREADS / 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t n = id * 32 + tx;
    float s = 0.0f;
    if (n < A.N) {
#pragma unroll 8
        for (int64_t r = ty; r < A.rows; r += kRows) s += A.part[r * A.N + n];
    }
    lds[ty * 32 + tx] = s;
    __syncthreads();
    if (ty == 0 && n < A.N) {
        for (int i = 1; i < kRows; ++i) s += lds[i * 32 + tx];
        if (A.wide)
            static_cast<float*>(A.out)[n] = s;
        else
            static_cast<T*>(A.out)[n] = T(s);
    }
}

template <class T>
__global__ __launch_bounds__(256) void k_sum_columns(Sums A) {
    __shared__ float lds[256];
    sum_columns<T, 256>(A, block_number(), lds);
}

// da = dh * up * act'(gate), db = dh * act(gate), rows of `ld` elements; C (4
// or 8) elements per thread.
template <class T, int C, int P>
__device__ __forceinline__ void gate_slope_block(const SlopeArgs& A, int64_t id, float scale) {
    const int64_t groups = A.ldz / C;
    id = id * 256 + threadIdx.x;
    if (id >= groups * A.M) return;
    const int64_t m = id / groups, n = (id - m * groups) * C;
    const int valid = A.N - n >= C ? C : A.N > n ? int(A.N - n) : 0;
    float d[C], a[C], b[C], oa[C], ob[C];
    load_row<T, C, true>(static_cast<const T*>(A.dy) + m * A.lddy + n, valid, d);
    load_row<T, C, true>(static_cast<const T*>(A.pre) + m * A.ldp + n, valid, a);
    load_row<T, C, true>(static_cast<const T*>(A.up) + m * A.ldu + n, valid, b);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        float value, slope;
        act_pair(A.act, a[i], value, slope);
        oa[i] = d[i] * b[i] * slope;
        ob[i] = d[i] * value;
    }
    scale_row<T, C>(oa, scale);
    scale_row<T, C>(ob, scale);
    // zeros in the padding
    store_pieces<T, C, P>(static_cast<T*>(A.dz) + m * A.ldz + n, A.low, oa);
    store_pieces<T, C, P>(static_cast<T*>(A.dz2) + m * A.ldz + n, A.low, ob);
}

// Rows at any even address to rows on 16 bytes, zeros up to their ends; 8
// elements per thread.
__device__ __forceinline__ void repack_block(const Repack& r, int64_t id) {
    id = id * 256 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i >= r.count) return;
        const int64_t per = (r.cols[i] + 7) / 8, have = per * r.rows[i];
        if (id < have) {
            const int64_t row = id / per, col = (id - row * per) * 8;
            const uint16_t* p = static_cast<const uint16_t*>(r.from[i]) + row * r.ld[i] + col;
            u32x4 v;
            if (col + 8 <= r.cols[i]) {
                v = reinterpret_cast<const Bytes16*>(p)->v;
            } else {
                uint16_t t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = col + e < r.cols[i] ? p[e] : uint16_t(0);
                __builtin_memcpy(&v, t, 16);
            }
            reinterpret_cast<u32x4*>(r.to[i])[id] = v;
            return;
        }
        id -= have;
    }
}

// What a call lays out before its products, in one launch.
template <class T, int P>
__global__ __launch_bounds__(256) void k_prepare(SlopeArgs A, int64_t slope_blocks, Repack r) {
    __shared__ float sums[4][512];
    const int64_t id = block_number();
    if (id >= slope_blocks) {
        repack_block(r, id - slope_blocks);
        return;
    }
    float scale = 1.0f;
    if constexpr (__is_same(T, _Float16)) {
        __shared__ float most[4];
        if (A.most) scale = dz_scale(A, most);
    }
    if (A.up && A.per == 4)
        gate_slope_block<T, 4, P>(A, id, scale);
    else if (A.up)
        gate_slope_block<T, 8, P>(A, id, scale);
    else
        slope_block<T, P>(A, id, sums, scale);
}

}  // namespace layers
}  // namespace dgc
