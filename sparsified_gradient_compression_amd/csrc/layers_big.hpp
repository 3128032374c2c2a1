// layers_big.hpp -- 256 x 256 outputs per workgroup: the products that are
// bound by the matrix units.
//
// Eight waves, two per SIMD, in two groups of four.  A group's waves lie on
// different SIMDs, and the groups run half a phase apart: while one multiplies
// (32 matrix instructions, 512 cycles), the other reads its next registers
// from LDS and orders tiles from memory, so a SIMD's matrix unit always has a
// wave to work for.  A barrier after every half phase keeps them so.
//
// LDS holds two tiles of 64 steps of k (128 KB), each as four regions: halves
// of 128 rows of a (A0, A1) and of b (B0, B1).  A tile takes two phases:
//
//   read A0, B0, B1, order A1 of the next tile            | multiply A0 x B
//   read A1, order A0, B0, B1 of the tile after the next  | multiply A1 x B
//
// Every region is ordered as soon as its last reads are over, memory goes
// straight to LDS, and it has three phases (3000 cycles) to come: at the end
// of each half phase of reads `vmcnt(8)`, four regions of two loads, is all
// the waiting there is.  Half phases of 16 matrix instructions leave the reads
// less time than they take (8192 x 8192 x 4096: 394 us, not 380).
//
// 8192^3 with bias and residual: 766-824 us from card to card, 1334-1435
// TFLOP/s; a gated block's forward pass, 8192 x 4096 x 12288: 1226-1249 us,
// 1320-1345; its dx, da and db in one piece, 1177 us, 1401, and dw (both operands
// turned on the way) 1318 us, 1252, in two pieces 2600-2700 and 2560-2670.  Bound
// by the matrix units but for 11 us per round of workgroups, while the outputs
// leave.
#pragma once

#include "layers_direct.hpp"

namespace dgc {
namespace layers {

constexpr int kRegion = 128 * kStep;  // elements of a region

__device__ __forceinline__ void half_phase_end() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

template <class T, int FORM, bool SPLIT>
__global__ __launch_bounds__(512, 2) void k_big(TileArgs A) {
    constexpr bool PAIR = FORM == kPair, ATR = FORM == kDw, BTR = FORM == kDx || FORM == kDw;
    typedef typename Arith<T>::v8 v8;
    __shared__ __align__(16) T a00[kRegion], a01[kRegion], a10[kRegion], a11[kRegion];
    __shared__ __align__(16) T b00[kRegion], b01[kRegion], b10[kRegion], b11[kRegion];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = wave >> 2, wn = wave & 3;

    const int64_t id = block_number();
    if (id >= all_blocks<FORM>(A)) return;
    const Spot at_tile = spot<FORM>(A, int(id));
    const int split = at_tile.split, z = at_tile.z;
    const int64_t m0 = at_tile.tm * 256, n0 = at_tile.tn * (PAIR ? 128 : 256);

    const int ksteps = int((A.K + kStep - 1) / kStep);
    const int total = all_steps<FORM, SPLIT>(A, ksteps);
    const int first = split * int(A.per);
    const int last = first + int(A.per) < total ? first + int(A.per) : total;

    Side<T, ATR, 4, false, 128, 8> sa[2];
    Side<T, BTR, 2, true, 128, 8> sb[2];
    const int64_t lda = A.lda[0], ldb = A.ldb[0];
    for (int h = 0; h < 2; ++h) {
        sa[h].init(lda, a_rows<FORM>(A) - m0 - h * 128, wave, lane, wm * 64);
        sb[h].init(ldb, A.N - n0 - (PAIR ? 0 : h * 128), wave, lane, wn * 32,
                   FORM == kDw ? A.fold : 0);
    }

    // Half h of tile t.  Beyond the last tile nothing is read, but the loads
    // are counted all the same.
    auto order_a = [&](int t, int h, T* lds) {
        const auto step = step_at<FORM, SPLIT>(A, t, ksteps);
        const int64_t k0 = step.k0, left = t < last ? A.K - k0 : 0;
        const T* p = static_cast<const T*>(A.a[FORM == kDw ? z : step.term]) + step.piece +
                     (ATR ? k0 * lda + m0 + h * 128 : (m0 + h * 128) * lda + k0);
        sa[h].order(left > 0 ? p : static_cast<const T*>(A.a[0]),
                    left < kStep ? int(left) : kStep, lds, wave);
    };
    auto order_b = [&](int t, int h, T* lds) {
        const auto step = step_at<FORM, SPLIT>(A, t, ksteps);
        const int64_t k0 = step.k0, left = t < last ? A.K - k0 : 0;
        const T* p = static_cast<const T*>(A.b[PAIR ? h : step.term]) +
                     (BTR ? k0 * ldb + n0 + h * 128 : (n0 + (PAIR ? 0 : h * 128)) * ldb + k0);
        sb[h].order(left > 0 ? p : static_cast<const T*>(A.b[0]),
                    left < kStep ? int(left) : kStep, lds, wave);
    };

    f32x4 acc[2][2][4][2];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i >> 3][(i >> 2) & 1][i & 3][j] = f32x4{0, 0, 0, 0};
    v8 fa[4][2], fb[2][2][2];

    auto read_a = [&](const T* lds) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i][s] = sa[0].get(lds, i, s);
    };
    auto read_b = [&](int h, const T* lds) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[h][j][s] = sb[0].get(lds, j, s);
    };
    auto read_end = [&]() {
        __builtin_amdgcn_s_waitcnt(wait_for(8, 0));
        half_phase_end();
    };
    auto multiply = [&](int ha) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[ha][hb][i][j] =
                            Arith<T>::mma(fb[hb][j][s], fa[i][s], acc[ha][hb][i][j]);
        __builtin_amdgcn_s_setprio(0);
        half_phase_end();
    };
    auto tile = [&](int t, T* la0, T* la1, T* lb0, T* lb1, T* other_a1) {
        read_b(0, lb0);
        read_a(la0);
        read_b(1, lb1);
        order_a(t + 1, 1, other_a1);
        read_end();
        multiply(0);
        read_a(la1);
        order_a(t + 2, 0, la0);
        order_b(t + 2, 0, lb0);
        order_b(t + 2, 1, lb1);
        read_end();
        multiply(1);
    };

    order_a(first, 0, a00);
    order_b(first, 0, b00);
    order_b(first, 1, b01);
    order_a(first, 1, a01);
    order_a(first + 1, 0, a10);
    order_b(first + 1, 0, b10);
    order_b(first + 1, 1, b11);
    read_end();
    if (wm == 1) half_phase_end();
    // by twos: with an odd count the last tile is one of zeros
    for (int t = first; t < last; t += 2) {
        tile(t, a00, a01, b00, b01, a11);
        tile(t + 1, a10, a11, b10, b11, a01);
    }
    if (wm == 0) half_phase_end();
    __builtin_amdgcn_s_waitcnt(0);

    __syncthreads();  // nobody reads a region any more, and no load is under way

    // 128 rows of outputs at a time, 16 in each region
    const auto at = [&](int r) {
        T* const lo = r < 32 ? (r < 16 ? a00 : a01) : (r < 48 ? a10 : a11);
        T* const hi = r < 96 ? (r < 80 ? b00 : b01) : (r < 112 ? b10 : b11);
        return reinterpret_cast<float*>(r < 64 ? lo : hi) + (r & 15) * 256;
    };
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const int r = wm * 64 + mt * 16 + (lane & 15);
            float* row = at(wm * 64 + mt * 16) + (lane & 15) * 256;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                put_tile<2, BTR>(row, r, j / 2 * 128 + wn * 32, j % 2, lane,
                                 acc[ha][j / 2][mt][j % 2]);
        }
        __syncthreads();
        put_rows<T, FORM, 128, 256, 512>(A, split, z, m0 + ha * 128, n0, 1, 0, at);
        if (ha == 0) __syncthreads();
    }
}

}  // namespace layers
}  // namespace dgc
