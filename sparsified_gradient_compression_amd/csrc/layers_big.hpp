// layers_big.hpp -- 256 x 256 outputs per workgroup: the products that are
// bound by the matrix units.
//
// Eight waves, two per SIMD, in two groups of four.  A group's waves lie on
// different SIMDs, and the groups run half a phase apart: while one multiplies
// (16 matrix instructions, 256 cycles), the other reads its next registers
// from LDS and orders tiles from memory, so a SIMD's matrix unit always has a
// wave to work for.  A barrier after every half phase keeps them so.
//
// LDS holds two tiles of 64 steps of k (128 KB), each as four regions: halves
// of 128 rows of a (A0, A1) and of b (B0, B1).  A tile takes four phases:
//
//   read A0 | A0 x first B half | read the second B half | A0 x it
//   read A1 | A1 x second half  | read the next tile's first half | A1 x first
//
// The half of b that the next tile starts with alternates, so that each phase
// reads 8 or 4 fragments and none waits for registers.  Every phase also
// orders one region of the tile after the next, into the region whose last
// reads are over: memory goes straight to LDS, six phases (3000 cycles) ahead
// of its use, and `vmcnt(12)` at the end of each read half phase is all the
// waiting there is (six regions of two loads are in flight beyond it).
#pragma once

#include "layers_tile.hpp"

namespace dgc {
namespace layers {

// A byte offset past every buffer descriptor's end: reads as zero.
constexpr uint32_t kOutside = 0x80000000u;

constexpr int kRegion = 128 * kStep;  // elements of a region

// s_waitcnt: at most 12 loads in flight, no LDS read.
constexpr int kWait12Lds0 = 12 | (7 << 4) | (0 << 8);

__device__ __forceinline__ void half_phase_end() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// How one side's regions come to LDS and to the registers.
//   TR:    stored with m (n) contiguous: region [64 k][128]
//   else:  stored with k contiguous:     region [128][64]
//   NT:    16-row tiles of a wave in a region; NSIDE: dealt by n_row<NT>
template <class T, bool TR, int NT, bool NSIDE>
struct Side {
    typedef typename Arith<T>::v8 v8;
    uint32_t at[2][2];  // byte offset of this lane's pieces: half, load; kOutside if none
    int k_at;           // first k of the lane's piece (TR: of load 0)
    int frag[TR ? NT : 2];

    // rows: how many rows (columns) exist from this tile's first on, per half
    __device__ __forceinline__ void init(int64_t ld, int64_t rows0, int64_t rows1, int wave,
                                         int lane, int base) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (TR) {
            const int k = wave * 4 + (lane >> 4);
            const int piece = ((((lane & 15) >> 1) ^ k_key<128>(k)) << 1) | (lane & 1);
            k_at = k;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const int64_t have = h ? rows1 : rows0;
                    at[h][l] = piece * 8 < have
                                   ? uint32_t((int64_t(k + 32 * l) * ld + h * 128 + piece * 8) * 2)
                                   : kOutside;
                }
            const int kk = g * 8 + (i >> 2);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                frag[j] = kk * 128 + ((((base >> 4) + j) ^ k_key<128>(kk)) << 4) + (i & 3) * 4;
        } else {
            const int r = wave * 8 + (lane >> 3);
            const int piece = (lane & 7) ^ row_key<NT, NSIDE>(r);
            k_at = piece * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const int64_t have = h ? rows1 : rows0;
                    const int row = r + 64 * l;
                    at[h][l] = row < have ? uint32_t((int64_t(row) * ld + piece * 8) * 2) : kOutside;
                }
            const int fr = base + (NSIDE ? n_row<NT>(i, 0) : i);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                frag[s] = fr * kStep + (((s * 4 + g) ^ row_key<NT, NSIDE>(fr)) << 3);
        }
    }

    // Order half h of a tile at `p` (its first row, its first k) of which
    // `left` steps of k exist, into region `lds`.
    __device__ __forceinline__ void order(const T* p, int left, int h, T* lds, int wave) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host's pass does not know 16-byte loads to LDS
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T*>(p), short(0), int(0x7FFFFFFF), 0x00020000);
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            const uint32_t v = k_at + (TR ? 32 * l : 0) < left ? at[h][l] : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (DGC_LDS void*)(lds + (l * 8 + wave) * 512), 16, int(v), 0, 0, 0);
        }
#endif
    }

    // Fragment j, steps 32 s .. 32 s + 31, of a region.
    __device__ __forceinline__ v8 get(const T* lds, int j, int s) const {
        if constexpr (TR) {
            union { s16x4 h[2]; v8 v; } u;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (DGC_LDS s16x4*)(const_cast<T*>(lds + frag[j] + s * 32 * 128 + h * 4 * 128)));
            return u.v;
        } else {
            return *reinterpret_cast<const v8*>(lds + frag[s] + j * (NSIDE ? 4 : 16) * kStep);
        }
    }
};

template <class T, int FORM>
__global__ __launch_bounds__(512, 2) void k_big(TileArgs A) {
    constexpr bool PAIR = FORM == kPair, ATR = FORM == kDw, BTR = FORM == kDx || FORM == kDw;
    typedef typename Arith<T>::v8 v8;
    __shared__ __align__(16) T a00[kRegion], a01[kRegion], a10[kRegion], a11[kRegion];
    __shared__ __align__(16) T b00[kRegion], b01[kRegion], b10[kRegion], b11[kRegion];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wm = wave >> 2, wn = wave & 3;

    const int64_t tiles = A.mt * A.nt;
    int64_t id = blockIdx.x;
    const int64_t per_split = tiles * (FORM == kDw ? A.parts : 1);
    const int split = int(id / per_split);
    id -= split * per_split;
    const int z = FORM == kDw ? int(id / tiles) : 0;
    id -= z * tiles;
    int64_t tm, tn;
    place(id, A.mt, A.nt, tm, tn);
    const int64_t m0 = tm * 256, n0 = tn * (PAIR ? 128 : 256);

    const int ksteps = int((A.K + kStep - 1) / kStep);
    const int total = ksteps * (FORM == kDx ? A.parts : 1);
    const int first = split * int(A.per);
    const int last = first + int(A.per) < total ? first + int(A.per) : total;

    Side<T, ATR, 4, false> sa;
    Side<T, BTR, 2, true> sb;
    const int64_t lda = A.lda[0], ldb = A.ldb[0];
    sa.init(lda, A.M - m0, A.M - m0 - 128, wave, lane, wm * 64);
    sb.init(ldb, A.N - n0, PAIR ? A.N - n0 : A.N - n0 - 128, wave, lane, wn * 32);

    // Half h of tile t.  Beyond the last tile nothing is read, but the loads
    // are counted all the same.
    auto order_a = [&](int t, int h, T* lds) {
        const int seg = FORM == kDx && t >= ksteps ? 1 : 0;
        const int64_t k0 = int64_t(t - seg * ksteps) * kStep;
        const int64_t left = t < last ? A.K - k0 : 0;
        const T* p = static_cast<const T*>(A.a[FORM == kDw ? z : seg]) +
                     (ATR ? k0 * lda + m0 : (m0 + h * 128) * lda + k0);
        sa.order(left > 0 ? p : static_cast<const T*>(A.a[0]), left < kStep ? int(left) : kStep,
                 h, lds, wave);
    };
    auto order_b = [&](int t, int h, T* lds) {
        const int seg = FORM == kDx && t >= ksteps ? 1 : 0;
        const int64_t k0 = int64_t(t - seg * ksteps) * kStep;
        const int64_t left = t < last ? A.K - k0 : 0;
        const T* p = static_cast<const T*>(A.b[PAIR ? h : seg]) +
                     (BTR ? k0 * ldb + n0 : (n0 + (PAIR ? 0 : h * 128)) * ldb + k0);
        sb.order(left > 0 ? p : static_cast<const T*>(A.b[0]), left < kStep ? int(left) : kStep,
                 h, lds, wave);
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
            for (int i = 0; i < 4; ++i) fa[i][s] = sa.get(lds, i, s);
    };
    auto read_b = [&](int h, const T* lds) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[h][j][s] = sb.get(lds, j, s);
    };
    auto read_end = [&]() {
        __builtin_amdgcn_s_waitcnt(kWait12Lds0);
        half_phase_end();
    };
    auto multiply = [&](int ha, int hb) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[ha][hb][i][j] = Arith<T>::mma(fb[hb][j][s], fa[i][s], acc[ha][hb][i][j]);
        __builtin_amdgcn_s_setprio(0);
        half_phase_end();
    };
    // Tile t, of the parity whose first half of b is f: its four regions, and
    // the next tile's first region of b.
    auto tile = [&](int t, int f, T* la0, T* la1, T* lbf, T* lbs, const T* next) {
        read_a(la0);
        order_b(t + 2, f, lbf);
        read_end();
        multiply(0, f);
        read_b(1 - f, lbs);
        order_a(t + 2, 0, la0);
        read_end();
        multiply(0, 1 - f);
        read_a(la1);
        order_b(t + 2, 1 - f, lbs);
        read_end();
        multiply(1, 1 - f);
        read_b(1 - f, next);
        order_a(t + 2, 1, la1);
        read_end();
        multiply(1, f);
    };

    order_b(first, 0, b00);
    order_a(first, 0, a00);
    order_b(first, 1, b01);
    order_a(first, 1, a01);
    order_b(first + 1, 1, b11);
    order_a(first + 1, 0, a10);
    order_b(first + 1, 0, b10);
    order_a(first + 1, 1, a11);
    read_end();
    read_b(0, b00);
    read_end();  // tile first + 2 may go there from now on
    if (wm == 1) half_phase_end();
    // by twos: with an odd count the last tile is one of zeros
    for (int t = first; t < last; t += 2) {
        tile(t, 0, a00, a01, b00, b01, b11);
        tile(t + 1, 1, a10, a11, b11, b10, b00);
    }
    if (wm == 0) half_phase_end();
    __builtin_amdgcn_s_waitcnt(0);

    __syncthreads();  // nobody reads a region any more, and no load is under way

    // 64 x 64 outputs of the wave at a time, in the 16 KB of one region
    T* const own = wave < 4 ? (wave < 2 ? (wave ? a01 : a00) : (wave & 1 ? a11 : a10))
                            : (wave < 6 ? (wave & 1 ? b01 : b00) : (wave & 1 ? b11 : b10));
    float* out = reinterpret_cast<float*>(own);
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                put_tile<4, 2, BTR>(out, mt, j / 2 * 32, j % 2, lane, acc[ha][j / 2][mt][j % 2]);
        const int64_t n = n0 + wn * 32;
        put_wave<T, FORM, 4, 4>(A, split, z, m0 + ha * 128 + wm * 64, n, PAIR ? n : n + 128, lane,
                                out);
    }
}

}  // namespace layers
}  // namespace dgc
