// layers_mid.hpp -- outputs of one or two hundred tiles, or few: bound by
// latency and by how many workgroups there are rather than by the matrix units.
//
// A ring of S tiles of 64 steps of k in LDS: loads go from memory straight
// there, S - 1 tiles ahead, and one barrier per tile both ends the reads of
// the oldest and shows the newest.  With KG > 1 as many groups of waves share
// the outputs and take the tiles of k in turn, each in a ring of its own, so
// that a long sum takes fewer steps; their sums meet in LDS.
//
// 2048 x 2048 x 8192 by 128 x 128 takes 72 us, 950 TFLOP/s: the matrix units
// are busy 45% of the time, LDS 34% (two bank conflicts in a hundred reads),
// the caches give 15 TB/s.  None is full; waves that read, multiply and wait
// for each other in step are what it costs.  Neither a ring of five tiles nor
// reads half a tile ahead change that (22.1 -> 22.1 and 23.2 us for 2048^3).
// 777 x 1000 x 2048 by 64 x 64: 10.1 us, most of it the first loads and the
// outputs' way out.
#pragma once

#include "layers_direct.hpp"
#include "layers_elem.hpp"

namespace dgc {
namespace layers {

// Shape of a workgroup: BM x BN outputs, KG groups of WM x WN waves, rings of
// S tiles.  EARLY: all reads of a tile go out before its products, not one by
// one among them, which is what the compiler makes of it: for the shape whose
// two workgroups share a compute unit and its few tiles under way (3000 x 1500
// x 3000: 50.1 -> 45.9 us, 2048 x 2048 x 8192 120 -> 109; by 128 x 128 with a
// ring of four 2048^3 takes 23.3 us so and 22.2 as it is).
template <int BM_, int BN_, int WM_, int WN_, int KG_, int S_, bool EARLY_ = false>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KG = KG_, S = S_;
    static constexpr bool EARLY = EARLY_;
    static constexpr int kThreads = WM * WN * KG * 64;
    static constexpr int kRing = KG * (BM + BN) * kStep;  // elements of a ring's tile
};
typedef Shape<32, 64, 2, 2, 4, 3> Shape32;
typedef Shape<64, 64, 2, 2, 2, 4> Shape64;
typedef Shape<64, 64, 2, 2, 1, 2> ShapeLight;
typedef Shape<128, 128, 2, 4, 1, 4> Shape128;
typedef Shape<128, 128, 2, 4, 1, 2, true> ShapePair;

// The ring's tiles are arrays of their own, so that a read of one is known
// not to wait for loads into another.
#define DGC_RING(T, SH)                                                        \
    __shared__ __align__(16) T s0[SH::kRing], s1[SH::kRing];                   \
    __shared__ __align__(16) T s2[SH::S > 2 ? SH::kRing : 8];                  \
    __shared__ __align__(16) T s3[SH::S > 3 ? SH::kRing : 8]

template <class T, int FORM, class SH, bool SPLIT>
__device__ __forceinline__ void mid_tile(const TileArgs& A, int id, T* s0, T* s1, T* s2,
                                         T* s3) {
    constexpr int BM = SH::BM, BN = SH::BN, WM = SH::WM, WN = SH::WN, KG = SH::KG, S = SH::S;
    constexpr bool PAIR = FORM == kPair, ATR = FORM == kDw, BTR = FORM == kDx || FORM == kDw;
    constexpr int W = WM * WN;
    constexpr int MT = BM / WM / 16, NTW = BN / WN / 16;  // 16 x 16 tiles of a wave
    constexpr int NT = PAIR ? NTW / 2 : NTW;              // ... of one product
    constexpr int RB = PAIR ? BN / 2 : BN;                // rows of a region of b
    constexpr int kTile = (BM + BN) * kStep;              // elements of both sides' tiles
    typedef typename Arith<T>::v8 v8;
    const int lane = threadIdx.x & 63;
    const int all = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int wave = all % W, group = all / W;
    const int wm = wave / WN, wn = wave % WN;

    const Spot at_tile = spot<FORM>(A, id);
    const int split = at_tile.split, z = at_tile.z;
    const int64_t m0 = at_tile.tm * BM, n0 = at_tile.tn * RB;

    const int ksteps = int((A.K + kStep - 1) / kStep);
    const int total = all_steps<FORM, SPLIT>(A, ksteps);
    const int first = split * int(A.per);
    const int last = first + int(A.per) < total ? first + int(A.per) : total;
    const int rounds = (last - first + KG - 1) / KG;

    Side<T, ATR, MT, false, BM, W> sa;
    Side<T, BTR, NT, true, RB, W> sb;
    const int64_t lda = A.lda[0], ldb = A.ldb[0];
    sa.init(lda, a_rows<FORM>(A) - m0, wave, lane, wm * MT * 16);
    sb.init(ldb, A.N - n0, wave, lane, wn * NT * 16, FORM == kDw ? A.fold : 0);
    constexpr int kLoads = decltype(sa)::kLoads + (PAIR ? 2 : 1) * decltype(sb)::kLoads;

    // The group's tile of round r; nothing is read beyond the last one.
    auto order = [&](int r, T* ring) {
        const int t = first + r * KG + group;
        const auto step = step_at<FORM, SPLIT>(A, t, ksteps);
        const int64_t more = t < last ? A.K - step.k0 : 0;
        const int left = more < kStep ? int(more) : kStep;
        const int64_t at = more > 0 ? step.k0 : 0;
        T* lds = ring + group * kTile;
        sa.order(static_cast<const T*>(A.a[FORM == kDw ? z : step.term]) + step.piece +
                     (ATR ? at * lda + m0 : m0 * lda + at), left, lds, wave);
#pragma unroll
        for (int w = 0; w < (PAIR ? 2 : 1); ++w)
            sb.order(static_cast<const T*>(A.b[PAIR ? w : step.term]) +
                         (BTR ? at * ldb + n0 : n0 * ldb + at), left,
                     lds + BM * kStep + w * RB * kStep, wave);
    };

    f32x4 acc[MT][NTW];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NTW; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    auto round = [&](int r, const T* use, T* fill) {
        __builtin_amdgcn_s_waitcnt(wait_for((S - 2) * kLoads, 15));
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (!SH::EARLY) order(r + S - 1, fill);
        const T* la = use + group * kTile;
        const T* lb = la + BM * kStep;
        v8 fa[2][MT], fb[2][NTW];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < NTW; ++j)
                fb[s][j] = sb.get(lb + (PAIR ? j / NT * RB * kStep : 0), PAIR ? j % NT : j, s);
#pragma unroll
            for (int i = 0; i < MT; ++i) fa[s][i] = sa.get(la, i, s);
        }
        if (SH::EARLY) {
            order(r + S - 1, fill);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NTW; ++j)
                    acc[i][j] = Arith<T>::mma(fb[s][j], fa[s][i], acc[i][j]);
            if (SH::EARLY) __builtin_amdgcn_sched_barrier(0);
        }
    };
    order(0, s0);
    if (S > 2) order(1, s1);
    if (S > 3) order(2, s2);
    for (int r = 0; r < rounds;) {
        round(r, s0, S == 2 ? s1 : S == 3 ? s2 : s3);
        if (++r >= rounds) break;
        round(r, s1, s0);
        if (++r >= rounds) break;
        if constexpr (S > 2) {
            round(r, s2, s1);
            if (++r >= rounds) break;
        }
        if constexpr (S > 3) {
            round(r, s3, s2);
            if (++r >= rounds) break;
        }
    }
    __builtin_amdgcn_s_waitcnt(wait_for(0, 0));
    __syncthreads();  // nobody reads the ring any more, and no load is under way

    // the outputs' 32-bit sums through LDS: as many rows as fit in a tile of
    // the ring, the others in the next
    constexpr int kFit = SH::kRing * int(sizeof(T)) / (BN * 4) / KG < BM
                             ? SH::kRing * int(sizeof(T)) / (BN * 4) / KG : BM;
    static_assert(KG == 1 ? 2 * kFit >= BM : kFit >= BM, "outputs fit the ring");
    constexpr int kGroupStride = BM * BN;
    const auto at = [&](int r) {
        return reinterpret_cast<float*>(r < kFit ? s0 : s1) + r % kFit * BN;
    };
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = (wm * MT + mt) * 16 + (lane & 15);
        float* row = at(r) + group * kGroupStride;
#pragma unroll
        for (int j = 0; j < NTW; ++j)
            put_tile<NT, BTR>(row, r, j / NT * (BN / 2) + wn * NT * 16, j % NT, lane, acc[mt][j]);
    }
    __syncthreads();
    put_rows<T, FORM, BM, BN, SH::kThreads>(A, split, z, m0, n0, KG, kGroupStride, at);
}

template <class T, int FORM, class SH, bool SPLIT>
__global__ __launch_bounds__(SH::kThreads) void k_mid(TileArgs A) {
    DGC_RING(T, SH);
    const int64_t id = block_number();
    if (id < all_blocks<FORM>(A)) mid_tile<T, FORM, SH, SPLIT>(A, int(id), s0, s1, s2, s3);
}

// Both gradients of a layer in one launch, and the column sums' last step.
template <class T, class SH, bool SPLIT>
__global__ __launch_bounds__(SH::kThreads) void k_mid_both(TileArgs dx, TileArgs dw,
                                                           int dx_blocks, int dw_blocks, Sums sums) {
    DGC_RING(T, SH);
    // each kind begins with the first die's workgroup
    const int64_t id = block_number(), dw0 = (dx_blocks + 7) & ~7, sum0 = dw0 + dw_blocks;
    if (id < dx_blocks)
        mid_tile<T, kDx, SH, SPLIT>(dx, int(id), s0, s1, s2, s3);
    else if (id >= dw0 && id < sum0)
        mid_tile<T, kDw, SH, SPLIT>(dw, int(id - dw0), s0, s1, s2, s3);
    else if (id >= sum0 && sums.out)
        sum_columns<T, SH::kThreads>(sums, id - sum0, reinterpret_cast<float*>(s0));
}

}  // namespace layers
}  // namespace dgc
