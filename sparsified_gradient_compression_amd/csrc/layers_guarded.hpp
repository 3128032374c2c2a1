// layers_guarded.hpp -- products whose operands' rows do not lie on 16 bytes:
// 64 x 64 outputs per workgroup, any strides, alignment and sizes.
//
// Four groups of four waves share the outputs and take the steps of 64 of k in
// turn, each with two LDS tiles of its own per side: the next one travels
// through the registers, with loads that are checked against the matrix, while
// this one is used.  Their sums meet in LDS.  Bound by those loads: 0.4 us per
// step and workgroup where rows lie on 16 bytes (2048^3: 47 us), 0.6 off them;
// four groups, since one step's loads alone leave the matrix units idle.
#pragma once

#include "layers_elem.hpp"

namespace dgc {
namespace layers {

// One side's pieces of a thread: 2 of the 512 of a tile of 64 rows by 64 k.
template <class T, bool TR>
struct Guarded {
    const T* p[2];   // of the piece in the group's first tile
    int have[2];     // TR: how many of its 8 columns exist; else 1 if its row does
    int k_at[2];     // its first k in a tile

    // fold (TR): steps of k from there on are the first ones again
    __device__ __forceinline__ void init(const T* base, int64_t ld, int64_t first, int64_t rows,
                                         int tid, int fold = 0) {
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            const int c = tid + l * 256;
            if constexpr (TR) {
                k_at[l] = c >> 3;
                const int64_t col = first + (c & 7) * 8;
                have[l] = rows - col >= 8 ? 8 : rows > col ? int(rows - col) : 0;
                p[l] = base + (fold && k_at[l] >= fold ? k_at[l] - fold : k_at[l]) * ld + col;
            } else {
                k_at[l] = (c & 7) * 8;
                have[l] = first + (c >> 3) < rows;
                p[l] = base + (first + (c >> 3)) * ld + k_at[l];
            }
        }
    }

    // `ahead` elements behind the first tile, `left` steps of k from there on
    __device__ __forceinline__ void load(int64_t ahead, int64_t left, u32x4* v) const {
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            int n = have[l];
            if constexpr (TR)
                n = k_at[l] < left ? n : 0;
            else
                n = !n || k_at[l] >= left ? 0 : left - k_at[l] >= 8 ? 8 : int(left - k_at[l]);
            const T* q = p[l] + ahead;
            v[l] = u32x4{0, 0, 0, 0};
            if (n == 8) {
                v[l] = reinterpret_cast<const Bytes16*>(q)->v;
            } else if (n > 0) {
                uint16_t t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[e] = e < n ? reinterpret_cast<const uint16_t*>(q)[e] : uint16_t(0);
                __builtin_memcpy(&v[l], t, 16);
            }
        }
    }

    template <int NT, bool NSIDE>
    static __device__ __forceinline__ void store(T* lds, int tid, const u32x4* v) {
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            const int c = tid + l * 256;
            *reinterpret_cast<u32x4*>(lds + piece_at<64, NT, TR, NSIDE>(c >> 3, c & 7)) = v[l];
        }
    }
};

constexpr int kGuardedGroups = 4;
constexpr int kGuardedSide = 64 * kStep;

template <class T, int FORM, bool SPLIT>
__device__ __forceinline__ void guarded_tile(const TileArgs& A, int id, T* smem) {
    constexpr bool PAIR = FORM == kPair, ATR = FORM == kDw, BTR = FORM == kDx || FORM == kDw;
    constexpr int KG = kGuardedGroups, MT = 2, NTW = 2, NT = PAIR ? 1 : 2;
    typedef typename Arith<T>::v8 v8;
    const int tid = threadIdx.x & 255, lane = threadIdx.x & 63;
    const int group = threadIdx.x >> 8, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    T* const sa = smem + group * 4 * kGuardedSide;  // two tiles of a, two of b
    T* const sb = sa + 2 * kGuardedSide;

    const Spot at_tile = spot<FORM>(A, id);
    const int split = at_tile.split, z = at_tile.z;
    const int64_t m0 = at_tile.tm * 64, n0 = at_tile.tn * (PAIR ? 32 : 64);

    const int64_t ksteps = (A.K + kStep - 1) / kStep;
    const int64_t total = all_steps<FORM, SPLIT>(A, ksteps);
    const int64_t first = split * A.per;
    const int64_t last = first + A.per < total ? first + A.per : total;
    const int64_t rounds = (last - first + KG - 1) / KG;

    Frags<T, ATR, MT, false, 64> fa;
    Frags<T, BTR, NT, true, 64> fb;
    fa.init(lane, wm * 32);
    fb.init(lane, wn * NT * 16);

    // both terms of kDx have pieces of their own; a pair's b is two half tiles
    Guarded<T, ATR> ga[FORM == kDx ? 2 : 1];
    Guarded<T, BTR> gb[FORM == kDx ? 2 : 1];
#pragma unroll
    for (int w = 0; w < (FORM == kDx ? 2 : 1); ++w) {
        if (w >= A.parts) break;
        ga[w].init(static_cast<const T*>(A.a[FORM == kDw ? z : w]), A.lda[FORM == kDw ? z : w],
                   m0, a_rows<FORM>(A), tid);
        if constexpr (!PAIR)
            gb[w].init(static_cast<const T*>(A.b[w]), A.ldb[w], n0, A.N, tid,
                       FORM == kDw ? A.fold : 0);
    }
    if constexpr (PAIR) {
#pragma unroll
        for (int l = 0; l < 2; ++l) {  // load l is product l's 32 rows
            const int row = tid >> 3;
            gb[0].k_at[l] = (tid & 7) * 8;
            gb[0].have[l] = n0 + row < A.N;
            gb[0].p[l] = static_cast<const T*>(A.b[l]) + (n0 + row) * A.ldb[l] + gb[0].k_at[l];
        }
    }

    u32x4 ra[2], rb[2];
    auto fetch = [&](int64_t r) {
        const int64_t t = first + r * KG + group;
        const auto step = step_at<FORM, SPLIT>(A, t, ksteps);
        const int64_t k0 = step.k0, left = t < last ? A.K - k0 : 0;
        if (FORM == kDx && step.term) {
            ga[FORM == kDx].load(step.piece + k0, left, ra);
            gb[FORM == kDx].load(k0 * A.ldb[1], left, rb);
        } else {
            ga[0].load(step.piece + (ATR ? k0 * A.lda[FORM == kDw ? z : 0] : k0), left, ra);
            gb[0].load(BTR ? k0 * A.ldb[0] : k0, left, rb);
        }
    };
    auto place_lds = [&](int buf) {
        Guarded<T, ATR>::template store<MT, false>(sa + buf * kGuardedSide, tid, ra);
        // a pair's halves are dealt to the matrix tiles within their 32 rows
        Guarded<T, BTR>::template store<NT, true>(sb + buf * kGuardedSide, tid, rb);
    };

    f32x4 acc[MT][NTW];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NTW; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    if (rounds > 0) {
        fetch(0);
        place_lds(0);
    }
    for (int64_t r = 0; r < rounds; ++r) {
        const int buf = int(r & 1);
        // tile r is in LDS, and nobody reads the other buffer any more
        __syncthreads();
        if (r + 1 < rounds) fetch(r + 1);
        const T* la = sa + buf * kGuardedSide;
        const T* lb = sb + buf * kGuardedSide;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v8 va[MT], vb[NTW];
#pragma unroll
            for (int j = 0; j < NTW; ++j)
                vb[j] = fb.get(lb + (PAIR ? j * 32 * kStep : 0), PAIR ? 0 : j, s);
#pragma unroll
            for (int i = 0; i < MT; ++i) va[i] = fa.get(la, i, s);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NTW; ++j) acc[i][j] = Arith<T>::mma(vb[j], va[i], acc[i][j]);
        }
        if (r + 1 < rounds) place_lds(buf ^ 1);
    }
    __syncthreads();
    float* const out = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = (wm * MT + mt) * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < NTW; ++j)
            put_tile<NT, BTR>(out + group * 4096 + r * 64, r, j / NT * 32 + wn * NT * 16, j % NT,
                              lane, acc[mt][j]);
    }
    __syncthreads();
    put_rows<T, FORM, 64, 64, 256 * KG>(A, split, z, m0, n0, KG, 4096,
                                        [&](int r) { return out + r * 64; });
}

constexpr int kGuardedThreads = 256 * kGuardedGroups;
constexpr int kGuardedLds = kGuardedGroups * 4 * kGuardedSide;

template <class T, int FORM, bool SPLIT>
__global__ __launch_bounds__(kGuardedThreads) void k_guarded(TileArgs A) {
    __shared__ __align__(16) T smem[kGuardedLds];
    const int64_t id = block_number();
    if (id < all_blocks<FORM>(A)) guarded_tile<T, FORM, SPLIT>(A, int(id), smem);
}

// Both gradients of a layer in one launch, and the column sums' last step.
template <class T, bool SPLIT>
__global__ __launch_bounds__(kGuardedThreads) void k_guarded_both(TileArgs dx, TileArgs dw,
                                                                  int dx_blocks, int dw_blocks,
                                                                  Sums sums) {
    __shared__ __align__(16) T smem[kGuardedLds];
    // each kind begins with the first die's workgroup
    const int64_t id = block_number(), dw0 = (dx_blocks + 7) & ~7, sum0 = dw0 + dw_blocks;
    if (id < dx_blocks)
        guarded_tile<T, kDx, SPLIT>(dx, int(id), smem);
    else if (id >= dw0 && id < sum0)
        guarded_tile<T, kDw, SPLIT>(dw, int(id - dw0), smem);
    else if (id >= sum0 && sums.out)
        sum_columns<T, kGuardedThreads>(sums, id - sum0, reinterpret_cast<float*>(smem));
}

}  // namespace layers
}  // namespace dgc
