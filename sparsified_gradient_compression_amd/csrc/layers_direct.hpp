// layers_direct.hpp -- operand tiles that go from memory straight to LDS.
#pragma once

#include "layers_tile.hpp"

namespace dgc {
namespace layers {

// A byte offset past every buffer descriptor's end: reads as zero.
constexpr uint32_t kOutside = 0x80000000u;

// s_waitcnt's operand: at most `loads` loads and `lds` LDS operations under way.
constexpr int wait_for(int loads, int lds) {
    return (loads & 15) | (loads >> 4) << 14 | 7 << 4 | lds << 8;
}

// How the regions of one side come to LDS and to the registers.  A region is
// 64 steps of k of R rows (columns), brought in by W waves.
//   TR:    stored with m (n) contiguous: [64 k][R] in LDS
//   else:  stored with k contiguous:     [R][64]
//   NT:    16-row tiles of a wave in a region; NSIDE: dealt by n_row<NT>
// The swizzle of piece_at is applied to the addresses in memory: a wave's load
// fills 1 KB of LDS in lane order.
template <class T, bool TR, int NT, bool NSIDE, int R, int W>
struct Side : Frags<T, TR, NT, NSIDE, R> {
    static constexpr int kLoads = R / (8 * W);    // of a wave, per region
    static constexpr int kRowsK = W * 512 / R;    // TR: steps of k per load of all waves
    uint32_t at[kLoads];  // byte offset of this lane's pieces; kOutside if none
    int k_at;             // first k of the lane's piece (TR: of load 0)

    // have: how many rows (columns) there are from the region's first on
    // fold (TR): steps of k from there on are the first ones again
    __device__ __forceinline__ void init(int64_t ld, int64_t have, int wave, int lane, int base,
                                         int fold = 0) {
        Frags<T, TR, NT, NSIDE, R>::init(lane, base);
        if constexpr (TR) {
            constexpr int kPer = R / 8;  // pieces of a step of k
            const int k = wave * (64 / kPer) + lane / kPer, p = lane % kPer;
            const int piece = (((p >> 1) ^ k_key<R>(k)) << 1) | (p & 1);
            k_at = k;
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                const int row = k + kRowsK * l, from = fold && row >= fold ? row - fold : row;
                at[l] = piece * 8 < have ? uint32_t((int64_t(from) * ld + piece * 8) * 2)
                                         : kOutside;
            }
        } else {
            const int r = wave * 8 + (lane >> 3);
            const int piece = (lane & 7) ^ row_key<NT, NSIDE>(r);
            k_at = piece * 8;
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                const int row = r + 8 * W * l;
                at[l] = row < have ? uint32_t((int64_t(row) * ld + piece * 8) * 2) : kOutside;
            }
        }
    }

    // Order the region at `p` (its first row, its first k) of which `left`
    // steps of k exist, into `lds`.
    __device__ __forceinline__ void order(const T* p, int left, T* lds, int wave) const {
#if defined(__HIP_DEVICE_COMPILE__)  // the host's pass does not know 16-byte loads to LDS
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T*>(p), short(0), int(0x7FFFFFFF), 0x00020000);
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
            const uint32_t v = k_at + (TR ? kRowsK * l : 0) < left ? at[l] : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (DGC_LDS void*)(lds + (l * W + wave) * 512), 16, int(v), 0, 0, 0);
        }
#endif
    }
};

}  // namespace layers
}  // namespace dgc
