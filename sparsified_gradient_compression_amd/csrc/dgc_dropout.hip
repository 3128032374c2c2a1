// dgc_dropout.hip -- dropout from a counter.  See include/dgc.h for the
// contract.
//
// The mask is a function of (seed, offset, row, column), so the backward pass
// makes it again and none is stored: a mask of bytes would add a quarter to a
// third to what the pass moves.  One Philox block gives 128 bits; an element
// takes 16 of them, so the eight elements that a lane loads at once cost one
// block, 40 of a lane's 32-bit multiplications: less than the bytes take.  Memory bounds it: 16384 x 4096 in bf16 with a residual 70 us
// (5.75 TB/s; an addition of two such matrices 67), 777 x 1001 in fp16 3.6 us.
#include <algorithm>

#include "tokens.hpp"

using namespace dgc::tokens;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostBlocks = 1 << 20;  // of a launch: workgroups take what is left in turn

struct Args {
    int64_t m, d;
    uint32_t kept;  // of 65536
    float scale;
    uint64_t seed, offset;
    const int64_t* step;
    const void* x;
    int64_t ldx;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    int across;           // lanes side by side on a row, a power of two
    int64_t spans, tasks;  // of `across` * 8 columns in a row; of all rows together
};

// Philox4x32-10.
__device__ __forceinline__ void philox(uint32_t* c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = uint64_t(0xD2511F53u) * c[0], q = uint64_t(0xCD9E8D57u) * c[2];
        const uint32_t c0 = uint32_t(q >> 32) ^ c[1] ^ k0, c2 = uint32_t(p >> 32) ^ c[3] ^ k1;
        c[1] = uint32_t(q);
        c[3] = uint32_t(p);
        c[0] = c0;
        c[2] = c2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// v: 8 elements of row r from column 8 * group on, residual: what is added to them.
template <bool RESIDUAL>
__device__ __forceinline__ void drop8(const Args& a, uint64_t offset, int64_t r, int64_t group, float* v,
                                      const float* residual) {
    uint32_t bits[4] = {uint32_t(group), uint32_t(r), uint32_t(offset), uint32_t(offset >> 32)};
    philox(bits, uint32_t(a.seed), uint32_t(a.seed >> 32));
#pragma unroll
    for (int i = 0; i < kRow; ++i) {
        const uint32_t u = i % 2 ? bits[i / 2] >> 16 : bits[i / 2] & 0xFFFF;
        v[i] = u < a.kept ? v[i] * a.scale : 0.0f;
        if (RESIDUAL) v[i] += residual[i];
    }
}

template <class T, bool RESIDUAL>
__global__ __launch_bounds__(kThreads) void k_dropout(Args a) {
    const uint64_t offset = a.offset + (a.step ? uint64_t(*a.step) : 0);
    const int tx = threadIdx.x & (a.across - 1), ty = threadIdx.x / a.across, rows = kThreads / a.across;
    for (int64_t task = blockIdx.x; task < a.tasks; task += gridDim.x) {
        const int64_t r = task / a.spans * rows + ty, group = task % a.spans * a.across + tx, c = group * kRow;
        const int valid = valid_of(a.d, c);
        if (r >= a.m || valid == 0) continue;
        const T* const x = static_cast<const T*>(a.x) + r * a.ldx + c;
        const T* const res = RESIDUAL ? static_cast<const T*>(a.residual) + r * a.ldr + c : nullptr;
        T* const y = static_cast<T*>(a.y) + r * a.ldy + c;
        float v[kRow], w[kRow];
        // (two ways through and through: a load behind a branch of its own would be
        // waited for there, before the next is on its way)
        if (valid == kRow) {
            const Eight<T> ex = read8(x);
            Eight<T> er;
            if (RESIDUAL) er = read8(res);
            widen(ex, v);
            if (RESIDUAL) widen(er, w);
            drop8<RESIDUAL>(a, offset, r, group, v, w);
            store8(y, kRow, v);
        } else {
            load8(x, valid, v);
            if (RESIDUAL) load8(res, valid, w);
            drop8<RESIDUAL>(a, offset, r, group, v, w);
            store8(y, valid, v);
        }
    }
}

}  // namespace

extern "C" int dgc_dropout(const dgc_dropout_args* a, hipStream_t stream) {
    if (!a || !type_ok(a->type) || !side_ok(a->m) || !side_ok(a->d) || !(a->p >= 0.0 && a->p <= 1.0))
        return DGC_EINVAL;
    const int64_t m = a->m, d = a->d;
    const int size = size_of(a->type);
    if (!mat_ok(a->x, a->ldx, m, d, size) || !optional_ok(a->residual, a->ldr, m, d, size) ||
        !mat_ok(a->y, a->ldy, m, d, size) || !optional_vec_ok(a->step, 1, 8))
        return DGC_EINVAL;
    if (m == 0 || d == 0) return DGC_OK;
    Args k{m,       d,           uint32_t(std::floor((1.0 - a->p) * 65536.0 + 0.5)), 0.0f, a->seed, a->offset,
           a->step, a->x,        a->ldx,
           a->residual, a->ldr,  a->y,
           a->ldy,  kThreads,    0,
           0};
    k.scale = k.kept ? float(65536.0 / k.kept) : 0.0f;
    while (k.across > 1 && k.across / 2 * kRow >= d) k.across /= 2;
    k.spans = cdiv(d, int64_t(k.across) * kRow);
    k.tasks = k.spans * cdiv(m, kThreads / k.across);
    return with_type(a->type, [&](auto t) {
        const auto kernel = k.residual ? k_dropout<decltype(t), true> : k_dropout<decltype(t), false>;
        kernel<<<dim3(unsigned(std::min(k.tasks, kMostBlocks))), kThreads, 0, stream>>>(k);
        return launched();
    });
}
