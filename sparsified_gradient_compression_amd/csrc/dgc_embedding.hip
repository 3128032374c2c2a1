// dgc_embedding.hip -- embedding look-up and the table's gradient.  See
// include/dgc.h for the contract of every function.
//
// The gradient sorts the tokens by id first, keeping their order among equal
// ids, so that a row's sum runs over neighbours in the sorted order and no two
// workgroups add to the same row: no atomics, and the same bits every run.
//   k_tiles   1024 ids of a workgroup sorted
//   k_merge   up to kFan sorted runs at a time made one: an id's place is its
//             own in its run plus, for each other run, how many lie before it
//   k_sum     units of kUnit sorted tokens: an id's sum over its tokens there.  An
//             id whose tokens go over a unit's ends leaves partial sums
//   k_join    adds these up
//   k_absent  zeros for the rows that no id names
#include <algorithm>

#include "tokens.hpp"

using namespace dgc::tokens;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostBlocks = 1 << 20;  // of a launch: workgroups take what is left in turn
constexpr int kTile = 1024, kSub = 256;
constexpr int kFan = 32;
constexpr int kUnit = 32;
constexpr int kAhead = 8;                 // tokens whose rows are under way together
constexpr int64_t kFillBytes = 64 << 10;  // of a workgroup's rows in k_absent

struct Lookup {
    int64_t m, vocab, d;
    int wide_index;
    const void* ids;
    const void* table;
    int64_t ldt;
    float scale;
    void* y;
    int64_t ldy;
    int across;            // lanes side by side on a row, a power of two
    int64_t spans, tasks;  // of `across` * 8 columns in a row; of all rows together
};

__device__ __forceinline__ int64_t id_at(const void* ids, int wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_lookup(Lookup a) {
    const int tx = threadIdx.x & (a.across - 1), ty = threadIdx.x / a.across, rows = kThreads / a.across;
    for (int64_t task = blockIdx.x; task < a.tasks; task += gridDim.x) {
        const int64_t r = task / a.spans * rows + ty, c = (task % a.spans * a.across + tx) * kRow;
        const int valid = valid_of(a.d, c);
        if (r >= a.m || valid == 0) continue;
        const int64_t id = id_at(a.ids, a.wide_index, r);
        float v[kRow] = {};
        if (id >= 0 && id < a.vocab) {
            load8(static_cast<const T*>(a.table) + id * a.ldt + c, valid, v);
#pragma unroll
            for (int i = 0; i < kRow; ++i) v[i] *= a.scale;
        }
        store8(static_cast<T*>(a.y) + r * a.ldy + c, valid, v);
    }
}

// ------------------------------------------------------------------ sorting

// How many of n ascending numbers are below k.
__device__ __forceinline__ int64_t below(const uint32_t* p, int64_t n, uint32_t k) {
    int64_t lo = 0;
    while (n > 0) {
        const int64_t half = n / 2;
        if (p[lo + half] < k) {
            lo += half + 1;
            n -= half + 1;
        } else {
            n = half;
        }
    }
    return lo;
}

struct Sort {
    int64_t m, vocab;
    int wide_index;
    const void* ids;
    uint32_t* key;  // ids in order; padding is `vocab`, behind all others
    uint32_t* pos;  // the tokens that they are of
};

constexpr uint32_t kBehind = 0x80000000u;  // more than any key

__global__ __launch_bounds__(kTile) void k_tiles(Sort a) {
    __shared__ uint32_t key[2][kTile];
    __shared__ uint16_t pos[2][kTile];
    const int i = threadIdx.x, sub = i / kSub * kSub;
    const int64_t first = int64_t(blockIdx.x) * kTile;
    uint32_t k = kBehind;
    if (first + i < a.m) {
        const int64_t id = id_at(a.ids, a.wide_index, first + i);
        k = id >= 0 && id < a.vocab ? uint32_t(id) : uint32_t(a.vocab);
    }
    key[0][i] = k;
    __syncthreads();
    // the place among 256, by counting; equal ones keep their order
    int rank = sub;
    for (int j = 0; j < kSub; j += 4) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(&key[0][sub + j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) rank += q[e] < k + (sub + j + e < i);
    }
    key[1][rank] = k;
    pos[1][rank] = uint16_t(i);
    __syncthreads();
    // the place among the four sorted quarters
    k = key[1][i];
    rank = i - sub;
    for (int s = 0; s < kTile; s += kSub)
        if (s != sub) rank += int(below(&key[1][s], kSub, k + (s < sub)));
    key[0][rank] = k;
    pos[0][rank] = pos[1][i];
    __syncthreads();
    if (first + i < a.m) {
        a.key[first + i] = key[0][i];
        a.pos[first + i] = uint32_t(first + pos[0][i]);
    }
}

struct Merge {
    int64_t m, run;  // runs of so many
    const uint32_t *key, *pos;
    uint32_t *key_out, *pos_out;
};

__global__ __launch_bounds__(kThreads) void k_merge(Merge a) {
    const int64_t runs = (a.m + a.run - 1) / a.run;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < a.m; i += int64_t(gridDim.x) * kThreads) {
        const int64_t r = i / a.run, first = r / kFan * kFan, last = first + kFan < runs ? first + kFan : runs;
        const uint32_t k = a.key[i];
        int64_t rank = i - r * a.run;
        for (int64_t s = first; s < last; ++s) {
            const int64_t at = s * a.run, n = a.m - at < a.run ? a.m - at : a.run;
            if (s != r) rank += below(a.key + at, n, k + (s < r));
        }
        a.key_out[first * a.run + rank] = k;
        a.pos_out[first * a.run + rank] = a.pos[i];
    }
}

// ------------------------------------------------------------------- adding

struct Sums {
    int64_t m, vocab, d;
    const uint32_t *key, *pos;
    const void* dy;
    int64_t lddy;
    float scale;
    int accumulate;
    void* dtable;
    int64_t lddt;
    float* part;  // [units][2][d]: of an id that came from before the unit, and of one that goes on behind it
    int64_t units;
    int across;
    int64_t spans, tasks;
    int64_t rows;  // of a workgroup in k_absent
};

template <class G>
__device__ __forceinline__ void finish8(const Sums& a, uint32_t id, int64_t c, int valid, const float* sum) {
    G* const p = static_cast<G*>(a.dtable) + int64_t(id) * a.lddt + c;
    float v[kRow], old[kRow];
    if (a.accumulate) load8(p, valid, old);
#pragma unroll
    for (int i = 0; i < kRow; ++i) v[i] = a.accumulate ? old[i] + a.scale * sum[i] : a.scale * sum[i];
    store8(p, valid, v);
}

template <class T, class G>
__global__ __launch_bounds__(kThreads) void k_sum(Sums a) {
    const int tx = threadIdx.x & (a.across - 1), ty = threadIdx.x / a.across, each = kThreads / a.across;
    for (int64_t task = blockIdx.x; task < a.tasks; task += gridDim.x) {
        const int64_t u = task / a.spans * each + ty, c = (task % a.spans * a.across + tx) * kRow;
        const int valid = valid_of(a.d, c);
        if (u >= a.units || valid == 0) continue;
        const int64_t begin = u * kUnit, end = begin + kUnit < a.m ? begin + kUnit : a.m;
        uint32_t id = a.key[begin];
        bool before = begin > 0 && a.key[begin - 1] == id;
        float sum[kRow] = {};
        float* const part = a.part + u * 2 * a.d + c;
        for (int64_t t = begin; t < end; t += kAhead) {
            Eight<T> row[kAhead];
            uint32_t key[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                key[j] = t + j < end ? a.key[t + j] : uint32_t(a.vocab);
                const int64_t from = t + j < end ? a.pos[t + j] : a.pos[begin];
                row[j] = read8(static_cast<const T*>(a.dy) + from * a.lddy + c, valid);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (key[j] != id) {
                    if (t + j < end) {
                        if (id < a.vocab) {
                            if (before)
                                store8(part, valid, sum);
                            else
                                finish8<G>(a, id, c, valid, sum);
                        }
                        before = false;
                        id = key[j];
#pragma unroll
                        for (int i = 0; i < kRow; ++i) sum[i] = 0.0f;
                    }
                }
                float v[kRow];
                widen(row[j], v);
                if (t + j < end)
#pragma unroll
                    for (int i = 0; i < kRow; ++i) sum[i] += v[i];
            }
        }
        if (id >= a.vocab) continue;
        if (before)
            store8(part, valid, sum);
        else if (end < a.m && a.key[end] == id)
            store8(part + a.d, valid, sum);
        else
            finish8<G>(a, id, c, valid, sum);
    }
}

// The id whose tokens begin in unit u and go on behind it, over all units that it
// reaches.
template <class G>
__global__ __launch_bounds__(kThreads) void k_join(Sums a) {
    const int tx = threadIdx.x & (a.across - 1), ty = threadIdx.x / a.across, each = kThreads / a.across;
    for (int64_t task = blockIdx.x; task < a.tasks; task += gridDim.x) {
        const int64_t u = task / a.spans * each + ty, c = (task % a.spans * a.across + tx) * kRow;
        const int valid = valid_of(a.d, c);
        const int64_t begin = u * kUnit, end = begin + kUnit;
        if (end >= a.m || valid == 0) continue;
        const uint32_t id = a.key[end - 1];
        if (id >= a.vocab || a.key[end] != id) continue;
        if (a.key[begin] == id && begin > 0 && a.key[begin - 1] == id) continue;  // begins earlier
        const int64_t last = (end + below(a.key + end, a.m - end, id + 1) - 1) / kUnit;
        double sum[kRow];
        float v[kRow];
        load8(a.part + (u * 2 + 1) * a.d + c, valid, v);
#pragma unroll
        for (int i = 0; i < kRow; ++i) sum[i] = double(v[i]);
#pragma unroll 4
        for (int64_t w = u + 1; w <= last; ++w) {
            load8(a.part + w * 2 * a.d + c, valid, v);
#pragma unroll
            for (int i = 0; i < kRow; ++i) sum[i] += double(v[i]);
        }
#pragma unroll
        for (int i = 0; i < kRow; ++i) v[i] = float(sum[i]);
        finish8<G>(a, id, c, valid, v);
    }
}

template <class G>
__global__ __launch_bounds__(kThreads) void k_absent(Sums a) {
    __shared__ uint8_t named[kThreads];
    const int64_t chunks = (a.vocab + a.rows - 1) / a.rows;
    for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
        const int64_t first = chunk * a.rows, mine = first + threadIdx.x;
        const int count = int(a.vocab - first < a.rows ? a.vocab - first : a.rows);
        __syncthreads();
        if (int(threadIdx.x) < count) {
            const int64_t at = below(a.key, a.m, uint32_t(mine));
            named[threadIdx.x] = at < a.m && a.key[at] == uint32_t(mine);
        }
        __syncthreads();
        const float zero[kRow] = {};
        for (int r = 0; r < count; ++r)
            if (!named[r])
                for (int64_t c = threadIdx.x * kRow; c < a.d; c += kThreads * kRow)
                    store8(static_cast<G*>(a.dtable) + (first + r) * a.lddt + c, valid_of(a.d, c), zero);
    }
}

// --------------------------------------------------------------------- host

struct Space {
    size_t key[2], pos[2], part, total;
};

Space space(int64_t m, int64_t d) {
    Space s{};
    const size_t list = round_up(size_t(m) * 4);
    for (int i = 0; i < 2; ++i) {
        s.key[i] = s.total;
        s.pos[i] = s.total + list;
        s.total += 2 * list;
    }
    s.part = s.total;
    if (m > kUnit) s.total += round_up(size_t(cdiv(m, kUnit)) * 2 * size_t(d) * 4);
    return s;
}

int across_of(int64_t d) {
    int across = kThreads;
    while (across > 1 && across / 2 * kRow >= d) across /= 2;
    return across;
}

dim3 grid(int64_t tasks) { return dim3(unsigned(std::min(tasks, kMostBlocks))); }

}  // namespace

extern "C" {

int dgc_embedding_workspace_bytes(int64_t m, int64_t vocab, int64_t d, int32_t backward, size_t* bytes) {
    if (!bytes || !side_ok(m) || !side_ok(vocab) || !side_ok(d) || (d > 0 && m > kMostArea / d)) return DGC_EINVAL;
    *bytes = backward && m > 0 && d > 0 ? space(m, d).total : 0;
    return DGC_OK;
}

int dgc_embedding(const dgc_embedding_args* a, hipStream_t stream) {
    if (!a || !type_ok(a->type) || !index_ok(a->index_type) || !side_ok(a->m) || !side_ok(a->vocab) ||
        !side_ok(a->d) || !std::isfinite(a->scale))
        return DGC_EINVAL;
    const int64_t m = a->m, d = a->d;
    const int size = size_of(a->type);
    if (!vec_ok(a->ids, m, size_of(a->index_type)) || !mat_ok(a->table, a->ldt, a->vocab, d, size) ||
        !mat_ok(a->y, a->ldy, m, d, size))
        return DGC_EINVAL;
    if (m == 0 || d == 0) return DGC_OK;
    Lookup k{m, a->vocab, d, a->index_type == DGC_INT64, a->ids, a->table, a->ldt, float(a->scale), a->y, a->ldy,
             across_of(d), 0, 0};
    k.spans = cdiv(d, int64_t(k.across) * kRow);
    k.tasks = k.spans * cdiv(m, kThreads / k.across);
    return with_type(a->type, [&](auto t) {
        k_lookup<decltype(t)><<<grid(k.tasks), kThreads, 0, stream>>>(k);
        return launched();
    });
}

int dgc_embedding_backward(const dgc_embedding_backward_args* a, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    if (!a || !type_ok(a->type) || (a->grad_type != a->type && a->grad_type != DGC_FP32) ||
        !index_ok(a->index_type) || !side_ok(a->m) || !side_ok(a->vocab) || !side_ok(a->d) ||
        !std::isfinite(a->scale) || (a->accumulate != 0 && a->accumulate != 1))
        return DGC_EINVAL;
    const int64_t m = a->m, d = a->d, vocab = a->vocab;
    const int gsize = size_of(a->grad_type);
    if (!mat_ok(a->dy, a->lddy, m, d, size_of(a->type)) || !vec_ok(a->ids, m, size_of(a->index_type)) ||
        !mat_ok(a->dtable, a->lddt, vocab, d, gsize) || (d > 0 && m > kMostArea / d))
        return DGC_EINVAL;
    const Space sp = space(m, d);
    int rc = space_ok(workspace, workspace_bytes, m > 0 && d > 0 ? sp.total : 0);
    if (rc != DGC_OK) return rc;
    if (vocab == 0 || d == 0 || (m == 0 && a->accumulate)) return DGC_OK;
    char* const ws = static_cast<char*>(workspace);
    uint32_t *key[2], *pos[2];
    for (int i = 0; i < 2; ++i) {
        key[i] = reinterpret_cast<uint32_t*>(ws + sp.key[i]);
        pos[i] = reinterpret_cast<uint32_t*>(ws + sp.pos[i]);
    }
    int in = 0;
    if (m > 0) {
        const Sort s{m, vocab, a->index_type == DGC_INT64, a->ids, key[0], pos[0]};
        k_tiles<<<dim3(unsigned(cdiv(m, kTile))), kTile, 0, stream>>>(s);
        for (int64_t run = kTile; run < m; run *= kFan, in ^= 1)
            k_merge<<<grid(cdiv(m, kThreads)), kThreads, 0, stream>>>(
                Merge{m, run, key[in], pos[in], key[in ^ 1], pos[in ^ 1]});
    }
    Sums k{m, vocab, d, key[in], pos[in], a->dy, a->lddy, float(a->scale), int(a->accumulate), a->dtable, a->lddt,
           reinterpret_cast<float*>(ws + sp.part), cdiv(m, kUnit), across_of(d), 0, 0, 0};
    k.spans = cdiv(d, int64_t(k.across) * kRow);
    k.tasks = k.spans * cdiv(k.units, kThreads / k.across);
    k.rows = std::max<int64_t>(1, std::min<int64_t>(kThreads, kFillBytes / (d * gsize)));
    return with_type(a->type, [&](auto t) {
        typedef decltype(t) T;
        const auto with = [&](auto g) {
            typedef decltype(g) G;
            if (!k.accumulate) k_absent<G><<<grid(cdiv(vocab, k.rows)), kThreads, 0, stream>>>(k);
            if (m > 0) k_sum<T, G><<<grid(k.tasks), kThreads, 0, stream>>>(k);
            if (m > kUnit) k_join<G><<<grid(k.tasks), kThreads, 0, stream>>>(k);
            return launched();
        };
        return a->grad_type == DGC_FP32 ? with(float()) : with(t);
    });
}

}  // extern "C"
