// dgc_recurrence.hip -- a gated linear recurrence along sequences, and its
// gradients.  See include/dgc.h for the contract of every function.
#include <algorithm>

#include "tokens.hpp"

using namespace dgc::tokens;

namespace {

constexpr int kLanes = 64;
constexpr int64_t kMostBlocks = 1 << 20;  // of a launch: workgroups take what is left in turn

struct Rows {
    int64_t m, d, batch;
    int wide_index;
    const void* offsets;  // or null: m / batch rows each
};

struct Forward {
    Rows s;
    const void* gate;
    int64_t ldg;
    const void* x;
    int64_t ldx;
    const float* h0;
    int64_t ldh0;
    void* h;
    int64_t ldh;
    float* state;
    int64_t lds;
};

struct Backward {
    Rows s;
    const void* dh;
    int64_t lddh;
    const void* gate;
    int64_t ldg;
    const void* x;
    int64_t ldx;
    const void* h;
    int64_t ldh;
    const float* h0;
    int64_t ldh0;
    const float* dstate;
    int64_t ldds;
    void* dgate;
    int64_t lddg;
    void* dx;
    int64_t lddx;
    float* dh0;
    int64_t lddh0;
};

// Where sequence b begins, within [0, m].
__device__ __forceinline__ int64_t row_of(const Rows& s, int64_t b) {
    if (!s.offsets) return s.m / s.batch * b;
    const int64_t r = s.wide_index ? static_cast<const int64_t*>(s.offsets)[b]
                                   : static_cast<const int32_t*>(s.offsets)[b];
    return r < 0 ? 0 : r > s.m ? s.m : r;
}

// f = sigmoid(z) and 1 - f, each accurate relative to itself.
__device__ __forceinline__ void gate_pair(float z, float& f, float& r) {
    const float e = expf(-fabsf(z)), s = 1.0f / (1.0f + e);
    f = z >= 0.0f ? s : e * s;
    r = z >= 0.0f ? e * s : s;
    if (z != z) f = r = z;
}

// A lane per column and sequence, row by row.
template <class T>
__global__ __launch_bounds__(kLanes) void k_forward(Forward a, int64_t strips) {
    const int64_t tasks = a.s.batch * strips;
    for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int64_t b = task / strips, c = task % strips * kLanes + threadIdx.x;
        if (c >= a.s.d) continue;
        float h = a.h0 ? a.h0[b * a.ldh0 + c] : 0.0f;
        const int64_t end = row_of(a.s, b + 1);
        for (int64_t t = row_of(a.s, b); t < end; ++t) {
            float f, r;
            gate_pair(float(static_cast<const T*>(a.gate)[t * a.ldg + c]), f, r);
            h = f * h + r * float(static_cast<const T*>(a.x)[t * a.ldx + c]);
            static_cast<T*>(a.h)[t * a.ldh + c] = T(h);
        }
        if (a.state) a.state[b * a.lds + c] = h;
    }
}

template <class T>
__global__ __launch_bounds__(kLanes) void k_backward(Backward a, int64_t strips) {
    const int64_t tasks = a.s.batch * strips;
    for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int64_t b = task / strips, c = task % strips * kLanes + threadIdx.x;
        if (c >= a.s.d) continue;
        float after = a.dstate ? a.dstate[b * a.ldds + c] : 0.0f;
        const int64_t begin = row_of(a.s, b);
        for (int64_t t = row_of(a.s, b + 1) - 1; t >= begin; --t) {
            float f, r;
            gate_pair(float(static_cast<const T*>(a.gate)[t * a.ldg + c]), f, r);
            const float x = float(static_cast<const T*>(a.x)[t * a.ldx + c]);
            const float h = t > begin ? float(static_cast<const T*>(a.h)[(t - 1) * a.ldh + c])
                                      : a.h0 ? a.h0[b * a.ldh0 + c] : 0.0f;
            const float g = float(static_cast<const T*>(a.dh)[t * a.lddh + c]) + after;
            if (a.dx) static_cast<T*>(a.dx)[t * a.lddx + c] = T(r * g);
            if (a.dgate) static_cast<T*>(a.dgate)[t * a.lddg + c] = T(g * (h - x) * (f * r));
            after = f * g;
        }
        if (a.dh0) a.dh0[b * a.lddh0 + c] = after;
    }
}

bool rows_ok(int64_t type, int64_t index_type, int64_t m, int64_t d, int64_t batch, const void* offsets) {
    if (!type_ok(type) || !side_ok(m) || !side_ok(d) || !side_ok(batch)) return false;
    if (offsets) return index_ok(index_type) && vec_ok(offsets, batch + 1, size_of(index_type));
    return batch == 0 ? m == 0 : m % batch == 0;
}

dim3 grid(int64_t tasks) { return dim3(unsigned(std::min(tasks, kMostBlocks))); }

}  // namespace

extern "C" {

int dgc_recurrence_workspace_bytes(int64_t m, int64_t d, int64_t batch, int32_t, size_t* bytes) {
    if (!bytes || !side_ok(m) || !side_ok(d) || !side_ok(batch) || (d > 0 && m > kMostArea / d)) return DGC_EINVAL;
    *bytes = 0;
    return DGC_OK;
}

int dgc_recurrence(const dgc_recurrence_args* a, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!a || !rows_ok(a->type, a->index_type, a->m, a->d, a->batch, a->offsets)) return DGC_EINVAL;
    const int64_t m = a->m, d = a->d, n = a->batch;
    const int size = size_of(a->type);
    if (!mat_ok(a->gate, a->ldg, m, d, size) || !mat_ok(a->x, a->ldx, m, d, size) ||
        !optional_ok(a->h0, a->ldh0, n, d, 4) || !mat_ok(a->h, a->ldh, m, d, size) ||
        !optional_ok(a->state, a->lds, n, d, 4))
        return DGC_EINVAL;
    if (n == 0 || d == 0) return DGC_OK;
    const Forward f{{m, d, n, a->index_type == DGC_INT64, a->offsets}, a->gate, a->ldg, a->x, a->ldx, a->h0, a->ldh0,
                    a->h, a->ldh, a->state, a->lds};
    const int64_t strips = cdiv(d, kLanes);
    return with_type(a->type, [&](auto t) {
        k_forward<decltype(t)><<<grid(n * strips), kLanes, 0, stream>>>(f, strips);
        return launched();
    });
}

int dgc_recurrence_backward(const dgc_recurrence_backward_args* a, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    if (!a || !rows_ok(a->type, a->index_type, a->m, a->d, a->batch, a->offsets)) return DGC_EINVAL;
    const int64_t m = a->m, d = a->d, n = a->batch;
    const int size = size_of(a->type);
    if (!mat_ok(a->dh, a->lddh, m, d, size) || !mat_ok(a->gate, a->ldg, m, d, size) ||
        !mat_ok(a->x, a->ldx, m, d, size) || !mat_ok(a->h, a->ldh, m, d, size) ||
        !optional_ok(a->h0, a->ldh0, n, d, 4) || !optional_ok(a->dstate, a->ldds, n, d, 4) ||
        !optional_ok(a->dgate, a->lddg, m, d, size) || !optional_ok(a->dx, a->lddx, m, d, size) ||
        !optional_ok(a->dh0, a->lddh0, n, d, 4))
        return DGC_EINVAL;
    if (n == 0 || d == 0) return DGC_OK;
    const Backward b{{m, d, n, a->index_type == DGC_INT64, a->offsets}, a->dh, a->lddh, a->gate, a->ldg, a->x, a->ldx,
                     a->h, a->ldh, a->h0, a->ldh0, a->dstate, a->ldds, a->dgate, a->lddg, a->dx, a->lddx, a->dh0,
                     a->lddh0};
    const int64_t strips = cdiv(d, kLanes);
    return with_type(a->type, [&](auto t) {
        k_backward<decltype(t)><<<grid(n * strips), kLanes, 0, stream>>>(b, strips);
        return launched();
    });
}

}  // extern "C"
