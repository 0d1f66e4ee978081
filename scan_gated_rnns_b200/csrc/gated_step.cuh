// gated_step.cuh -- one token of the gated linear recurrence for each of M
// requests, on a pool of fp32 states that the call updates in place.
#pragma once

#include "gated_math.cuh"

namespace sgr {
namespace gated {

struct StepParams {
    const void *f, *v;
    void *h;
    int64_t f_rs, v_rs, h_rs;
    float *state;                  // (n_slots, D), rows state_rs apart
    int64_t state_rs, n_slots;
    const void *slots;             // M slot numbers, or null: row i has slot i
    int slot_bytes;                // 4 or 8
    int64_t rows, D;
    int64_t d_blocks;              // blocks per row
    int zero_padding;
};

__device__ __forceinline__ int64_t slot_at(const StepParams &p, int64_t i) {
    return p.slot_bytes == 8 ? static_cast<const int64_t *>(p.slots)[i]
                             : int64_t(static_cast<const int32_t *>(p.slots)[i]);
}

// V channels (consecutive, V elements aligned) of one row.
template <typename IO, int GATE, int V>
__device__ __forceinline__ void step_row(const StepParams &p, int64_t row, int64_t d, float (&st)[V]) {
    float f[V], v[V], y[V];
    const IO *fp = static_cast<const IO *>(p.f) + row * p.f_rs + d;
    const IO *vp = static_cast<const IO *>(p.v) + row * p.v_rs + d;
    IO *hp = static_cast<IO *>(p.h) + row * p.h_rs + d;
    if constexpr (V == 1) {
        f[0] = Conv<IO, 1>::in(*reinterpret_cast<const typename Raw<IO, 1>::type *>(fp));
        v[0] = Conv<IO, 1>::in(*reinterpret_cast<const typename Raw<IO, 1>::type *>(vp));
    } else if constexpr (sizeof(IO) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(fp)), b = __ldcs(reinterpret_cast<const float4 *>(vp));
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        v[0] = b.x; v[1] = b.y; v[2] = b.z; v[3] = b.w;
    } else {
        const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(fp)), b = __ldcs(reinterpret_cast<const uint2 *>(vp));
        const float2 f0 = Conv<IO, 2>::in(a.x), f1 = Conv<IO, 2>::in(a.y);
        const float2 v0 = Conv<IO, 2>::in(b.x), v1 = Conv<IO, 2>::in(b.y);
        f[0] = f0.x; f[1] = f0.y; f[2] = f1.x; f[3] = f1.y;
        v[0] = v0.x; v[1] = v0.y; v[2] = v1.x; v[3] = v1.y;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float a, b;
        gate_pair<GATE, IO>(f[i], v[i], a, b);
        y[i] = st[i] = fmaf(a, st[i], b);
    }
    if constexpr (V == 1) {
        *reinterpret_cast<typename Raw<IO, 1>::type *>(hp) = Conv<IO, 1>::out(y[0]);
    } else if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<float4 *>(hp) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
        *reinterpret_cast<uint2 *>(hp) = make_uint2(Conv<IO, 2>::out(make_float2(y[0], y[1])),
                                                    Conv<IO, 2>::out(make_float2(y[2], y[3])));
    }
}

// A block takes 256 V channels of one row.  Rows that name a slot already
// named by an earlier row are taken by that row's block, in row order: a slot
// that appears twice receives two tokens one after the other, and no two
// blocks ever touch the same state.
template <typename IO, int GATE, int V>
__global__ void __launch_bounds__(256) gated_step_kernel(const StepParams p) {
    const int64_t row = blockIdx.x / p.d_blocks;
    const int64_t d = ((blockIdx.x - row * p.d_blocks) * blockDim.x + threadIdx.x) * V;
    int64_t slot = row;
    bool again = false;
    if (p.slots) {
        slot = slot_at(p, row);
        bool before = false, after = false;
        for (int64_t j = threadIdx.x; j < p.rows; j += blockDim.x) {
            if (j != row && slot_at(p, j) == slot) {
                if (j < row) before = true;
                else after = true;
            }
        }
        const bool taken = __syncthreads_or(before);
        again = __syncthreads_or(after);
        if (slot < 0 || slot >= p.n_slots) {              // padding
            if (p.zero_padding) {
                for (int i = 0; i < V; ++i)
                    if (d + i < p.D)
                        *reinterpret_cast<typename Raw<IO, 1>::type *>(static_cast<IO *>(p.h) + row * p.h_rs + d + i) = 0;
            }
            return;
        }
        if (taken) return;
    }
    if (d >= p.D) return;
    float *sp = p.state + slot * p.state_rs + d;
    float st[V];
    if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(sp);
        st[0] = x.x; st[1] = x.y; st[2] = x.z; st[3] = x.w;
    } else {
        st[0] = *sp;
    }
    step_row<IO, GATE, V>(p, row, d, st);
    if (again) {
        for (int64_t j = row + 1; j < p.rows; ++j)
            if (slot_at(p, j) == slot) step_row<IO, GATE, V>(p, j, d, st);
    }
    if constexpr (V == 4) {
        *reinterpret_cast<float4 *>(sp) = make_float4(st[0], st[1], st[2], st[3]);
    } else {
        *sp = st[0];
    }
}

}  // namespace gated
}  // namespace sgr
