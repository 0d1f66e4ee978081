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

template <int V> struct Values { float x[V]; };

// V channels (consecutive, V elements aligned) of an operand's row.
template <typename IO, int V>
__device__ __forceinline__ Values<V> load_values(const void *base, int64_t off) {
    const IO *at = static_cast<const IO *>(base) + off;
    Values<V> y;
    if constexpr (V == 1) {
        y.x[0] = Conv<IO, 1>::in(*reinterpret_cast<const typename Raw<IO, 1>::type *>(at));
    } else if constexpr (sizeof(IO) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(at));
        y.x[0] = a.x; y.x[1] = a.y; y.x[2] = a.z; y.x[3] = a.w;
    } else {
        const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(at));
        const float2 lo = Conv<IO, 2>::in(a.x), hi = Conv<IO, 2>::in(a.y);
        y.x[0] = lo.x; y.x[1] = lo.y; y.x[2] = hi.x; y.x[3] = hi.y;
    }
    return y;
}
template <typename IO, int V>
__device__ __forceinline__ void store_values(void *base, int64_t off, const Values<V> &y) {
    IO *at = static_cast<IO *>(base) + off;
    if constexpr (V == 1) {
        *reinterpret_cast<typename Raw<IO, 1>::type *>(at) = Conv<IO, 1>::out(y.x[0]);
    } else if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<float4 *>(at) = make_float4(y.x[0], y.x[1], y.x[2], y.x[3]);
    } else {
        *reinterpret_cast<uint2 *>(at) = make_uint2(Conv<IO, 2>::out(make_float2(y.x[0], y.x[1])),
                                                    Conv<IO, 2>::out(make_float2(y.x[2], y.x[3])));
    }
}

// A block takes 256 V U channels of one row.  Rows that name a slot already
// named by an earlier row are taken by that row's block, in row order: a slot
// that appears twice receives two tokens one after the other, and no two
// blocks ever touch the same state.  The row's operands are on their way while
// the slots are looked through, by every block the whole list: nothing beside
// the rest up to some thousand rows, then quadratic (1024 bf16 channels: 4096
// rows 25 us against 12 without slots, 32768 rows 890 against 91).  U vectors a
// thread keep enough bytes in flight
// (509 rows of 4096 bf16 channels, states in fp32: 9.2 us, 10.6 with one; their
// 29 MB take 4.5 us from memory, the rest is the start and the slots' search).
template <typename IO, int GATE, int V, int U>
__global__ void __launch_bounds__(256) gated_step_kernel(const StepParams p) {
    const int64_t row = blockIdx.x / p.d_blocks;
    const int64_t d0 = ((blockIdx.x - row * p.d_blocks) * U * 256 + threadIdx.x) * V;
    Values<V> f[U], v[U], st[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t d = d0 + u * 256 * V;
        if (d < p.D) {
            f[u] = load_values<IO, V>(p.f, row * p.f_rs + d);
            v[u] = load_values<IO, V>(p.v, row * p.v_rs + d);
        }
    }
    int64_t slot = row;
    bool again = false;
    if (p.slots) {
        slot = slot_at(p, row);
        bool before = false, after = false;
        for (int64_t j = threadIdx.x; j < p.rows; j += 256) {
            if (j != row && slot_at(p, j) == slot) {
                if (j < row) before = true;
                else after = true;
            }
        }
        const bool taken = __syncthreads_or(before);
        again = __syncthreads_or(after);
        if (slot < 0 || slot >= p.n_slots) {              // padding
            if (p.zero_padding) {
                Values<V> zero;
#pragma unroll
                for (int i = 0; i < V; ++i) zero.x[i] = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (d0 + u * 256 * V < p.D) store_values<IO, V>(p.h, row * p.h_rs + d0 + u * 256 * V, zero);
            }
            return;
        }
        if (taken) return;
    }
    float *sp = p.state + slot * p.state_rs;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t d = d0 + u * 256 * V;
        if (d >= p.D) continue;
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(sp + d);
            st[u].x[0] = x.x; st[u].x[1] = x.y; st[u].x[2] = x.z; st[u].x[3] = x.w;
        } else {
            st[u].x[0] = sp[d];
        }
    }
    auto token = [&](int64_t r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t d = d0 + u * 256 * V;
            if (d >= p.D) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float a, b;
                gate_pair<GATE>(f[u].x[i], v[u].x[i], a, b);
                st[u].x[i] = fmaf(a, st[u].x[i], b);
            }
            store_values<IO, V>(p.h, r * p.h_rs + d, st[u]);
        }
    };
    token(row);
    if (again) {
        for (int64_t j = row + 1; j < p.rows; ++j) {
            if (slot_at(p, j) != slot) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t d = d0 + u * 256 * V;
                if (d < p.D) {
                    f[u] = load_values<IO, V>(p.f, j * p.f_rs + d);
                    v[u] = load_values<IO, V>(p.v, j * p.v_rs + d);
                }
            }
            token(j);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t d = d0 + u * 256 * V;
        if (d >= p.D) continue;
        if constexpr (V == 4) {
            *reinterpret_cast<float4 *>(sp + d) = make_float4(st[u].x[0], st[u].x[1], st[u].x[2], st[u].x[3]);
        } else {
            sp[d] = st[u].x[0];
        }
    }
}

}  // namespace gated
}  // namespace sgr
