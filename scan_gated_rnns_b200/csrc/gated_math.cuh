// gated_math.cuh -- element arithmetic of the gated linear recurrence
// (gated_scan, gated_scan_backward, gated_step): vectors of one or two
// channels, storage types, and the two gates.
//
//   GATE_SIGMOID: a = sigmoid(f),       z = sigmoid(-f) = 1 - a, h' = a h + z v
//   GATE_LOG:     a = exp(min(f, 0)),                            h' = a h + v
//
// All arithmetic and every state is fp32; 16-bit inputs widen exactly and
// outputs round to nearest-even once, at the store.  NaN in f or v reaches
// every later state of its sequence and channel, and nothing else.
#pragma once

#include "scan_engine.cuh"

#include <cuda_fp16.h>

namespace sgr {
namespace gated {

enum { GATE_SIGMOID = 0, GATE_LOG = 1 };

// ------------------------------------------------ one or two channels
template <int E> struct FVec;
template <> struct FVec<1> { using type = float; };
template <> struct FVec<2> { using type = float2; };

__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
template <class F> __device__ __forceinline__ float vmap(float a, F f) { return f(a); }
template <class F> __device__ __forceinline__ float2 vmap(float2 a, F f) { return make_float2(f(a.x), f(a.y)); }
template <class F> __device__ __forceinline__ float vmap(float a, float b, F f) { return f(a, b); }
template <class F> __device__ __forceinline__ float2 vmap(float2 a, float2 b, F f) {
    return make_float2(f(a.x, b.x), f(a.y, b.y));
}
template <class F> __device__ __forceinline__ float vmap(float a, float b, float c, F f) { return f(a, b, c); }
template <class F> __device__ __forceinline__ float2 vmap(float2 a, float2 b, float2 c, F f) {
    return make_float2(f(a.x, b.x, c.x), f(a.y, b.y, c.y));
}
template <class T> __device__ __forceinline__ T vset(float x);
template <> __device__ __forceinline__ float vset<float>(float x) { return x; }
template <> __device__ __forceinline__ float2 vset<float2>(float x) { return make_float2(x, x); }

// minimum that keeps NaN
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ------------------------------------------------------------- storage
// E consecutive elements of type IO, as they lie in memory.
template <typename IO, int E> struct Raw;
template <> struct Raw<float, 1> { using type = uint32_t; };
template <> struct Raw<__nv_bfloat16, 1> { using type = uint16_t; };
template <> struct Raw<__nv_bfloat16, 2> { using type = uint32_t; };
template <> struct Raw<__half, 1> { using type = uint16_t; };
template <> struct Raw<__half, 2> { using type = uint32_t; };

template <typename IO, int E> struct Conv;
template <> struct Conv<float, 1> {
    static __device__ __forceinline__ float in(uint32_t r) { return __uint_as_float(r); }
    static __device__ __forceinline__ uint32_t out(float x) { return __float_as_uint(x); }
};
template <> struct Conv<__nv_bfloat16, 1> {
    static __device__ __forceinline__ float in(uint16_t r) { return __uint_as_float(uint32_t(r) << 16); }
    static __device__ __forceinline__ uint16_t out(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <> struct Conv<__nv_bfloat16, 2> {
    static __device__ __forceinline__ float2 in(uint32_t r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t out(float2 x) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <> struct Conv<__half, 1> {
    static __device__ __forceinline__ float in(uint16_t r) { return __half2float(__ushort_as_half(r)); }
    static __device__ __forceinline__ uint16_t out(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
template <> struct Conv<__half, 2> {
    static __device__ __forceinline__ float2 in(uint32_t r) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&r));
    }
    static __device__ __forceinline__ uint32_t out(float2 x) {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// --------------------------------------------------------------- gates

// sigmoid(-|f|) in [0, 1/2] with the sign bit set where f >= 0.  The smaller
// of the two probabilities is computed with its own relative accuracy and the
// larger is 1 minus it (exact to an fp32 rounding, since the smaller is at
// most 1/2), so neither a nor 1 - a loses bits when the gate closes on one
// side; one register holds both.  2 MUFU operations.
__device__ __forceinline__ float signed_small(float f) {
    const float e = fast_exp2(fabsf(f) * kNegLog2e);          // exp(-|f|)
    const float s = e * fast_rcp(1.f + e);
    return __uint_as_float(__float_as_uint(s) | (~__float_as_uint(f) & 0x80000000u));
}
// (a, z) from it
__device__ __forceinline__ void split_small(float s, float &a, float &z) {
    const float u = fabsf(s), w = 1.f - u;
    const bool pos = __float_as_uint(s) >> 31;
    a = pos ? w : u;
    z = pos ? u : w;
}
__device__ __forceinline__ void split_small(float2 s, float2 &a, float2 &z) {
    split_small(s.x, a.x, z.x);
    split_small(s.y, a.y, z.y);
}

// The same pair for the scan, E channels at a time, in one value that keeps
// the smaller probability's own bits: hold_gate once per element, open_gate
// wherever a and z are needed.  fp32 I/O: signed_small as above.  16-bit I/O:
// the states are fp32 and the gradients z g and a z (h - v) g of an open gate
// are small numbers that 16 bits hold, so z must not come from 1 - a (1 % off
// at f = 12, 0 from f = 17 on); but the two channels of a thread go through
// packed arithmetic: with c = 1 where p < 0, a = c + p and z = (1 - c) - p
// are each the held value or one rounding from 1.  The 2^-126 keeps p from
// being a zero without a side (there the hardware's 2^x ends as well).  bf16
// 32768 x 4096 in 23 sequences forward, 16384 x 2048 backward: 181 and 98 us;
// with split_small's selects 201 and 100; 1 - a 165 and 85, and wrong.
template <typename IO, class V> __device__ __forceinline__ V hold_gate(V f) {
    if constexpr (sizeof(IO) == 4) {
        return vmap(f, [](float x) { return signed_small(x); });
    } else {
        const V x = vmul(f, vset<V>(kNegLog2e));
        const V e = vmap(x, [](float t) { return fast_exp2(-fabsf(t)); });          // exp(-|f|)
        const V s = vfma(e, vmap(vadd(e, vset<V>(1.f)), [](float t) { return fast_rcp(t); }), vset<V>(1.17549435e-38f));
        return vmap(s, x, [](float u, float t) {                                    // negative where f >= 0
            return __uint_as_float(__float_as_uint(u) | (__float_as_uint(t) & 0x80000000u));
        });
    }
}
__device__ __forceinline__ float one_if_negative(float p) {
    float c;
    asm("set.lt.f32.f32 %0, %1, 0f00000000;" : "=f"(c) : "f"(p));
    return c;
}
template <typename IO, class V> __device__ __forceinline__ void open_gate(V p, V &a, V &z) {
    if constexpr (sizeof(IO) == 4) {
        split_small(p, a, z);
    } else {
        const V c = vmap(p, [](float x) { return one_if_negative(x); });
        a = vadd(c, p);
        z = vfma(p, vset<V>(-1.f), vfma(c, vset<V>(-1.f), vset<V>(1.f)));
    }
}

// exp(min(f, 0)).  Decays near 1 carry an fp32 state over thousands of steps,
// whatever the type of f, where the MUFU's 2^x would drift (2^-22 a step, not
// centred); for f > -1/4 the Taylor series 1 + f + ... + f^7 / 7!, whose rest
// is below 2^-31, keeps the error at fp32's rounding of a.  Below -1/4 memory
// is a few steps and the MUFU's error stays where it is.  Packed for two
// channels: bf16 32768 x 4096 in 23 sequences 166 us, 186 a channel at a time,
// 158 by the MUFU alone.
template <class V> __device__ __forceinline__ V log_decay(V f) {
    const V x = vmap(f, [](float t) { return min_nan(t, 0.f); });
    const V far = vmap(vmul(x, vset<V>(-kNegLog2e)), [](float t) { return fast_exp2(t); });
    V p = vset<V>(1.f / 5040.f);
    p = vfma(p, x, vset<V>(1.f / 720.f));
    p = vfma(p, x, vset<V>(1.f / 120.f));
    p = vfma(p, x, vset<V>(1.f / 24.f));
    p = vfma(p, x, vset<V>(1.f / 6.f));
    p = vfma(p, x, vset<V>(0.5f));
    p = vfma(p, x, vset<V>(1.f));
    const V near = vfma(p, x, vset<V>(1.f));
    return vmap(x, near, far, [](float t, float n, float g) { return t > -0.25f ? n : g; });
}

// (f, v) -> (a, b) of h' = a h + b
template <int GATE, class V>
__device__ __forceinline__ void gate_pair(V f, V v, V &a, V &b) {
    if constexpr (GATE == GATE_SIGMOID) {
        V z;
        split_small(vmap(f, [](float x) { return signed_small(x); }), a, z);
        b = vmul(z, v);
    } else {
        a = log_decay(f);
        b = v;
    }
}

}  // namespace gated
}  // namespace sgr
