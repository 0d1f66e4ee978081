// int8_projection.cuh -- products of 8-bit integers with a scale for each
// token (row of x) and each channel (row of w):
//   y[m, n] = (sum_k x[m, k] w[n, k]) s_x[m] s_w[n] + bias[n]
// The sum is exact in int32 (rows of at most 2^17 - 1 values); scales, bias
// and the one rounding to the output type are fp32.
#pragma once

#include "gated_math.cuh"

namespace sgr {
namespace i8 {

using gated::Conv;
using gated::Raw;

constexpr float kScaleFloor = 7.888609052210118e-31f;      // 2^-100

struct ProjectParams {
    const int8_t *x, *w;
    int64_t x_rs, w_rs;            // row strides, bytes
    const float *x_scale, *w_scale, *bias;
    void *y;
    int64_t y_rs;                  // elements
    int64_t M, N, K;
    uint32_t epilogue_polls;       // polls of the pair kernel's epilogue for a product,
    uint64_t epilogue_ns;          // and how long it goes on behind them
};

template <typename OUT>
__device__ __forceinline__ void put(const ProjectParams &p, int64_t m, int64_t n, int acc, float sx, float sw, float b) {
    using R = typename Raw<OUT, 1>::type;
    reinterpret_cast<R *>(p.y)[m * p.y_rs + n] = Conv<OUT, 1>::out(fmaf(float(acc) * sx, sw, b));
}

// ---------------------------------------------------------- quantisation
//
// s = max |x| times 1/127, both in fp32 (at least 2^-100), q = x / s to the
// nearest whole number, ties to even.  The quotient is decided exactly: with q0 = rint(x (1 / s)),
// off by one at most, the signs of the fused x - (q0 +- 1/2) s, which fma
// rounds but never changes, say on which side of the half the quotient lies.
// A row that holds an infinity or NaN gets the scale NaN and zeros, so its
// outputs are NaN.
__device__ __forceinline__ int quantize_one(float x, float s, float inv) {
    float q = rintf(x * inv);
    const bool odd = int(q) & 1;
    const float up = fmaf(-(q + 0.5f), s, x), down = fmaf(-(q - 0.5f), s, x);
    if (up > 0.f || (up == 0.f && odd)) q += 1.f;
    else if (down < 0.f || (down == 0.f && odd)) q -= 1.f;
    return int(q);
}

// N values at once: t = x (1 / s) + 3 2^22 leaves a whole number in its low
// bits.  x (1 / s) is off from the quotient by at most 127 2^-23 (the hardware's
// 1 / s), so where it is more than 2^-15 away from a half the whole number is
// right; a group with a quotient nearer to one (one in two thousand) is
// decided exactly.  Packs four to a word.
template <int N>
__device__ __forceinline__ void quantize_words(const float2 (&x)[N / 2], float s, float inv, uint32_t (&w)[N / 4]) {
    const float2 i2 = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f), minus = make_float2(-1.f, -1.f);
    float2 t[N / 2];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        t[i] = __ffma2_rn(x[i], i2, magic);
        const float2 d = __ffma2_rn(x[i], i2, __ffma2_rn(t[i], minus, magic));
        far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
    }
    if (far > 0.5f - 1.f / 32768.f) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 v = x[i];
            t[i] = make_float2(__int_as_float(quantize_one(v.x, s, inv)), __int_as_float(quantize_one(v.y, s, inv)));
        }
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint32_t lo = __byte_perm(__float_as_uint(t[2 * i].x), __float_as_uint(t[2 * i].y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(t[2 * i + 1].x), __float_as_uint(t[2 * i + 1].y), 0x0040);
        w[i] = __byte_perm(lo, hi, 0x5410);
    }
}

struct QuantParams {
    const void *x;
    int64_t x_rs;                  // elements
    int8_t *q;
    int64_t q_rs;                  // bytes
    float *scale;
    int64_t rows, K;
};

// (scale, the hardware's 1 / scale) of a row whose largest |x| is m; the second
// is 0 for a row that is not finite.
__device__ __forceinline__ float2 row_scale(float m) {
    if (!(m <= 3.402823466e38f)) return make_float2(__int_as_float(0x7fffffff), 0.f);
    const float s = fmaxf(m * (1.f / 127.f), kScaleFloor);
    return make_float2(s, fast_rcp(s));
}

// One row per TPR threads of a block of 256, held in registers between the
// maximum and the rounding: NV vectors of 16 bytes a thread, so the row is
// read once.  Rows that do not fit (NV = 0) or do not start on 16-byte
// boundaries are read twice, element by element.  Short rows take a warp
// each, longer ones four warps or the block: a row's barrier passes under the
// others' loads.  8192 rows of 4096 bf16: 31 us, 15 of them memory's (a warp a
// row, 16 vectors a lane, needed 245 registers and 117 us).
template <typename IO> __device__ __forceinline__ void unpack16(const uint4 &x, float2 (&v)[8 / sizeof(IO)]) {
    if constexpr (sizeof(IO) == 4) {
        v[0] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
        v[1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
    } else {
        v[0] = Conv<IO, 2>::in(x.x);
        v[1] = Conv<IO, 2>::in(x.y);
        v[2] = Conv<IO, 2>::in(x.z);
        v[3] = Conv<IO, 2>::in(x.w);
    }
}
// Largest |x| as bits: magnitudes of one type order as whole numbers do, NaN
// above all.  16-bit types two at a time, the halves joined at the end.
template <typename H2> __device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    const H2 m = __hmax2_nan(*reinterpret_cast<const H2 *>(&a), __habs2(*reinterpret_cast<const H2 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <typename IO> __device__ __forceinline__ uint32_t max_bits(uint32_t m, const uint4 &x) {
    if constexpr (sizeof(IO) == 4) {
        const uint32_t k = 0x7fffffffu;
        return max(max(max(m, x.x & k), max(x.y & k, x.z & k)), x.w & k);
    } else {
        using H2 = typename std::conditional<std::is_same<IO, __half>::value, __half2, __nv_bfloat162>::type;
        return max_pair<H2>(max_pair<H2>(max_pair<H2>(max_pair<H2>(m, x.x), x.y), x.z), x.w);
    }
}
template <typename IO> __device__ __forceinline__ uint32_t join_bits(uint32_t m) {
    return sizeof(IO) == 4 ? m : max(m & 0xffffu, m >> 16);
}
template <typename IO> __device__ __forceinline__ float max_value(uint32_t m) {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(m);
    else return Conv<IO, 1>::in(uint16_t(m));
}

template <typename IO, int TPR, int NV>
__global__ void __launch_bounds__(256, NV >= 4 ? 4 : 6) int8_quantize_kernel(const QuantParams p) {
    constexpr int VEC = 16 / sizeof(IO), ROWS = 256 / TPR;
    __shared__ uint32_t s_max[2][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    const int part = threadIdx.x % TPR;
    using W = typename Raw<IO, 1>::type;
    asm volatile("griddepcontrol.launch_dependents;");     // a product behind it may set up now
    // a block reduction holds a barrier, so every thread of the block stays in the loop
    for (int64_t row0 = int64_t(blockIdx.x) * ROWS; row0 < p.rows; row0 += int64_t(gridDim.x) * ROWS) {
        const int64_t row = row0 + threadIdx.x / TPR;
        const bool on = row < p.rows;
        const IO *x = static_cast<const IO *>(p.x) + (on ? row : 0) * p.x_rs;
        uint4 raw[NV > 0 ? NV : 1];
        uint32_t bits = 0;
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t k = int64_t(i * TPR + part) * VEC;
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if (on && k + VEC <= p.K) {
                    raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x + k));
                } else if (on && k < p.K) {
                    for (int j = 0; j < int(p.K - k); ++j) {
                        const uint32_t e = reinterpret_cast<const W *>(x)[k + j];
                        const int at = j * int(sizeof(IO));
                        const uint32_t y = sizeof(IO) == 4 ? e : e << (8 * (at & 3));
                        if (at < 4) raw[i].x |= y;
                        else if (at < 8) raw[i].y |= y;
                        else if (at < 12) raw[i].z |= y;
                        else raw[i].w |= y;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) bits = max_bits<IO>(bits, raw[i]);
            bits = join_bits<IO>(bits);
        } else if (on) {
            for (int64_t k = part; k < p.K; k += TPR)
                bits = max(bits, uint32_t(reinterpret_cast<const W *>(x)[k]) & (sizeof(IO) == 4 ? 0x7fffffffu : 0x7fffu));
        }
        bits = __reduce_max_sync(0xffffffffu, bits);
        if constexpr (TPR > 32) {
            constexpr int PER = TPR / 32;                  // warps of a row
            if (lane == 0) s_max[turn][warp] = bits;
            __syncthreads();                               // one a row: the next writes the other half
            bits = __reduce_max_sync(0xffffffffu, s_max[turn][warp / PER * PER + lane % PER]);
            turn ^= 1;
        }
        const float2 s = row_scale(max_value<IO>(bits));
        if (!on) continue;
        if (part == 0) p.scale[row] = s.x;
        int8_t *q = p.q + row * p.q_rs;
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t k = int64_t(i * TPR + part) * VEC;
                uint32_t w[VEC / 4] = {};
                if (s.y != 0.f) {
                    float2 v[VEC / 2];
                    unpack16<IO>(raw[i], v);
                    quantize_words<VEC>(v, s.x, s.y, w);
                }
                if (k + VEC <= p.K) {
                    if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(q + k) = make_uint2(w[0], w[1]);
                    else *reinterpret_cast<uint32_t *>(q + k) = w[0];
                } else {
                    for (int j = 0; j < int(p.K - k); ++j) q[k + j] = int8_t(w[j / 4] >> (8 * (j % 4)));
                }
            }
        } else {
            for (int64_t k = part; k < p.K; k += TPR)
                q[k] = s.y == 0.f ? int8_t(0) : int8_t(quantize_one(Conv<IO, 1>::in(reinterpret_cast<const W *>(x)[k]), s.x, s.y));
        }
    }
}

// -------------------------------------------------- product, any layout
//
// 64 x 64 outputs per block of 256 threads, 64 bytes of K at a time through
// shared memory, four-byte dot products.  Rows may start at any byte.  Bound by
// the integer pipe: 8192 x 4096 x 8192 7.5 ms, so for odd layouts only.
__device__ __forceinline__ int load_word(const int8_t *row, int64_t k, int64_t K) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k + i < K) v |= uint32_t(uint8_t(row[k + i])) << (8 * i);
    return int(v);
}

template <typename OUT>
__global__ void __launch_bounds__(256) int8_project_any_kernel(const ProjectParams p) {
    __shared__ int s_x[64][17], s_w[64][17];
    const unsigned across = unsigned((p.N + 63) / 64);
    const int64_t m0 = int64_t(blockIdx.x / across) * 64, n0 = int64_t(blockIdx.x % across) * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 64) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i >> 4, c = i & 15;
            s_x[r][c] = m0 + r < p.M ? load_word(p.x + (m0 + r) * p.x_rs, k0 + 4 * c, p.K) : 0;
            s_w[r][c] = n0 + r < p.N ? load_word(p.w + (n0 + r) * p.w_rs, k0 + 4 * c, p.K) : 0;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(s_x[ty + 16 * i][c], s_w[tx + 16 * j][c], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty + 16 * i;
        if (m >= p.M) continue;
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx + 16 * j;
            if (n < p.N) put<OUT>(p, m, n, acc[i][j], p.x_scale[m], p.w_scale[n], p.bias ? p.bias[n] : 0.f);
        }
    }
}

}  // namespace i8
}  // namespace sgr
