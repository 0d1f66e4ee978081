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
};

template <typename OUT>
__device__ __forceinline__ void put(const ProjectParams &p, int64_t m, int64_t n, int acc, float sx, float sw, float b) {
    using R = typename Raw<OUT, 1>::type;
    reinterpret_cast<R *>(p.y)[m * p.y_rs + n] = Conv<OUT, 1>::out(fmaf(float(acc) * sx, sw, b));
}

// ---------------------------------------------------------- quantisation
//
// s = max |x| / 127 (at least 2^-100), q = x / s to the nearest whole number,
// ties to even.  The quotient is decided exactly: with q0 = rint(x (1 / s)),
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

struct QuantParams {
    const void *x;
    int64_t x_rs;                  // elements
    int8_t *q;
    int64_t q_rs;                  // bytes
    float *scale;
    int64_t rows, K;
};

// largest |x| of a row: NaN where one is NaN
__device__ __forceinline__ float absmax(float m, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
    return r;
}

// (scale, 1 / scale) of a row whose largest |x| is m
__device__ __forceinline__ float2 row_scale(float m) {
    if (!(m <= 3.402823466e38f)) return make_float2(__int_as_float(0x7fffffff), 0.f);
    const float s = fmaxf(__fdiv_rn(m, 127.f), kScaleFloor);
    return make_float2(s, __fdiv_rn(1.f, s));
}

// One row per TPR threads of a block of 256, held in registers between the
// maximum and the rounding: NV vectors of 16 bytes a thread, so the row is
// read once.  Rows that do not fit (NV = 0) or do not start on 16-byte
// boundaries are read twice, element by element.
template <typename IO> __device__ __forceinline__ void unpack16(uint4 x, float (&v)[16 / sizeof(IO)]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(IO) == 4) {
            v[i] = __uint_as_float(w[i]);
        } else {
            const float2 t = Conv<IO, 2>::in(w[i]);
            v[2 * i] = t.x;
            v[2 * i + 1] = t.y;
        }
    }
}

template <typename IO, int TPR, int NV>
__global__ void __launch_bounds__(256) int8_quantize_kernel(const QuantParams p) {
    constexpr int VEC = 16 / sizeof(IO), ROWS = 256 / TPR;
    __shared__ float s_max[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = threadIdx.x % TPR;
    // a block reduction holds a barrier, so every thread of the block stays in the loop
    for (int64_t row0 = int64_t(blockIdx.x) * ROWS; row0 < p.rows; row0 += int64_t(gridDim.x) * ROWS) {
        const int64_t row = row0 + threadIdx.x / TPR;
        const bool on = row < p.rows;
        const IO *x = static_cast<const IO *>(p.x) + (on ? row : 0) * p.x_rs;
        using W = typename Raw<IO, 1>::type;
        float v[NV > 0 ? NV : 1][VEC];
        float m = 0.f;
        if constexpr (NV > 0) {
            uint4 raw[NV];
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
            for (int i = 0; i < NV; ++i) {
                unpack16<IO>(raw[i], v[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) m = absmax(m, v[i][j]);
            }
        } else if (on) {
            for (int64_t k = part; k < p.K; k += TPR) m = absmax(m, Conv<IO, 1>::in(reinterpret_cast<const W *>(x)[k]));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = absmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        if constexpr (TPR > 32) {
            if (lane == 0) s_max[warp] = m;
            __syncthreads();
            m = s_max[0];
#pragma unroll
            for (int w = 1; w < 8; ++w) m = absmax(m, s_max[w]);
            __syncthreads();
        }
        const float2 s = row_scale(m);
        if (!on) continue;
        if (part == 0) p.scale[row] = s.x;
        int8_t *q = p.q + row * p.q_rs;
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t k = int64_t(i * TPR + part) * VEC;
                uint32_t w[VEC / 4];
#pragma unroll
                for (int j = 0; j < VEC / 4; ++j) {
                    w[j] = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        w[j] |= uint32_t(uint8_t(s.y == 0.f ? 0 : quantize_one(v[i][4 * j + b], s.x, s.y))) << (8 * b);
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
// shared memory, four-byte dot products.  Rows may start at any byte.
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
    const int64_t m0 = int64_t(blockIdx.y) * 64, n0 = int64_t(blockIdx.x) * 64;
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
