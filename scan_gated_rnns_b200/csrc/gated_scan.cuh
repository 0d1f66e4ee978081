// gated_scan.cuh -- the gated linear recurrence h_t = a_t h_{t-1} + b_t over
// rows of packed sequences, forward and backward, for sm_100a.
//
// Rows of all sequences lie one behind another; a sequence begins at a row
// that is a "start", where the state is replaced by the sequence's initial
// state.  The steps of a run of rows compose to one affine map (A, B),
// h -> A h + B, or, where the run holds a start, to the constant B: such a
// map is a "cut", written A = -0 (products of the non-negative a keep the
// sign), and is never multiplied with what came before, so nothing that an
// earlier sequence held (infinities, NaN) reaches a later one.
//
// A tile is kTR rows x TC channels (128 bytes of a row).  Data warp w owns
// rows [16 w, 16 w + 16), lane l channels [E l, E l + E): a thread folds its
// 16 rows in registers, the seven folds of a channel meet in shared memory,
// and the carry warp finds the state that enters the tile; the threads then
// replay their rows from it.  Inputs are read once and outputs written once.
//
// The carry between tiles of one channel strip: each publishes its map (flag
// 1), finds the nearest earlier tile whose final state is published (flag 2),
// applies the maps between, oldest first, and publishes its own final state.
// The arithmetic is the sequential S_q = A_q S_{q-1} + B_q wherever that
// state came from, so results do not depend on timing.  Blocks take tiles by
// ticket in the order they run, so a wait is always for a tile that a running
// block holds; waits are bounded.
#pragma once

#include "gated_math.cuh"

namespace sgr {
namespace gated {

constexpr int kWarps = 7;                  // data warps; the eighth carries
constexpr int kRows = 16;                  // rows per data warp and thread
constexpr int kTR = kWarps * kRows;        // rows per tile, and between saved states
constexpr int kThreads = (kWarps + 1) * 32;
constexpr uint32_t kFlagMap = 1, kFlagState = 2;

struct GatedParams {
    const void *f, *v, *dh;                // (rows, D), unit stride along D
    int64_t f_rs, v_rs, dh_rs;             // row strides, elements
    void *h, *df, *dv;
    int64_t h_rs, df_rs, dv_rs;
    const float *h0;                       // (n_seqs, D) rows h0_ss apart, or null: zero
    int64_t h0_ss;
    float *h_last;                         // (n_seqs, D) or null
    const float *dh_last;                  // (n_seqs, D) or null
    float *dh0;                            // (n_seqs, D) or null
    float *states;                         // (n_chunks, D): forward: state entering each chunk
    const void *cu;                        // n_seqs + 1 row bounds, or null: sequences of seq_rows rows
    int cu_bytes;                          // 4 or 8
    uint32_t seq_rows;
    int64_t rows, D, n_seqs;
    int64_t n_strips, n_chunks, n_tiles;
    int zero_padding;                      // outputs of rows in no sequence: 0 written, else left
    float *carry;                          // backward: (n_chunks, D) as states, in processing order
    float2 *maps;                          // [n_tiles][TC]
    uint32_t *flags;                       // [n_strips][n_chunks], zero at launch
    uint32_t *ticket;                      // zero at launch, or null: tile = blockIdx.x
    uint32_t *status;                      // or null (one chunk: nothing waits)
    uint32_t spin_limit;
};

__device__ __forceinline__ int64_t cu_at(const GatedParams &p, int64_t i) {
    return p.cu_bytes == 8 ? static_cast<const int64_t *>(p.cu)[i] : int64_t(static_cast<const int32_t *>(p.cu)[i]);
}

__device__ __forceinline__ bool is_cut(float A) { return __float_as_uint(A) >> 31; }
// the map (A, B) applied to a state, and `then` after `first`
__device__ __forceinline__ float apply_map(float A, float B, float h) { return is_cut(A) ? B : fmaf(A, h, B); }
__device__ __forceinline__ float2 then_map(float2 first, float2 then) {
    return make_float2(first.x * then.x, is_cut(then.x) ? then.y : fmaf(then.x, first.y, then.y));
}

// What the carry warp tells the data warps of a tile.
struct TileInfo {
    int64_t tile;
    int64_t lo, hi;                        // rows that lie in sequences
    int start[kTR], end[kTR];              // sequence that starts (ends) at the row, or -1
};

// Fill the table of the tile of rows [row0, row0 + kTR) (whole warp).  Bounds
// that are not ascending give wrong sequences but never a row or a sequence
// outside the buffers.
__device__ __forceinline__ void fill_info(const GatedParams &p, int64_t row0, TileInfo &t, int lane) {
    const int64_t row_end = row0 + kTR < p.rows ? row0 + kTR : p.rows;
    if (p.cu == nullptr) {
        for (int r = lane; r < kTR; r += 32) {
            const uint32_t n = uint32_t(row0 + r), s = n / p.seq_rows, k = n - s * p.seq_rows;
            const bool in = row0 + r < p.rows;
            t.start[r] = in && k == 0 ? int(s) : -1;
            t.end[r] = in && k + 1 == p.seq_rows ? int(s) : -1;
        }
        if (lane == 0) { t.lo = 0; t.hi = p.rows; }
        __syncwarp();
        return;
    }
    for (int r = lane; r < kTR; r += 32) t.start[r] = t.end[r] = -1;
    if (lane == 0) {
        const int64_t lo = cu_at(p, 0), hi = cu_at(p, p.n_seqs);
        t.lo = lo;
        t.hi = hi < p.rows ? hi : p.rows;
    }
    // bounds at or below row0, by a 33-way search: the last of them begins the
    // sequence that holds row0
    int64_t lo = 0, hi = p.n_seqs + 1;
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32;
        const int64_t i = lo + (lane + 1) * step - 1;
        const bool below = i < hi && cu_at(p, i) <= row0;
        const int n = __popc(__ballot_sync(0xffffffffu, below));
        const int64_t next = lo + n * step;
        const int64_t top = lo + (n + 1) * step - 1;
        lo = next < hi ? next : hi;
        hi = top < hi ? top : hi;
    }
    __syncwarp();
    for (int64_t s = (lo > 0 ? lo - 1 : 0) + lane;; s += 32) {
        bool more = false;
        if (s < p.n_seqs) {
            const int64_t b = cu_at(p, s), e = cu_at(p, s + 1);
            more = b < row_end;
            if (b < e) {
                if (b >= row0 && b < row_end) t.start[b - row0] = int(s);
                if (e > row0 && e <= row_end) t.end[e - 1 - row0] = int(s);
            }
        }
        if (!__any_sync(0xffffffffu, more)) break;
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t ld_acquire_u32(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release_u32(uint32_t *p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ float ld_relaxed_f32(const float *p) {
    float v;
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_relaxed_f2(const float2 *p) {
    const uint64_t v = ld_relaxed_u64(reinterpret_cast<const uint64_t *>(p));
    return make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
}

// The carry of one tile (carry warp): q its place in processing order along
// its strip, tot the tile's maps of this lane's E channels.  Publishes,
// waits, and returns the entering states; `carry` row q + 1 receives the
// final ones.  Tiles whose first row (in processing order) is a start enter
// with 0, which they never use.
template <int E>
__device__ __forceinline__ void carry_tile_state(const GatedParams &p, float *carry, int64_t strip, int64_t q, int lane,
                                                 bool fresh, const float2 (&tot)[E], float (&hin)[E]) {
    constexpr int TC = 32 * E;
    const int64_t d0 = strip * TC + lane * E;
    uint32_t *flags = p.flags + strip * p.n_chunks;
    const bool last = q + 1 == p.n_chunks;
    const bool cut = __any_sync(0xffffffffu, is_cut(tot[0].x));    // a start cuts all channels alike
#pragma unroll
    for (int e = 0; e < E; ++e) hin[e] = 0.f;
    auto publish_state = [&] {
        if (last) return;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d0 + e < p.D) carry[(q + 1) * p.D + d0 + e] = apply_map(tot[e].x, tot[e].y, hin[e]);
        __syncwarp();
        if (lane == 0) st_release_u32(flags + q, kFlagState);
    };
    if (fresh || q == 0) {
        publish_state();
        return;
    }
    if (cut) {
        publish_state();
    } else if (!last) {
#pragma unroll
        for (int e = 0; e < E; ++e) p.maps[(q * p.n_strips + strip) * TC + lane * E + e] = tot[e];
        __syncwarp();
        if (lane == 0) st_release_u32(flags + q, kFlagMap);
    }
    // the nearest published state among the 32 tiles before, all nearer maps there
    int k = -1;
    for (uint32_t polls = 0;; ++polls) {
        const int64_t i = q - 1 - lane;
        const uint32_t fl = i >= 0 ? ld_acquire_u32(flags + i) : 0u;
        const uint32_t state = __ballot_sync(0xffffffffu, fl == kFlagState);
        const uint32_t any = __ballot_sync(0xffffffffu, fl != 0u);
        if (state != 0u) {
            k = __ffs(state) - 1;
            const uint32_t nearer = (1u << k) - 1u;
            if ((any & nearer) == nearer) break;
        }
        if (polls >= p.spin_limit) {
            k = -1;
            break;
        }
        if (polls > 4) __nanosleep(64);
    }
    __syncwarp();
    if (k < 0) {
        if (lane == 0) atomicOr(p.status, kTimeoutBit);
#pragma unroll
        for (int e = 0; e < E; ++e) hin[e] = __int_as_float(0x7fffffff);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d0 + e < p.D) hin[e] = ld_relaxed_f32(carry + (q - k) * p.D + d0 + e);
        for (int j = k; j > 0; j -= 4) {
            float2 m[4][E];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    m[u][e] = j - u > 0 ? ld_relaxed_f2(p.maps + ((q - j + u) * p.n_strips + strip) * TC + lane * E + e)
                                        : make_float2(1.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (j - u > 0) {
#pragma unroll
                    for (int e = 0; e < E; ++e) hin[e] = apply_map(m[u][e].x, m[u][e].y, hin[e]);
                }
            }
        }
    }
    if (!cut) publish_state();
}

// Final (and gradient of initial) states of sequences without rows, which no
// tile visits: dst = src, or 0.
__device__ __forceinline__ void empty_sequences(const GatedParams &p, float *dst, const float *src, int64_t src_ss) {
    if (dst == nullptr || (p.cu == nullptr && p.rows > 0)) return;
    for (int64_t s = blockIdx.x; s < p.n_seqs; s += gridDim.x) {
        if (p.cu && cu_at(p, s) < cu_at(p, s + 1)) continue;
        for (int64_t d = threadIdx.x; d < p.D; d += blockDim.x) dst[s * p.D + d] = src ? src[s * src_ss + d] : 0.f;
    }
}

// E floats at a row of states, for this lane's channels
template <int E>
__device__ __forceinline__ typename FVec<E>::type state_row(const float *base, int64_t off, int64_t d0, int64_t D) {
    if constexpr (E == 1) {
        return base && d0 < D ? base[off + d0] : 0.f;
    } else {
        float2 x = make_float2(0.f, 0.f);
        if (base && d0 < D) x.x = base[off + d0];
        if (base && d0 + 1 < D) x.y = base[off + d0 + 1];
        return x;
    }
}
template <int E>
__device__ __forceinline__ void put_state_row(float *base, int64_t off, int64_t d0, int64_t D, typename FVec<E>::type x) {
    if constexpr (E == 1) {
        if (d0 < D) base[off + d0] = x;
    } else {
        if (d0 < D) base[off + d0] = x.x;
        if (d0 + 1 < D) base[off + d0 + 1] = x.y;
    }
}

// Streaming load and store of one thread's E channels of a row.  E = 2 is
// chosen only for even D, strides and 4-byte aligned bases, so a pair never
// straddles the last channel.
template <typename IO, int E>
__device__ __forceinline__ typename Raw<IO, E>::type load_raw(const void *base, int64_t off) {
    return __ldcs(reinterpret_cast<const typename Raw<IO, E>::type *>(static_cast<const IO *>(base) + off));
}
template <typename IO, int E>
__device__ __forceinline__ void store_raw(void *base, int64_t off, typename Raw<IO, E>::type x) {
    __stcs(reinterpret_cast<typename Raw<IO, E>::type *>(static_cast<IO *>(base) + off), x);
}

// ------------------------------------------------------------- forward
template <typename IO, int E, int GATE>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_kernel(const GatedParams p) {
    using V = typename FVec<E>::type;
    using R = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    constexpr int TC = 32 * E;
    __shared__ TileInfo s_info[2];
    __shared__ V s_A[kWarps][32], s_B[kWarps][32], s_in[kWarps][32];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n_tiles = p.n_tiles;
    auto prepare = [&](int par, bool first) {             // carry warp: the next tile and its table
        int64_t tile = n_tiles;
        if (p.ticket) {
            uint32_t t = 0;
            if (lane == 0) t = atomicAdd(p.ticket, 1u);
            tile = __shfl_sync(0xffffffffu, t, 0);
        } else if (first) {
            tile = blockIdx.x;
        }
        if (tile < n_tiles) fill_info(p, int64_t(uint32_t(tile) / uint32_t(p.n_strips)) * kTR, s_info[par], lane);
        if (lane == 0) s_info[par].tile = tile;
        __syncwarp();
    };
    if (warp == kWarps) prepare(0, true);
    for (int par = 0;; par ^= 1) {
        __syncthreads();                                  // the table is there; the last tile's is free
        const TileInfo &info = s_info[par];
        const int64_t tile = info.tile;
        if (tile >= n_tiles) break;
        const int64_t chunk = uint32_t(tile) / uint32_t(p.n_strips), strip = tile - chunk * p.n_strips;
        if (warp < kWarps) {
            const int64_t row0 = chunk * kTR + warp * kRows;
            const int64_t d0 = strip * TC + lane * E;
            const bool dvalid = d0 < p.D;
            R rf[kRows], rv[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const bool ok = dvalid && row0 + r < p.rows;
                rf[r] = ok ? load_raw<IO, E>(p.f, (row0 + r) * p.f_rs + d0) : R(0);
                rv[r] = ok ? load_raw<IO, E>(p.v, (row0 + r) * p.v_rs + d0) : R(0);
            }
            // rows of this warp that start or end a sequence, and that lie in one
            const int rr = lane & 15;
            const uint32_t starts = __ballot_sync(0xffffffffu, info.start[warp * kRows + rr] >= 0) & 0xffffu;
            const uint32_t ends = __ballot_sync(0xffffffffu, info.end[warp * kRows + rr] >= 0) & 0xffffu;
            const uint32_t live =
                __ballot_sync(0xffffffffu, row0 + rr >= info.lo && row0 + rr < info.hi) & 0xffffu;
            V a[kRows], b[kRows];
            V A = vset<V>(1.f), B = vset<V>(0.f);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                gate_pair<GATE, IO>(C::in(rf[r]), C::in(rv[r]), a[r], b[r]);
                if (starts >> r & 1u) {
                    A = vset<V>(-0.f);
                    B = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                }
                B = vfma(a[r], B, b[r]);
                A = vmul(A, a[r]);
            }
            s_A[warp][lane] = A;
            s_B[warp][lane] = B;
            named_barrier_arrive(1, kThreads);
            named_barrier_sync(2, kThreads);
            V h = s_in[warp][lane];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (starts >> r & 1u) h = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                h = vfma(a[r], h, b[r]);
                if (live >> r & 1u) {
                    if (dvalid) store_raw<IO, E>(p.h, (row0 + r) * p.h_rs + d0, C::out(h));
                } else if (p.zero_padding && dvalid && row0 + r < p.rows) {
                    store_raw<IO, E>(p.h, (row0 + r) * p.h_rs + d0, R(0));
                }
                if (ends >> r & 1u) {
                    if (p.h_last) put_state_row<E>(p.h_last, info.end[warp * kRows + r] * p.D, d0, p.D, h);
                }
            }
        } else {
            prepare(par ^ 1, false);
            named_barrier_sync(1, kThreads);
            float2 pre[kWarps][E], tot[E];
#pragma unroll
            for (int e = 0; e < E; ++e) tot[e] = make_float2(1.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *A = reinterpret_cast<const float *>(&s_A[w][lane]);
                const float *B = reinterpret_cast<const float *>(&s_B[w][lane]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    pre[w][e] = make_float2(A[e], B[e]);
                    tot[e] = then_map(tot[e], pre[w][e]);
                }
            }
            float hin[E];
            carry_tile_state<E>(p, p.states, strip, chunk, lane, info.start[0] >= 0, tot, hin);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                float *in = reinterpret_cast<float *>(&s_in[w][lane]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    in[e] = hin[e];
                    hin[e] = apply_map(pre[w][e].x, pre[w][e].y, hin[e]);
                }
            }
            named_barrier_arrive(2, kThreads);
        }
    }
    empty_sequences(p, p.h_last, p.h0, p.h0_ss);
}

// ------------------------------------------------------------ backward
//
// g_t = dh_t + a_{t+1} g_{t+1} within a sequence (its last row adds dh_last);
// with r_t = a_t g_t, the flow into the row before, the reverse pass is the
// recurrence r_t = a_t r_{t+1} + a_t dh_t, run over the tiles from the last.
//   GATE_SIGMOID: dv = z g, df = a z (h_{t-1} - v) g
//   GATE_LOG:     dv = g,   df = [f <= 0] a h_{t-1} g
// and dh0 of a sequence is r at its first row.  h_{t-1} is recomputed from
// the fp32 state that entered the tile, saved by the forward pass (one row of
// D per kTR rows), instead of being read back: the outputs h are not needed,
// so the pass reads three arrays and not four, and the states have not been
// rounded to 16 bits.
template <typename IO, int E, int GATE>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_backward_kernel(const GatedParams p) {
    using V = typename FVec<E>::type;
    using R = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    constexpr int TC = 32 * E;
    __shared__ TileInfo s_info[2];
    __shared__ V s_A[kWarps][32], s_B[kWarps][32];        // forward maps
    __shared__ V s_RA[kWarps][32], s_RB[kWarps][32];      // reverse maps
    __shared__ V s_in[kWarps][32];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n_tiles = p.n_tiles;
    auto prepare = [&](int par, bool first) {
        int64_t tile = n_tiles;
        if (p.ticket) {
            uint32_t t = 0;
            if (lane == 0) t = atomicAdd(p.ticket, 1u);
            tile = __shfl_sync(0xffffffffu, t, 0);
        } else if (first) {
            tile = blockIdx.x;
        }
        if (tile < n_tiles) fill_info(p, (p.n_chunks - 1 - uint32_t(tile) / uint32_t(p.n_strips)) * kTR, s_info[par], lane);
        if (lane == 0) s_info[par].tile = tile;
        __syncwarp();
    };
    if (warp == kWarps) prepare(0, true);
    for (int par = 0;; par ^= 1) {
        __syncthreads();
        const TileInfo &info = s_info[par];
        const int64_t tile = info.tile;
        if (tile >= n_tiles) break;
        const int64_t q = uint32_t(tile) / uint32_t(p.n_strips), strip = tile - q * p.n_strips, chunk = p.n_chunks - 1 - q;
        if (warp < kWarps) {
            const int64_t row0 = chunk * kTR + warp * kRows;
            const int64_t d0 = strip * TC + lane * E;
            const bool dvalid = d0 < p.D;
            R rf[kRows], rv[kRows], rg[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const bool ok = dvalid && row0 + r < p.rows;
                rf[r] = ok ? load_raw<IO, E>(p.f, (row0 + r) * p.f_rs + d0) : R(0);
                rv[r] = ok ? load_raw<IO, E>(p.v, (row0 + r) * p.v_rs + d0) : R(0);
                rg[r] = ok ? load_raw<IO, E>(p.dh, (row0 + r) * p.dh_rs + d0) : R(0);
            }
            V h = info.start[0] >= 0 || chunk == 0 ? vset<V>(0.f) : state_row<E>(p.states, chunk * p.D, d0, p.D);
            const int rr = lane & 15;
            const uint32_t starts = __ballot_sync(0xffffffffu, info.start[warp * kRows + rr] >= 0) & 0xffffu;
            const uint32_t ends = __ballot_sync(0xffffffffu, info.end[warp * kRows + rr] >= 0) & 0xffffu;
            const uint32_t live =
                __ballot_sync(0xffffffffu, row0 + rr >= info.lo && row0 + rr < info.hi) & 0xffffu;
            // s: the gate of each row (GATE_SIGMOID: signed small probability; GATE_LOG: a,
            // negated where f > 0, which has no gradient)
            V s[kRows];
            V A = vset<V>(1.f), B = vset<V>(0.f);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                V a, b;
                const V f = C::in(rf[r]), v = C::in(rv[r]);
                if constexpr (GATE == GATE_SIGMOID) {
                    V z;
                    s[r] = vmap(f, [](float x) { return signed_small(x); });
                    split_small(s[r], a, z);
                    b = vmul(z, v);
                } else {
                    s[r] = vmap(f, [](float x) {
                        const float t = log_decay<sizeof(IO) == 4>(x);
                        return x > 0.f ? -t : t;
                    });
                    a = vmap(s[r], [](float x) { return fabsf(x); });
                    b = v;
                }
                if (starts >> r & 1u) {
                    A = vset<V>(-0.f);
                    B = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                }
                B = vfma(a, B, b);
                A = vmul(A, a);
            }
            V RA = vset<V>(1.f), RB = vset<V>(0.f);
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                V a, z;
                if constexpr (GATE == GATE_SIGMOID) split_small(s[r], a, z);
                else a = vmap(s[r], [](float x) { return fabsf(x); });
                if (ends >> r & 1u) {
                    RA = vset<V>(-0.f);
                    RB = state_row<E>(p.dh_last, info.end[warp * kRows + r] * p.D, d0, p.D);
                }
                RB = vmul(a, vadd(RB, C::in(rg[r])));
                RA = vmul(RA, a);
            }
            s_A[warp][lane] = A;
            s_B[warp][lane] = B;
            s_RA[warp][lane] = RA;
            s_RB[warp][lane] = RB;
            named_barrier_arrive(1, kThreads);
            named_barrier_sync(3, kWarps * 32);           // the data warps' maps are there
            for (int w = 0; w < warp; ++w) {
                const V a = s_A[w][lane], b = s_B[w][lane];
                h = vmap(a, b, h, [](float x, float y, float z) { return apply_map(x, y, z); });
            }
            V c[kRows];                                   // df = c g
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (starts >> r & 1u) h = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                const V v = C::in(rv[r]);
                if constexpr (GATE == GATE_SIGMOID) {
                    V a, z;
                    split_small(s[r], a, z);
                    c[r] = vmul(vmul(a, z), vadd(h, vmul(v, vset<V>(-1.f))));
                    h = vfma(a, h, vmul(z, v));
                } else {
                    c[r] = vmap(s[r], h, [](float x, float y) { return is_cut(x) ? 0.f : x * y; });
                    h = vfma(vmap(s[r], [](float x) { return fabsf(x); }), h, v);
                }
            }
            named_barrier_sync(2, kThreads);
            V flow = s_in[warp][lane];
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                if (ends >> r & 1u) flow = state_row<E>(p.dh_last, info.end[warp * kRows + r] * p.D, d0, p.D);
                const V g = vadd(flow, C::in(rg[r]));
                V a, gv;
                if constexpr (GATE == GATE_SIGMOID) {
                    V z;
                    split_small(s[r], a, z);
                    gv = vmul(z, g);
                } else {
                    a = vmap(s[r], [](float x) { return fabsf(x); });
                    gv = g;
                }
                if (dvalid && row0 + r < p.rows) {
                    if (live >> r & 1u) {
                        store_raw<IO, E>(p.df, (row0 + r) * p.df_rs + d0, C::out(vmul(c[r], g)));
                        store_raw<IO, E>(p.dv, (row0 + r) * p.dv_rs + d0, C::out(gv));
                    } else {
                        store_raw<IO, E>(p.df, (row0 + r) * p.df_rs + d0, R(0));
                        store_raw<IO, E>(p.dv, (row0 + r) * p.dv_rs + d0, R(0));
                    }
                }
                flow = vmul(a, g);
                if (starts >> r & 1u) {
                    if (p.dh0) put_state_row<E>(p.dh0, info.start[warp * kRows + r] * p.D, d0, p.D, flow);
                }
            }
        } else {
            prepare(par ^ 1, false);
            named_barrier_sync(1, kThreads);
            float2 pre[kWarps][E], tot[E];
#pragma unroll
            for (int e = 0; e < E; ++e) tot[e] = make_float2(1.f, 0.f);
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                const float *A = reinterpret_cast<const float *>(&s_RA[w][lane]);
                const float *B = reinterpret_cast<const float *>(&s_RB[w][lane]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    pre[w][e] = make_float2(A[e], B[e]);
                    tot[e] = then_map(tot[e], pre[w][e]);
                }
            }
            float hin[E];
            carry_tile_state<E>(p, p.carry, strip, q, lane, info.end[kTR - 1] >= 0, tot, hin);
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                float *in = reinterpret_cast<float *>(&s_in[w][lane]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    in[e] = hin[e];
                    hin[e] = apply_map(pre[w][e].x, pre[w][e].y, hin[e]);
                }
            }
            named_barrier_arrive(2, kThreads);
        }
    }
    empty_sequences(p, p.dh0, p.dh_last, p.D);
}

}  // namespace gated
}  // namespace sgr
