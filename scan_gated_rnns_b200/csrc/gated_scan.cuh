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
// The carry between tiles of one channel strip: each publishes its map, finds
// the nearest earlier tile whose final state is published, applies the maps
// between, oldest first, and publishes its own final state.  The arithmetic
// is the sequential S_q = A_q S_{q-1} + B_q wherever that state came from, so
// results do not depend on timing.  A map is one 64-bit word, a state one
// 32-bit word per channel, all of them ~0 before the launch and valid once
// they are not (arithmetic never gives that NaN), so a look-back is one round
// trip to L2, without flags or fences.  Blocks take tiles by ticket in the
// order they run, so a wait is always for a tile that a running block holds;
// waits are bounded.
//
// Persistent blocks, two per SM.  The carry warp also keeps a ring of kSlots
// tiles filled by the tensor memory accelerator (TMA; rows that start on
// 16-byte boundaries; else the data warps load from memory themselves), and
// hands each tile's table of sequence starts and ends over with it.
#pragma once

#include "gated_math.cuh"

namespace sgr {
namespace gated {

constexpr int kWarps = 7;                  // data warps; the eighth carries
constexpr int kRows = 16;                  // rows per data warp and thread
constexpr int kTR = kWarps * kRows;        // rows per tile, and between saved states
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kSlots = 3;                  // forward ring
constexpr int kBwdSlots = 2;               // backward ring
constexpr uint32_t kNone = 0xffffffffu;    // a word not yet published

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
    float *states;                         // (n_chunks, D): state entering each chunk, or null (forward)
    const void *cu;                        // n_seqs + 1 row bounds, or null: sequences of seq_rows rows
    int cu_bytes;                          // 4 or 8
    uint32_t seq_rows;
    int64_t rows, D, n_seqs;
    int64_t n_strips, n_chunks, n_tiles;
    int zero_padding;                      // outputs of rows in no sequence: 0 written, else left
    uint64_t *maps;                        // [n_tiles][TC] words (A, B), ~0 at launch
    uint32_t *carry;                       // [n_tiles][TC] words: state leaving each tile, ~0 at launch
    uint32_t *ticket;                      // ~0 at launch, or null: tile = blockIdx.x
    uint32_t *status;                      // ~0 at launch; SGR_ERR_TIMEOUT once a wait ran out; may be null
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

__device__ __forceinline__ uint32_t ld_relaxed_u32(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed_u32(uint32_t *p, uint32_t v) {
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint64_t pack_map(float2 m) {
    return (uint64_t(__float_as_uint(m.y)) << 32) | __float_as_uint(m.x);
}

// The carry of one tile (carry warp): q its place in processing order along
// its strip, tot the tile's maps of this lane's E channels.  Publishes,
// waits, and returns the entering states.  Tiles whose first row (in
// processing order) is a start enter with 0, which they never use.  The
// window holds the words of the W tiles before: all are read in one round
// trip, and again only those not yet published.  W tiles are what one hop of
// the chain advances (about 1 us); 16 (8 with two channels a lane) fit the
// registers that the data warps' threads leave.
template <int E>
__device__ __forceinline__ void carry_tile_state(const GatedParams &p, int64_t strip, int64_t q, int lane, bool fresh,
                                                 const float2 (&tot)[E], float (&hin)[E]) {
    constexpr int TC = 32 * E;
    constexpr int W = E == 1 ? 16 : 8;
    const int64_t step = p.n_strips * TC;                          // from a tile's words to the next chunk's
    const int64_t at = q * step + strip * TC + lane * E;
    const bool last = q + 1 == p.n_chunks;
    bool cut = true;                                               // a start cuts all channels alike
#pragma unroll
    for (int e = 0; e < E; ++e) {
        hin[e] = 0.f;
        cut = cut && is_cut(tot[e].x);
    }
    auto publish_state = [&] {
        if (last) return;
#pragma unroll
        for (int e = 0; e < E; ++e) st_relaxed_u32(p.carry + at + e, __float_as_uint(apply_map(tot[e].x, tot[e].y, hin[e])));
    };
    if (fresh || q == 0) {
        publish_state();
        return;
    }
    if (cut) {
        publish_state();
    } else if (!last) {
#pragma unroll
        for (int e = 0; e < E; ++e) st_relaxed_u64(p.maps + at + e, pack_map(tot[e]));
    }
    uint64_t m[W][E];
    uint32_t st[W][E];
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            m[i][e] = ~uint64_t(0);
            st[i][e] = kNone;
        }
    }
    int k = -1;                                                    // nearest published state, maps there before it
    for (uint32_t polls = 0;; ++polls) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (q - 1 - i < 0) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (st[i][e] == kNone) st[i][e] = ld_relaxed_u32(p.carry + at + e - (i + 1) * step);
                if (i < W - 1 && m[i][e] == ~uint64_t(0)) m[i][e] = ld_relaxed_u64(p.maps + at + e - (i + 1) * step);
            }
        }
        bool there = true;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            bool s_ok = true, m_ok = true;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s_ok = s_ok && st[i][e] != kNone;
                m_ok = m_ok && m[i][e] != ~uint64_t(0);
            }
            if (there && k < 0 && s_ok) k = i;
            there = there && m_ok;
        }
        if (__all_sync(0xffffffffu, k >= 0) || polls >= p.spin_limit) break;
        if (polls > 8) __nanosleep(32);
    }
    if (k < 0) {
        atomicExch(p.status, 5u);                                  // SGR_ERR_TIMEOUT
#pragma unroll
        for (int e = 0; e < E; ++e) hin[e] = __int_as_float(0x7fffffff);
    } else {
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (i == k) hin[e] = __uint_as_float(st[i][e]);
                else if (i < k)
                    hin[e] = apply_map(__uint_as_float(uint32_t(m[i][e])), __uint_as_float(uint32_t(m[i][e] >> 32)), hin[e]);
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


// The tiles of a block, handed from the carry warp to the data warps through
// a ring: tile n lies in slot n % S, its table in s_info[n % (S + 1)] (read
// until the tile's replay is over, one tile longer than the slot).
template <int S> struct Ring {
    uint64_t full[S];
    TileInfo info[S + 1];
};

template <typename IO, int E, int OPS, int S, bool TMA>
struct SmemShape {
    static constexpr int TC = 32 * E;
    static constexpr uint32_t op_bytes = kTR * TC * sizeof(IO);
    static constexpr uint32_t slot_bytes = OPS * op_bytes;
    static constexpr uint32_t bytes = TMA ? S * slot_bytes + 128 : 0;
};

// The carry warp's side of the ring.  A tile is taken in three parts, so that
// none of them delays the carry: next() draws its ticket, issue() starts its
// copies as soon as the slot is free, finish() writes its table and lets the
// data warps have it.  `reverse` counts chunks from the last.
template <int S, int OPS, uint32_t OP_BYTES, int TC, bool TMA>
struct Feed {
    const GatedParams &p;
    Ring<S> &ring;
    const int lane;
    const bool reverse;
    const uint32_t slots;
    const CUtensorMap *maps[3];
    int64_t tile;                          // drawn, not yet finished; n_tiles: no more

    __device__ __forceinline__ void next(bool first) {
        if (p.ticket) {
            if (!first && tile >= p.n_tiles) return;
            uint32_t t = 0;
            if (lane == 0) t = atomicAdd(p.ticket, 1u) + 1u;
            tile = __shfl_sync(0xffffffffu, t, 0);
        } else {
            tile = first ? int64_t(blockIdx.x) : p.n_tiles;
        }
    }
    __device__ __forceinline__ int64_t row0() const {
        const uint32_t q = uint32_t(tile) / uint32_t(p.n_strips);
        return int64_t(reverse ? uint32_t(p.n_chunks) - 1 - q : q) * kTR;
    }
    __device__ __forceinline__ void issue(int n) {
        if constexpr (TMA) {
            if (lane == 0 && tile < p.n_tiles) {
                const uint32_t strip = uint32_t(tile) % uint32_t(p.n_strips);
                const uint32_t bar = smem_addr(&ring.full[n % S]);
                const uint32_t dst = slots + uint32_t(n % S) * (OPS * OP_BYTES);
                asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(OPS * OP_BYTES)
                             : "memory");
#pragma unroll
                for (int i = 0; i < OPS; ++i)
                    tma_load_2d(dst + i * OP_BYTES, maps[i], int(strip) * TC, int(row0()), bar);
            }
            __syncwarp();
        }
    }
    __device__ __forceinline__ void finish(int n) {
        TileInfo &info = ring.info[n % (S + 1)];
        if (tile < p.n_tiles) fill_info(p, row0(), info, lane);
        if (lane == 0) info.tile = tile;
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&ring.full[n % S])) : "memory");
    }
};

// Data warp: wait for tile n.  The table is always there in the end (the
// carry warp's own waits are bounded); false means that copies are missing,
// and the tile's outputs become NaN.
__device__ __forceinline__ bool wait_tile(uint64_t *full, int n, int S, uint32_t &limit, uint32_t *status) {
    if (mbar_wait(smem_addr(&full[n % S]), uint32_t((n / S) & 1), limit)) return true;
    limit = 1;
    if (status) atomicExch(status, 5u);                               // SGR_ERR_TIMEOUT
    return false;
}
constexpr uint32_t kTileWait = 1u << 24;

struct RowMasks {
    uint32_t starts, ends, live;           // bit r: row r of the warp starts / ends a sequence, lies in one
};
__device__ __forceinline__ RowMasks row_masks(const TileInfo &info, int64_t row0, int warp, int lane) {
    const int rr = lane & 15;
    RowMasks k;
    k.starts = __ballot_sync(0xffffffffu, info.start[warp * kRows + rr] >= 0) & 0xffffu;
    k.ends = __ballot_sync(0xffffffffu, info.end[warp * kRows + rr] >= 0) & 0xffffu;
    k.live = __ballot_sync(0xffffffffu, row0 + rr >= info.lo && row0 + rr < info.hi) & 0xffffu;
    return k;
}

// The carry warp's part of a tile once the data warps' maps are in shared
// memory: the entering state of each warp.  DIR +1: warps in order, -1: from
// the last.
template <int E, int DIR, class V>
__device__ __forceinline__ void carry_warps(const GatedParams &p, const V (&sA)[kWarps][32], const V (&sB)[kWarps][32],
                                            V (&sin)[kWarps][32], int64_t strip, int64_t q, int lane, bool fresh,
                                            float *entering, int64_t d0) {
    float2 pre[kWarps][E], tot[E];
#pragma unroll
    for (int e = 0; e < E; ++e) tot[e] = make_float2(1.f, 0.f);
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        const int w = DIR > 0 ? j : kWarps - 1 - j;
        const float *A = reinterpret_cast<const float *>(&sA[w][lane]);
        const float *B = reinterpret_cast<const float *>(&sB[w][lane]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            pre[j][e] = make_float2(A[e], B[e]);
            tot[e] = then_map(tot[e], pre[j][e]);
        }
    }
    float hin[E];
    carry_tile_state<E>(p, strip, q, lane, fresh, tot, hin);
    if (entering) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d0 + e < p.D) entering[q * p.D + d0 + e] = hin[e];
    }
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        const int w = DIR > 0 ? j : kWarps - 1 - j;
        float *in = reinterpret_cast<float *>(&sin[w][lane]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            in[e] = hin[e];
            hin[e] = apply_map(pre[j][e].x, pre[j][e].y, hin[e]);
        }
    }
}

// ------------------------------------------------------------- forward
template <typename IO, int E, int GATE, bool TMA>
__global__ void __launch_bounds__(kThreads, 2)
gated_scan_kernel(const GatedParams p, const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_v) {
    using V = typename FVec<E>::type;
    using R = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    using Shape = SmemShape<IO, E, 2, kSlots, TMA>;
    constexpr int TC = 32 * E;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Ring<kSlots> ring;
    __shared__ V s_A[2][kWarps][32], s_B[2][kWarps][32], s_in[2][kWarps][32];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) mbar_init(smem_addr(&ring.full[s]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (warp < kWarps) {
        uint32_t limit = kTileWait;
        for (int n = 0;; ++n) {
            const int par = n & 1;
            const bool got = wait_tile(ring.full, n, kSlots, limit, p.status);
            const TileInfo &info = ring.info[n % (kSlots + 1)];
            const int64_t tile = info.tile;
            if (tile >= p.n_tiles) break;
            const uint32_t chunk = uint32_t(tile) / uint32_t(p.n_strips), strip = uint32_t(tile) - chunk * uint32_t(p.n_strips);
            const int64_t row0 = int64_t(chunk) * kTR + warp * kRows;
            const int64_t d0 = int64_t(strip) * TC + lane * E;
            const bool dvalid = d0 < p.D;
            const RowMasks k = row_masks(info, row0, warp, lane);
            R rf[kRows], rv[kRows];
            if constexpr (TMA) {
                const R *sf = reinterpret_cast<const R *>(smem + (n % kSlots) * Shape::slot_bytes) + warp * kRows * 32 + lane;
                const R *sv = sf + kTR * 32;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    rf[r] = sf[r * 32];
                    rv[r] = sv[r * 32];
                }
            } else {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const bool ok = dvalid && row0 + r < p.rows;
                    rf[r] = ok ? load_raw<IO, E>(p.f, (row0 + r) * p.f_rs + d0) : R(0);
                    rv[r] = ok ? load_raw<IO, E>(p.v, (row0 + r) * p.v_rs + d0) : R(0);
                }
            }
            V a[kRows], b[kRows];
            V A = vset<V>(1.f), B = vset<V>(0.f);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                gate_pair<GATE, IO>(C::in(rf[r]), C::in(rv[r]), a[r], b[r]);
                if (k.starts >> r & 1u) {
                    A = vset<V>(-0.f);
                    B = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                }
                B = vfma(a[r], B, b[r]);
                A = vmul(A, a[r]);
            }
            if (!got) {
                A = B = vset<V>(__int_as_float(0x7fffffff));
#pragma unroll
                for (int r = 0; r < kRows; ++r) b[r] = B;
            }
            s_A[par][warp][lane] = A;
            s_B[par][warp][lane] = B;
            named_barrier_arrive(1 + par, kThreads);
            named_barrier_sync(3 + par, kThreads);
            V h = s_in[par][warp][lane];
            char *dst = static_cast<char *>(p.h) + (row0 * p.h_rs + d0) * int64_t(sizeof(IO));
            const int64_t pitch = p.h_rs * int64_t(sizeof(IO));
            if (k.starts == 0u && k.ends == 0u && k.live == 0xffffu) {
                if (dvalid) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        h = vfma(a[r], h, b[r]);
                        __stcs(reinterpret_cast<R *>(dst), C::out(h));
                        dst += pitch;
                    }
                }
            } else {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    if (k.starts >> r & 1u) h = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                    h = vfma(a[r], h, b[r]);
                    if (dvalid && row0 + r < p.rows) {
                        if (k.live >> r & 1u) __stcs(reinterpret_cast<R *>(dst), C::out(h));
                        else if (p.zero_padding) __stcs(reinterpret_cast<R *>(dst), R(0));
                    }
                    dst += pitch;
                    if ((k.ends >> r & 1u) && p.h_last) put_state_row<E>(p.h_last, info.end[warp * kRows + r] * p.D, d0, p.D, h);
                }
            }
        }
    } else {
        Feed<kSlots, 2, Shape::op_bytes, TC, TMA> feed{p, ring, lane, false, smem_addr(smem), {&map_f, &map_v, nullptr}, 0};
        for (int n = 0; n < kSlots; ++n) {
            feed.next(n == 0);
            feed.issue(n);
            feed.finish(n);
        }
        feed.next(false);
        for (int n = 0;; ++n) {
            const int par = n & 1;
            const TileInfo &info = ring.info[n % (kSlots + 1)];
            const int64_t tile = info.tile;
            if (tile >= p.n_tiles) break;
            const uint32_t chunk = uint32_t(tile) / uint32_t(p.n_strips), strip = uint32_t(tile) - chunk * uint32_t(p.n_strips);
            const bool fresh = info.start[0] >= 0;
            named_barrier_sync(1 + par, kThreads);         // the maps are there, and the slot has been read
            feed.issue(n + kSlots);
            carry_warps<E, 1>(p, s_A[par], s_B[par], s_in[par], strip, chunk, lane, fresh, p.states,
                              int64_t(strip) * TC + lane * E);
            named_barrier_arrive(3 + par, kThreads);
            feed.finish(n + kSlots);
            feed.next(false);
        }
    }
    __syncthreads();
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
//
// The tile's slot is read three times (folds, forward replay, reverse
// replay), so it is refilled once the next tile's maps are in; the registers
// hold the gates and the factors of df.
template <int GATE, typename IO, class V>
__device__ __forceinline__ V bwd_gate(V f) {
    // GATE_SIGMOID: signed small probability; GATE_LOG: a, negated where f > 0, which has no gradient
    if constexpr (GATE == GATE_SIGMOID) return vmap(f, [](float x) { return signed_small(x); });
    else
        return vmap(f, [](float x) {
            const float t = log_decay<sizeof(IO) == 4>(x);
            return x > 0.f ? -t : t;
        });
}
template <int GATE, class V>
__device__ __forceinline__ V bwd_a(V s) {
    if constexpr (GATE == GATE_SIGMOID) {
        V a, z;
        split_small(s, a, z);
        return a;
    } else {
        return vmap(s, [](float x) { return fabsf(x); });
    }
}

template <typename IO, int E, int GATE, bool TMA>
__global__ void __launch_bounds__(kThreads, 2)
gated_scan_backward_kernel(const GatedParams p, const __grid_constant__ CUtensorMap map_f,
                           const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_dh) {
    using V = typename FVec<E>::type;
    using R = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    using Shape = SmemShape<IO, E, 3, kBwdSlots, TMA>;
    constexpr int TC = 32 * E;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Ring<kBwdSlots> ring;
    __shared__ V s_A[kWarps][32], s_B[kWarps][32];                    // forward maps
    __shared__ V s_RA[2][kWarps][32], s_RB[2][kWarps][32];            // reverse maps
    __shared__ V s_in[2][kWarps][32];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kBwdSlots; ++s) mbar_init(smem_addr(&ring.full[s]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (warp < kWarps) {
        uint32_t limit = kTileWait;
        for (int n = 0;; ++n) {
            const int par = n & 1;
            const bool got = wait_tile(ring.full, n, kBwdSlots, limit, p.status);
            const TileInfo &info = ring.info[n % (kBwdSlots + 1)];
            const int64_t tile = info.tile;
            if (tile >= p.n_tiles) break;
            const uint32_t q = uint32_t(tile) / uint32_t(p.n_strips), strip = uint32_t(tile) - q * uint32_t(p.n_strips);
            const uint32_t chunk = uint32_t(p.n_chunks) - 1 - q;
            const int64_t row0 = int64_t(chunk) * kTR + warp * kRows;
            const int64_t d0 = int64_t(strip) * TC + lane * E;
            const bool dvalid = d0 < p.D;
            V h = info.start[0] >= 0 || chunk == 0 ? vset<V>(0.f) : state_row<E>(p.states, chunk * p.D, d0, p.D);
            const RowMasks k = row_masks(info, row0, warp, lane);
            [[maybe_unused]] R gv[TMA ? 1 : kRows], gg[TMA ? 1 : kRows];
            const R *sf = reinterpret_cast<const R *>(smem + (n % kBwdSlots) * Shape::slot_bytes) + warp * kRows * 32 + lane;
            if constexpr (!TMA) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const bool ok = dvalid && row0 + r < p.rows;
                    gv[r] = ok ? load_raw<IO, E>(p.v, (row0 + r) * p.v_rs + d0) : R(0);
                    gg[r] = ok ? load_raw<IO, E>(p.dh, (row0 + r) * p.dh_rs + d0) : R(0);
                }
            }
            auto in_f = [&](int r) {
                if constexpr (TMA) return C::in(sf[r * 32]);
                else return C::in(dvalid && row0 + r < p.rows ? load_raw<IO, E>(p.f, (row0 + r) * p.f_rs + d0) : R(0));
            };
            auto in_v = [&](int r) {
                if constexpr (TMA) return C::in(sf[(kTR + r) * 32]);
                else return C::in(gv[r]);
            };
            auto in_g = [&](int r) {
                if constexpr (TMA) return C::in(sf[(2 * kTR + r) * 32]);
                else return C::in(gg[r]);
            };
            V s[kRows];
            V A = vset<V>(1.f), B = vset<V>(0.f);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                s[r] = bwd_gate<GATE, IO>(in_f(r));
                V a, b = in_v(r);
                if constexpr (GATE == GATE_SIGMOID) {
                    V z;
                    split_small(s[r], a, z);
                    b = vmul(z, b);
                } else {
                    a = bwd_a<GATE>(s[r]);
                }
                if (k.starts >> r & 1u) {
                    A = vset<V>(-0.f);
                    B = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                }
                B = vfma(a, B, b);
                A = vmul(A, a);
            }
            V RA = vset<V>(1.f), RB = vset<V>(0.f);
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                const V a = bwd_a<GATE>(s[r]);
                if (k.ends >> r & 1u) {
                    RA = vset<V>(-0.f);
                    RB = state_row<E>(p.dh_last, info.end[warp * kRows + r] * p.D, d0, p.D);
                }
                RB = vmul(a, vadd(RB, in_g(r)));
                RA = vmul(RA, a);
            }
            if (!got) {
                A = B = RA = RB = vset<V>(__int_as_float(0x7fffffff));
#pragma unroll
                for (int r = 0; r < kRows; ++r) s[r] = B;
            }
            s_A[warp][lane] = A;
            s_B[warp][lane] = B;
            s_RA[par][warp][lane] = RA;
            s_RB[par][warp][lane] = RB;
            named_barrier_arrive(1 + par, kThreads);
            named_barrier_sync(5, kWarps * 32);                       // the data warps' maps are there
            for (int w = 0; w < warp; ++w)
                h = vmap(s_A[w][lane], s_B[w][lane], h, [](float x, float y, float z) { return apply_map(x, y, z); });
            V c[kRows];                                               // df = c g
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (k.starts >> r & 1u) h = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, d0, p.D);
                const V v = in_v(r);
                if constexpr (GATE == GATE_SIGMOID) {
                    V a, z;
                    split_small(s[r], a, z);
                    c[r] = vmul(vmul(a, z), vfma(v, vset<V>(-1.f), h));
                    h = vfma(a, h, vmul(z, v));
                } else {
                    c[r] = vmap(s[r], h, [](float x, float y) { return is_cut(x) ? 0.f : x * y; });
                    h = vfma(bwd_a<GATE>(s[r]), h, v);
                }
            }
            named_barrier_sync(3 + par, kThreads);
            V flow = s_in[par][warp][lane];
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                if (k.ends >> r & 1u) flow = state_row<E>(p.dh_last, info.end[warp * kRows + r] * p.D, d0, p.D);
                const V g = vadd(flow, in_g(r));
                V a, dv = g;
                if constexpr (GATE == GATE_SIGMOID) {
                    V z;
                    split_small(s[r], a, z);
                    dv = vmul(z, g);
                } else {
                    a = bwd_a<GATE>(s[r]);
                }
                if (dvalid && row0 + r < p.rows) {
                    const bool live = k.live >> r & 1u;
                    store_raw<IO, E>(p.df, (row0 + r) * p.df_rs + d0, live ? C::out(vmul(c[r], g)) : R(0));
                    store_raw<IO, E>(p.dv, (row0 + r) * p.dv_rs + d0, live ? C::out(dv) : R(0));
                }
                flow = vmul(a, g);
                if ((k.starts >> r & 1u) && p.dh0) put_state_row<E>(p.dh0, info.start[warp * kRows + r] * p.D, d0, p.D, flow);
            }
        }
    } else {
        Feed<kBwdSlots, 3, Shape::op_bytes, TC, TMA> feed{p, ring, lane, true, smem_addr(smem), {&map_f, &map_v, &map_dh}, 0};
        for (int n = 0; n < kBwdSlots; ++n) {
            feed.next(n == 0);
            feed.issue(n);
            feed.finish(n);
        }
        feed.next(false);
        for (int n = 0;; ++n) {
            const int par = n & 1;
            const TileInfo &info = ring.info[n % (kBwdSlots + 1)];
            const int64_t tile = info.tile;
            if (tile >= p.n_tiles) break;
            const uint32_t q = uint32_t(tile) / uint32_t(p.n_strips), strip = uint32_t(tile) - q * uint32_t(p.n_strips);
            const bool fresh = info.end[kTR - 1] >= 0;
            named_barrier_sync(1 + par, kThreads);         // every data warp has left tile n - 1 behind
            if (n >= 1) feed.issue(n + kBwdSlots - 1);     // ... whose slot takes this one
            carry_warps<E, -1>(p, s_RA[par], s_RB[par], s_in[par], strip, q, lane, fresh, nullptr, 0);
            named_barrier_arrive(3 + par, kThreads);
            if (n >= 1) {
                feed.finish(n + kBwdSlots - 1);
                feed.next(false);
            }
        }
    }
    __syncthreads();
    empty_sequences(p, p.dh0, p.dh_last, p.D);
}

}  // namespace gated
}  // namespace sgr
