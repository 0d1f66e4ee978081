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
// rows [8 w, 8 w + 8), lane l channels [E l, E l + E): a thread folds its 8
// rows, the folds of a channel meet in shared memory, and a carry warp finds
// the state that enters the tile; the threads then replay their rows from it.
// Inputs are read from memory once and outputs written once.
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
// One persistent block per SM.  The feeding warp keeps a ring of tiles in
// shared memory filled by the tensor memory accelerator (TMA; rows that start
// on 16-byte boundaries, else the data warps load from memory themselves) and
// writes each tile's table of sequence starts and ends.  A tile's state takes
// two or three microseconds to arrive, longer than its arithmetic, so the
// data warps fold tile n and then replay tile n - kLag, evaluating its gates
// again from the ring: the second evaluation costs less than holding two
// values per element in registers across the wait, which left room for two
// tiles per SM only (bf16 32768 x 4096, sigmoid: 307 us that way).
#pragma once

#include "gated_math.cuh"

namespace sgr {
namespace gated {

constexpr int kWarps = 13;                 // data warps
constexpr int kRows = 8;                   // rows per data warp and thread
constexpr int kTR = kWarps * kRows;        // rows per tile, and between saved states
constexpr int kCarryWarps = 2;             // tiles in turn
constexpr int kThreads = (kWarps + kCarryWarps + 1) * 32;   // the last warp feeds the ring
constexpr int kSlots = 6, kLag = 2;        // forward: tiles in shared memory, tiles between fold and replay
constexpr int kBwdSlots = 4, kBwdLag = 1;  // backward
constexpr uint32_t kTileWait = 1u << 16;   // polls of a wait inside the block (each suspends for tens of us)
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
    return is_cut(then.x) ? then : make_float2(first.x * then.x, fmaf(then.x, first.y, then.y));
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
// registers.
// `between` runs once the tile's own words are out.
template <int E, class Between>
__device__ __forceinline__ void carry_tile_state(const GatedParams &p, int64_t strip, int64_t q, int lane, bool fresh,
                                                 const float2 (&tot)[E], float (&hin)[E], Between between) {
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
        between();
        return;
    }
    if (cut) {
        publish_state();
    } else if (!last) {
#pragma unroll
        for (int e = 0; e < E; ++e) st_relaxed_u64(p.maps + at + e, pack_map(tot[e]));
    }
    between();
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


// ------------------------------------------------------ inside a block
//
// Tile n of the block lies in slot n % S from its copies until every data
// warp has replayed it; its maps and entering states in entry n % Q, Q =
// lag + 1: a data warp folds tile n after its replay of tile n - Q, which it
// began with that tile's states.  Every wait is bounded; one that runs out
// poisons the tile (NaN) and records it, and nothing else waits on it.
template <typename V, int S, int Q, int MAPS> struct Block {
    uint64_t full[S], empty[S];            // copies and table there; replayed by every data warp
    uint64_t maps[Q], in[Q];               // maps there; entering states there
    TileInfo info[S];
    V A[MAPS][Q][kWarps][32], B[MAPS][Q][kWarps][32];
    V enter[MAPS][Q][kWarps][32];
};
template <class B, int S, int Q> __device__ __forceinline__ void init_block(B &blk) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_addr(&blk.full[i]), 1);
            mbar_init(smem_addr(&blk.empty[i]), kWarps);
        }
        for (int i = 0; i < Q; ++i) {
            mbar_init(smem_addr(&blk.maps[i]), kWarps);
            mbar_init(smem_addr(&blk.in[i]), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// wait for use u of a barrier (its phases are uses 0, 1, 2, ...)
struct Waiter {
    uint32_t *status;
    uint32_t limit;
    __device__ __forceinline__ bool operator()(uint64_t *bar, int u) {
        if (mbar_wait(smem_addr(bar), uint32_t(u & 1), limit)) return true;
        limit = 1;
        if (status) atomicExch(status, 5u);                           // SGR_ERR_TIMEOUT
        return false;
    }
};

template <typename IO, int E, int OPS, int S, bool TMA>
struct SmemShape {
    static constexpr int TC = 32 * E;
    static constexpr uint32_t op_bytes = kTR * TC * sizeof(IO);
    static constexpr uint32_t slot_bytes = OPS * op_bytes;
    static constexpr uint32_t ring_bytes = TMA ? S * slot_bytes : 0;
};

// The feeding warp: draws tickets, starts the copies of a tile when its slot
// is free, writes its table and hands both over.  `reverse` counts chunks
// from the last.  Ends with one entry for each carry warp whose tile is
// n_tiles, so that each of them comes upon one.
template <int S, int OPS, uint32_t OP_BYTES, int TC, bool TMA, class B>
__device__ __forceinline__ void feed(const GatedParams &p, B &blk, uint32_t slots, int lane, bool reverse,
                                     const CUtensorMap *m0, const CUtensorMap *m1, const CUtensorMap *m2) {
    Waiter wait{p.status, kTileWait};
    int ends = 0;
    for (int n = 0; ends < kCarryWarps; ++n) {
        int64_t tile = p.n_tiles;
        if (ends > 0) {
        } else if (p.ticket) {
            uint32_t t = 0;
            if (lane == 0) t = atomicAdd(p.ticket, 1u) + 1u;
            tile = __shfl_sync(0xffffffffu, t, 0);
        } else if (n == 0) {
            tile = blockIdx.x;
        }
        const bool more = tile < p.n_tiles;
        if (n >= S) wait(&blk.empty[n % S], n / S - 1);
        TileInfo &info = blk.info[n % S];
        if (more) {
            const uint32_t q = uint32_t(tile) / uint32_t(p.n_strips), strip = uint32_t(tile) - q * uint32_t(p.n_strips);
            const int64_t row0 = int64_t(reverse ? uint32_t(p.n_chunks) - 1 - q : q) * kTR;
            if constexpr (TMA) {
                if (lane == 0) {
                    const uint32_t bar = smem_addr(&blk.full[n % S]);
                    const uint32_t dst = slots + uint32_t(n % S) * (OPS * OP_BYTES);
                    // the data warps' reads of the slot came before the copies into it
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(OPS * OP_BYTES)
                                 : "memory");
                    tma_load_2d(dst, m0, int(strip) * TC, int(row0), bar);
                    tma_load_2d(dst + OP_BYTES, m1, int(strip) * TC, int(row0), bar);
                    if constexpr (OPS == 3) tma_load_2d(dst + 2 * OP_BYTES, m2, int(strip) * TC, int(row0), bar);
                }
                __syncwarp();
            }
            fill_info(p, row0, info, lane);
        }
        if (lane == 0) info.tile = tile;
        __syncwarp();
        if (lane == 0) arrive(&blk.full[n % S]);
        if (!more) ++ends;
    }
}

// A carry warp: tiles c, c + kCarryWarps, ... of the block.  Forward (DIR +1):
// warps in order; the state entering each chunk is kept in p.states if given.
// Backward (DIR -1): warps from the last, and beside them (map 1) the states
// of the forward recurrence within the tile, from p.states.
template <int E, int S, int Q, int DIR, class B>
__device__ __forceinline__ void carry_loop(const GatedParams &p, B &blk, int c, int lane) {
    Waiter wait{p.status, kTileWait};
    for (int n = c;; n += kCarryWarps) {
        wait(&blk.full[n % S], n / S);
        const TileInfo &info = blk.info[n % S];
        const int64_t tile = info.tile;
        if (tile >= p.n_tiles) return;
        const uint32_t q = uint32_t(tile) / uint32_t(p.n_strips), strip = uint32_t(tile) - q * uint32_t(p.n_strips);
        const bool fresh = DIR > 0 ? info.start[0] >= 0 : info.end[kTR - 1] >= 0;
        const int e0 = n % Q;
        const int64_t d0 = int64_t(strip) * 32 * E + lane * E;
        float hf[E];
        if constexpr (DIR < 0) {
            const uint32_t chunk = uint32_t(p.n_chunks) - 1 - q;
            const bool begins = info.start[0] >= 0 || chunk == 0;
#pragma unroll
            for (int e = 0; e < E; ++e) hf[e] = begins || d0 + e >= p.D ? 0.f : p.states[int64_t(chunk) * p.D + d0 + e];
        }
        wait(&blk.maps[e0], n / Q);
        auto map_of = [&](int k, int w, int e) {
            return make_float2(reinterpret_cast<const float *>(&blk.A[k][e0][w][lane])[e],
                               reinterpret_cast<const float *>(&blk.B[k][e0][w][lane])[e]);
        };
        // the states entering each warp from those entering the tile
        auto enter = [&](int k, bool up, float (&h)[E]) {
#pragma unroll
            for (int j = 0; j < kWarps; ++j) {
                const int w = up ? j : kWarps - 1 - j;
                float *in = reinterpret_cast<float *>(&blk.enter[k][e0][w][lane]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float2 m = map_of(k, w, e);
                    in[e] = h[e];
                    h[e] = apply_map(m.x, m.y, h[e]);
                }
            }
        };
        float2 tot[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            tot[e] = map_of(0, DIR > 0 ? 0 : kWarps - 1, e);
#pragma unroll
            for (int j = 1; j < kWarps; ++j) tot[e] = then_map(tot[e], map_of(0, DIR > 0 ? j : kWarps - 1 - j, e));
        }
        float hin[E];
        carry_tile_state<E>(p, strip, q, lane, fresh, tot, hin, [&] {
            if constexpr (DIR < 0) enter(1, true, hf);
        });
        const float first[2] = {hin[0], hin[E - 1]};
        enter(0, DIR > 0, hin);
        __syncwarp();
        if (lane == 0) arrive(&blk.in[e0]);
        if constexpr (DIR > 0) {
            if (p.states) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (d0 + e < p.D) p.states[q * p.D + d0 + e] = first[e];
            }
        }
    }
}

// What a data warp knows of a tile: its place and, per row of the warp (bit
// r), whether the row starts or ends a sequence and lies in one.
struct WarpTile {
    int64_t row0, d0;
    uint32_t q, chunk;
    uint32_t starts, ends, live;
    int slot;
    bool dvalid;
};
template <int TC>
__device__ __forceinline__ WarpTile warp_tile(const GatedParams &p, const TileInfo &info, int slot, bool reverse, int warp,
                                              int lane, int E) {
    WarpTile t;
    const uint32_t tile = uint32_t(info.tile);
    t.slot = slot;
    t.q = tile / uint32_t(p.n_strips);
    t.chunk = reverse ? uint32_t(p.n_chunks) - 1 - t.q : t.q;
    t.row0 = int64_t(t.chunk) * kTR + warp * kRows;
    t.d0 = int64_t(tile - t.q * uint32_t(p.n_strips)) * TC + lane * E;
    t.dvalid = t.d0 < p.D;
    const int rr = lane & (kRows - 1);
    constexpr uint32_t all = (1u << kRows) - 1u;
    t.starts = __ballot_sync(0xffffffffu, info.start[warp * kRows + rr] >= 0) & all;
    t.ends = __ballot_sync(0xffffffffu, info.end[warp * kRows + rr] >= 0) & all;
    t.live = __ballot_sync(0xffffffffu, t.row0 + rr >= info.lo && t.row0 + rr < info.hi) & all;
    return t;
}

// The thread's rows of operand OP of a tile: from the slot, or from memory
// (read twice then, the second time from a cache).
template <typename IO, int E, bool TMA, class Shape, int OP>
__device__ __forceinline__ void tile_rows(const GatedParams &p, const unsigned char *smem, const WarpTile &t, int warp,
                                          int lane, const void *base, int64_t rs, typename Raw<IO, E>::type (&x)[kRows]) {
    using R = typename Raw<IO, E>::type;
    if constexpr (TMA) {
        const R *src = reinterpret_cast<const R *>(smem + t.slot * Shape::slot_bytes + OP * Shape::op_bytes) +
                       warp * kRows * 32 + lane;
#pragma unroll
        for (int r = 0; r < kRows; ++r) x[r] = src[r * 32];
    } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const bool ok = t.dvalid && t.row0 + r < p.rows;
            x[r] = ok ? *reinterpret_cast<const R *>(static_cast<const IO *>(base) + (t.row0 + r) * rs + t.d0) : R(0);
        }
    }
}

// ------------------------------------------------------------- forward
template <typename IO, int E, bool TMA> struct ForwardShape {
    using Ring = SmemShape<IO, E, 2, kSlots, TMA>;
    using Blk = Block<typename FVec<E>::type, kSlots, kLag + 1, 1>;
    static constexpr uint32_t smem_bytes = Ring::ring_bytes + sizeof(Blk);
};

template <typename IO, int E, int GATE, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
gated_scan_kernel(const GatedParams p, const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_v) {
    using V = typename FVec<E>::type;
    using R = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    using Shape = typename ForwardShape<IO, E, TMA>::Ring;
    using Blk = typename ForwardShape<IO, E, TMA>::Blk;
    constexpr int S = kSlots, Q = kLag + 1, TC = 32 * E;
    extern __shared__ __align__(128) unsigned char smem[];
    Blk &blk = *reinterpret_cast<Blk *>(smem + Shape::ring_bytes);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    init_block<Blk, S, Q>(blk);
    if (warp < kWarps) {
        Waiter wait{p.status, kTileWait};
        int n_end = 1 << 30;                               // tiles of the block, once known
        for (int n = 0; n < n_end + kLag; ++n) {
            if (n < n_end) {
                const bool got = wait(&blk.full[n % S], n / S);
                const TileInfo &info = blk.info[n % S];
                if (info.tile >= p.n_tiles) {
                    n_end = n;
                } else {
                    const WarpTile t = warp_tile<TC>(p, info, n % S, false, warp, lane, E);
                    R rf[kRows], rv[kRows];
                    tile_rows<IO, E, TMA, Shape, 0>(p, smem, t, warp, lane, p.f, p.f_rs, rf);
                    tile_rows<IO, E, TMA, Shape, 1>(p, smem, t, warp, lane, p.v, p.v_rs, rv);
                    V A = vset<V>(1.f), B = vset<V>(0.f);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        V a, b;
                        gate_pair<GATE, IO>(C::in(rf[r]), C::in(rv[r]), a, b);
                        if (t.starts >> r & 1u) {
                            A = vset<V>(-0.f);
                            B = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, t.d0, p.D);
                        }
                        B = vfma(a, B, b);
                        A = vmul(A, a);
                    }
                    if (!got) A = B = vset<V>(__int_as_float(0x7fffffff));
                    blk.A[0][n % Q][warp][lane] = A;
                    blk.B[0][n % Q][warp][lane] = B;
                    __syncwarp();
                    if (lane == 0) arrive(&blk.maps[n % Q]);
                }
            }
            const int m = n - kLag;
            if (m < 0 || m >= n_end) continue;
            const bool got = wait(&blk.in[m % Q], m / Q);
            const TileInfo &info = blk.info[m % S];
            const WarpTile t = warp_tile<TC>(p, info, m % S, false, warp, lane, E);
            R rf[kRows], rv[kRows];
            tile_rows<IO, E, TMA, Shape, 0>(p, smem, t, warp, lane, p.f, p.f_rs, rf);
            tile_rows<IO, E, TMA, Shape, 1>(p, smem, t, warp, lane, p.v, p.v_rs, rv);
            V h = got ? blk.enter[0][m % Q][warp][lane] : vset<V>(__int_as_float(0x7fffffff));
            char *dst = static_cast<char *>(p.h) + (t.row0 * p.h_rs + t.d0) * int64_t(sizeof(IO));
            const int64_t pitch = p.h_rs * int64_t(sizeof(IO));
            if (t.starts == 0u && t.ends == 0u && t.live == (1u << kRows) - 1u) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    V a, b;
                    gate_pair<GATE, IO>(C::in(rf[r]), C::in(rv[r]), a, b);
                    h = vfma(a, h, b);
                    if (t.dvalid) __stcs(reinterpret_cast<R *>(dst), C::out(h));
                    dst += pitch;
                }
            } else {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    V a, b;
                    gate_pair<GATE, IO>(C::in(rf[r]), C::in(rv[r]), a, b);
                    if (t.starts >> r & 1u) h = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, t.d0, p.D);
                    h = vfma(a, h, b);
                    if (t.dvalid && t.row0 + r < p.rows) {
                        if (t.live >> r & 1u) __stcs(reinterpret_cast<R *>(dst), C::out(h));
                        else if (p.zero_padding) __stcs(reinterpret_cast<R *>(dst), R(0));
                    }
                    dst += pitch;
                    if ((t.ends >> r & 1u) && p.h_last)
                        put_state_row<E>(p.h_last, info.end[warp * kRows + r] * p.D, t.d0, p.D, h);
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&blk.empty[m % S]);
        }
    } else if (warp < kWarps + kCarryWarps) {
        carry_loop<E, S, Q, 1>(p, blk, warp - kWarps, lane);
    } else {
        feed<S, 2, Shape::op_bytes, TC, TMA>(p, blk, smem_addr(smem), lane, false, &map_f, &map_v, nullptr);
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
// (a, z) of it; z is 1 for GATE_LOG
template <int GATE, class V>
__device__ __forceinline__ void bwd_split(V s, V &a, V &z) {
    if constexpr (GATE == GATE_SIGMOID) {
        split_small(s, a, z);
    } else {
        a = vmap(s, [](float x) { return fabsf(x); });
        z = vset<V>(1.f);
    }
}

template <typename IO, int E, bool TMA> struct BackwardShape {
    using Ring = SmemShape<IO, E, 3, kBwdSlots, TMA>;
    using Blk = Block<typename FVec<E>::type, kBwdSlots, kBwdLag + 1, 2>;       // maps 0: reverse, 1: forward
    static constexpr uint32_t smem_bytes = Ring::ring_bytes + sizeof(Blk);
};

template <typename IO, int E, int GATE, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
gated_scan_backward_kernel(const GatedParams p, const __grid_constant__ CUtensorMap map_f,
                           const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_dh) {
    using V = typename FVec<E>::type;
    using R = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    using Shape = typename BackwardShape<IO, E, TMA>::Ring;
    using Blk = typename BackwardShape<IO, E, TMA>::Blk;
    constexpr int S = kBwdSlots, Q = kBwdLag + 1, TC = 32 * E;
    extern __shared__ __align__(128) unsigned char smem[];
    Blk &blk = *reinterpret_cast<Blk *>(smem + Shape::ring_bytes);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    init_block<Blk, S, Q>(blk);
    if (warp < kWarps) {
        Waiter wait{p.status, kTileWait};
        int n_end = 1 << 30;
        for (int n = 0; n < n_end + kBwdLag; ++n) {
            if (n < n_end) {
                const bool got = wait(&blk.full[n % S], n / S);
                const TileInfo &info = blk.info[n % S];
                if (info.tile >= p.n_tiles) {
                    n_end = n;
                } else {
                    const WarpTile t = warp_tile<TC>(p, info, n % S, true, warp, lane, E);
                    R rf[kRows], rv[kRows], rg[kRows];
                    tile_rows<IO, E, TMA, Shape, 0>(p, smem, t, warp, lane, p.f, p.f_rs, rf);
                    tile_rows<IO, E, TMA, Shape, 1>(p, smem, t, warp, lane, p.v, p.v_rs, rv);
                    tile_rows<IO, E, TMA, Shape, 2>(p, smem, t, warp, lane, p.dh, p.dh_rs, rg);
                    V a[kRows];
                    V A = vset<V>(1.f), B = vset<V>(0.f);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        V b;
                        gate_pair<GATE, IO>(C::in(rf[r]), C::in(rv[r]), a[r], b);
                        if (t.starts >> r & 1u) {
                            A = vset<V>(-0.f);
                            B = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, t.d0, p.D);
                        }
                        B = vfma(a[r], B, b);
                        A = vmul(A, a[r]);
                    }
                    V RA = vset<V>(1.f), RB = vset<V>(0.f);
#pragma unroll
                    for (int r = kRows - 1; r >= 0; --r) {
                        if (t.ends >> r & 1u) {
                            RA = vset<V>(-0.f);
                            RB = state_row<E>(p.dh_last, info.end[warp * kRows + r] * p.D, t.d0, p.D);
                        }
                        RB = vmul(a[r], vadd(RB, C::in(rg[r])));
                        RA = vmul(RA, a[r]);
                    }
                    if (!got) A = B = RA = RB = vset<V>(__int_as_float(0x7fffffff));
                    blk.A[0][n % Q][warp][lane] = RA;
                    blk.B[0][n % Q][warp][lane] = RB;
                    blk.A[1][n % Q][warp][lane] = A;
                    blk.B[1][n % Q][warp][lane] = B;
                    __syncwarp();
                    if (lane == 0) arrive(&blk.maps[n % Q]);
                }
            }
            const int m = n - kBwdLag;
            if (m < 0 || m >= n_end) continue;
            const TileInfo &info = blk.info[m % S];
            const WarpTile t = warp_tile<TC>(p, info, m % S, true, warp, lane, E);
            R rv[kRows], rg[kRows];
            V s[kRows], c[kRows];                                     // df = c g
            {
                R rf[kRows];
                tile_rows<IO, E, TMA, Shape, 0>(p, smem, t, warp, lane, p.f, p.f_rs, rf);
#pragma unroll
                for (int r = 0; r < kRows; ++r) s[r] = bwd_gate<GATE, IO>(C::in(rf[r]));
            }
            tile_rows<IO, E, TMA, Shape, 1>(p, smem, t, warp, lane, p.v, p.v_rs, rv);
            const bool got = wait(&blk.in[m % Q], m / Q);
            V h = blk.enter[1][m % Q][warp][lane];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (t.starts >> r & 1u) h = state_row<E>(p.h0, info.start[warp * kRows + r] * p.h0_ss, t.d0, p.D);
                const V v = C::in(rv[r]);
                V a, z;
                bwd_split<GATE>(s[r], a, z);
                if constexpr (GATE == GATE_SIGMOID) {
                    c[r] = vmul(vmul(a, z), vfma(v, vset<V>(-1.f), h));
                    h = vfma(a, h, vmul(z, v));
                } else {
                    c[r] = vmap(s[r], h, [](float x, float y) { return is_cut(x) ? 0.f : x * y; });
                    h = vfma(a, h, v);
                }
            }
            tile_rows<IO, E, TMA, Shape, 2>(p, smem, t, warp, lane, p.dh, p.dh_rs, rg);
            V flow = got ? blk.enter[0][m % Q][warp][lane] : vset<V>(__int_as_float(0x7fffffff));
#pragma unroll
            for (int r = kRows - 1; r >= 0; --r) {
                if (t.ends >> r & 1u) flow = state_row<E>(p.dh_last, info.end[warp * kRows + r] * p.D, t.d0, p.D);
                const V g = vadd(flow, C::in(rg[r]));
                V a, z;
                bwd_split<GATE>(s[r], a, z);
                if (t.dvalid && t.row0 + r < p.rows) {
                    const bool live = t.live >> r & 1u;
                    store_raw<IO, E>(p.df, (t.row0 + r) * p.df_rs + t.d0, live ? C::out(vmul(c[r], g)) : R(0));
                    store_raw<IO, E>(p.dv, (t.row0 + r) * p.dv_rs + t.d0,
                                     live ? C::out(GATE == GATE_SIGMOID ? vmul(z, g) : g) : R(0));
                }
                flow = vmul(a, g);
                if ((t.starts >> r & 1u) && p.dh0)
                    put_state_row<E>(p.dh0, info.start[warp * kRows + r] * p.D, t.d0, p.D, flow);
            }
            __syncwarp();
            if (lane == 0) arrive(&blk.empty[m % S]);
        }
    } else if (warp < kWarps + kCarryWarps) {
        carry_loop<E, S, Q, -1>(p, blk, warp - kWarps, lane);
    } else {
        feed<S, 3, Shape::op_bytes, TC, TMA>(p, blk, smem_addr(smem), lane, true, &map_f, &map_v, &map_dh);
    }
    __syncthreads();
    empty_sequences(p, p.dh0, p.dh_last, p.D);
}

}  // namespace gated
}  // namespace sgr
