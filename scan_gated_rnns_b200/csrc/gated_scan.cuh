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
// A tile is TR rows x TC channels (128 bytes of a row).  Each data warp owns R
// consecutive rows of it, lane l channels [E l, E l + E): a thread folds its
// rows, the folds of a channel meet in shared memory, and a carry warp finds
// the state that enters the tile; the threads then replay their rows from it.
// Inputs are read from memory once and outputs written once.
//
// The carry between tiles of one channel strip: each publishes its map, finds
// the nearest earlier tile whose final state is published, applies the maps
// between, oldest first, and publishes its own final state.  The arithmetic
// is the sequential S_q = A_q S_{q-1} + B_q wherever that state came from, so
// results do not depend on timing.  To have the state there when it is asked
// for, the rows are cut at sequence starts into segments of about equal length
// and the segments are worked on side by side, so that a tile's predecessor is
// a round of blocks older (with one segment the 64 strips of bf16 32768 x 4096
// in 23 sequences waited 2.6 us a tile, half of that for the predecessor's own
// fold).  A map, and then in its place the state, is one 64-bit word per
// channel, ~0 before the launch and valid once it is not (arithmetic never
// gives that NaN), so a look-back is one round trip to L2, without flags or
// fences.  Blocks take tiles by ticket in the order they run, so a wait is
// always for a tile that a running block holds; waits are bounded.
//
// One persistent block per SM.  The feeding warp keeps a ring of tiles in
// shared memory filled by the tensor memory accelerator (TMA; rows that start
// on 16-byte boundaries, else the data warps load from memory themselves) and
// writes each tile's table of sequence starts and ends.  A tile's state takes
// two or three microseconds to arrive, longer than its arithmetic, so the
// data warps fold tile n and then replay tile n - 1.  Across the wait a thread
// keeps one register per element, the gate; the values are read again from
// the ring.  (Both coefficients in registers left room for one tile at a time
// in each of two blocks per SM, which spent half its time waiting, 307 us on
// bf16 32768 x 4096; evaluating the gates twice was bound by instruction
// issue, 50 per element, 311 us.)
//
// Measured (B200, SM clock 1965 MHz; bytes = f, v in and h out, or f, v, dh in
// and df, dv out, over the 6549 GB/s of a copy): forward fp32 131072 x 512
// 155 us (0.79), fp32 8 x 4096 x 1024 77 us (0.80), bf16 32768 x 4096 in 23
// sequences 186 us (0.66; log gate 166, 0.74); backward fp32 8 x 4096 x 1024
// 125 us (0.82), bf16 16384 x 2048 98 us (0.52; log gate 88).  Bound by: the
// wait for the carried state where one long sequence keeps the segments at
// one; memory at about 5.6 TB/s and some 10 us of start and end in fp32; in
// 16 bits by too little independent work for 15 warps: schedulers issue in 40
// (forward) and 48 % (backward) of the cycles, and a warp spends 37 and 27 % of
// its time behind barriers and loads, 12 and 17 % behind fixed latencies, 10
// and 7 % behind instruction fetch.
#pragma once

#include "gated_math.cuh"

#include <limits.h>

namespace sgr {
namespace gated {

constexpr int kWarps = 12;                 // data warps
constexpr int kCarryWarps = 2;             // tiles in turn
constexpr int kThreads = (kWarps + kCarryWarps + 1) * 32;   // the last warp feeds the ring
constexpr int kRows = 16, kBwdRows = 8;    // rows per data warp and thread, forward and backward
constexpr int kTR = kWarps * kRows;        // rows per forward tile
constexpr int kBwdTR = kWarps * kBwdRows;  // rows per backward tile, and between saved states
constexpr int kSlots = 4, kBwdSlots = 5;   // tiles in shared memory
constexpr int kQ = 2;                      // tiles between fold and the end of their replay
constexpr uint32_t kCopyWait = 1u << 16;   // polls, of about 4 us, of a lost block for its copies in flight
static_assert(kTR == 2 * kBwdTR, "a forward tile holds two saved states");
constexpr int kSegs = 32;                  // most segments: one per lane of the feeding warp
constexpr uint64_t kNone = ~uint64_t(0);    // a word not yet published

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
    float *states;                         // state entering every kBwdTR rows of each segment, or null (forward)
    const void *cu;                        // n_seqs + 1 row bounds, or null: sequences of seq_rows rows
    int cu_bytes;                          // 4 or 8
    uint32_t seq_rows;
    int64_t rows, D, n_seqs;
    int64_t n_strips;
    int n_segs;                            // at most kSegs
    int zero_padding;                      // outputs of rows in no sequence: 0 written, else left
    uint64_t *words;                       // [chunks][n_strips][TC] what tiles hand on, ~0 at launch
    uint32_t *ticket;                      // ~0 at launch, or null: one chunk, tile = blockIdx.x
    uint32_t *status;                      // 0 at launch; SGR_ERR_TIMEOUT once a wait ran out; may be null
    uint32_t spin_limit;                   // polls of a look-back, one to three us each
    uint32_t tile_wait;                    // polls, of about 4 us, of a wait inside a block
    int64_t drop_tile;                     // testing: the tile of these words (word * n_strips + strip) hands nothing on
    int window;                            // chunks of a strip and segment that blocks may hold at a time
};

// bound i, clamped to what rows can be
__device__ __forceinline__ int cu_at(const GatedParams &p, int64_t i) {
    const int64_t b = p.cu_bytes == 8 ? static_cast<const int64_t *>(p.cu)[i] : int64_t(static_cast<const int32_t *>(p.cu)[i]);
    return int(b < -1 ? -1 : (b > p.rows + 1 ? p.rows + 1 : b));
}
// The bounds as the feeding warp reads them: from shared memory, where they
// are copied once if they fit (every tile looks them up, and a chain of loads
// from L2 took longer than the tile).
constexpr int kBoundsHeld = 1024;
struct Bounds {
    const GatedParams &p;
    const int *held;                       // or null
    __device__ __forceinline__ int operator()(int64_t i) const { return held ? held[i] : cu_at(p, i); }
};

__device__ __forceinline__ bool is_cut(float A) { return __float_as_uint(A) >> 31; }
// the map (A, B) applied to a state, and `then` after `first`
__device__ __forceinline__ float apply_map(float A, float B, float h) { return is_cut(A) ? B : fmaf(A, h, B); }
__device__ __forceinline__ float2 then_map(float2 first, float2 then) {
    return is_cut(then.x) ? then : make_float2(first.x * then.x, fmaf(then.x, first.y, then.y));
}

// What the feeding warp tells the others of a tile.
template <int TR> struct TileInfo {
    int64_t row0, row_end;                 // its rows (fewer than TR at the end of a segment)
    int64_t state_row;                     // place of its first row's state in `states`
    int there;                             // 0: no more tiles
    int strip, place, word;                // strip; chunk in processing order within the segment, and of all
    int last;                              // nothing of its segment follows
    int cut;                               // a sequence starts (1) or ends (2) in the tile
    uint4 masks[kWarps];                   // of each data warp's rows: starts, ends, in a sequence; .w: all plain
    int start[TR], end[TR];                // sequence that starts (ends) at the row, or -1
};

// Fill the table of the tile of rows [row0, row_end) (whole warp).  Bounds
// that are not ascending give wrong sequences but never a row or a sequence
// outside the buffers.
template <int TR>
__device__ __forceinline__ void fill_info(const GatedParams &p, const Bounds &cu, int64_t row0, int64_t row_end,
                                          TileInfo<TR> &t, int lane) {
    constexpr int R = TR / kWarps;
    int64_t lo_row = 0, hi_row = p.rows;   // rows that lie in sequences
    constexpr uint32_t all = (1u << R) - 1u;
    // most tiles lie inside one sequence: nothing starts or ends in them, and no row is looked at
    auto plain = [&] {
        if (lane < kWarps) t.masks[lane] = make_uint4(0u, 0u, all, 1u);
        if (lane == 0) {
            t.cut = 0;
            t.start[0] = t.end[TR - 1] = -1;
        }
    };
    if (p.cu == nullptr) {
        const uint32_t s0 = uint32_t(row0) / p.seq_rows, k0 = uint32_t(row0) - s0 * p.seq_rows;
        if (k0 > 0 && k0 + TR < p.seq_rows) return plain();
        uint32_t s = uint32_t(row0 + lane) / p.seq_rows, k = uint32_t(row0 + lane) - s * p.seq_rows;
        for (int r = lane; r < TR; r += 32) {
            const bool in = row0 + r < row_end;
            t.start[r] = in && k == 0 ? int(s) : -1;
            t.end[r] = in && k + 1 == p.seq_rows ? int(s) : -1;
            k += 32;
            if (k >= p.seq_rows) {
                const uint32_t over = k / p.seq_rows;
                s += over;
                k -= over * p.seq_rows;
            }
        }
    } else {
        // bounds at or below row0, by a 33-way search: the last of them begins the
        // sequence that holds row0
        int lo = 0, hi = int(p.n_seqs) + 1;
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32;
            const int64_t i = int64_t(lo) + int64_t(lane + 1) * step - 1;
            const bool below = i < hi && cu(i) <= row0;
            const int n = __popc(__ballot_sync(0xffffffffu, below));
            const int64_t next = int64_t(lo) + int64_t(n) * step;
            const int64_t top = int64_t(lo) + int64_t(n + 1) * step - 1;
            lo = int(next < hi ? next : hi);
            hi = int(top < hi ? top : hi);
        }
        if (lo > 0 && lo <= p.n_seqs && cu(lo - 1) < row0 && cu(lo) > row0 + TR && row0 + TR <= row_end) return plain();
        lo_row = cu(0);
        const int64_t last = cu(p.n_seqs);
        hi_row = last < p.rows ? last : p.rows;
        for (int r = lane; r < TR; r += 32) t.start[r] = t.end[r] = -1;
        __syncwarp();
        for (int64_t s = (lo > 0 ? lo - 1 : 0) + lane;; s += 32) {
            bool more = false;
            if (s < p.n_seqs) {
                const int64_t b = cu(s), e = cu(s + 1);
                more = b < row_end;
                if (b < e) {
                    if (b >= row0 && b < row_end) t.start[b - row0] = int(s);
                    if (e > row0 && e <= row_end) t.end[e - 1 - row0] = int(s);
                }
            }
            if (!__any_sync(0xffffffffu, more)) break;
        }
    }
    __syncwarp();
    int cut = 0;
#pragma unroll
    for (int r0 = 0; r0 < TR; r0 += 32) {
        const int r = r0 + lane;
        const uint32_t starts = __ballot_sync(0xffffffffu, r < TR && t.start[r < TR ? r : 0] >= 0);
        const uint32_t ends = __ballot_sync(0xffffffffu, r < TR && t.end[r < TR ? r : 0] >= 0);
        const uint32_t live = __ballot_sync(0xffffffffu, r < TR && row0 + r >= lo_row && row0 + r < hi_row && row0 + r < row_end);
        cut |= (starts ? 1 : 0) | (ends ? 2 : 0);
        if (lane < 32 / R && r0 / R + lane < kWarps) {
            const uint32_t a = starts >> (lane * R) & all, b = ends >> (lane * R) & all, c = live >> (lane * R) & all;
            t.masks[r0 / R + lane] = make_uint4(a, b, c, a == 0u && b == 0u && c == all);
        }
    }
    if (lane == 0) t.cut = cut;
}

// A tile's word for a channel: its map (A, B), and later the state behind it,
// which is the map that cuts, (-0, state).
__device__ __forceinline__ uint64_t word_of(float A, float B) {
    return (uint64_t(__float_as_uint(B)) << 32) | __float_as_uint(A);
}
__device__ __forceinline__ float word_a(uint64_t w) { return __uint_as_float(uint32_t(w)); }
__device__ __forceinline__ float word_b(uint64_t w) { return __uint_as_float(uint32_t(w >> 32)); }

// The words of this lane's E channels: each is read whole.
template <int E> __device__ __forceinline__ void load_words(const uint64_t *p, uint64_t (&m)[E]) {
    if constexpr (E == 1) {
        m[0] = ld_relaxed_u64(p);
    } else {
        asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(m[0]), "=l"(m[1]) : "l"(p) : "memory");
    }
}
template <int E> __device__ __forceinline__ bool words_in(const uint64_t (&m)[E]) {
    bool ok = m[0] != kNone;
    if constexpr (E == 2) ok = ok && m[1] != kNone;
    return ok;
}
// they are states (of words that are in)
template <int E> __device__ __forceinline__ bool words_cut(const uint64_t (&m)[E]) {
    bool ok = is_cut(word_a(m[0]));
    if constexpr (E == 2) ok = ok && is_cut(word_a(m[1]));
    return ok;
}
template <int E> __device__ __forceinline__ void apply_words(const uint64_t (&m)[E], float (&h)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) h[e] = apply_map(word_a(m[e]), word_b(m[e]), h[e]);
}

// The carry of one tile (carry warp): q its place in processing order within
// its segment, word that of its words, mute: it hands nothing on, tot the
// tile's maps of this lane's E channels.  Publishes, waits, and returns the
// entering states.  Tiles whose first row (in processing order) is a start
// enter with 0, which they never use.  One round trip reads the words of the
// kNear tiles before for every channel, and those of up to 32 more for the
// strip's first channel; if the state is among the far ones, a second round
// trip reads the rest of the channels.  No word is read that lies further back
// than the blocks can hold tiles of the strip (p.window), and where those are
// few the first round reads the tile before alone: an older word has left L2
// for memory, and a load from there, behind the streams, took 2.7 us.
// `meanwhile` runs under the first round.
constexpr int kNear = 4;
template <int E, class Meanwhile>
__device__ __forceinline__ void carry_tile_state(const GatedParams &p, int64_t strip, int q, int word, bool mute, int lane,
                                                 bool fresh, bool cut, const float2 (&tot)[E], float (&hin)[E],
                                                 Meanwhile meanwhile) {
    constexpr int TC = 32 * E;
    const int64_t step = p.n_strips * TC;                          // from a tile's words to the next chunk's
    const int64_t at = word * step + strip * TC + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) hin[e] = 0.f;
    auto publish_state = [&] {
        if (mute) return;
#pragma unroll
        for (int e = 0; e < E; ++e) st_relaxed_u64(p.words + at + e, word_of(-0.f, apply_map(tot[e].x, tot[e].y, hin[e])));
    };
    if (fresh) {
        publish_state();
        meanwhile();
        return;
    }
    if (cut) {                                                     // a start within: the state does not depend on what enters
        publish_state();
    } else if (!mute) {
#pragma unroll
        for (int e = 0; e < E; ++e) st_relaxed_u64(p.words + at + e, word_of(tot[e].x, tot[e].y));
    }
    bool found = false;
    for (uint32_t polls = 0; !found; ++polls) {
        uint64_t m[kNear][E];
        const int reach = polls == 0 && p.window <= 8 ? 1 : (q < p.window ? q : p.window);
#pragma unroll
        for (int i = 0; i < kNear; ++i) {
            m[i][0] = kNone;
            if (i < reach) load_words<E>(p.words + at - (i + 1) * step, m[i]);
        }
        const int far = 1 + kNear + lane;                          // this lane probes the tile that far before
        uint64_t probe = kNone;
        if (far <= reach) probe = ld_relaxed_u64(p.words + (word - far) * step + strip * TC);
        if (polls == 0) meanwhile();
        int k = -1;                                                // nearest state, maps there before it
        bool there = true;
#pragma unroll
        for (int i = 0; i < kNear; ++i) {
            there = there && words_in<E>(m[i]);
            if (there && k < 0 && words_cut<E>(m[i])) k = i;
        }
        if (__all_sync(0xffffffffu, k >= 0)) {
#pragma unroll
            for (int i = kNear - 1; i >= 0; --i)
                if (i <= k) apply_words<E>(m[i], hin);
            found = true;
        } else if (__all_sync(0xffffffffu, there)) {
            const uint32_t in = __ballot_sync(0xffffffffu, probe != kNone);
            const uint32_t state = __ballot_sync(0xffffffffu, probe != kNone && is_cut(word_a(probe)));
            const int j = state ? __ffs(state) - 1 : 0;
            const uint32_t nearer = (1u << j) - 1u;
            if (state && (in & nearer) == nearer) {
                bool ok = true;
                for (int i0 = j; i0 >= 0; i0 -= 4) {               // the state, then the maps of the far tiles, oldest first
                    uint64_t w[4][E];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (i0 - u >= 0) load_words<E>(p.words + at - (kNear + i0 - u + 1) * step, w[u]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (i0 - u >= 0) {
                            ok = ok && words_in<E>(w[u]);
                            if (i0 - u == j) ok = ok && words_cut<E>(w[u]);
                            apply_words<E>(w[u], hin);
                        }
                    }
                }
#pragma unroll
                for (int i = kNear - 1; i >= 0; --i) apply_words<E>(m[i], hin);
                found = __all_sync(0xffffffffu, ok);
            }
        }
        if (!found && polls >= p.spin_limit) {
            if (lane == 0) atomicExch(p.status, 5u);               // SGR_ERR_TIMEOUT
#pragma unroll
            for (int e = 0; e < E; ++e) hin[e] = __int_as_float(0x7fffffff);
            found = true;
        }
    }
    if (!cut) publish_state();
}

// Final (and gradient of initial) states of sequences without rows, which no
// tile visits: dst = src, or 0.
__device__ __forceinline__ void empty_sequences(const GatedParams &p, float *dst, const float *src, int64_t src_ss) {
    if (dst == nullptr || (p.cu == nullptr && p.rows > 0)) return;
    // 32 sequences a warp at a time, so that many bounds are on their way at
    // once: 4096 rows in 30000 sequences, 64 channels, take 46 us, and 224 us
    // with a sequence a block at a time
    constexpr int kAll = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t s0 = (int64_t(blockIdx.x) * kAll + warp) * 32; s0 < p.n_seqs; s0 += int64_t(gridDim.x) * kAll * 32) {
        const int64_t mine = s0 + lane;
        const bool none = mine < p.n_seqs && !(p.cu && cu_at(p, mine) < cu_at(p, mine + 1));
        for (uint32_t left = __ballot_sync(0xffffffffu, none); left; left &= left - 1) {
            const int64_t s = s0 + __ffs(left) - 1;
            for (int64_t d = lane; d < p.D; d += 32) dst[s * p.D + d] = src ? src[s * src_ss + d] : 0.f;
        }
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

// The scan is launched as the dependent of the kernel that sets its workspace
// to ~0 (programmatic launch), so that its blocks are set up by the time the
// words are: whoever touches the workspace waits here first.
__device__ __forceinline__ void workspace_ready() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// All of it to ~0, but the status word (the first) to 0.
__global__ void __launch_bounds__(256) gated_clear_kernel(uint4 *p, int64_t n) {
    asm volatile("griddepcontrol.launch_dependents;");
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
        p[i] = make_uint4(i ? ~0u : 0u, ~0u, ~0u, ~0u);
}

// ------------------------------------------------------ inside a block
//
// Tile n of the block lies in slot n % S from its copies until every data
// warp has replayed it; its maps and entering states in entry n % kQ: a data
// warp folds tile n after its replay of tile n - 2, which it began with that
// tile's states.  Every wait is bounded.  Each of these depends, through a
// warp or two of the block, on at most one look-back that may run to its own
// end, so their bound is twice as many polls, each longer.  Should one run
// out all the same, the block is lost: a warp whose wait failed leaves its loop
// without an arrival, so that no barrier ever counts a phase that did not
// happen and a wait that succeeds has found what it waited for; once all have
// left, the block writes NaN for every tile it had not finished and for those
// it can still draw, and hands NaN on (give_up).
template <typename V, int S, int TR, int MAPS> struct Block {
    uint64_t full[S], empty[S];            // copies and table there; replayed by every data warp
    uint64_t maps[kQ], in[kQ];             // maps there; entering states there
    TileInfo<TR> info[S];
    // maps of the data warps, then (by the carry warp) of everything before
    // each of them in the tile; the forward maps of a backward tile (1) turn
    // into the states entering each warp, in A
    V A[MAPS][kQ][kWarps][32], B[MAPS][kQ][kWarps][32];
    V enter[kQ][32];                       // states entering the tile
    int bounds[kBoundsHeld];
    int lost;                              // a wait ran out
    int fed, done[kWarps];                 // tiles handed over; replayed by each data warp (at its end)
    uint32_t ticket;                       // the feeding warp's last, in hand or behind the end
};
template <int S, class B> __device__ __forceinline__ void init_block(B &blk) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_addr(&blk.full[i]), 1);
            mbar_init(smem_addr(&blk.empty[i]), kWarps);
        }
        for (int i = 0; i < kQ; ++i) {
            mbar_init(smem_addr(&blk.maps[i]), kWarps);
            mbar_init(smem_addr(&blk.in[i]), 1);
        }
        blk.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Wait of a warp for use u of a barrier (its phases are uses 0, 1, 2, ...), all
// lanes together: the result is the warp's, and each poll suspends it for up to
// 4 us (75 ns where some lanes of a warp poll alone).  (Lanes that poll by
// themselves and vote behind it: 189 us for bf16 32768 x 4096 forward, 186 so;
// a limit by the clock 197.)
struct Waiter {
    int *lost;
    uint32_t limit;
    __device__ __forceinline__ bool operator()(uint64_t *bar, int u) const {
        const uint32_t at = smem_addr(bar), phase = uint32_t(u & 1);
        bool ok = mbar_try_wait(at, phase);
        if (__builtin_expect(__all_sync(0xffffffffu, ok), 1)) return true;
        uint32_t polls = 1;
        do {
            ok = __all_sync(0xffffffffu, mbar_try_wait(at, phase));
        } while (!ok && ++polls < limit);
        if (!ok) *lost = 1;
        return ok;
    }
};
__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fffffff); }

template <typename IO, int E, int OPS, int S, int TR, bool TMA>
struct SmemShape {
    static constexpr int TC = 32 * E;
    static constexpr uint32_t op_bytes = TR * TC * sizeof(IO);
    static constexpr uint32_t slot_bytes = OPS * op_bytes;
    static constexpr uint32_t ring_bytes = TMA ? S * slot_bytes : 0;
    static_assert(op_bytes % 128 == 0 && TR <= 256, "copy boxes");
};

// The segments, one per lane of the feeding warp: rows [start, start + len),
// n chunks of TR rows.  Segment g begins at the sequence bound nearest to
// rows g / n_segs, segment 0 at row 0.  A tile is found from its ticket in
// order of the place within the segment, then the segment, then the strip.
template <int TR> struct Segments {
    int64_t start, len;
    int n, word0, state0;                  // chunks; chunks and kept states of the segments before
    int total;                             // chunks of all
    int c, below;                          // place reached, and chunks at lower places

    __device__ __forceinline__ void init(const GatedParams &p, const Bounds &cu, int lane) {
        int64_t at = p.rows;
        if (lane == 0) {
            at = 0;
        } else if (lane < p.n_segs) {
            const int64_t ideal = p.rows / p.n_segs * lane;
            if (p.cu == nullptr) {
                at = (ideal + p.seq_rows / 2) / p.seq_rows * p.seq_rows;
            } else {
                int64_t lo = 0, hi = p.n_seqs + 1;                 // bounds at or below the ideal one
                while (lo < hi) {
                    const int64_t mid = (lo + hi) / 2;
                    if (cu(mid) <= ideal) lo = mid + 1;
                    else hi = mid;
                }
                const int64_t up = lo <= p.n_seqs ? cu(lo) : cu(p.n_seqs);
                const int64_t down = lo > 0 ? cu(lo - 1) : up;
                at = ideal - down <= up - ideal ? down : up;
            }
            if (at < 0) at = 0;
            if (at > p.rows) at = p.rows;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {                         // ascending whatever the bounds are
            const int64_t x = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o && x > at) at = x;
        }
        start = at;
        const int64_t next = __shfl_down_sync(0xffffffffu, at, 1);
        len = lane >= p.n_segs ? 0 : (lane == p.n_segs - 1 ? p.rows : next) - start;
        n = int((len + TR - 1) / TR);
        const int k = int((len + kBwdTR - 1) / kBwdTR);
        int a = n, b = k;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) {
                a += x;
                b += y;
            }
        }
        word0 = a - n;
        state0 = b - k;
        total = __shfl_sync(0xffffffffu, a, 31);
        c = below = 0;
    }
    // the segment of chunk `k` in processing order (k ascends from call to call, below total); c is its place
    __device__ __forceinline__ int find(int k, int lane) {
        uint32_t live = __ballot_sync(0xffffffffu, n > c);
        while (k >= below + __popc(live)) {
            const int cnt = __popc(live);
            const int shortest = __reduce_min_sync(0xffffffffu, n > c ? n : INT_MAX);
            const int want = (k - below) / cnt, most = shortest - c;
            const int steps = want < most ? want : most;
            c += steps;
            below += steps * cnt;
            live = __ballot_sync(0xffffffffu, n > c);
        }
        const int rank = __popc(live & ((1u << lane) - 1u));
        return __ffs(__ballot_sync(0xffffffffu, n > c && rank == k - below)) - 1;
    }
};

// A tile load that says its lines will not be wanted again, so that the words
// that blocks hand one another stay in L2.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}

// The tile of a ticket (whole warp); false behind the last.  `reverse`: places
// count from the segment's end.
template <int TR> struct TileAt {
    int64_t row0, row_end;
    int strip, place, word, state, last;

    __device__ __forceinline__ bool find(const GatedParams &p, Segments<TR> &seg, uint32_t tile, int lane, bool reverse) {
        const uint32_t k = tile / uint32_t(p.n_strips);
        const bool there = k < uint32_t(seg.total);
        int g = 0;
        if (there) g = seg.find(int(k), lane);
        const int count = __shfl_sync(0xffffffffu, seg.n, g);
        const int c = reverse ? count - 1 - seg.c : seg.c;                      // chunk of the segment
        const int64_t from = __shfl_sync(0xffffffffu, seg.start, g), end = from + __shfl_sync(0xffffffffu, seg.len, g);
        strip = int(tile - k * uint32_t(p.n_strips));
        place = seg.c;
        word = __shfl_sync(0xffffffffu, seg.word0, g) + seg.c;
        state = __shfl_sync(0xffffffffu, seg.state0, g) + c * (TR / kBwdTR);
        last = seg.c + 1 == count;
        row0 = from + int64_t(c) * TR;
        row_end = row0 + TR < end ? row0 + TR : end;
        return there;
    }
    __device__ __forceinline__ void put(TileInfo<TR> &info) const {
        info.row0 = row0;
        info.row_end = row_end;
        info.state_row = state;
        info.strip = strip;
        info.place = place;
        info.word = word;
        info.last = last;
    }
};

// The feeding warp: draws tickets, starts the copies of a tile when its slot
// is free, writes its table and hands both over.  Ends with one entry for each
// carry warp that says so, so that each of them comes upon one; a lost block's
// when its copies in flight have landed.
template <int S, int OPS, int TR, uint32_t OP_BYTES, int TC, bool TMA, class B>
__device__ __forceinline__ void feed(const GatedParams &p, B &blk, uint32_t slots, int lane, bool reverse,
                                     const CUtensorMap *m0, const CUtensorMap *m1, const CUtensorMap *m2) {
    const Waiter wait{&blk.lost, p.tile_wait};
    const bool held = p.cu != nullptr && p.n_seqs < kBoundsHeld;
    if (held)
        for (int i = lane; i <= int(p.n_seqs); i += 32) blk.bounds[i] = cu_at(p, i);
    const Bounds bounds{p, held ? blk.bounds : nullptr};
    __syncwarp();
    Segments<TR> seg;
    seg.init(p, bounds, lane);
    // the next ticket is drawn a tile ahead, so that its round trip passes under the work on this one
    uint32_t ticket = 0;
    if (p.ticket) {
        workspace_ready();
        if (lane == 0) ticket = atomicAdd(p.ticket, 1u) + 1u;
    } else {
        ticket = blockIdx.x;
    }
    uint64_t once;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    int ends = 0, n = 0;
    for (; ends < kCarryWarps; ++n) {
        TileAt<TR> at;
        const bool more = at.find(p, seg, __shfl_sync(0xffffffffu, ticket, 0), lane, reverse) && ends == 0;
        if (n >= S && !wait(&blk.empty[n % S], n / S - 1)) break;
        TileInfo<TR> &info = blk.info[n % S];
        if (more) {
            if (lane == 0) {
                if constexpr (TMA) {
                    const uint32_t bar = smem_addr(&blk.full[n % S]);
                    const uint32_t dst = slots + uint32_t(n % S) * (OPS * OP_BYTES);
                    // the data warps' reads of the slot came before the copies into it
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(OPS * OP_BYTES)
                                 : "memory");
                    load_tile(dst, m0, at.strip * TC, int(at.row0), bar, once);
                    load_tile(dst + OP_BYTES, m1, at.strip * TC, int(at.row0), bar, once);
                    if constexpr (OPS == 3) load_tile(dst + 2 * OP_BYTES, m2, at.strip * TC, int(at.row0), bar, once);
                }
                ticket = p.ticket ? atomicAdd(p.ticket, 1u) + 1u : uint32_t(p.n_strips);
                at.put(info);
            }
            __syncwarp();
            fill_info<TR>(p, bounds, at.row0, at.row_end, info, lane);
        } else {
            ++ends;
        }
        if (lane == 0) info.there = more;
        __syncwarp();
        if (lane == 0) arrive(&blk.full[n % S]);
    }
    if (lane == 0) {
        blk.fed = n;
        blk.ticket = ticket;
    }
    if (ends < kCarryWarps)
        for (int m = n > S ? n - S : 0; m < n; ++m) mbar_wait(smem_addr(&blk.full[m % S]), uint32_t(m / S & 1), kCopyWait);
}

// Maps of a channel's E elements composed: `then` after `first`.
template <class V> __device__ __forceinline__ void compose(V &A, V &B, V a, V b, bool cuts) {
    if (cuts) {
        if constexpr (sizeof(V) == 4) {
            const float2 m = then_map(make_float2(A, B), make_float2(a, b));
            A = m.x;
            B = m.y;
        } else {
            const float2 x = then_map(make_float2(A.x, B.x), make_float2(a.x, b.x));
            const float2 y = then_map(make_float2(A.y, B.y), make_float2(a.y, b.y));
            A = make_float2(x.x, y.x);
            B = make_float2(x.y, y.y);
        }
    } else {
        B = vfma(a, B, b);
        A = vmul(A, a);
    }
}
template <class V> __device__ __forceinline__ V apply_vec(V A, V B, V h) {
    return vmap(A, B, h, [](float x, float y, float z) { return apply_map(x, y, z); });
}

// A carry warp: tiles c, c + kCarryWarps, ... of the block.  It is one warp's
// dependent instructions that set the pace here, so before the wait it only
// composes the warps' maps (leaving in their place the maps of what precedes
// each warp) and publishes, and behind it stores one state per channel.
// Forward (DIR +1): warps in order; the states entering the tile and its
// second half are kept in p.states if given.  Backward (DIR -1): warps from
// the last, and under the wait (map 1) the states of the forward recurrence
// within the tile, from p.states.
template <int E, int S, int TR, int DIR, class B>
__device__ __forceinline__ void carry_loop(const GatedParams &p, B &blk, int c, int lane) {
    using V = typename FVec<E>::type;
    const Waiter wait{&blk.lost, p.tile_wait};
    workspace_ready();
    for (int n = c;; n += kCarryWarps) {
        if (!wait(&blk.full[n % S], n / S)) return;
        const TileInfo<TR> &info = blk.info[n % S];
        if (!info.there) return;
        const int64_t strip = info.strip, state = info.state_row;
        const int q = info.place, word = info.word;
        const bool fresh = q == 0 || (DIR > 0 ? info.start[0] : info.end[TR - 1]) >= 0, last = info.last;
        const bool mute = last || int64_t(word) * p.n_strips + strip == p.drop_tile;
        const bool halves = info.row0 + kBwdTR < info.row_end;
        const bool cut = info.cut & (DIR > 0 ? 1 : 2), begins = info.cut & 1;
        const int e0 = n % kQ;
        const int64_t d0 = strip * 32 * E + lane * E;
        V hf = vset<V>(0.f);
        if constexpr (DIR < 0) {
            if (info.start[0] < 0 && !last) hf = state_row<E>(p.states, state * p.D, d0, p.D);
        }
        if (!wait(&blk.maps[e0], n / kQ)) return;
        V A[kWarps], B_[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            A[w] = blk.A[0][e0][w][lane];
            B_[w] = blk.B[0][e0][w][lane];
        }
        V tA = A[DIR > 0 ? 0 : kWarps - 1], tB = B_[DIR > 0 ? 0 : kWarps - 1];
#pragma unroll
        for (int j = 1; j < kWarps; ++j) {
            const int w = DIR > 0 ? j : kWarps - 1 - j;
            const V a = A[w], b = B_[w];
            blk.A[0][e0][w][lane] = tA;
            blk.B[0][e0][w][lane] = tB;
            compose(tA, tB, a, b, cut);
        }
        float2 tot[E];
        float hin[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            tot[e] = make_float2(reinterpret_cast<const float *>(&tA)[e], reinterpret_cast<const float *>(&tB)[e]);
        carry_tile_state<E>(p, strip, q, word, mute, lane, fresh, cut, tot, hin, [&] {
            if constexpr (DIR < 0) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const V a = blk.A[1][e0][w][lane], b = blk.B[1][e0][w][lane];
                    blk.A[1][e0][w][lane] = hf;
                    hf = begins ? apply_vec(a, b, hf) : vfma(a, hf, b);
                }
            }
        });
        V h;
#pragma unroll
        for (int e = 0; e < E; ++e) reinterpret_cast<float *>(&h)[e] = hin[e];
        blk.enter[e0][lane] = h;
        __syncwarp();
        if constexpr (DIR > 0) {
            // read before the data warps may go on to overwrite the maps
            const V half = p.states ? apply_vec(blk.A[0][e0][kWarps / 2][lane], blk.B[0][e0][kWarps / 2][lane], h) : h;
            if (lane == 0) arrive(&blk.in[e0]);
            if (p.states) {
                put_state_row<E>(p.states, state * p.D, d0, p.D, h);
                if (halves) put_state_row<E>(p.states, (state + 1) * p.D, d0, p.D, half);
            }
        } else {
            if (lane == 0) arrive(&blk.in[e0]);
        }
    }
}

// What a lost block still does (all of it, its loops ended): NaN for the tiles
// that not every data warp has replayed, whose tables are still in their
// slots, then for the ticket in hand and all it can draw; and NaN handed on, so
// that no other block waits for these tiles.
template <typename IO, int E, int S, int TR, int DIR, class B>
__device__ __noinline__ void give_up(const GatedParams &p, B &blk, int warp, int lane) {
    using V = typename FVec<E>::type;
    using W = typename Raw<IO, E>::type;
    constexpr int R = TR / kWarps;
    const V bad = vset<V>(nan_value());
    const W out = Conv<IO, E>::out(bad);
    auto spoil = [&](const TileInfo<TR> &info) {
        const int64_t d0 = int64_t(info.strip) * 32 * E + lane * E;
        if (warp < kWarps) {
            const uint4 k = info.masks[warp];
            for (int r = 0; r < R; ++r) {
                const int64_t row = info.row0 + warp * R + r;
                if (row >= info.row_end) break;
                const bool live = k.z >> r & 1u;
                if (d0 < p.D && (live || p.zero_padding)) {
                    if constexpr (DIR > 0) {
                        reinterpret_cast<W *>(static_cast<char *>(p.h) + (row * p.h_rs + d0) * int64_t(sizeof(IO)))[0] = live ? out : W(0);
                    } else {
                        reinterpret_cast<W *>(static_cast<char *>(p.df) + (row * p.df_rs + d0) * int64_t(sizeof(IO)))[0] = live ? out : W(0);
                        reinterpret_cast<W *>(static_cast<char *>(p.dv) + (row * p.dv_rs + d0) * int64_t(sizeof(IO)))[0] = live ? out : W(0);
                    }
                }
                if constexpr (DIR > 0) {
                    if ((k.y >> r & 1u) && p.h_last) put_state_row<E>(p.h_last, info.end[warp * R + r] * p.D, d0, p.D, bad);
                } else {
                    if ((k.x >> r & 1u) && p.dh0) put_state_row<E>(p.dh0, info.start[warp * R + r] * p.D, d0, p.D, bad);
                }
            }
        } else if (warp == kWarps) {
            if (DIR > 0 && p.states) {
                put_state_row<E>(p.states, info.state_row * p.D, d0, p.D, bad);
                if (info.row0 + kBwdTR < info.row_end) put_state_row<E>(p.states, (info.state_row + 1) * p.D, d0, p.D, bad);
            }
            if (p.words && !info.last) {
                const int64_t at = (info.word * p.n_strips + info.strip) * 32 * E + lane * E;
                for (int e = 0; e < E; ++e) st_relaxed_u64(p.words + at + e, word_of(-0.f, nan_value()));
            }
        }
    };
    workspace_ready();
    if (threadIdx.x == 0 && p.status) atomicExch(p.status, 5u);      // SGR_ERR_TIMEOUT
    int from = blk.fed;
    for (int w = 0; w < kWarps; ++w) from = blk.done[w] < from ? blk.done[w] : from;
    for (int n = from; n < blk.fed; ++n)
        if (blk.info[n % S].there) spoil(blk.info[n % S]);
    const Bounds bounds{p, nullptr};
    Segments<TR> seg;
    seg.init(p, bounds, lane);
    uint32_t ticket = blk.ticket;
    for (;;) {
        __syncthreads();
        if (warp == kThreads / 32 - 1) {
            TileAt<TR> at;
            const bool more = at.find(p, seg, __shfl_sync(0xffffffffu, ticket, 0), lane, DIR < 0);
            if (more) {
                if (lane == 0) {
                    ticket = p.ticket ? atomicAdd(p.ticket, 1u) + 1u : uint32_t(p.n_strips);
                    at.put(blk.info[0]);
                }
                __syncwarp();
                fill_info<TR>(p, bounds, at.row0, at.row_end, blk.info[0], lane);
            }
            if (lane == 0) blk.info[0].there = more;
        }
        __syncthreads();
        if (!blk.info[0].there) break;
        spoil(blk.info[0]);
    }
}

// The state entering data warp w (in processing order the first: the tile's own)
template <int FIRST, class B, class V>
__device__ __forceinline__ V entering(const B &blk, int e0, int warp, int lane, V h) {
    return warp == FIRST ? h : apply_vec(blk.A[0][e0][warp][lane], blk.B[0][e0][warp][lane], h);
}

// The thread's rows of an operand: from the slot, or from memory, all of them
// asked for at once (a row's branches would set its load behind the row
// before: 61 rows of 1001 fp16 17.6 us, and 16.5 so).
template <typename IO, int E, bool TMA, int R> struct RowReader;
template <typename IO, int E, int R> struct RowReader<IO, E, true, R> {
    using Word = typename Raw<IO, E>::type;
    const Word *src;                       // the warp's first row
    __device__ __forceinline__ typename FVec<E>::type operator()(int r) const { return Conv<IO, E>::in(src[r * 32]); }
};
template <typename IO, int E, int R> struct RowReader<IO, E, false, R> {
    using Word = typename Raw<IO, E>::type;
    Word x[R];
    __device__ __forceinline__ typename FVec<E>::type operator()(int r) const { return Conv<IO, E>::in(x[r]); }
};
template <typename IO, int E, bool TMA, int R, class Shape, int OP>
__device__ __forceinline__ RowReader<IO, E, TMA, R> reader(const GatedParams &p, const unsigned char *smem, int slot, int warp,
                                                           int lane, int64_t row, int64_t d0, const void *base, int64_t rs) {
    using Word = typename Raw<IO, E>::type;
    RowReader<IO, E, TMA, R> y;
    if constexpr (TMA) {
        y.src = reinterpret_cast<const Word *>(smem + slot * Shape::slot_bytes + OP * Shape::op_bytes) + warp * R * 32 + lane;
    } else {
        const int64_t left = d0 < p.D ? p.rows - row : 0;
        const char *from = static_cast<const char *>(base) + (row * rs + d0) * int64_t(sizeof(IO));
#pragma unroll
        for (int r = 0; r < R; ++r)
            y.x[r] = r < left ? *reinterpret_cast<const Word *>(from + r * rs * int64_t(sizeof(IO))) : Word(0);
    }
    return y;
}

// ------------------------------------------------------------- forward
//
// What a thread keeps of an element between fold and replay, and the step.
template <int GATE, typename IO, class V>
__device__ __forceinline__ V fwd_gate(V f) {
    if constexpr (GATE == GATE_LOG) {
        return log_decay(f);
    } else {
        return hold_gate<IO>(f);
    }
}
template <int GATE, typename IO, class V>
__device__ __forceinline__ void fwd_step(V g, V v, V &a, V &b) {
    if constexpr (GATE == GATE_LOG) {
        a = g;
        b = v;
    } else {
        V z;
        open_gate<IO>(g, a, z);
        b = vmul(z, v);
    }
}

template <typename IO, int E, bool TMA> struct ForwardShape {
    using Ring = SmemShape<IO, E, 2, kSlots, kTR, TMA>;
    using Blk = Block<typename FVec<E>::type, kSlots, kTR, 1>;
    static constexpr uint32_t smem_bytes = Ring::ring_bytes + sizeof(Blk);
};

template <typename IO, int E, int GATE, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
gated_scan_kernel(const __grid_constant__ GatedParams p, const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_v) {
    using V = typename FVec<E>::type;
    using W = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    using Shape = typename ForwardShape<IO, E, TMA>::Ring;
    using Blk = typename ForwardShape<IO, E, TMA>::Blk;
    constexpr int S = kSlots, R = kRows, TC = 32 * E;
    extern __shared__ __align__(128) unsigned char smem[];
    Blk &blk = *reinterpret_cast<Blk *>(smem + Shape::ring_bytes);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    init_block<S>(blk);
    if (warp < kWarps) {
        const Waiter wait{&blk.lost, p.tile_wait};
        V gate[2][R];
        // tile n: gates into registers, the warp's map to shared memory; false behind the last tile
        // and where a wait ran out
        auto fold = [&](int n, V (&g)[R]) {
            if (!wait(&blk.full[n % S], n / S)) return false;
            const TileInfo<kTR> &info = blk.info[n % S];
            if (!info.there) return false;
            const int64_t row = info.row0 + warp * R, d0 = int64_t(info.strip) * TC + lane * E;
            const auto f = reader<IO, E, TMA, R, Shape, 0>(p, smem, n % S, warp, lane, row, d0, p.f, p.f_rs);
            const auto v = reader<IO, E, TMA, R, Shape, 1>(p, smem, n % S, warp, lane, row, d0, p.v, p.v_rs);
            const uint4 k = info.masks[warp];
            V A = vset<V>(1.f), B = vset<V>(0.f);
            if (k.x == 0u) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    V a, b;
                    g[r] = fwd_gate<GATE, IO>(f(r));
                    fwd_step<GATE, IO>(g[r], v(r), a, b);
                    B = vfma(a, B, b);
                    A = vmul(A, a);
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    V a, b;
                    g[r] = fwd_gate<GATE, IO>(f(r));
                    fwd_step<GATE, IO>(g[r], v(r), a, b);
                    if (k.x >> r & 1u) {
                        A = vset<V>(-0.f);
                        B = state_row<E>(p.h0, info.start[warp * R + r] * p.h0_ss, d0, p.D);
                    }
                    B = vfma(a, B, b);
                    A = vmul(A, a);
                }
            }
            blk.A[0][n % kQ][warp][lane] = A;
            blk.B[0][n % kQ][warp][lane] = B;
            __syncwarp();
            if (lane == 0) arrive(&blk.maps[n % kQ]);
            return true;
        };
        auto replay = [&](int n, const V (&g)[R]) {
            const TileInfo<kTR> &info = blk.info[n % S];
            const int64_t row = info.row0 + warp * R, d0 = int64_t(info.strip) * TC + lane * E;
            const auto v = reader<IO, E, TMA, R, Shape, 1>(p, smem, n % S, warp, lane, row, d0, p.v, p.v_rs);
            const uint4 k = info.masks[warp];
            const bool dvalid = d0 < p.D;
            char *dst = static_cast<char *>(p.h) + (row * p.h_rs + d0) * int64_t(sizeof(IO));
            const int64_t pitch = p.h_rs * int64_t(sizeof(IO));
            if (!wait(&blk.in[n % kQ], n / kQ)) return false;
            V h = entering<0>(blk, n % kQ, warp, lane, blk.enter[n % kQ][lane]);
            if (k.w) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    V a, b;
                    fwd_step<GATE, IO>(g[r], v(r), a, b);
                    h = vfma(a, h, b);
                    if (dvalid) __stcs(reinterpret_cast<W *>(dst), C::out(h));
                    dst += pitch;
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    V a, b;
                    fwd_step<GATE, IO>(g[r], v(r), a, b);
                    if (k.x >> r & 1u) h = state_row<E>(p.h0, info.start[warp * R + r] * p.h0_ss, d0, p.D);
                    h = vfma(a, h, b);
                    if (dvalid && row + r < info.row_end) {
                        if (k.z >> r & 1u) __stcs(reinterpret_cast<W *>(dst), C::out(h));
                        else if (p.zero_padding) __stcs(reinterpret_cast<W *>(dst), W(0));
                    }
                    dst += pitch;
                    if ((k.y >> r & 1u) && p.h_last) put_state_row<E>(p.h_last, info.end[warp * R + r] * p.D, d0, p.D, h);
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&blk.empty[n % S]);
            return true;
        };
        // one copy of either body: with two, for registers that need not move, the warps
        // spent a fifth of their time waiting for instructions
        int done = 0;
#pragma unroll 1
        for (int n = 0;; ++n) {
            const bool more = fold(n, gate[0]);
            if (n > 0) {
                if (!replay(n - 1, gate[1])) break;
                done = n;
            }
            if (!more) break;
#pragma unroll
            for (int r = 0; r < R; ++r) gate[1][r] = gate[0][r];
        }
        if (lane == 0) blk.done[warp] = done;
    } else if (warp < kWarps + kCarryWarps) {
        carry_loop<E, S, kTR, 1>(p, blk, warp - kWarps, lane);
    } else {
        feed<S, 2, kTR, Shape::op_bytes, TC, TMA>(p, blk, smem_addr(smem), lane, false, &map_f, &map_v, nullptr);
    }
    __syncthreads();
    if (blk.lost) give_up<IO, E, S, kTR, 1>(p, blk, warp, lane);
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
// D per kBwdTR rows), instead of being read back: the outputs h are not
// needed, so the pass reads three arrays and not four, and the states have
// not been rounded to 16 bits.
//
// What a thread keeps of a gate: GATE_SIGMOID as forward; GATE_LOG: a, negated
// where f > 0, which has no gradient.
template <int GATE, typename IO, class V>
__device__ __forceinline__ V bwd_gate(V f) {
    if constexpr (GATE == GATE_SIGMOID) return fwd_gate<GATE, IO>(f);
    else return vmap(log_decay(f), f, [](float t, float x) { return x > 0.f ? -t : t; });
}
// (a, z) of it; z is 1 for GATE_LOG
template <int GATE, typename IO, class V>
__device__ __forceinline__ void bwd_split(V s, V &a, V &z) {
    if constexpr (GATE == GATE_SIGMOID) {
        open_gate<IO>(s, a, z);
    } else {
        a = vmap(s, [](float x) { return fabsf(x); });
        z = vset<V>(1.f);
    }
}

// df of a row from c = a z (h - v) or a h: where f > 0 it is 0, whatever c and
// g are (a product would make NaN of an infinite one).
template <int GATE, class V> __device__ __forceinline__ V bwd_df(V s, V c, V g) {
    const V y = vmul(c, g);
    if constexpr (GATE == GATE_SIGMOID) return y;
    else return vmap(s, y, [](float t, float u) { return is_cut(t) ? 0.f : u; });
}

template <typename IO, int E, bool TMA> struct BackwardShape {
    using Ring = SmemShape<IO, E, 3, kBwdSlots, kBwdTR, TMA>;
    using Blk = Block<typename FVec<E>::type, kBwdSlots, kBwdTR, 2>;            // maps 0: reverse, 1: forward
    static constexpr uint32_t smem_bytes = Ring::ring_bytes + sizeof(Blk);
};

template <typename IO, int E, int GATE, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
gated_scan_backward_kernel(const __grid_constant__ GatedParams p, const __grid_constant__ CUtensorMap map_f,
                           const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_dh) {
    using V = typename FVec<E>::type;
    using W = typename Raw<IO, E>::type;
    using C = Conv<IO, E>;
    using Shape = typename BackwardShape<IO, E, TMA>::Ring;
    using Blk = typename BackwardShape<IO, E, TMA>::Blk;
    constexpr int S = kBwdSlots, R = kBwdRows, TC = 32 * E;
    extern __shared__ __align__(128) unsigned char smem[];
    Blk &blk = *reinterpret_cast<Blk *>(smem + Shape::ring_bytes);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    init_block<S>(blk);
    if (warp < kWarps) {
        const Waiter wait{&blk.lost, p.tile_wait};
        V gate[2][R];
        auto fold = [&](int n, V (&s)[R]) {
            if (!wait(&blk.full[n % S], n / S)) return false;
            const TileInfo<kBwdTR> &info = blk.info[n % S];
            if (!info.there) return false;
            const int64_t row = info.row0 + warp * R, d0 = int64_t(info.strip) * TC + lane * E;
            const auto f = reader<IO, E, TMA, R, Shape, 0>(p, smem, n % S, warp, lane, row, d0, p.f, p.f_rs);
            const auto v = reader<IO, E, TMA, R, Shape, 1>(p, smem, n % S, warp, lane, row, d0, p.v, p.v_rs);
            const auto dh = reader<IO, E, TMA, R, Shape, 2>(p, smem, n % S, warp, lane, row, d0, p.dh, p.dh_rs);
            const uint4 k = info.masks[warp];
            V A = vset<V>(1.f), B = vset<V>(0.f), RA = vset<V>(1.f), RB = vset<V>(0.f);
            // rows without a branch, so that their loads and gates run side by side (with a
            // branch for starts and ends in each: 148 us for this pass on bf16 16384 x 2048)
            {
                V a[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    V z;
                    s[r] = bwd_gate<GATE, IO>(f(r));
                    bwd_split<GATE, IO>(s[r], a[r], z);
                    B = vfma(a[r], B, GATE == GATE_SIGMOID ? vmul(z, v(r)) : v(r));
                    A = vmul(A, a[r]);
                }
#pragma unroll
                for (int r = R - 1; r >= 0; --r) {
                    RB = vmul(a[r], vadd(RB, dh(r)));
                    RA = vmul(RA, a[r]);
                }
            }
            if (!k.w) {                                               // few tiles: the folds again, row by row
                A = RA = vset<V>(1.f);
                B = RB = vset<V>(0.f);
#pragma unroll (TMA ? 1 : R)
                for (int r = 0; r < R; ++r) {
                    V a, z;
                    bwd_split<GATE, IO>(bwd_gate<GATE, IO>(f(r)), a, z);
                    if (k.x >> r & 1u) {
                        A = vset<V>(-0.f);
                        B = state_row<E>(p.h0, info.start[warp * R + r] * p.h0_ss, d0, p.D);
                    }
                    B = vfma(a, B, GATE == GATE_SIGMOID ? vmul(z, v(r)) : v(r));
                    A = vmul(A, a);
                }
#pragma unroll (TMA ? 1 : R)
                for (int r = R - 1; r >= 0; --r) {
                    V a, z;
                    bwd_split<GATE, IO>(bwd_gate<GATE, IO>(f(r)), a, z);
                    if (k.y >> r & 1u) {
                        RA = vset<V>(-0.f);
                        RB = state_row<E>(p.dh_last, info.end[warp * R + r] * p.D, d0, p.D);
                    }
                    RB = vmul(a, vadd(RB, dh(r)));
                    RA = vmul(RA, a);
                }
            }
            blk.A[0][n % kQ][warp][lane] = RA;
            blk.B[0][n % kQ][warp][lane] = RB;
            blk.A[1][n % kQ][warp][lane] = A;
            blk.B[1][n % kQ][warp][lane] = B;
            __syncwarp();
            if (lane == 0) arrive(&blk.maps[n % kQ]);
            return true;
        };
        auto replay = [&](int n, const V (&s)[R]) {
            const TileInfo<kBwdTR> &info = blk.info[n % S];
            const int64_t row = info.row0 + warp * R, d0 = int64_t(info.strip) * TC + lane * E;
            const auto v = reader<IO, E, TMA, R, Shape, 1>(p, smem, n % S, warp, lane, row, d0, p.v, p.v_rs);
            const auto dh = reader<IO, E, TMA, R, Shape, 2>(p, smem, n % S, warp, lane, row, d0, p.dh, p.dh_rs);
            const uint4 k = info.masks[warp];
            const bool dvalid = d0 < p.D;
            if (!wait(&blk.in[n % kQ], n / kQ)) return false;
            V h = blk.A[1][n % kQ][warp][lane];
            V c[R];                                                   // df = c g
            auto forward = [&](auto plain) {
                constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (!PLAIN && (k.x >> r & 1u)) h = state_row<E>(p.h0, info.start[warp * R + r] * p.h0_ss, d0, p.D);
                    const V x = v(r);
                    V a, z;
                    bwd_split<GATE, IO>(s[r], a, z);
                    if constexpr (GATE == GATE_SIGMOID) {
                        c[r] = vmul(vmul(a, z), vfma(x, vset<V>(-1.f), h));
                        h = vfma(a, h, vmul(z, x));
                    } else {
                        c[r] = vmul(s[r], h);
                        h = vfma(a, h, x);
                    }
                }
            };
            if (k.w) forward(std::true_type{});
            else forward(std::false_type{});
            V flow = entering<kWarps - 1>(blk, n % kQ, warp, lane, blk.enter[n % kQ][lane]);
            char *pf = static_cast<char *>(p.df) + ((row + R - 1) * p.df_rs + d0) * int64_t(sizeof(IO));
            char *pv = static_cast<char *>(p.dv) + ((row + R - 1) * p.dv_rs + d0) * int64_t(sizeof(IO));
            const int64_t pitch_f = p.df_rs * int64_t(sizeof(IO)), pitch_v = p.dv_rs * int64_t(sizeof(IO));
            if (k.w) {
#pragma unroll
                for (int r = R - 1; r >= 0; --r) {
                    const V g = vadd(flow, dh(r));
                    V a, z;
                    bwd_split<GATE, IO>(s[r], a, z);
                    if (dvalid) {
                        __stcs(reinterpret_cast<W *>(pf), C::out(bwd_df<GATE>(s[r], c[r], g)));
                        __stcs(reinterpret_cast<W *>(pv), C::out(GATE == GATE_SIGMOID ? vmul(z, g) : g));
                    }
                    pf -= pitch_f;
                    pv -= pitch_v;
                    flow = vmul(a, g);
                }
            } else {
#pragma unroll
                for (int r = R - 1; r >= 0; --r) {
                    if (k.y >> r & 1u) flow = state_row<E>(p.dh_last, info.end[warp * R + r] * p.D, d0, p.D);
                    const V g = vadd(flow, dh(r));
                    V a, z;
                    bwd_split<GATE, IO>(s[r], a, z);
                    if (dvalid && row + r < info.row_end) {
                        const bool live = k.z >> r & 1u;
                        __stcs(reinterpret_cast<W *>(pf), live ? C::out(bwd_df<GATE>(s[r], c[r], g)) : W(0));
                        __stcs(reinterpret_cast<W *>(pv), live ? C::out(GATE == GATE_SIGMOID ? vmul(z, g) : g) : W(0));
                    }
                    pf -= pitch_f;
                    pv -= pitch_v;
                    flow = vmul(a, g);
                    if ((k.x >> r & 1u) && p.dh0) put_state_row<E>(p.dh0, info.start[warp * R + r] * p.D, d0, p.D, flow);
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&blk.empty[n % S]);
            return true;
        };
        // one copy of either body: with two, for registers that need not move, the warps
        // spent a fifth of their time waiting for instructions
        int done = 0;
#pragma unroll 1
        for (int n = 0;; ++n) {
            const bool more = fold(n, gate[0]);
            if (n > 0) {
                if (!replay(n - 1, gate[1])) break;
                done = n;
            }
            if (!more) break;
#pragma unroll
            for (int r = 0; r < R; ++r) gate[1][r] = gate[0][r];
        }
        if (lane == 0) blk.done[warp] = done;
    } else if (warp < kWarps + kCarryWarps) {
        carry_loop<E, S, kBwdTR, -1>(p, blk, warp - kWarps, lane);
    } else {
        feed<S, 3, kBwdTR, Shape::op_bytes, TC, TMA>(p, blk, smem_addr(smem), lane, true, &map_f, &map_v, &map_dh);
    }
    __syncthreads();
    if (blk.lost) give_up<IO, E, S, kBwdTR, -1>(p, blk, warp, lane);
    empty_sequences(p, p.dh0, p.dh_last, p.D);
}

}  // namespace gated
}  // namespace sgr
