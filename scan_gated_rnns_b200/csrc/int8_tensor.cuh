// int8_tensor.cuh -- the 8-bit projection on the 5th-generation tensor cores
// (tcgen05.mma kind::i8, signed operands, int32 accumulators in tensor
// memory), for rows that start on 16-byte boundaries.
//
// The product is taken transposed: the MMA's M side is channels (rows of w),
// its N side tokens (rows of x), so that few tokens still fill the M side and
// a warp that reads the accumulator holds 32 consecutive channels of a token.
// Both operands are K-major, 128 bytes of K a stage with the 128-byte
// swizzle, staged by the tensor memory accelerator; bytes past K, M and N
// arrive as zeros and add nothing.  Waits are bounded: a tile whose wait ran
// out gets NaN outputs.
#pragma once

#include "int8_projection.cuh"

namespace sgr {
namespace i8 {

constexpr int kKB = 128;                       // K bytes per stage
// Bounded waits.  A poll of an mbarrier suspends a whole warp for 4 us, but
// returns after 75 ns where only some of its lanes poll, as they do here: a
// wait polls kPolls times and then goes on by the clock.
constexpr uint32_t kPolls = 1u << 10;
constexpr uint64_t kWaitNs = 500000000;
__device__ __forceinline__ uint64_t timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t phase, uint32_t polls = kPolls, uint64_t ns = kWaitNs) {
    if (mbar_wait(bar, phase, polls)) return true;
    const uint64_t t0 = timer_ns();
    for (uint32_t i = 0; i < 1u << 28 && timer_ns() - t0 < ns; ++i)
        if (mbar_try_wait(bar, phase)) return true;
    return false;
}
// the copies still in flight at the end: at once, if `ok`; else they were
// started a wait's length ago at least
__device__ __forceinline__ void wait_at_end(uint32_t bar, uint32_t phase, bool ok) {
    if (ok) wait_for(bar, phase);
    else mbar_wait(bar, phase, kPolls);
}

// kind::i8 instruction descriptor: s8 x s8 -> s32, both K-major
constexpr uint32_t idesc(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// K-major operand with the 128-byte swizzle: rows of 128 bytes, groups of 8
// rows 1024 bytes apart (shared-memory matrix descriptor, version 1)
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3FFF) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}

template <int CTAS>
__device__ __forceinline__ void mma_i8(uint32_t acc, uint64_t a, uint64_t b, uint32_t id, bool add) {
    if constexpr (CTAS == 1) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(acc), "l"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u));
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(acc), "l"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u));
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the same shared-memory address in block `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// 32 consecutive accumulator columns of this thread's lane (lane quarter of
// the warp); completes with tmem_wait
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// The kernel this one was launched behind as a dependent has ended and its
// writes are there; returns at once where there is none.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16 accumulator columns of this thread's lane; completes with tmem_wait
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Four channels of a token, together where they lie on a boundary of their
// size and inside the row.
template <typename OUT>
__device__ __forceinline__ void put4(const ProjectParams &p, int64_t m, int64_t n, int4 acc, float sx, const float (&sw)[4],
                                     const float (&b)[4]) {
    const float y[4] = {fmaf(float(acc.x) * sx, sw[0], b[0]), fmaf(float(acc.y) * sx, sw[1], b[1]),
                        fmaf(float(acc.z) * sx, sw[2], b[2]), fmaf(float(acc.w) * sx, sw[3], b[3])};
    using W = typename Raw<OUT, 1>::type;
    W *at = reinterpret_cast<W *>(p.y) + m * p.y_rs + n;
    if (n + 4 <= p.N && (reinterpret_cast<uintptr_t>(at) & (4 * sizeof(OUT) - 1)) == 0) {
        if constexpr (sizeof(OUT) == 4) {
            *reinterpret_cast<float4 *>(at) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
            *reinterpret_cast<uint2 *>(at) = make_uint2(Conv<OUT, 2>::out(make_float2(y[0], y[1])),
                                                        Conv<OUT, 2>::out(make_float2(y[2], y[3])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < p.N) at[i] = Conv<OUT, 1>::out(y[i]);
    }
}

// ------------------------------------------------- few tokens: split K
//
// One block per tile of 128 channels x NT tokens and per part of K; the C
// blocks that share a tile form a cluster, each multiplies its part of K, and
// then each sums one slice of the tile's tokens over the cluster's shared
// memories and writes it.  The sums are whole numbers, so their order does
// not matter.  With few tokens the weights' bytes are the work, and the split
// is what spreads them over all SMs.
//
// Behind int8_quantize in one call the kernel is launched as its dependent
// (programmatic launch): its blocks set up and start the copies of the weights
// while the tokens are still being quantised, and wait for that kernel's end
// before anything of x is touched.  Measured: 8 x 1024 x 2048 8 us, 120 x 4096
// x 8192 17 us (its 33.5 MB of weights take 5 us from memory), 1111 x 1000 x
// 1502 to fp32 13.8 us; bound by the start of a block, its few stages and the
// cluster's two barriers, one after the other.
template <int NT>
struct SplitShape {
    static constexpr uint32_t a_bytes = 128 * kKB, b_bytes = NT * kKB, stage_bytes = a_bytes + b_bytes;
    static constexpr int stages = NT >= 128 ? 3 : (NT >= 64 ? 4 : (NT >= 32 ? 5 : 6));   // two blocks per SM
    static constexpr uint32_t smem_bytes = 1024 + stages * stage_bytes + 128;
    static constexpr uint32_t columns = NT < 32 ? 32 : NT;
    static_assert(NT * 128 * 4 <= int(stages * stage_bytes), "a tile of sums fits the ring");
};

template <int NT, typename OUT>
__global__ void __launch_bounds__(128, 2) int8_project_split_kernel(const ProjectParams p, int n_channel_tiles, int C,
                                                                    const __grid_constant__ CUtensorMap map_w,
                                                                    const __grid_constant__ CUtensorMap map_x) {
    using S = SplitShape<NT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::stages * S::stage_bytes);   // full, empty, done
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + 2 * S::stages + 1);
    int *s_bad = reinterpret_cast<int *>(s_tmem + 1);
    const uint32_t ring = smem_addr(smem);
    auto full = [&](int s) { return smem_addr(&bars[s]); };
    auto empty = [&](int s) { return smem_addr(&bars[S::stages + s]); };
    const uint32_t done = smem_addr(&bars[2 * S::stages]);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / C, rank = blockIdx.x - tile * C;
    const int ct = tile % n_channel_tiles, tt = tile / n_channel_tiles;
    const int n_kb = int((p.K + kKB - 1) / kKB);
    const int kb0 = int(int64_t(rank) * n_kb / C), kb1 = int(int64_t(rank + 1) * n_kb / C);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * S::stages + 1; ++i) mbar_init(smem_addr(&bars[i]), 1);
        *s_bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(s_tmem)), "r"(S::columns));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tmem = *s_tmem;

    if (warp == 0 && lane == 0) {
        int g = 0;
        // the first stages' weights, before x may be there
        for (; g < S::stages && kb0 + g < kb1; ++g) {
            mbar_expect_tx(full(g), S::stage_bytes);
            tma_load_2d(ring + uint32_t(g) * S::stage_bytes, &map_w, (kb0 + g) * kKB, ct * 128, full(g));
        }
        grid_dependency_wait();
        bool ok = true;
        for (int i = 0; i < g; ++i)
            tma_load_2d(ring + uint32_t(i) * S::stage_bytes + S::a_bytes, &map_x, (kb0 + i) * kKB, tt * NT, full(i));
        for (int kb = kb0 + g; kb < kb1; ++kb, ++g) {
            const int s = g % S::stages;
            if (!wait_for(empty(s), uint32_t((g / S::stages - 1) & 1))) {
                *s_bad = 1;
                ok = false;
                break;
            }
            const uint32_t dst = ring + uint32_t(s) * S::stage_bytes;
            mbar_expect_tx(full(s), S::stage_bytes);
            tma_load_2d(dst, &map_w, kb * kKB, ct * 128, full(s));
            tma_load_2d(dst + S::a_bytes, &map_x, kb * kKB, tt * NT, full(s));
        }
        // never leave with copies in flight
        for (int k = g > S::stages ? g - S::stages : 0; k < g; ++k)
            wait_at_end(full(k % S::stages), uint32_t((k / S::stages) & 1), ok);
    } else if (warp == 1 && lane == 0) {
        int g = 0;
        grid_dependency_wait();                                    // no wait's time passes while tokens are quantised
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = g % S::stages;
            if (!wait_for(full(s), uint32_t((g / S::stages) & 1))) {
                *s_bad = 1;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;");
            const uint32_t a = ring + uint32_t(s) * S::stage_bytes;
            const uint64_t da = sw128_desc(a), db = sw128_desc(a + S::a_bytes);
#pragma unroll
            for (int k = 0; k < kKB / 32; ++k)
                mma_i8<1>(tmem, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc(128, NT), g > 0 || k > 0);
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                         ::"r"(empty(s)) : "memory");
        }
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(done) : "memory");
    }
    __syncwarp();
    grid_dependency_wait();                                        // the tokens and their scales
    if (!wait_for(done, 0)) *s_bad = 1;
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;");

    const int64_t n = int64_t(ct) * 128 + threadIdx.x;
    const bool nvalid = n < p.N;
    const float sw = nvalid ? p.w_scale[n] : 0.f;
    const float b = nvalid && p.bias ? p.bias[n] : 0.f;
    const uint32_t taddr = tmem + (uint32_t(warp * 32) << 16);
    const int64_t tok0 = int64_t(tt) * NT;
    if (C == 1) {
        const bool bad = *s_bad != 0;
#pragma unroll 1
        for (int t0 = 0; t0 < NT; t0 += 16) {
            if (tok0 + t0 >= p.M) break;
            uint32_t r[16];
            tmem_ld16(taddr + t0, r);
            tmem_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t m = tok0 + t0 + i;
                if (m < p.M && nvalid) {
                    const float sx = bad ? __int_as_float(0x7fffffff) : p.x_scale[m];
                    put<OUT>(p, m, n, int(r[i]), sx, sw, b);
                }
            }
        }
    } else {
        int *sum = reinterpret_cast<int *>(smem);                   // [NT][128], over the ring
#pragma unroll 1
        for (int t0 = 0; t0 < NT; t0 += 16) {
            if (tok0 + t0 >= p.M) break;
            uint32_t r[16];
            tmem_ld16(taddr + t0, r);
            tmem_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[(t0 + i) * 128 + threadIdx.x] = kb1 > kb0 ? int(r[i]) : 0;
        }
        cluster_sync();
        bool bad = false;
        for (int c = 0; c < C; ++c) {
            int x;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(map_rank(smem_addr(s_bad), c)));
            bad = bad || x != 0;
        }
        // this block's share of the tile's tokens, four channels a thread, four tokens in flight
        const int live = int(p.M - tok0 < NT ? p.M - tok0 : NT);
        const int lo = rank * live / C, hi = (rank + 1) * live / C;
        const int64_t n4 = int64_t(ct) * 128 + 4 * lane;
        float w4[4], b4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w4[i] = n4 + i < p.N ? p.w_scale[n4 + i] : 0.f;
            b4[i] = n4 + i < p.N && p.bias ? p.bias[n4 + i] : 0.f;
        }
        for (int t0 = lo + warp; t0 < hi; t0 += 16) {
            int4 acc[4];
            float sx[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                acc[u] = make_int4(0, 0, 0, 0);
                sx[u] = t0 + 4 * u < hi ? p.x_scale[tok0 + t0 + 4 * u] : 0.f;
                if (bad) sx[u] = __int_as_float(0x7fffffff);
            }
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (t0 + 4 * u < hi) {
                        int4 x;
                        asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                     : "r"(map_rank(smem_addr(sum + (t0 + 4 * u) * 128 + 4 * lane), c)));
                        acc[u].x += x.x;
                        acc[u].y += x.y;
                        acc[u].z += x.z;
                        acc[u].w += x.w;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (t0 + 4 * u < hi) put4<OUT>(p, tok0 + t0 + 4 * u, n4, acc[u], sx[u], w4, b4);
            }
        }
        cluster_sync();                                             // a peer may still be reading
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::columns));
    }
}

// ------------------------------------------ many tokens: pairs of SMs
//
// Persistent pairs of blocks (a cluster of two), each pair on tiles of 256
// channels x 256 tokens: block r stages channels [128 r, +128) and tokens
// [128 r, +128) of the tile, one MMA (cta_group::2, issued by block 0) reads
// both blocks' shared memory and leaves each block its 128 channels x 256
// tokens.  Against a tile of 128 x 256 per SM this needs two thirds of the
// bytes from L2 for the same product, which is what bounds an 8-bit product
// of this size first.  Two accumulators: the epilogue of a tile runs under
// the next one's product.  A warp of the epilogue whose wait runs out writes
// NaN from there on and hands no accumulator back, so that the products stop
// and the other warps' waits run out in turn.  Measured: 8192 x 4096 x 8192 to bf16 198 us, 2.8
// POP/s, 0.85 of twice the bf16 rate of a large library product; the tensor
// cores' rate under the power limit bounds it.
namespace pair {
constexpr int kStages = 6;
constexpr uint32_t kHalf = 128 * kKB;                      // one operand's share per block and stage
constexpr uint32_t kStageBytes = 2 * kHalf;
constexpr int kTok = 256, kCh = 256;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (4 + kEpiWarps) * 32;
constexpr uint32_t kScaleAt = kStages * kStageBytes + 256;
constexpr uint32_t kSmemBytes = 1024 + kScaleAt + kEpiWarps * 128 * 4;
static_assert(kSmemBytes <= 227 * 1024, "one block per SM");
}  // namespace pair

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"(uint16_t(3)) : "memory");
}

template <typename OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair::kThreads, 1)
int8_project_pair_kernel(const ProjectParams p, int n_channel_tiles, int n_tiles,
                         const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x) {
    using namespace pair;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    // full[S] and acc_empty[2] are used in block 0, empty[S] and acc_full[2] in both
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + 2 * kStages + 4);
    const uint32_t ring = smem_addr(smem);
    auto full = [&](int s) { return smem_addr(&bars[s]); };
    auto empty = [&](int s) { return smem_addr(&bars[kStages + s]); };
    auto acc_full = [&](int a) { return smem_addr(&bars[2 * kStages + a]); };
    auto acc_empty = [&](int a) { return smem_addr(&bars[2 * kStages + 2 + a]); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = int(gridDim.x) / 2, first = int(blockIdx.x) / 2;
    const int n_kb = int((p.K + kKB - 1) / kKB);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kStages + 2; ++i) mbar_init(smem_addr(&bars[i]), 1);
        for (int a = 0; a < 2; ++a) mbar_init(acc_empty(a), 2 * kEpiWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(s_tmem)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        if (lane == 0) {
            // both blocks: own share of each stage; the bytes of both count on block 0's barrier
            int64_t g = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += pairs) {
                const int ct = tile % n_channel_tiles, tt = tile / n_channel_tiles;
                const int wy = ct * kCh + int(rank) * 128, xy = tt * kTok + int(rank) * 128;
                for (int kb = 0; kb < n_kb; ++kb, ++g) {
                    const int s = int(g % kStages);
                    if (g >= kStages && !wait_for(empty(s), uint32_t((g / kStages - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = ring + uint32_t(s) * kStageBytes;
                    const uint32_t bar = map_rank(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), 2 * kStageBytes);
                    tma_load_2d_pair(dst, &map_w, kb * kKB, wy, bar);
                    tma_load_2d_pair(dst + kHalf, &map_x, kb * kKB, xy, bar);
                }
            }
            // never leave with copies in flight: the last stages have been read once they are empty again
            for (int64_t k = g > kStages ? g - kStages : 0; k < g; ++k)
                wait_at_end(empty(int(k % kStages)), uint32_t((k / kStages) & 1), ok);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            int64_t g = 0;
            int n = 0;
            bool ok = true;
            for (int tile = first; tile < n_tiles && ok; tile += pairs, ++n) {
                const int a = n & 1;
                if (n >= 2 && !wait_for(acc_empty(a), uint32_t((n / 2 - 1) & 1))) break;
                asm volatile("tcgen05.fence::after_thread_sync;");
                for (int kb = 0; kb < n_kb; ++kb, ++g) {
                    const int s = int(g % kStages);
                    if (!wait_for(full(s), uint32_t((g / kStages) & 1))) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;");
                    const uint32_t at = ring + uint32_t(s) * kStageBytes;
                    const uint64_t da = sw128_desc(at), db = sw128_desc(at + kHalf);
#pragma unroll
                    for (int k = 0; k < kKB / 32; ++k)
                        mma_i8<2>(tmem + uint32_t(a * kTok), da + uint64_t(2 * k), db + uint64_t(2 * k),
                                  idesc(kCh, kTok), kb > 0 || k > 0);
                    commit_pair(empty(s));
                }
                commit_pair(acc_full(a));
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // epilogue: lane quarter q, tokens 128 half .. 128 half + 127
        const int q = warp & 3, half = (warp - 4) >> 2;
        float *s_sx = reinterpret_cast<float *>(smem + kScaleAt) + (warp - 4) * 128;
        int it = 0;
        bool lost = false;
        for (int tile = first; tile < n_tiles; tile += pairs, ++it) {
            const int ct = tile % n_channel_tiles, tt = tile / n_channel_tiles, a = it & 1;
            const int64_t n = int64_t(ct) * kCh + int64_t(rank) * 128 + q * 32 + lane;
            const int64_t tok0 = int64_t(tt) * kTok + half * 128;
            const bool nvalid = n < p.N;
            const float sw = nvalid ? p.w_scale[n] : 0.f;
            const float b = nvalid && p.bias ? p.bias[n] : 0.f;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = tok0 + lane + 32 * i;
                s_sx[lane + 32 * i] = m < p.M ? p.x_scale[m] : 0.f;
            }
            if (!lost && !wait_for(acc_full(a), uint32_t((it / 2) & 1), p.epilogue_polls, p.epilogue_ns)) lost = true;
            lost = __any_sync(0xffffffffu, lost);
            asm volatile("tcgen05.fence::after_thread_sync;");
            const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + uint32_t(a * kTok + half * 128);
#pragma unroll 1
            for (int t0 = 0; t0 < 128; t0 += 32) {
                uint32_t r[32];
                tmem_ld32(taddr + t0, r);
                tmem_wait();
                // the accumulator has been read; a warp that gave up never says so, or its
                // arrivals would hand accumulators on that others still read
                if (t0 == 96 && !lost) {
                    asm volatile("tcgen05.fence::before_thread_sync;");
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                                     ::"r"(map_rank(acc_empty(a), 0)) : "memory");
                }
                const int live = int(p.M - (tok0 + t0) < 32 ? p.M - (tok0 + t0) : 32);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float sx = lost ? __int_as_float(0x7fffffff) : s_sx[t0 + i];
                    if (i < live && nvalid) put<OUT>(p, tok0 + t0 + i, n, int(r[i]), sx, sw, b);
                }
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    cluster_sync();                                                // both blocks are done with both memories
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

}  // namespace i8
}  // namespace sgr
