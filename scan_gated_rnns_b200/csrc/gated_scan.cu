// gated_scan.cu -- host side of gated_scan, gated_scan_backward and
// gated_step (include/scan_gated_rnns.h): argument checks, the choice of
// kernel, the workspace and the launches.  No allocation, no synchronisation.
#include "gated_scan.cuh"
#include "gated_step.cuh"
#include "host_checks.h"

#include <algorithm>
#include <cstring>
#include <limits>

namespace {

using namespace sgr;
using namespace sgr::gated;
using sgr::host::Span;

constexpr size_t kHeader = 256;             // status word at 0, ticket at 64 (its own sector)
constexpr size_t kTicketAt = 64;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1 - kTR;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Workspace: header, then the words through which tiles hand their maps and
// final states on.  All of it is set to ~0, the status word to 0, on the
// stream before the launch.
// The rows fall into segments, each of whole chunks, so up to segs - 1 chunks
// come on top of the rows' own.
struct Layout {
    int64_t n_strips, n_chunks, n_tiles;
    size_t total;
};
Layout layout(int64_t rows, int64_t D, int tc, int tr, int segs) {
    Layout l;
    l.n_strips = (D + tc - 1) / tc;
    l.n_chunks = rows <= tr ? 1 : (rows + tr - 1) / tr + segs - 1;
    l.n_tiles = l.n_strips * l.n_chunks;
    l.total = kHeader + size_t(l.n_tiles) * tc * 8;
    return l;
}

// Segments to work on side by side: enough that a tile's predecessor is two
// rounds of blocks older, and none shorter than eight tiles (each ends in a
// partial one).  A function of the sizes alone: both directions share it, and
// with it the places of the kept states.
int segments(int64_t rows, int64_t D, int64_t n_seqs, int esz) {
    constexpr int64_t kBlocks = 148;
    const int64_t strips = (D * esz + 127) / 128;
    return int(std::max<int64_t>(1, std::min<int64_t>({int64_t(kSegs), (2 * kBlocks + strips - 1) / strips,
                                                       rows / (8 * kTR), n_seqs})));
}

bool sizes_ok(int64_t rows, int64_t D) {
    int64_t n = 0;
    // 16 bytes an element covers the workspace and every dense array
    return rows <= kMaxRows && D <= (int64_t(1) << 31) - 64 && host::mul_ok(rows, D, &n) && host::mul_ok(n, 16, &n) &&
           ((rows + kBwdTR - 1) / kBwdTR + kSegs) * ((D + 31) / 32) <= std::numeric_limits<int>::max() / 2;
}

// Tensor map of (rows, D) for boxes of 128 bytes x tr rows; what lies past
// the edges reads as zero.
bool tile_map(CUtensorMap *map, const void *base, int64_t rows, int64_t D, int64_t rs, int esz, int tr) {
    const cuuint64_t dims[2] = {cuuint64_t(D), cuuint64_t(rows)};
    const cuuint64_t row_bytes = rows > 1 ? cuuint64_t(rs) * esz : align_up(size_t(D) * esz, 16);
    const cuuint32_t box[2] = {cuuint32_t(128 / esz), cuuint32_t(tr)};
    return host::encode_rows(map, esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, base,
                             dims, row_bytes, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}
bool mappable(const void *base, int64_t rows, int64_t D, int64_t rs, int esz) {
    return host::aligned(base, 16) && (rows <= 1 || (rs * esz % 16 == 0 && rs >= D && rs * esz < (int64_t(1) << 40)));
}

// `behind`: as the dependent of the launch before, which cleared the workspace.
template <class Kernel, class... Args>
cudaError_t launch_behind(Kernel kernel, unsigned grid, size_t bytes, bool behind, cudaStream_t s, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename IO, int E, int GATE, bool TMA>
cudaError_t launch(GatedParams p, bool backward, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = host::sm_count(dev);
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int tr = backward ? kBwdTR : kTR;
    const int64_t chunks = (p.rows + tr - 1) / tr;
    const int64_t tiles = p.n_strips * (chunks + p.n_segs - 1);
    const unsigned grid = unsigned(std::max<int64_t>(1, p.ticket ? std::min<int64_t>(tiles, sms) : tiles));
    const int64_t held = int64_t(grid) * (backward ? kBwdSlots : kSlots);
    p.window = int(std::min<int64_t>(kNear + 32, held / (p.n_strips * p.n_segs) + 2));
    CUtensorMap m[3];
    std::memset(m, 0, sizeof(m));
    if (TMA) {
        const int esz = sizeof(IO);
        if (!tile_map(&m[0], p.f, p.rows, p.D, p.f_rs, esz, tr) || !tile_map(&m[1], p.v, p.rows, p.D, p.v_rs, esz, tr) ||
            (backward && !tile_map(&m[2], p.dh, p.rows, p.D, p.dh_rs, esz, tr)))
            return cudaErrorInvalidValue;
    }
    if (backward) {
        constexpr uint32_t bytes = BackwardShape<IO, E, TMA>::smem_bytes;
        auto kernel = gated_scan_backward_kernel<IO, E, GATE, TMA>;
        static_assert(bytes <= 227 * 1024, "one block per SM");
        if ((e = host::allow_smem<gated_scan_backward_kernel<IO, E, GATE, TMA>>(int(bytes))) != cudaSuccess) return e;
        e = launch_behind(kernel, grid, bytes, p.ticket != nullptr, s, p, m[0], m[1], m[2]);
    } else {
        constexpr uint32_t bytes = ForwardShape<IO, E, TMA>::smem_bytes;
        auto kernel = gated_scan_kernel<IO, E, GATE, TMA>;
        static_assert(bytes <= 227 * 1024, "one block per SM");
        if ((e = host::allow_smem<gated_scan_kernel<IO, E, GATE, TMA>>(int(bytes))) != cudaSuccess) return e;
        e = launch_behind(kernel, grid, bytes, p.ticket != nullptr, s, p, m[0], m[1]);
    }
    return e;
}

template <typename IO, int E, bool TMA>
cudaError_t launch_gate(const GatedParams &p, int gate, bool backward, cudaStream_t s) {
    return gate == GATE_SIGMOID ? launch<IO, E, GATE_SIGMOID, TMA>(p, backward, s)
                                : launch<IO, E, GATE_LOG, TMA>(p, backward, s);
}
template <typename IO, int E>
cudaError_t launch_e(const GatedParams &p, int gate, bool backward, bool tma, cudaStream_t s) {
    return tma ? launch_gate<IO, E, true>(p, gate, backward, s) : launch_gate<IO, E, false>(p, gate, backward, s);
}

cudaError_t launch_any(const GatedParams &p, sgr_dtype_t dtype, int gate, int E, bool backward, cudaStream_t s) {
    const int esz = host::float_size(dtype);
    const bool tma = p.rows > 0 && mappable(p.f, p.rows, p.D, p.f_rs, esz) && mappable(p.v, p.rows, p.D, p.v_rs, esz) &&
                     (!backward || mappable(p.dh, p.rows, p.D, p.dh_rs, esz)) && (esz == 4 || E == 2);
    if (dtype == SGR_F32) return launch_e<float, 1>(p, gate, backward, tma, s);
    if (dtype == SGR_BF16)
        return E == 2 ? launch_e<__nv_bfloat16, 2>(p, gate, backward, tma, s)
                      : launch_gate<__nv_bfloat16, 1, false>(p, gate, backward, s);
    return E == 2 ? launch_e<__half, 2>(p, gate, backward, tma, s) : launch_gate<__half, 1, false>(p, gate, backward, s);
}

sgr_status_t run(GatedParams &p, sgr_dtype_t dtype, sgr_gate_t gate, bool backward, void *ws, size_t ws_bytes,
                 cudaStream_t stream) {
    const int esz = host::float_size(dtype);
    if (esz == 0 || (gate != SGR_GATE_SIGMOID && gate != SGR_GATE_LOG)) return SGR_ERR_INVALID_ARG;
    if (p.rows < 0 || p.D < 0 || p.n_seqs < 0 || p.h0_ss < 0) return SGR_ERR_INVALID_ARG;
    if (p.cu ? (p.cu_bytes != 4 && p.cu_bytes != 8) : (p.rows > 0 && (p.n_seqs == 0 || p.rows % p.n_seqs != 0)))
        return SGR_ERR_INVALID_ARG;
    if (p.D == 0 || (p.rows == 0 && p.n_seqs == 0)) return SGR_OK;
    if (p.f_rs < 0 || p.v_rs < 0 || p.h_rs < 0 || p.dh_rs < 0 || p.df_rs < 0 || p.dv_rs < 0) return SGR_ERR_INVALID_ARG;
    // the search for bounds adds up to 32 to their number, in 32 bits
    if (!sizes_ok(p.rows, p.D) || p.n_seqs > std::numeric_limits<int>::max() - 63) return SGR_ERR_UNSUPPORTED;
    const int tr = backward ? kBwdTR : kTR;
    const int64_t n_chunks = (p.rows + tr - 1) / tr, n_states = sgr_gated_chunks(p.rows);
    if (p.rows > 0) {
        if (!p.f || !p.v) return SGR_ERR_INVALID_ARG;
        if (backward ? (!p.dh || !p.df || !p.dv || (n_chunks > 1 && !p.states)) : !p.h) return SGR_ERR_INVALID_ARG;
        // written rows may not share elements with one another
        if (p.rows > 1 && (backward ? (p.df_rs < p.D || p.dv_rs < p.D) : p.h_rs < p.D)) return SGR_ERR_INVALID_ARG;
    }
    int64_t b_f, b_v, b_dh, b_h, b_df, b_dv, b_h0, b_seq, b_cu, b_st;
    if (!host::span_ok(p.rows, p.D, p.f_rs, esz, &b_f) || !host::span_ok(p.rows, p.D, p.v_rs, esz, &b_v) ||
        !host::span_ok(p.rows, p.D, p.dh_rs, esz, &b_dh) || !host::span_ok(p.rows, p.D, p.h_rs, esz, &b_h) ||
        !host::span_ok(p.rows, p.D, p.df_rs, esz, &b_df) || !host::span_ok(p.rows, p.D, p.dv_rs, esz, &b_dv) ||
        !host::span_ok(p.n_seqs, p.D, p.h0_ss, 4, &b_h0) || !host::span_ok(p.n_seqs, p.D, p.D, 4, &b_seq) ||
        !host::mul_ok(p.n_seqs + 1, p.cu_bytes, &b_cu) || !host::span_ok(n_states, p.D, p.D, 4, &b_st))
        return SGR_ERR_UNSUPPORTED;
    // Two channels a thread where every row starts on a 4-byte boundary.
    int E = 1;
    if (esz == 2) {
        const int64_t odd = p.D | (p.rows > 1 ? (p.f_rs | p.v_rs | p.dh_rs | p.h_rs | p.df_rs | p.dv_rs) : 0);
        bool four = true;
        for (const void *q : {p.f, p.v, p.dh, static_cast<const void *>(p.h), static_cast<const void *>(p.df),
                              static_cast<const void *>(p.dv)})
            four = four && host::aligned(q, 4);
        E = (odd & 1) == 0 && four ? 2 : 1;
    }
    p.n_segs = segments(p.rows, p.D, p.n_seqs, esz);
    const Layout l = layout(p.rows, p.D, 32 * E, tr, p.n_segs);
    p.n_strips = l.n_strips;
    p.seq_rows = p.cu ? 1u : uint32_t(p.rows / std::max<int64_t>(1, p.n_seqs));
    p.spin_limit = host::wait_limit();
    p.drop_tile = host::drop_tile();
    p.tile_wait = host::block_wait_limit() ? host::block_wait_limit() : 2 * std::min(p.spin_limit, uint32_t(1) << 30);
    Span out[4], in[8];
    if (backward) {
        out[0] = {p.df, b_df};
        out[1] = {p.dv, b_dv};
        out[2] = {p.dh0, b_seq};
        out[3] = {ws, n_chunks > 1 ? int64_t(l.total) : 0};
    } else {
        out[0] = {p.h, b_h};
        out[1] = {p.h_last, b_seq};
        out[2] = {p.states, b_st};
        out[3] = {ws, n_chunks > 1 ? int64_t(l.total) : 0};
    }
    const Span ins[8] = {{p.f, b_f}, {p.v, b_v}, {p.dh, b_dh}, {p.h0, b_h0}, {p.dh_last, b_seq}, {p.cu, b_cu},
                         {backward ? p.states : nullptr, b_st}, {nullptr, 0}};
    std::copy(ins, ins + 8, in);
    if (host::any_overlap(out, in)) return SGR_ERR_INVALID_ARG;
    if (n_chunks > 1) {
        if (!ws || ws_bytes < l.total || !host::aligned(ws, 16)) return SGR_ERR_WORKSPACE;
        char *w = static_cast<char *>(ws);
        p.status = reinterpret_cast<uint32_t *>(w);
        p.ticket = reinterpret_cast<uint32_t *>(w + kTicketAt);
        p.words = reinterpret_cast<uint64_t *>(w + kHeader);
        // nothing of an earlier call is read
        const int64_t n = int64_t(l.total / 16);
        gated_clear_kernel<<<unsigned(std::min<int64_t>((n + 255) / 256, 148 * 4)), 256, 0, stream>>>(
            reinterpret_cast<uint4 *>(w), n);
        if (cudaGetLastError() != cudaSuccess) return SGR_ERR_CUDA;
    }
    return launch_any(p, dtype, gate == SGR_GATE_LOG ? GATE_LOG : GATE_SIGMOID, E, backward, stream) == cudaSuccess
               ? SGR_OK
               : SGR_ERR_CUDA;
}

template <typename IO, int V, int U>
void launch_step(const StepParams &p, int gate, unsigned grid, cudaStream_t s) {
    if (gate == SGR_GATE_SIGMOID) gated_step_kernel<IO, GATE_SIGMOID, V, U><<<grid, 256, 0, s>>>(p);
    else gated_step_kernel<IO, GATE_LOG, V, U><<<grid, 256, 0, s>>>(p);
}
template <typename IO>
void launch_step_any(const StepParams &p, int gate, int V, int U, unsigned grid, cudaStream_t s) {
    if (V == 1) launch_step<IO, 1, 1>(p, gate, grid, s);
    else if (U == 1) launch_step<IO, 4, 1>(p, gate, grid, s);
    else launch_step<IO, 4, 4>(p, gate, grid, s);
}

}  // namespace

extern "C" {

int64_t sgr_gated_chunks(int64_t rows) { return rows <= 0 ? 0 : rows <= kBwdTR ? 1 : (rows + kBwdTR - 1) / kBwdTR + kSegs - 1; }

size_t sgr_gated_workspace_size(int64_t rows, int64_t D) {
    if (rows <= kBwdTR || D <= 0 || !sizes_ok(rows, D)) return 0;
    return std::max(layout(rows, D, 32, kBwdTR, kSegs).total, layout(rows, D, 64, kBwdTR, kSegs).total);
}

sgr_status_t gated_scan(const void *f, int64_t f_row_stride, const void *v, int64_t v_row_stride, const float *h0,
                        int64_t h0_seq_stride, const void *cu_seqlens, int cu_bytes, int64_t n_seqs, void *h,
                        int64_t h_row_stride, float *h_last, float *states, int64_t rows, int64_t D, sgr_gate_t gate,
                        sgr_dtype_t dtype, int zero_padding, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    GatedParams p;
    std::memset(&p, 0, sizeof(p));
    p.f = f; p.f_rs = f_row_stride; p.v = v; p.v_rs = v_row_stride;
    p.h0 = h0; p.h0_ss = h0 ? h0_seq_stride : 0;
    p.cu = cu_seqlens; p.cu_bytes = cu_seqlens ? cu_bytes : 0; p.n_seqs = n_seqs;
    p.h = h; p.h_rs = h_row_stride; p.h_last = h_last; p.states = states;
    p.rows = rows; p.D = D; p.zero_padding = zero_padding;
    return run(p, dtype, gate, false, workspace, ws_bytes, stream);
}

sgr_status_t gated_scan_backward(const void *f, int64_t f_row_stride, const void *v, int64_t v_row_stride,
                                 const float *h0, int64_t h0_seq_stride, const void *cu_seqlens, int cu_bytes,
                                 int64_t n_seqs, const float *states, const void *dh, int64_t dh_row_stride,
                                 const float *dh_last, void *df, int64_t df_row_stride, void *dv,
                                 int64_t dv_row_stride, float *dh0, int64_t rows, int64_t D, sgr_gate_t gate,
                                 sgr_dtype_t dtype, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    GatedParams p;
    std::memset(&p, 0, sizeof(p));
    p.f = f; p.f_rs = f_row_stride; p.v = v; p.v_rs = v_row_stride;
    p.h0 = h0; p.h0_ss = h0 ? h0_seq_stride : 0;
    p.cu = cu_seqlens; p.cu_bytes = cu_seqlens ? cu_bytes : 0; p.n_seqs = n_seqs;
    p.states = const_cast<float *>(states);
    p.dh = dh; p.dh_rs = dh_row_stride; p.dh_last = dh_last;
    p.df = df; p.df_rs = df_row_stride; p.dv = dv; p.dv_rs = dv_row_stride; p.dh0 = dh0;
    p.rows = rows; p.D = D; p.zero_padding = 1;
    return run(p, dtype, gate, true, workspace, ws_bytes, stream);
}

sgr_status_t gated_step(const void *f, int64_t f_row_stride, const void *v, int64_t v_row_stride, float *state,
                        int64_t state_row_stride, int64_t n_slots, const void *slots, int slot_bytes, void *h,
                        int64_t h_row_stride, int64_t rows, int64_t D, sgr_gate_t gate, sgr_dtype_t dtype,
                        int zero_padding, cudaStream_t stream) {
    const int esz = host::float_size(dtype);
    if (esz == 0 || (gate != SGR_GATE_SIGMOID && gate != SGR_GATE_LOG)) return SGR_ERR_INVALID_ARG;
    if (rows < 0 || D < 0 || n_slots < 0 || f_row_stride < 0 || v_row_stride < 0 || h_row_stride < 0 ||
        state_row_stride < 0)
        return SGR_ERR_INVALID_ARG;
    if (rows == 0 || D == 0) return SGR_OK;
    if (!f || !v || !h || (n_slots > 0 && !state)) return SGR_ERR_INVALID_ARG;
    if (slots ? (slot_bytes != 4 && slot_bytes != 8) : n_slots < rows) return SGR_ERR_INVALID_ARG;
    if ((rows > 1 && h_row_stride < D) || (n_slots > 1 && state_row_stride < D)) return SGR_ERR_INVALID_ARG;
    int64_t b_f, b_v, b_h, b_s, b_slots;
    if (!host::span_ok(rows, D, f_row_stride, esz, &b_f) || !host::span_ok(rows, D, v_row_stride, esz, &b_v) ||
        !host::span_ok(rows, D, h_row_stride, esz, &b_h) || !host::span_ok(n_slots, D, state_row_stride, 4, &b_s) ||
        !host::mul_ok(rows, slots ? slot_bytes : 0, &b_slots))
        return SGR_ERR_UNSUPPORTED;
    const Span out[2] = {{h, b_h}, {state, b_s}}, in[3] = {{f, b_f}, {v, b_v}, {slots, b_slots}};
    if (host::any_overlap(out, in)) return SGR_ERR_INVALID_ARG;
    StepParams p;
    p.f = f; p.f_rs = f_row_stride; p.v = v; p.v_rs = v_row_stride; p.h = h; p.h_rs = h_row_stride;
    p.state = state; p.state_rs = state_row_stride; p.n_slots = n_slots; p.slots = slots; p.slot_bytes = slot_bytes;
    p.rows = rows; p.D = D; p.zero_padding = zero_padding;
    // four channels a thread where every row allows 16-byte states and 4-element operands
    const int64_t strides = D | f_row_stride | v_row_stride | h_row_stride | state_row_stride;
    const bool four = strides % 4 == 0 && host::aligned(f, 4 * esz) && host::aligned(v, 4 * esz) &&
                      host::aligned(h, 4 * esz) && host::aligned(state, 16);
    const int V = four ? 4 : 1;
    // four vectors a thread once one each would give every SM more than two blocks
    const int64_t one = (D + 256 * V - 1) / (256 * V);
    const int U = four && one >= 4 && rows * one > 2 * 148 ? 4 : 1;
    p.d_blocks = (one + U - 1) / U;
    int64_t grid = 0;
    if (!host::mul_ok(rows, p.d_blocks, &grid) || grid > std::numeric_limits<int>::max()) return SGR_ERR_UNSUPPORTED;
    if (dtype == SGR_F32) launch_step_any<float>(p, gate, V, U, unsigned(grid), stream);
    else if (dtype == SGR_BF16) launch_step_any<__nv_bfloat16>(p, gate, V, U, unsigned(grid), stream);
    else launch_step_any<__half>(p, gate, V, U, unsigned(grid), stream);
    return cudaGetLastError() == cudaSuccess ? SGR_OK : SGR_ERR_CUDA;
}

}  // extern "C"
