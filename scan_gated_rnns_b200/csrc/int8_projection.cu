// int8_projection.cu -- host side of int8_quantize and int8_projection
// (include/scan_gated_rnns.h): argument checks, the choice of kernel, the
// workspace and the launches.  No allocation, no synchronisation.
#include "host_checks.h"
#include "int8_projection.cuh"
#include "int8_tensor.cuh"

#include <algorithm>
#include <limits>

namespace {

using namespace sgr;
using namespace sgr::i8;
using sgr::host::Span;

constexpr int64_t kMaxK = (int64_t(1) << 17) - 1;      // 128 * 128 * K stays below 2^31
constexpr int64_t kMaxDim = std::numeric_limits<int>::max() - 4096;

inline int64_t pad16(int64_t n) { return (n + 15) / 16 * 16; }

// Workspace of a product whose x is not 8-bit: the quantised rows, then their scales.
size_t quant_bytes(int64_t M, int64_t K) { return size_t(M) * size_t(pad16(K)); }
size_t scale_at(int64_t M, int64_t K) { return (quant_bytes(M, K) + 255) / 256 * 256; }

template <typename IO, int TPR, int NV>
void launch_quantize(const QuantParams &p, cudaStream_t s) {
    const int64_t blocks = (p.rows + 256 / TPR - 1) / (256 / TPR);
    int8_quantize_kernel<IO, TPR, NV><<<unsigned(std::min<int64_t>(blocks, 148 * 32)), 256, 0, s>>>(p);
}
// Up to 4 vectors a thread: a warp a row (bf16: 1024 values), four warps
// (4096), a block (8192).  Fewer rows than SMs take a block each up to there,
// for the latency.
template <typename IO>
void quantize_rows(const QuantParams &p, cudaStream_t s) {
    constexpr int VEC = 16 / sizeof(IO);
    const bool vec = host::aligned(p.x, 16) && host::aligned(p.q, 16) &&
                     (p.rows <= 1 || (p.x_rs * int64_t(sizeof(IO)) % 16 == 0 && p.q_rs % 16 == 0));
    const int64_t n = (p.K + VEC - 1) / VEC;
    const bool few = p.rows <= 148;
    if (!vec || n > 4 * 256) launch_quantize<IO, 256, 0>(p, s);
    else if (n <= 32) launch_quantize<IO, 32, 1>(p, s);
    else if (n <= 128 && !few) launch_quantize<IO, 32, 4>(p, s);
    else if (n <= 256 && few) launch_quantize<IO, 256, 1>(p, s);
    else if (n <= 512 && few) launch_quantize<IO, 256, 2>(p, s);
    else if (n <= 512) launch_quantize<IO, 128, 4>(p, s);
    else launch_quantize<IO, 256, 4>(p, s);
}

sgr_status_t quantize(const QuantParams &p, sgr_dtype_t dtype, cudaStream_t s) {
    if (dtype == SGR_F32) quantize_rows<float>(p, s);
    else if (dtype == SGR_BF16) quantize_rows<__nv_bfloat16>(p, s);
    else quantize_rows<__half>(p, s);
    return cudaGetLastError() == cudaSuccess ? SGR_OK : SGR_ERR_CUDA;
}

// Tensor map of 8-bit rows for boxes of 128 bytes x `box` rows, 128-byte
// swizzle; bytes past the rows' ends read as zero.
bool row_map(CUtensorMap *map, const int8_t *base, int64_t rows, int64_t K, int64_t rs, int box) {
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    const cuuint32_t boxes[2] = {cuuint32_t(kKB), cuuint32_t(box)};
    return host::encode_rows(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, dims, cuuint64_t(rows > 1 ? rs : pad16(K)),
                             boxes, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows that a tensor map can describe.
bool mappable(const int8_t *base, int64_t rows, int64_t rs) {
    return host::aligned(base, 16) && (rows <= 1 || (rs % 16 == 0 && rs > 0 && rs < (int64_t(1) << 40)));
}

template <int NT, typename OUT>
cudaError_t launch_split(const ProjectParams &p, int sms, bool behind, cudaStream_t s) {
    using S = SplitShape<NT>;
    const int64_t ct = (p.N + 127) / 128, tt = (p.M + NT - 1) / NT, n_kb = (p.K + kKB - 1) / kKB;
    if (ct * tt > std::numeric_limits<int>::max() / 8) return cudaErrorInvalidConfiguration;
    // as many parts of K as two blocks per SM take at once
    int C = 1;
    while (C < 8 && 2 * C <= n_kb && ct * tt * 2 * C <= 2 * sms) C *= 2;
    CUtensorMap map_w, map_x;
    if (!row_map(&map_w, p.w, p.N, p.K, p.w_rs, 128) || !row_map(&map_x, p.x, p.M, p.K, p.x_rs, NT))
        return cudaErrorInvalidValue;
    auto kernel = int8_project_split_kernel<NT, OUT>;
    const cudaError_t e = host::allow_smem<int8_project_split_kernel<NT, OUT>>(int(S::smem_bytes));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ct * tt * C));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = S::smem_bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, int(ct), C, map_w, map_x);
}

template <typename OUT>
cudaError_t launch_pair(const ProjectParams &p, int sms, cudaStream_t s) {
    const int64_t ct = (p.N + pair::kCh - 1) / pair::kCh, tt = (p.M + pair::kTok - 1) / pair::kTok;
    if (ct * tt > std::numeric_limits<int>::max() / 2) return cudaErrorInvalidConfiguration;
    CUtensorMap map_w, map_x;
    if (!row_map(&map_w, p.w, p.N, p.K, p.w_rs, 128) || !row_map(&map_x, p.x, p.M, p.K, p.x_rs, 128))
        return cudaErrorInvalidValue;
    auto kernel = int8_project_pair_kernel<OUT>;
    const cudaError_t e = host::allow_smem<int8_project_pair_kernel<OUT>>(int(pair::kSmemBytes));
    if (e != cudaSuccess) return e;
    const unsigned grid = 2 * unsigned(std::min<int64_t>(ct * tt, sms / 2));
    kernel<<<grid, pair::kThreads, pair::kSmemBytes, s>>>(p, int(ct), int(ct * tt), map_w, map_x);
    return cudaGetLastError();
}

// `behind`: the quantising kernel of this call was the last launch on the stream.
template <typename OUT>
cudaError_t launch_tensor(const ProjectParams &p, int sms, bool behind, cudaStream_t s) {
    const int64_t pairs = ((p.N + 255) / 256) * ((p.M + 255) / 256);
    if (p.M > 128 && 2 * pairs >= sms / 2) return launch_pair<OUT>(p, sms, s);
    if (p.M <= 16) return launch_split<16, OUT>(p, sms, behind, s);
    if (p.M <= 32) return launch_split<32, OUT>(p, sms, behind, s);
    if (p.M <= 64) return launch_split<64, OUT>(p, sms, behind, s);
    return launch_split<128, OUT>(p, sms, behind, s);
}

sgr_status_t product(const ProjectParams &p, sgr_dtype_t out, bool behind, cudaStream_t s) {
    if (mappable(p.w, p.N, p.w_rs) && mappable(p.x, p.M, p.x_rs)) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SGR_ERR_CUDA;
        const int sms = host::sm_count(dev);
        if (sms <= 1) return SGR_ERR_CUDA;
        const cudaError_t e = out == SGR_F32    ? launch_tensor<float>(p, sms, behind, s)
                              : out == SGR_BF16 ? launch_tensor<__nv_bfloat16>(p, sms, behind, s)
                                                : launch_tensor<__half>(p, sms, behind, s);
        return e == cudaSuccess ? SGR_OK : SGR_ERR_CUDA;
    }
    const int64_t tiles = ((p.N + 63) / 64) * ((p.M + 63) / 64);
    if (tiles > std::numeric_limits<int>::max()) return SGR_ERR_UNSUPPORTED;
    const dim3 grid{unsigned(tiles)};
    if (out == SGR_F32) int8_project_any_kernel<float><<<grid, 256, 0, s>>>(p);
    else if (out == SGR_BF16) int8_project_any_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else int8_project_any_kernel<__half><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SGR_OK : SGR_ERR_CUDA;
}

}  // namespace

extern "C" {

sgr_status_t int8_quantize(const void *x, int64_t x_row_stride, int8_t *q, int64_t q_row_stride, float *scale,
                           int64_t rows, int64_t K, sgr_dtype_t dtype, cudaStream_t stream) {
    const int esz = host::float_size(dtype);
    if (esz == 0 || rows < 0 || K < 0 || x_row_stride < 0 || q_row_stride < 0) return SGR_ERR_INVALID_ARG;
    if (rows == 0) return SGR_OK;
    if (!scale || (K > 0 && (!x || !q))) return SGR_ERR_INVALID_ARG;
    if (rows > 1 && q_row_stride < K) return SGR_ERR_INVALID_ARG;
    int64_t b_x, b_q, b_s;
    if (!host::span_ok(rows, K, x_row_stride, esz, &b_x) || !host::span_ok(rows, K, q_row_stride, 1, &b_q) ||
        !host::mul_ok(rows, 4, &b_s))
        return SGR_ERR_UNSUPPORTED;
    const Span out[2] = {{q, b_q}, {scale, b_s}}, in[1] = {{x, b_x}};
    if (host::any_overlap(out, in)) return SGR_ERR_INVALID_ARG;
    return quantize({x, x_row_stride, q, q_row_stride, scale, rows, K}, dtype, stream);
}

size_t sgr_int8_workspace_size(int64_t rows, int64_t K, sgr_dtype_t x_dtype) {
    int64_t n = 0;
    if (rows <= 0 || K <= 0 || K > kMaxK || host::float_size(x_dtype) == 0 || !host::mul_ok(rows, pad16(K) + 4, &n))
        return 0;
    return scale_at(rows, K) + size_t(rows) * 4;
}

sgr_status_t int8_projection(const void *x, int64_t x_row_stride, sgr_dtype_t x_dtype, const float *x_scale,
                             const int8_t *w, int64_t w_row_stride, const float *w_scale, const float *bias, void *y,
                             int64_t y_row_stride, sgr_dtype_t y_dtype, int64_t rows, int64_t K, int64_t N,
                             void *workspace, size_t ws_bytes, cudaStream_t stream) {
    const int xsz = x_dtype == SGR_I8 ? 1 : host::float_size(x_dtype);
    const int ysz = host::float_size(y_dtype);
    if (xsz == 0 || ysz == 0 || rows < 0 || K < 0 || N < 0 || x_row_stride < 0 || w_row_stride < 0 || y_row_stride < 0)
        return SGR_ERR_INVALID_ARG;
    if (rows == 0 || N == 0) return SGR_OK;
    if (K == 0 || !x || !w || !w_scale || !y || (x_dtype == SGR_I8) != (x_scale != nullptr)) return SGR_ERR_INVALID_ARG;
    if (rows > 1 && y_row_stride < N) return SGR_ERR_INVALID_ARG;
    if (K > kMaxK || rows > kMaxDim || N > kMaxDim) return SGR_ERR_UNSUPPORTED;
    int64_t b_x, b_w, b_y, b_q;
    if (!host::span_ok(rows, K, x_row_stride, xsz, &b_x) || !host::span_ok(N, K, w_row_stride, 1, &b_w) ||
        !host::span_ok(rows, N, y_row_stride, ysz, &b_y) || !host::mul_ok(rows, pad16(K) + 4, &b_q))
        return SGR_ERR_UNSUPPORTED;
    const size_t need = sgr_int8_workspace_size(rows, K, x_dtype);
    const Span out[2] = {{y, b_y}, {need ? workspace : nullptr, int64_t(need)}};
    const Span in[5] = {{x, b_x}, {w, b_w}, {x_scale, rows * 4}, {w_scale, N * 4}, {bias, N * 4}};
    if (host::any_overlap(out, in)) return SGR_ERR_INVALID_ARG;
    if (need && (!workspace || ws_bytes < need || !host::aligned(workspace, 16))) return SGR_ERR_WORKSPACE;
    ProjectParams p;
    p.x = static_cast<const int8_t *>(x); p.x_rs = x_row_stride; p.x_scale = x_scale;
    p.w = w; p.w_rs = w_row_stride; p.w_scale = w_scale; p.bias = bias;
    p.y = y; p.y_rs = y_row_stride; p.M = rows; p.N = N; p.K = K;
    const uint32_t hook = host::block_wait_limit();
    p.epilogue_polls = hook ? hook : kPolls;
    p.epilogue_ns = hook ? 0 : kWaitNs;
    if (x_dtype != SGR_I8) {
        int8_t *q = static_cast<int8_t *>(workspace);
        float *scale = reinterpret_cast<float *>(static_cast<char *>(workspace) + scale_at(rows, K));
        const sgr_status_t st = quantize({x, x_row_stride, q, pad16(K), scale, rows, K}, x_dtype, stream);
        if (st != SGR_OK) return st;
        p.x = q; p.x_rs = pad16(K); p.x_scale = scale;
    }
    return product(p, y_dtype, x_dtype != SGR_I8, stream);
}

}  // extern "C"
