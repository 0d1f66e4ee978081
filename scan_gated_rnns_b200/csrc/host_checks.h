// host_checks.h -- argument checks shared by the host sides of the gated
// recurrence and the 8-bit projection.
#pragma once

#include "scan_gated_rnns.h"

#include <cuda.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

namespace sgr {
namespace host {

// a * b for sizes and strides, false if it passes int64
inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// bytes that `rows` rows of n elements, rs elements apart, span from the first
// to the last; false if they pass int64
inline bool span_ok(int64_t rows, int64_t n, int64_t rs, int64_t esz, int64_t *bytes) {
    int64_t x = 0;
    if (rows <= 0 || n <= 0) {
        *bytes = 0;
        return true;
    }
    return mul_ok(rows - 1, rs, &x) && !__builtin_add_overflow(x, n, &x) && mul_ok(x, esz, bytes);
}

inline bool overlaps(const void *a, int64_t na, const void *b, int64_t nb) {
    if (!a || !b || na <= 0 || nb <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + uintptr_t(nb) && y < x + uintptr_t(na);
}

// An array of rows as a call gives it, with the bytes it spans.
struct Span {
    const void *p;
    int64_t n;
};
template <int N, int M>
inline bool any_overlap(const Span (&outs)[N], const Span (&ins)[M]) {
    for (int i = 0; i < N; ++i) {
        for (int j = 0; j < M; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
        for (int j = i + 1; j < N; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
    }
    return false;
}

// SMs of a device; 0 if the runtime does not say
inline int sm_count(int dev) {
    static std::atomic<int> cache[64];
    if (dev < 0 || dev >= 64) return 0;
    int v = cache[dev].load();
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) v = 0;
        cache[dev].store(v);
    }
    return v;
}

// cuTensorMapEncodeTiled, through the runtime; null if the driver lacks it
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled() {
    static std::atomic<EncodeTiledFn> fn{nullptr};
    EncodeTiledFn f = fn.load();
    if (f == nullptr) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || ptr == nullptr)
            return nullptr;
        f = reinterpret_cast<EncodeTiledFn>(ptr);
        fn.store(f);
    }
    return f;
}

// A tensor map of (rows, elements of a row).  The driver's encoder wants the
// device's context current on the calling thread, and a thread that has made
// no launch yet (a backward pass on its own thread) may not have it so: then
// the device is set, as launches do by themselves, and the map encoded again.
inline bool encode_rows(CUtensorMap *map, CUtensorMapDataType type, const void *base, const cuuint64_t (&dims)[2],
                        cuuint64_t row_bytes, const cuuint32_t (&box)[2], CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t es[2] = {1u, 1u};
    const auto encode = [&] {
        return enc(map, type, 2, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    int dev = 0;
    return encode() || (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode());
}

// Dynamic shared memory of a kernel, set once per kernel and device.
template <auto KERNEL>
inline cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// The testing hooks of the chunk hand-off (sgr_set_wait_limit,
// sgr_set_block_wait_limit, sgr_set_drop_publish), as they are set now.
uint32_t wait_limit();
uint32_t block_wait_limit();
int64_t drop_tile();

inline int float_size(sgr_dtype_t t) { return t == SGR_F32 ? 4 : (t == SGR_BF16 || t == SGR_F16 ? 2 : 0); }

}  // namespace host
}  // namespace sgr
