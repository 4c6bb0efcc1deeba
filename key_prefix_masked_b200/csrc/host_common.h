// host_common.h -- host helpers shared by the library's translation units: tensor maps,
// strides, the device check, the process-wide test settings, and the device flags that
// attn_get_device_status collects from each of them.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <stdint.h>

#include <atomic>
#include <mutex>

#include "attn_prefix.h"

namespace attn {

constexpr unsigned STATUS_TIMEOUT = 1u;
constexpr unsigned STATUS_KVLEN = 2u;
constexpr unsigned STATUS_LAYOUT = 4u;   // dynamic shared memory not 1024-byte aligned
constexpr unsigned STATUS_CACHE = 8u;    // a page, slot or query range outside its bounds

// The sticky flags of paged.cu's kernels: read, and cleared; false on a CUDA error.
bool read_paged_flags(unsigned* flags);
bool clear_paged_flags();

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Test hooks (attn_set_wait_limit_ns, attn_set_debug_flags): process-wide settings read
// by every launch that starts after they are written, from any host thread.
inline std::atomic<unsigned long long> g_wait_ns{1000000000ull};
inline std::atomic<unsigned> g_debug{0u};

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Element strides of one [B, H, T, D] operand (d contiguous).
struct Strides {
    long long b, h, t;
};
inline Strides contiguous(int H, int T, int D) {
    return {static_cast<long long>(H) * T * D, static_cast<long long>(T) * D, static_cast<long long>(D)};
}
// Caller strides, or the contiguous [B,H,T,D] layout for NULL.  Every stride must be a
// non-negative multiple of 8 elements (16-byte rows for TMA and vector stores), and a
// row may not overlap the next one (t >= D).
inline bool resolve_strides(const attn_strides* in, int H, int T, int D, Strides* out) {
    if (in == nullptr) {
        *out = contiguous(H, T, D);
        return true;
    }
    if (in->b < 0 || in->h < 0 || in->t < D || (in->b & 7) || (in->h & 7) || (in->t & 7)) return false;
    *out = {static_cast<long long>(in->b), static_cast<long long>(in->h), static_cast<long long>(in->t)};
    return true;
}

// Device must be compute capability 10.0 (B200 / sm_100a).  Cached per device ordinal
// (0 = not looked up yet, 1 = supported, 2 = not supported); host threads may race on an
// entry, and every one of them writes the same value.
inline attn_status check_device() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    if (dev < 0 || dev >= 64) return ATTN_ERR_UNSUPPORTED;
    int c = cached[dev].load(std::memory_order_relaxed);
    if (c == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
            cudaGetLastError();
            return ATTN_ERR_CUDA;
        }
        c = (major == 10 && minor == 0) ? 1 : 2;
        cached[dev].store(c, std::memory_order_relaxed);
    }
    return c == 1 ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

// A tensor map of up to five dims, innermost first (strides in bytes, of dims 1 and up).
inline bool encode_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
    return enc(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A [B, H, T, D] bf16 tensor at element strides s (d contiguous) as a 4-D TMA map with
// dims (D, T, H, B); a box is box_rows rows x box_cols columns of box_outer b's of one h.
inline bool make_map(CUtensorMap* map, const void* base, int B, int H, int T, int D, const Strides& s, int box_cols,
                     int box_rows, CUtensorMapSwizzle swz, int box_outer = 1) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(H),
                                static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s.t) * 2ull, static_cast<cuuint64_t>(s.h) * 2ull,
                                   static_cast<cuuint64_t>(s.b) * 2ull};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u,
                               static_cast<cuuint32_t>(box_outer)};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, swz);
}

}  // namespace attn
