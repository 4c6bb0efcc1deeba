// cache.cuh -- writing rows to the pages of a key/value cache and reading them back.
// Included by paged.cu inside namespace attn.
//
// Quantised rows: e4m3 codes with one power-of-two scale 2^e per row, e the least exponent
// with amax / 2^e <= 448.  x / 2^e only shifts the exponent, so the one rounding is that
// to e4m3, and every code * 2^e is a bf16 number (4 significant bits; e >= -117 keeps the
// smallest code, 2^-9, above bf16's smallest normal number; at e = 120 codes end at 240,
// since 256 * 2^120 would be infinite).  Whoever reads the row, in
// whatever order it scales, computes with the same values.  A free fp32 scale would use
// the top binade of e4m3 fully, but a floating-point code gains no precision from that, and
// each reader would round once more.
//
// Both kernels are copies: HBM bounds them.  A lane moves 8 elements (16 bytes of bf16, 8
// bytes of codes) and has several rows in flight.

constexpr int CACHE_THREADS = 256;
constexpr int CACHE_WRITE_U = 2;      // rows in flight per thread
constexpr int CACHE_READ_U = 4;       // (K and V each)
constexpr int SCALE_EXP_MIN = -117, SCALE_EXP_MAX = 120;
constexpr int SCALE_NAN = 255;

struct CacheView {
    uint8_t* data[2];             // k, v
    uint8_t* scale[2];
    long long sp[2], sh[2], st[2];   // strides in BYTES: page, head, slot
    int num_pages, page_size, Hkv, D;
    int e4m3;
};

// 2^(code - 127), NaN for code 255
__device__ __forceinline__ float scale_value(uint32_t code) {
    return code == SCALE_NAN ? __uint_as_float(0x7fc00000u) : __uint_as_float(code << 23);
}
// Scale code of a row whose largest magnitude has the bf16 pattern `amax` (sign clear).
// amax = (1 + M/128) 2^(E-127) and 448 = 1.75 * 2^8, so e = E - 127 - 8, plus 1 where
// M > 96 (1 + 96/128 = 1.75).  Patterns from 0x7f80 on are infinities and NaN.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
    if (amax >= 0x7f80u) return SCALE_NAN;
    if (amax == 0u) return 127u;
    const int e = static_cast<int>(amax >> 7) - 127 - 8 + ((amax & 0x7fu) > 96u ? 1 : 0);
    return static_cast<uint32_t>(min(max(e, SCALE_EXP_MIN), SCALE_EXP_MAX) + 127);
}
// Eight bf16 values (four words) to eight e4m3 codes of magnitude <= top; inv = 2^-e.
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv, float top) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = make_float2(fminf(fmaxf(__uint_as_float(w[i] << 16) * inv, -top), top),
                                     fminf(fmaxf(__uint_as_float(w[i] & 0xffff0000u) * inv, -top), top));
        h[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
// Eight e4m3 codes to eight bf16 values code * scale (exact for scales the writer makes).
__device__ __forceinline__ uint4 dequantise8(const uint2& c, float scale) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = ((i < 2 ? c.x : c.y) >> (16 * (i & 1))) & 0xffffu;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        o[i] = pack_bf16(f.x * scale, f.y * scale);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

struct CacheWriteParams {
    CacheView c;
    const __nv_bfloat16* src[2];
    long long st[2], sh[2];   // element strides of the new rows: token, head
    const int32_t* slots;
    long long rows;           // T * 2 * Hkv: (token, k or v, head), head fastest
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(CACHE_THREADS) cache_write_kernel(const CacheWriteParams p) {
    constexpr int LPR = D / 8;
    constexpr int RPI = CACHE_THREADS / LPR;
    const int lane = threadIdx.x % LPR;
    const long long r0 = static_cast<long long>(blockIdx.x) * (RPI * CACHE_WRITE_U) + threadIdx.x / LPR;
    const int per_token = 2 * p.c.Hkv;
    uint4 x[CACHE_WRITE_U];
    int slot[CACHE_WRITE_U], kv[CACHE_WRITE_U], head[CACHE_WRITE_U];
#pragma unroll
    for (int u = 0; u < CACHE_WRITE_U; ++u) {
        const long long r = r0 + u * RPI;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        slot[u] = -1;
        if (r < p.rows) {
            const long long t = r / per_token;
            const int rest = static_cast<int>(r - t * per_token);
            kv[u] = rest >= p.c.Hkv;
            head[u] = kv[u] ? rest - p.c.Hkv : rest;
            x[u] = __ldg(reinterpret_cast<const uint4*>(p.src[kv[u]] + t * p.st[kv[u]] + head[u] * p.sh[kv[u]]) + lane);
            slot[u] = __ldg(p.slots + t);
            if (slot[u] >= p.c.num_pages * p.c.page_size) {
                if (lane == 0) atomicOr(&g_paged_status, STATUS_CACHE);
                slot[u] = -1;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < CACHE_WRITE_U; ++u) {
        uint32_t code = 0u;
        if constexpr (E4M3) {
            // largest magnitude of the row, as bf16 patterns (ordered like the numbers, NaN on top)
            uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                                  __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
#pragma unroll
            for (int k = LPR / 2; k > 0; k >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, k));
            code = scale_code(max(m & 0xffffu, m >> 16));
        }
        if (slot[u] < 0) continue;
        const int page = slot[u] / p.c.page_size, row = slot[u] - page * p.c.page_size;
        uint8_t* dst = p.c.data[kv[u]] + page * p.c.sp[kv[u]] + head[u] * p.c.sh[kv[u]] + row * p.c.st[kv[u]];
        if constexpr (E4M3) {
            uint2 q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);   // NaN
            if (code != SCALE_NAN) q = quantise8(x[u], __uint_as_float((254u - code) << 23), code == SCALE_EXP_MAX + 127 ? 240.0f : 448.0f);
            reinterpret_cast<uint2*>(dst)[lane] = q;
            if (lane == 0)
                p.c.scale[kv[u]][(static_cast<long long>(page) * p.c.Hkv + head[u]) * p.c.page_size + row] =
                    static_cast<uint8_t>(code);
        } else {
            reinterpret_cast<uint4*>(dst)[lane] = x[u];
        }
    }
}

struct CacheReadParams {
    CacheView c;
    __nv_bfloat16* dst[2];
    long long sb[2], sh[2], st[2];   // element strides of the output
    const int32_t* table;
    long long table_stride;
    const int32_t* kv_len;
    int max_pages, Tk, n_rb;         // row blocks per (b, h)
};

// One block: rows [rb * RPI * U, ...) of element b, head h, K and V.
template <int D, bool E4M3>
__global__ void __launch_bounds__(CACHE_THREADS) cache_read_kernel(const CacheReadParams p) {
    constexpr int LPR = D / 8;
    constexpr int RPI = CACHE_THREADS / LPR;
    const int lane = threadIdx.x % LPR;
    const int rb = static_cast<int>(blockIdx.x % p.n_rb);
    const int bh = static_cast<int>(blockIdx.x / p.n_rb);
    const int b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
    const int kv = paged_kv_len(p.kv_len, b, static_cast<int>(min(static_cast<long long>(p.Tk),
                                static_cast<long long>(p.max_pages) * p.c.page_size)), rb == 0 && h == 0);
    const long long j0 = static_cast<long long>(rb) * (RPI * CACHE_READ_U) + threadIdx.x / LPR;
    using Raw = typename std::conditional<E4M3, uint2, uint4>::type;
    Raw x[CACHE_READ_U][2];
    float sc[CACHE_READ_U][2];
#pragma unroll
    for (int u = 0; u < CACHE_READ_U; ++u) {
        const long long j = j0 + u * RPI;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[u][w] = Raw{};
            sc[u][w] = 0.0f;
        }
        if (j >= kv) continue;
        const int pj = static_cast<int>(j) / p.c.page_size, row = static_cast<int>(j) - pj * p.c.page_size;
        const int page = __ldg(p.table + b * p.table_stride + pj);
        if (page < 0 || page >= p.c.num_pages) {
            if (lane == 0) atomicOr(&g_paged_status, STATUS_CACHE);
            continue;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[u][w] = __ldg(reinterpret_cast<const Raw*>(p.c.data[w] + page * p.c.sp[w] + h * p.c.sh[w] + row * p.c.st[w]) + lane);
            if constexpr (E4M3)
                sc[u][w] = scale_value(__ldg(p.c.scale[w] + (static_cast<long long>(page) * p.c.Hkv + h) * p.c.page_size + row));
        }
    }
#pragma unroll
    for (int u = 0; u < CACHE_READ_U; ++u) {
        const long long j = j0 + u * RPI;
        if (j >= kv) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 o;
            if constexpr (E4M3) o = dequantise8(x[u][w], sc[u][w]);
            else o = x[u][w];
            reinterpret_cast<uint4*>(p.dst[w] + b * p.sb[w] + h * p.sh[w] + j * p.st[w])[lane] = o;
        }
    }
}
