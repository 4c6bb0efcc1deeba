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
// Both kernels are copies: HBM bounds them.  A lane moves 8 elements (16 bytes of bf16; 16
// codes, 32 bytes of bf16, where codes are read) and has several rows in flight.  Measured: 131072
// tokens of 8 heads of 128 into random slots, bf16 172 us (6.2 TB/s), e4m3 182 us (4.4 TB/s: scattered
// lines of 128 bytes, and twice the instructions per byte, mostly the ALU's); 64 sequences of 4001
// such rows read back, bf16 320 us (6.6 TB/s), e4m3 283 us (5.6 TB/s).

constexpr int CACHE_THREADS = 128;     // (256: e4m3 1 to 3 % slower)
template <bool E4M3>
constexpr int CACHE_WRITE_U = E4M3 ? 2 : 4;   // rows in flight per thread (e4m3 at 4: up to 10 % slower, at 1: 11 %)
constexpr int CACHE_READ_U = 2;       // (K and V each)
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
// Eight bf16 values (four words) to eight e4m3 codes; inv = 2^-e.  `last`: e = 120, where codes
// end at 240 (below that exponent none exceeds 448), that is magnitudes at 240 * 2^120 (0x7f70).
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv, bool last) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (last) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (w[i] & 0x80008000u) | __vminu2(w[i] & 0x7fff7fffu, 0x7f707f70u);
    }
    uint32_t h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = mul2(make_float2(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i] & 0xffff0000u)), make_float2(inv, inv));
        const float2 b = mul2(make_float2(__uint_as_float(w[2 * i + 1] << 16), __uint_as_float(w[2 * i + 1] & 0xffff0000u)), make_float2(inv, inv));
        asm("{\n.reg .b16 lo, hi;\ncvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\nmov.b32 %0, {lo, hi};\n}\n"
            : "=r"(h[i])
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    }
    return make_uint2(h[0], h[1]);
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
    long long st[2], sh[2];     // strides of the new rows: token (elements), head (bytes)
    const int32_t* slots;
    int page_shift;             // log2(page_size), -1 if it is no power of two
    int parts, rows_per_part;   // warps per token, and of its 2 Hkv rows (k heads, v heads) each
    long long tasks;            // tokens * parts
};

// A warp takes a token's rows (or a part of them), so the slot is looked up and taken apart once.
template <int D, bool E4M3>
__global__ void __launch_bounds__(CACHE_THREADS) cache_write_kernel(const CacheWriteParams p) {
    constexpr int LPR = D / 8;
    constexpr int RPW = 32 / LPR;
    constexpr int U = CACHE_WRITE_U<E4M3>;
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const long long task = static_cast<long long>(blockIdx.x) * (CACHE_THREADS / 32) + (threadIdx.x >> 5);
    if (task >= p.tasks) return;
    const long long t = task / p.parts;
    const int begin = static_cast<int>(task - t * p.parts) * p.rows_per_part, end = min(2 * p.c.Hkv, begin + p.rows_per_part);
    const int slot = __ldg(p.slots + t);
    if (slot < 0) return;
    if (slot >= p.c.num_pages * p.c.page_size) {
        if (lane == 0) atomicOr(&g_paged_status, STATUS_CACHE);
        return;
    }
    const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.c.page_size, row = slot - page * p.c.page_size;
    // the token's first row at its source and in the pages, for k and v; a head further costs one multiply
    const uint8_t* src[2];
    uint8_t* dst[2];
    uint8_t* scale[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        src[w] = reinterpret_cast<const uint8_t*>(p.src[w] + t * p.st[w]) + 16 * l;
        dst[w] = p.c.data[w] + page * p.c.sp[w] + row * p.c.st[w] + (E4M3 ? 8 : 16) * l;
        if (E4M3) scale[w] = p.c.scale[w] + static_cast<long long>(page) * p.c.Hkv * p.c.page_size + row;
    }
#pragma unroll 1
    for (int r0 = begin + lane / LPR; r0 - lane / LPR < end; r0 += U * RPW) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RPW;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < end) {
                const bool w = r >= p.c.Hkv;
                x[u] = __ldg(reinterpret_cast<const uint4*>((w ? src[1] : src[0]) + (w ? r - p.c.Hkv : r) * (w ? p.sh[1] : p.sh[0])));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RPW;
            uint32_t code = 0u;
            if constexpr (E4M3) {
                // largest magnitude of the row, as bf16 patterns (ordered like the numbers, NaN on top)
                uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                                      __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
#pragma unroll
                for (int k = LPR / 2; k > 0; k >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, k));
                code = scale_code(max(m & 0xffffu, m >> 16));
            }
            if (r >= end) continue;
            const bool w = r >= p.c.Hkv;
            const int head = w ? r - p.c.Hkv : r;
            uint8_t* to = (w ? dst[1] : dst[0]) + head * (w ? p.c.sh[1] : p.c.sh[0]);
            if constexpr (E4M3) {
                uint2 q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);   // NaN
                if (code != SCALE_NAN) q = quantise8(x[u], __uint_as_float((254u - code) << 23), code == SCALE_EXP_MAX + 127);
                *reinterpret_cast<uint2*>(to) = q;
                if (l == 0) (w ? scale[1] : scale[0])[static_cast<long long>(head) * p.c.page_size] = static_cast<uint8_t>(code);
            } else {
                *reinterpret_cast<uint4*>(to) = x[u];
            }
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
    int page_shift;                  // log2(page_size), -1 if it is no power of two
};

// One block: rows [rb * RPI * U, ...) of element b, head h, K and V.
template <int D, bool E4M3>
__global__ void __launch_bounds__(CACHE_THREADS) cache_read_kernel(const CacheReadParams p) {
    constexpr int PER = E4M3 ? 16 : 8;        // elements per lane: 16 bytes loaded
    constexpr int LPR = D / PER;
    constexpr int RPI = CACHE_THREADS / LPR;
    const int lane = threadIdx.x % LPR;
    const int rb = static_cast<int>(blockIdx.x % p.n_rb);
    const int bh = static_cast<int>(blockIdx.x / p.n_rb);
    const int b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
    const int kv = paged_kv_len(p.kv_len, b, static_cast<int>(min(static_cast<long long>(p.Tk),
                                static_cast<long long>(p.max_pages) * p.c.page_size)), rb == 0 && h == 0);
    const long long j0 = static_cast<long long>(rb) * (RPI * CACHE_READ_U) + threadIdx.x / LPR;
    uint4 x[CACHE_READ_U][2];
    uint32_t sc[CACHE_READ_U][2];
#pragma unroll
    for (int u = 0; u < CACHE_READ_U; ++u) {
        const long long j = j0 + u * RPI;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[u][w] = make_uint4(0u, 0u, 0u, 0u);
            sc[u][w] = 0u;
        }
        if (j >= kv) continue;
        const int pj = p.page_shift >= 0 ? static_cast<int>(j) >> p.page_shift : static_cast<int>(j) / p.c.page_size;
        const int row = static_cast<int>(j) - pj * p.c.page_size;
        const int page = __ldg(p.table + b * p.table_stride + pj);
        if (page < 0 || page >= p.c.num_pages) {
            if (lane == 0) atomicOr(&g_paged_status, STATUS_CACHE);
            continue;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            x[u][w] = __ldg(reinterpret_cast<const uint4*>(p.c.data[w] + page * p.c.sp[w] + h * p.c.sh[w] + row * p.c.st[w]) + lane);
            if constexpr (E4M3) sc[u][w] = __ldg(p.c.scale[w] + (static_cast<long long>(page) * p.c.Hkv + h) * p.c.page_size + row);
        }
    }
#pragma unroll
    for (int u = 0; u < CACHE_READ_U; ++u) {
        const long long j = j0 + u * RPI;
        if (j >= kv) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4* dst = reinterpret_cast<uint4*>(p.dst[w] + b * p.sb[w] + h * p.sh[w] + j * p.st[w]);
            if constexpr (E4M3) {
                const float f = scale_value(sc[u][w]);
                dst[2 * lane] = dequantise8(make_uint2(x[u][w].x, x[u][w].y), f);
                dst[2 * lane + 1] = dequantise8(make_uint2(x[u][w].z, x[u][w].w), f);
            } else {
                dst[lane] = x[u][w];
            }
        }
    }
}
