// paged_rows.cuh -- attention over pages for few query rows per key head (at most 16):
// single tokens of grouped heads, and short chunks.  Included by paged.cu inside namespace attn.
//
// What bounds it: every key and value row is read once, with at most 16 query rows to use it,
// so HBM does.  The kernel is built around keeping loads in flight:
//
// - The keys of all (sequence, key head) pairs are cut into tiles of 64 to 256, laid end to end,
//   and dealt to the CTAs in equal contiguous runs, so a batch of ragged lengths keeps every
//   SM busy to the end (each CTA finds its run with a scan over kv_len).  A pair whose tiles
//   fall to several CTAs is put together by paged_rows_combine_kernel, by log-sum-exp weights.
// - Each of a CTA's four warps takes a quarter of a tile's keys through a ring of shared memory of
//   its own, so no warp waits for another inside a run.  bf16 rows come by 16-byte cp.async
//   (keys behind the sequence and pages that do not exist are filled with zeros).
// - 16 rows and 16 keys make one m16n8k16 tile: S = Q K^T (two MMAs per 16 dims), and
//   P, already in the A layout, times V.  mma.sync is enough here: at HBM's rate the
//   tensor work of a tile is a small part of its load time.
// - e4m3 rows halve the bytes, and the instructions per byte become the bound (the first
//   form of this path, cp.async and five integer operations per pair of codes, ran 944
//   instructions per 16-key tile and reached 2.8 TB/s).  So the tiles come by TMA, issued by one
//   lane, and the codes go to the tensor cores as f16, which holds them exactly: one cvt
//   per pair of K, a byte permute and a cvt per pair of V (which transposes it on the way).  To
//   load 16 codes of one key at once, the head dims are taken in a permuted order, the same
//   for Q and K.  Q is scaled to f16 by a power of two per row (its largest element in [2^14, 2^15),
//   so what f16 drops is below 2^-39 of it); the key rows' scales multiply the scores; the
//   value rows' scales 2^e multiply the weights, relative to E, the largest e seen: a weight
//   times 2^(e-E) stays below 2^15.  Where e lies more than 12 below E in a tile, f16 would drop
//   bits of such weights, and the tile's V is widened to bf16 instead, exactly: a code's bits moved
//   to a bf16's place are the value times 2^-120, and one packed multiply by 2^(120+e-E) does the rest.
// - The running maximum moves only when a score exceeds it by 2^8 (a vote per tile): the
//   weights stay below 2^8 (2^15 where they become f16) and the result is the same up to rounding.
// Measured: 64 ragged sequences up to 32768 keys (32 heads on 8, D 128, bf16; six draws of the lengths) 6.4 to 6.6
// TB/s, 630 us for a million keys in all; 32 up to 65536 (64 on 8, e4m3) 4.2 to 4.6 TB/s, 450 to 490 us for a million,
// where the ALU pipe is at 47 % and each warp waits out its own instruction latencies (eight warps an SM: a ring of
// 96 KB and 244 registers).

constexpr int PR_THREADS = 128;
constexpr int PR_WARPS = 4;
constexpr int PR_ROWS = 16;                // query rows per CTA
constexpr float PR_RESCALE_LOG2 = 8.0f;    // how far a score may exceed the running maximum's reference

template <int D, bool E4M3>
struct RowsCfg {
    // Keys per warp and tile: what a tile costs besides its keys (waits, copies, votes) is most of an
    // e4m3 tile of 16 keys (528 instructions at D = 128).
    static constexpr int WK = !E4M3 || D == 256 ? 16 : D == 128 ? 32 : 64, TK = PR_WARPS * WK, NT = WK / 8;
    static constexpr int ROW = D * (E4M3 ? 1 : 2);      // bytes of one row
    static constexpr int CPR = ROW / 16;                // 16-byte chunks per row
    static constexpr int HALF = WK * ROW;            // K or V part of a stage
    static constexpr int STAGE = 2 * HALF;
    // e4m3: the swizzle span that TMA applies to a row (128 bytes at most: column blocks at D = 256)
    static constexpr int SW = ROW < 128 ? ROW : 128;
    static constexpr int BLOCK = WK * SW;               // a column block of a tile
    // about 96 KB of rings per CTA (two CTAs per SM), 192 KB where a stage is 16 KB (one)
    static constexpr int NST_RAW = 24576 / (2 * HALF);
    static constexpr int NST = NST_RAW < 3 ? 3 : NST_RAW > 8 ? 8 : NST_RAW;
    static constexpr int RING = PR_WARPS * NST * STAGE;
    static constexpr int MERGE = PR_WARPS * PR_ROWS * (D + 4) * 4;   // reuses the ring
    // e4m3, behind the ring: each warp's barriers, and the K and V scale bytes of each stage
    static constexpr int BARS = E4M3 ? PR_WARPS * NST * 8 : 0, SCALES = E4M3 ? PR_WARPS * NST * 2 * WK : 0;
    static constexpr int AREA = (RING > MERGE ? RING : MERGE) + 127 & ~127;
    static constexpr int SMEM = AREA + BARS + SCALES;
    static constexpr int PER_SM = SMEM > 110 * 1024 ? 1 : 2;
    // e4m3: weights are kept 2^7 high, at most 2^15, so that f16 drops less than 2^-32 of a weight of one
    static constexpr float HIGH_LOG2 = E4M3 ? 7.0f : 0.0f;
};

// Byte offset of 16-byte chunk c of row r in a stage's K or V part.  bf16: ldmatrix takes one
// chunk of 8 rows, and the permutation puts those into different banks.  e4m3: what TMA's
// swizzle of SW bytes makes of column blocks; the reads of V (4 bytes of rows 2 q4, q4 = 0..3)
// then touch every bank once, those of K (16 bytes a lane, two rows to a quarter warp) twice.
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t rows_swizzle(int r, int c) {
    using C = RowsCfg<D, E4M3>;
    constexpr int CPR = C::CPR;
    if constexpr (E4M3) {
        if constexpr (CPR >= 8) return static_cast<uint32_t>((c >> 3) * C::BLOCK + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        else if constexpr (CPR == 4) return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
        else return static_cast<uint32_t>(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
    } else {
        constexpr int RPL = CPR >= 8 ? 1 : 8 / CPR;            // rows per 128-byte line
        const int line = r * CPR / 8 + (CPR >= 8 ? c >> 3 : 0);
        const int pos = (CPR >= 8 ? c & 7 : (r % RPL) * CPR + c) ^ (CPR >= 8 ? r & 7 : (r >> 1) & 3);
        return static_cast<uint32_t>(line * 128 + pos * 16);
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool fill) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(fill ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The two e4m3 codes in the low or the high half of w as two f16 values, exactly.
__device__ __forceinline__ uint32_t codes_f16_lo(uint32_t w) {
    uint32_t d;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t w) {
    uint32_t d;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Two e4m3 codes in bytes 1 and 3 of t (other bytes: anything) as bf16 values times 2^-120: sign
// to bit 15, exponent and mantissa (a magnitude) to bits 10..4.  Times 2^(120 + e) they are the row's
// values, but the two codes of NaN would be 480: what nan_codes gives (all ones in their places: the sum's
// sign bit, spread over the half by prmt) is or-ed to the product.
__device__ __forceinline__ uint32_t code_magnitudes(uint32_t t) { return (t >> 4) & 0x07f007f0u; }
__device__ __forceinline__ uint32_t code_signs(uint32_t t) { return t & 0x80008000u; }
__device__ __forceinline__ uint32_t nan_codes(uint32_t magnitudes) {
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, 0xbb99;\n" : "=r"(d) : "r"(magnitudes + 0x78107810u));
    return d;
}
__device__ __forceinline__ uint32_t widen2(uint32_t t, uint32_t f) {
    const uint32_t m = code_magnitudes(t);
    return mul_bf16x2(code_signs(t) | m, f) | nan_codes(m);
}
// bf16 pattern of 2^(120 + e) cut to 2^127, for a scale code e + 127; NaN for 255.
__device__ __forceinline__ uint32_t scale_factor(uint32_t code) {
    return code == SCALE_NAN ? 0x7fffu : min(code + 120u, 254u) << 7;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Tiles of sequence b for one key head: at least one where it has query rows, so that empty
// sequences get their zeros.
__device__ __forceinline__ int rows_units(const PagedParams& p, int b, bool report = false) {
    const int n = query_range(p, b, report).n;
    const int kv = paged_kv_len(p.kv_len, b, p.kv_cap, report);
    if (n == 0) return 0;
    return max(1, tiles_of(kv, p.tile_keys));
}

// The deal: `total` units per key head over the batch, `per` of all heads' units to a CTA.
struct RowsDeal {
    long long total, per;
    __device__ __forceinline__ long long all(int Hkv) const { return total * Hkv; }
};
// Block-wide sum over the batch (PR_THREADS threads).
__device__ __forceinline__ RowsDeal rows_deal(const PagedParams& p, int n_ctas, long long* s_sum, bool report) {
    long long sum = 0;
    for (int b = threadIdx.x; b < p.B; b += PR_THREADS) sum += rows_units(p, b, report);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    RowsDeal d;
    d.total = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    __syncthreads();
    d.per = max(static_cast<long long>(p.min_units), (d.all(p.c.Hkv) + n_ctas - 1) / n_ctas);
    return d;
}
// Calls f(b, units of one key head before b) on the one thread whose sequence b holds `unit`, counted over all
// heads of the sequences in turn.
template <typename F>
__device__ __forceinline__ void rows_scan(const PagedParams& p, long long* s_sum, long long unit, F f) {
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += PR_THREADS) {
        const int b = b0 + threadIdx.x;
        const long long n = b < p.B ? rows_units(p, b) : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if ((threadIdx.x & 31) >= o) incl += t;
        }
        if ((threadIdx.x & 31) == 31) s_sum[threadIdx.x >> 5] = incl;
        __syncthreads();
        for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) incl += s_sum[w];
        const long long all = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
        incl += base;
        if (n > 0 && (incl - n) * p.c.Hkv <= unit && unit < incl * p.c.Hkv) f(b, incl - n);
        base += all;
        __syncthreads();
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(PR_THREADS, RowsCfg<D, E4M3>::PER_SM)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedParams p,
                      const int n_ctas) {
    using C = RowsCfg<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_sum[PR_WARPS];
    __shared__ long long s_first;
    __shared__ int s_b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q4 = lane & 3, r8 = lane >> 2;

    allow_next_kernel();
    const RowsDeal deal = rows_deal(p, n_ctas, s_sum, blockIdx.x == 0);
    const long long all = deal.all(p.c.Hkv);
    long long unit = blockIdx.x * deal.per;
    const long long unit_end = min(all, unit + deal.per);
    if (unit >= all) {
        if (tid == 0) p.shared_at[blockIdx.x].n = 0;
        return;
    }
    rows_scan(p, s_sum, unit, [&](int b, long long before) {
        s_b = b;
        s_first = before;
    });
    int b = s_b;
    long long rem = unit - s_first * p.c.Hkv;
    const uint32_t ring = smem_u32(smem) + warp * C::NST * C::STAGE;
    // e4m3: this warp's barriers and scale bytes
    const uint32_t bars = smem_u32(smem) + C::AREA + warp * C::NST * 8;
    uint8_t* const scales = smem + C::AREA + C::BARS + warp * C::NST * 2 * C::WK;
    // e4m3: where this lane's 16 (8) bytes of keys r8, r8 + 8, ... begin in a K tile, and its 4 bytes of
    // rows 2 q4, + 1, + 8, + 9, ... in a V tile.  The swizzle only flips address bits, so further chunks
    // of the row are an exclusive or away.
    uint32_t k_off[C::NT], v_off[C::NT * 2];
    if constexpr (E4M3) {
#pragma unroll
        for (int n = 0; n < C::NT; ++n) k_off[n] = D >= 64 ? rows_swizzle<D, true>(8 * n + r8, q4) : rows_swizzle<D, true>(8 * n + r8, q4 >> 1) + (q4 & 1) * 8;
#pragma unroll
        for (int k = 0; k < 2 * C::NT; ++k) v_off[k] = rows_swizzle<D, true>(2 * q4 + (k & 1) + 8 * (k >> 1), r8 >> 2) + (r8 & 3) * 4;
    }
    uint32_t item = 0;       // e4m3: tiles consumed, over all segments
    bool ok = true;          // e4m3: no wait has run out
    if constexpr (E4M3) {
        if (lane == 0) {
            for (int s = 0; s < C::NST; ++s) mbar_init(bars + 8 * s, 1 + C::WK / 4);   // the byte count's arrival and the scale copies'
            fence_mbar_init();
        }
        __syncwarp();
    }

    while (unit < unit_end) {
        int units = rows_units(p, b);
        while (units == 0) units = rows_units(p, ++b);   // a later one exists: unit < all
        const int h = static_cast<int>(rem / units);
        const int tile0 = static_cast<int>(rem - static_cast<long long>(h) * units);
        const int tile1 = static_cast<int>(min(static_cast<long long>(units), tile0 + (unit_end - unit)));
        if (tid == 0 && unit == blockIdx.x * deal.per) p.shared_at[blockIdx.x] = {b, h, tile0, tile0 > 0 ? units : 0, deal.per};
        const QueryRange qr = query_range(p, b, false);
        const int kv = paged_kv_len(p.kv_len, b, p.kv_cap, false);
        const int rows = min(qr.n, p.max_q) * p.G;

        // ---- Q fragments (rows beyond the last one: zeros) and what each of the two rows sees
        uint32_t qf[D / 16][4];
        int seen[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = r8 + 8 * e;
            const int i = r / p.G;
            seen[e] = r < rows ? (p.causal ? min(kv, max(0, kv - qr.n + i + 1)) : kv) : 0;
            const __nv_bfloat16* src = p.q + (qr.t0 + (r < rows ? i : 0)) * p.q_t + (h * p.G + (r < rows ? r - i * p.G : 0)) * p.q_h;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                uint2 v = make_uint2(0u, 0u);
                if (r < rows) {
                    if constexpr (E4M3) {
                        // dims in the order the e4m3 rows are loaded: lane q4 holds D/4 of them in runs of
                        // 16 (8 at D = 32), four of a run per step
                        constexpr int RUN = D >= 64 ? 16 : 8;
                        const int d = (s / (RUN / 4)) * (RUN * 4) + q4 * RUN + (s % (RUN / 4)) * 4;
                        v = *reinterpret_cast<const uint2*>(src + d);
                    } else {
                        v.x = *reinterpret_cast<const uint32_t*>(src + s * 16 + q4 * 2);
                        v.y = *reinterpret_cast<const uint32_t*>(src + s * 16 + q4 * 2 + 8);
                    }
                }
                qf[s][e] = v.x;
                qf[s][2 + e] = v.y;
            }
        }
        float row_mul[2] = {p.scale_log2, p.scale_log2};   // what turns a row's products into log2 scores
        if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t top = 0u;                         // the row's largest magnitude, as a bf16 pattern
#pragma unroll
                for (int s = 0; s < D / 16; ++s) top = __vmaxu2(top, __vmaxu2(qf[s][e] & 0x7fff7fffu, qf[s][2 + e] & 0x7fff7fffu));
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // amax in [2^k, 2^(k+1)): times 2^(14-k).  Rows of zeros, infinities and NaN, and exponents
                // whose power is no normal fp32 number, are cut to what is.
                const int up = top == 0u || top >= 0x7f80u ? 0 : min(14 + 127 - static_cast<int>(top >> 7), 126);
                const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                row_mul[e] *= __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int x = e; x < 4; x += 2)
                        qf[s][x] = pack_f16(__uint_as_float(qf[s][x] << 16) * f, __uint_as_float(qf[s][x] & 0xffff0000u) * f);
            }
        }
        const int all_seen = p.causal ? max(0, kv - qr.n + 1) : kv;   // keys that every row sees

        // ---- loads: this warp's WK keys of tile t, in groups of eight, each within one page
        const int32_t* table = p.table + b * p.table_stride;
        auto page_of = [&](int t) {   // lane g < WK / 8: the page of the 8-key group, -1: none
            const int key = key_at(t, C::TK, warp * C::WK + (lane & (C::WK / 8 - 1)) * 8);
            int page = -1;
            if (t < tile1 && key < kv) {
                page = __ldg(table + page_index(p, key));
                if (page < 0 || page >= p.c.num_pages) {
                    if (lane < C::WK / 8) atomicOr(&g_paged_status, STATUS_CACHE);
                    page = -1;
                }
            }
            return page;
        };
        auto load = [&](int t, int page_l, int slot) {
          if constexpr (E4M3) {
            const uint32_t dst = ring + slot * C::STAGE, bar = bars + 8 * slot;
            const int key0 = t * C::TK + warp * C::WK;
            const int g_l = lane & (C::WK / 8 - 1);        // this lane's 8-row group
            const int row_l = key0 + 8 * g_l - page_index(p, key0 + 8 * g_l) * p.c.page_size;
            // box g (box_rows rows, all in one page) by the lane that looked its first group up
            if (lane == 0) mbar_arrive_expect_tx(bar, C::STAGE);
            __syncwarp();
            if (lane < C::WK / 8 && (lane * 8 & (p.box_rows - 1)) == 0) {
#pragma unroll
                for (int b2 = 0; b2 < C::ROW / C::SW; ++b2)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        tma_load_4d(dst + w * C::HALF + b2 * C::BLOCK + lane * 8 * C::SW, w ? &tm_v : &tm_k, b2 * C::SW, row_l, h,
                                    page_l < 0 ? p.c.num_pages : page_l, bar);
            }
            if (lane < C::WK / 4) {      // scale bytes: K, then V, of each 8-row group
                const int w = lane / (C::WK / 8);
                const uint8_t* src = p.c.scale[w];
                if (page_l >= 0) src += (static_cast<long long>(page_l) * p.c.Hkv + h) * p.c.page_size + row_l;
                cp_async8(smem_u32(scales) + slot * 2 * C::WK + 8 * lane, src, page_l >= 0);
                cp_async_mbar_arrive_noinc(bar);
            }
          } else {
            const uint32_t dst = ring + slot * C::STAGE;
            const int key0 = t * C::TK + warp * C::WK;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int page = __shfl_sync(0xffffffffu, page_l, g);
                const int k0 = key0 + 8 * g;
                const int r0 = k0 - k0 / p.c.page_size * p.c.page_size;
                const int n = page < 0 ? 0 : kv - k0;   // rows of the group that exist
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint8_t* src = p.c.data[w];
                    if (page >= 0) src += page * p.c.sp[w] + h * p.c.sh[w] + r0 * p.c.st[w];
#pragma unroll
                    for (int x = 0; x < 8 * C::CPR / 32 + (8 * C::CPR % 32 != 0); ++x) {
                        const int idx = x * 32 + lane;
                        const int r = idx / C::CPR, c = idx % C::CPR;
                        if (8 * C::CPR % 32 == 0 || idx < 8 * C::CPR)
                            cp_async16(dst + w * C::HALF + rows_swizzle<D, E4M3>(8 * g + r, c), src + (r < n ? r * p.c.st[w] + c * 16 : 0), r < n);
                    }
                }
            }
          }
        };
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

        int page_next = page_of(tile0);
#pragma unroll 1
        for (int s = 0; s < C::NST - 1; ++s) {
            const int pg = page_next;
            page_next = page_of(tile0 + s + 1);
            if (tile0 + s < tile1) load(tile0 + s, pg, E4M3 ? static_cast<int>((item + s) % C::NST) : s);
            if constexpr (!E4M3) cp_commit();
        }
        int slot = E4M3 ? static_cast<int>(item % C::NST) : 0;
        int e_ref = -1000;       // e4m3: E + 127, the largest scale code of a value row so far
#pragma unroll 1
        for (int t = tile0; t < tile1; ++t) {
            __syncwarp();   // every lane is done with the slot that is filled next
            {
                const int tn = t + C::NST - 1;
                const int pg = page_next;
                page_next = page_of(tn + 1);
                if (tn < tile1) load(tn, pg, slot == 0 ? C::NST - 1 : slot - 1);
                if constexpr (!E4M3) cp_commit();
            }
            if constexpr (E4M3) {
                ok = ok && chunk_wait_warp(bars + 8 * slot, (item / C::NST) & 1u, nullptr, p.wait_ns);
                if (!ok) break;
                ++item;
            } else {
                cp_wait<C::NST - 1>();
                __syncwarp();
            }
            const uint32_t kb = ring + slot * C::STAGE, vb = kb + C::HALF;
            const int key0 = t * C::TK + warp * C::WK;
            float s[C::NT][4];
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
            float ks[C::NT][2];      // e4m3: 2^e of keys 8 n + 2 q4, + 1
            uint32_t vc[C::NT / 2];  // e4m3: the scale codes of the value rows, a byte each: tiles 2 i, 2 i + 1
            bool odd_codes = false;  // a scale code of NaN in the tile
            if constexpr (E4M3) {
                const uint8_t* sc = scales + slot * 2 * C::WK + 2 * q4;
                uint32_t kc[C::NT / 2];
                bool odd = false;
#pragma unroll
                for (int i = 0; i < C::NT / 2; ++i) {
                    kc[i] = *reinterpret_cast<const uint16_t*>(sc + 16 * i) | static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(sc + 16 * i + 8)) << 16;
                    vc[i] = *reinterpret_cast<const uint16_t*>(sc + C::WK + 16 * i) | static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(sc + C::WK + 16 * i + 8)) << 16;
                }
                if (kv - key0 < C::WK) {
                    // rows of a page behind the sequence hold anything: value codes of NaN, scale bytes
                    const int left = max(0, kv - key0);
                    for (int x = lane; x < (C::WK - left) * C::CPR; x += 32)
                        *reinterpret_cast<uint4*>(smem + (vb - smem_u32(smem)) + rows_swizzle<D, true>(left + x / C::CPR, x % C::CPR)) = make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // before TMA writes there again
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < C::NT / 2; ++i)
#pragma unroll
                        for (int b2 = 0; b2 < 4; ++b2)
                            if (16 * i + 2 * q4 + (b2 & 1) + 8 * (b2 >> 1) >= left) vc[i] &= ~(255u << 8 * b2);
                }
#pragma unroll
                for (int i = 0; i < C::NT / 2; ++i) odd |= (__vcmpeq4(kc[i], 0xffffffffu) | __vcmpeq4(vc[i], 0xffffffffu)) != 0u;
                odd_codes = __any_sync(0xffffffffu, odd);
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int b2 = 0; b2 < 2; ++b2) {
                        const uint32_t code = (kc[n >> 1] >> (16 * (n & 1) + 8 * b2)) & 255u;
                        ks[n][b2] = odd_codes ? scale_value(code) : __uint_as_float(code << 23);
                    }
                constexpr int RUN = D >= 64 ? 16 : 8;
#pragma unroll
                for (int c = 0; c < D / (RUN * 4); ++c) {
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        uint32_t w[RUN / 4];
                        const uint32_t at = kb + (D == 256 ? (c >> 1) * C::BLOCK : 0) + (k_off[n] ^ ((D == 256 ? c & 1 : c) << 6));
                        if constexpr (RUN == 16)
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
                        else
                            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
#pragma unroll
                        for (int e = 0; e < RUN / 4; ++e) mma16816_f16(s[n], qf[c * (RUN / 4) + e], codes_f16_lo(w[e]), codes_f16_hi(w[e]));
                    }
                }
            } else {
#pragma unroll
                for (int st = 0; st < D / 16; ++st) {
                    uint32_t kf[4];   // keys 0-7 dims 0-7, 8-15; keys 8-15 dims 0-7, 8-15
                    ldsm4(kb + rows_swizzle<D, false>((lane & 7) + ((lane >> 4) << 3), st * 2 + ((lane >> 3) & 1)), kf);
                    mma16816(s[0], qf[st], kf[0], kf[1]);
                    mma16816(s[1], qf[st], kf[2], kf[3]);
                }
            }
            // ---- scores in the log2 domain, masked by selection
            float x[C::NT][4];
            const bool masked = all_seen - key0 < C::WK;   // uniform
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y = s[n][e] * row_mul[e >> 1];
                    if constexpr (E4M3) y *= ks[n][e & 1];
                    if (masked && key0 + 8 * n + 2 * q4 + (e & 1) >= seen[e >> 1]) y = -INFINITY;
                    x[n][e] = y;
                    mx[e >> 1] = fmaxf(mx[e >> 1], y);
                }
            // m: the reference of the weights 2^(x - m), HIGH_LOG2 below a maximum of the scores so far
            constexpr float LAZY = PR_RESCALE_LOG2 + C::HIGH_LOG2;
            if (__any_sync(0xffffffffu, mx[0] > m[0] + LAZY || mx[1] > m[1] + LAZY)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mn = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
                    mn = fmaxf(m[e], mn - C::HIGH_LOG2);
                    const float f = m[e] == -INFINITY ? 0.0f : exp2_approx(m[e] - mn);
                    m[e] = mn;
                    l[e] *= f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][2 * e] *= f;
                        o[i][2 * e + 1] *= f;
                    }
                }
            }
            uint32_t pf[C::NT / 2][4];   // A fragments of 16 keys each
            const float m0 = m[0] == -INFINITY ? 0.0f : m[0], m1 = m[1] == -INFINITY ? 0.0f : m[1];
            float wt[C::NT][4];
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    wt[n][e] = exp2_approx(x[n][e] - (e < 2 ? m0 : m1));
                    l[e >> 1] += wt[n][e];
                }
            // ---- O += P V
            if constexpr (E4M3) {
                // E over the tile's rows.  Codes of NaN do not count (their weights become NaN), nor do rows
                // that are not there (code 0 above).
                uint32_t c4[C::NT / 2], top = 0u;
#pragma unroll
                for (int i = 0; i < C::NT / 2; ++i) {
                    c4[i] = odd_codes ? vc[i] & ~__vcmpeq4(vc[i], 0xffffffffu) : vc[i];
                    top = __vmaxu4(top, c4[i]);
                }
                top = __vmaxu4(top, top >> 16);
                top = __reduce_max_sync(0xffffffffu, max(top & 255u, (top >> 8) & 255u));
                if (static_cast<int>(top) > e_ref) {
                    const int up = static_cast<int>(top) - e_ref;
                    const float f = up > 126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                    e_ref = static_cast<int>(top);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][e] *= f;
                }
                // 2^(e - E) multiplies the f16 weights, or (wide) the bf16 values
                bool far = false;
                int de[C::NT][2];
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int b2 = 0; b2 < 2; ++b2) {
                        de[n][b2] = static_cast<int>((c4[n >> 1] >> (16 * (n & 1) + 8 * b2)) & 255u) - e_ref;
                        far |= de[n][b2] < -12;
                    }
                // (rows that are not there ask for the wide form too: a sequence's last tile)
                const bool wide = __any_sync(0xffffffffu, far);
                uint32_t vsc[C::NT];
#pragma unroll
                for (int n = 0; n < C::NT; ++n) {
                    float vm[2];
                    vsc[n] = 0u;
                    if (wide) {
                        vm[0] = vm[1] = 1.0f;
                        vsc[n] = static_cast<uint32_t>(max(247 + de[n][0], 0)) << 7 | static_cast<uint32_t>(max(247 + de[n][1], 0)) << 23;
                    } else {
                        vm[0] = __uint_as_float(static_cast<uint32_t>(127 + de[n][0]) << 23);
                        vm[1] = __uint_as_float(static_cast<uint32_t>(127 + de[n][1]) << 23);
                    }
                    if (odd_codes) {
#pragma unroll
                        for (int b2 = 0; b2 < 2; ++b2)
                            if (((vc[n >> 1] >> (16 * (n & 1) + 8 * b2)) & 255u) == SCALE_NAN) vm[b2] = __uint_as_float(0x7fc00000u);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) wt[n][e] *= vm[e & 1];
                    uint32_t(&pw)[4] = pf[n >> 1];
                    pw[2 * (n & 1)] = wide ? pack_bf16(wt[n][0], wt[n][1]) : pack_f16(wt[n][0], wt[n][1]);
                    pw[2 * (n & 1) + 1] = wide ? pack_bf16(wt[n][2], wt[n][3]) : pack_f16(wt[n][2], wt[n][3]);
                }
                auto pv = [&](auto is_wide) {
#pragma unroll
                    for (int g = 0; g < D / 32; ++g) {
#pragma unroll
                        for (int i = 0; i < C::NT / 2; ++i) {
                            uint32_t w[4];   // keys 16 i + 2 q4, + 1, + 8, + 9: dims 32 g + 4 r8 + {0..3}
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                asm volatile("ld.shared.b32 %0, [%1];"
                                             : "=r"(w[k])
                                             : "r"(vb + (D == 256 ? (g >> 2) * C::BLOCK : 0) + (v_off[4 * i + k] ^ ((D == 256 ? g & 3 : g) << 5))));
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if constexpr (decltype(is_wide)::value)
                                    mma16816(o[4 * g + e], pf[i], widen2(__byte_perm(w[0], w[1], e << 4 | (4 + e) << 12), vsc[2 * i]),
                                             widen2(__byte_perm(w[2], w[3], e << 4 | (4 + e) << 12), vsc[2 * i + 1]));
                                else
                                    mma16816_f16(o[4 * g + e], pf[i], codes_f16_lo(__byte_perm(w[0], w[1], e | (4 + e) << 4)),
                                                 codes_f16_lo(__byte_perm(w[2], w[3], e | (4 + e) << 4)));
                            }
                        }
                    }
                };
                if (wide) pv(std::true_type{});
                else pv(std::false_type{});
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    pf[0][2 * n] = pack_bf16(wt[n][0], wt[n][1]);
                    pf[0][2 * n + 1] = pack_bf16(wt[n][2], wt[n][3]);
                }
#pragma unroll
                for (int st = 0; st < D / 16; ++st) {
                    uint32_t vf[4];   // dims 0-7: keys 0-7, 8-15; dims 8-15: keys 0-7, 8-15
                    ldsm4_trans(vb + rows_swizzle<D, false>(lane & 15, st * 2 + (lane >> 4)), vf);
                    mma16816(o[2 * st], pf[0], vf[0], vf[1]);
                    mma16816(o[2 * st + 1], pf[0], vf[2], vf[3]);
                }
            }
            slot = slot + 1 == C::NST ? 0 : slot + 1;
        }
        if constexpr (!E4M3) cp_wait<0>();
        if constexpr (E4M3) {
            if (!ok) {   // copies that were issued must land before the memory is used otherwise
                const uint64_t d0 = global_timer_ns();
                while (global_timer_ns() - d0 < 2000000ull) {
                }
            }
        }

        // ---- the four warps' results into one: m, l and o / l of each warp through shared memory
        // (divided first: sums of values near bf16's largest would not fit fp32)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            float f = l[e] == 0.0f ? 0.0f : 1.0f / l[e];
            if (E4M3 && e_ref > -1000) f *= __uint_as_float(static_cast<uint32_t>(e_ref) << 23);   // O is in units of 2^E
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][2 * e] *= f;
                o[i][2 * e + 1] *= f;
            }
        }
        __syncthreads();   // every warp is done with its ring
        float* so = reinterpret_cast<float*>(smem);                      // [4][16][D + 2]
        float* sm = so + PR_WARPS * PR_ROWS * (D + 2);                   // [4][16][2]: m, l
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = r8 + 8 * e;
            float* dst = so + (warp * PR_ROWS + r) * (D + 2);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                if constexpr (E4M3) {
                    // n-tile 4 g + t holds dims 32 g + 4 n + t, this lane n = 2 q4 and 2 q4 + 1
                    const int d = (i >> 2) * 32 + (i & 3) + 8 * q4;
                    dst[d] = o[i][2 * e];
                    dst[d + 4] = o[i][2 * e + 1];
                } else {
                    *reinterpret_cast<float2*>(dst + i * 8 + q4 * 2) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
                }
            }
            if (q4 == 0) {
                sm[(warp * PR_ROWS + r) * 2] = m[e];
                sm[(warp * PR_ROWS + r) * 2 + 1] = l[e];
            }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == units;
        const long long part = 2LL * blockIdx.x + (tile0 == 0 ? 1 : 0);
        for (int idx = tid; idx < rows * (D / 4); idx += PR_THREADS) {
            const int r = idx / (D / 4), d = idx % (D / 4) * 4;
            float mm = -INFINITY, ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < PR_WARPS; ++w) mm = fmaxf(mm, sm[(w * PR_ROWS + r) * 2]);
#pragma unroll
            for (int w = 0; w < PR_WARPS; ++w) {
                const float mw = sm[(w * PR_ROWS + r) * 2];
                const float f = (mw == -INFINITY ? 0.0f : exp2_approx(mw - mm)) * sm[(w * PR_ROWS + r) * 2 + 1];
                ll += f;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += f * so[(w * PR_ROWS + r) * (D + 2) + d + e];
            }
            const bool some = mm != -INFINITY || ll != 0.0f;   // (a NaN sum counts as some)
            const float inv = some ? 1.0f / ll : 0.0f;
            const float lse = some ? (mm + log2f(ll)) * 0.69314718055994530942f : -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] *= inv;
            if (whole) {
                const int i = r / p.G, hq = h * p.G + r - i * p.G;
                *reinterpret_cast<uint2*>(p.out + (qr.t0 + i) * p.out_t + hq * p.out_h + d) =
                    make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
                if (d == 0 && p.lse != nullptr) p.lse[static_cast<long long>(qr.t0 + i) * p.Hq + hq] = lse;
            } else {
                *reinterpret_cast<float4*>(p.part_out + (part * PR_ROWS + r) * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (d == 0) p.part_lse[part * PR_ROWS + r] = lse;
            }
        }
        if constexpr (E4M3) {
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // the merge's accesses, before TMA writes there
            if (__syncthreads_or(!ok)) return;
        } else {
            __syncthreads();
        }
        unit += tile1 - tile0;
        rem += tile1 - tile0;
        if (rem >= static_cast<long long>(units) * p.c.Hkv) {
            rem = 0;
            ++b;
        }
    }
}

// Puts together the pairs that several CTAs of paged_rows_kernel worked on.  Block (c, r) looks at
// the border between the runs of CTAs c and c + 1, and takes row r; the first border inside a pair
// does the pair.  CTA c's part is slot 2c where the pair's tiles reach its run's start from an
// earlier CTA, 2c + 1 where the pair begins in its run.  A single long sequence has hundreds of
// parts: the block's groups of D / 4 threads take them in turn (16 rows of one sequence of 20000 keys,
// 4 key heads, D 128: 46 us a call, 79 with a block for all rows whose threads
// each walked all parts).
template <int D>
__global__ void __launch_bounds__(PR_THREADS) paged_rows_combine_kernel(const PagedParams p) {
    constexpr int LANES = D / 4, GROUPS = PR_THREADS / LANES;
    __shared__ float s_max[PR_WARPS], s_sum[GROUPS];
    __shared__ float4 s_acc[PR_THREADS];
    const int tid = threadIdx.x, r = blockIdx.y;
    wait_for_main_kernel();   // every block, so that this grid never ends before that one
    const SharedAt s = p.shared_at[blockIdx.x + 1];
    if (s.n == 0) return;
    const int b = s.b, h = s.h;
    const long long u0 = (blockIdx.x + 1) * s.per - s.t0, c0 = u0 / s.per, c1 = (u0 + s.n - 1) / s.per;
    if (c0 != blockIdx.x) return;
    const QueryRange qr = query_range(p, b, false);
    if (r >= min(qr.n, p.max_q) * p.G) return;
    auto slot = [&](long long c) { return 2 * c + (c == c0 ? 1 : 0); };
    float M = -INFINITY;
    for (long long c = c0 + tid; c <= c1; c += PR_THREADS) M = fmaxf(M, __ldcg(p.part_lse + slot(c) * PR_ROWS + r));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const int g = tid / LANES, d = tid % LANES * 4;
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (long long c = c0 + g; c <= c1; c += GROUPS) {
        const float lc = __ldcg(p.part_lse + slot(c) * PR_ROWS + r);
        const float w = lc == -INFINITY ? 0.0f : expf(lc - M);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_out + (slot(c) * PR_ROWS + r) * D + d));
        sum += w;
        acc.x += w * v.x;
        acc.y += w * v.y;
        acc.z += w * v.z;
        acc.w += w * v.w;
    }
    s_acc[tid] = acc;
    if (d == 0) s_sum[g] = sum;
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) {
        const float4 v = s_acc[k * LANES + tid];
        sum += s_sum[k];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
    }
    const bool some = sum != 0.0f;
    const float inv = some ? 1.0f / sum : 0.0f;
    const int i = r / p.G, hq = h * p.G + r - i * p.G;
    *reinterpret_cast<uint2*>(p.out + (qr.t0 + i) * p.out_t + hq * p.out_h + d) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (d == 0 && p.lse != nullptr) p.lse[static_cast<long long>(qr.t0 + i) * p.Hq + hq] = some ? M + logf(sum) : -INFINITY;
}
