// paged_chunk.cuh -- attention over pages for many query rows per key head, head dims 32,
// 64 and 128: chunks of prompts.  Included by paged.cu inside namespace attn.
//
// Rows: the G query heads of a key head see the same keys, so a 128-row tile is 128 / G tokens
// times G heads (row = token * G + head, loaded by one 4-D TMA box per 64 dims).  A CTA
// works on two such tiles of consecutive tokens, one per softmax warpgroup, against the same
// 128-key tiles of K and V: while one tile's scores are in its softmax warps, the tensor
// pipe runs the other tile's MMAs, and each K/V byte brought to shared memory serves 256 rows.
//
// TMEM: S_0, S_1 (128 columns each), O_0, O_1.  MMA order per key tile j at D = 128: PV_0(j),
// S_0(j+1), PV_1(j), S_1(j+1), P_g stored over S_g; one thread's MMAs run in issue order, so "S_g(j)
// ready" also means PV_g(j-1) is complete and the group may rescale O_g.  At D <= 64 P_0 and P_1 have
// columns of their own and the order is S_0(j+1), S_1(j+1), PV_0(j), PV_1(j); every PV is
// announced on a barrier, which a group waits for before it writes P_g (or O_g) again.
//
// The work, (sequence, key head, token tile, key tile), is laid end to end and dealt to
// one persistent CTA per SM in equal contiguous runs, like the few-row kernel's: ragged
// batches and causal triangles leave no SM idle at the end, and only a run's first and last
// token tile can be shared with another CTA; paged_chunk_combine_kernel puts those together.
//
// K and V are copied by TMA, in boxes of the largest power of two of rows (up to 128) that divides
// the page size, each box from its page; a box behind the sequence or of a page that does
// not exist has its page coordinate outside the pool and reads as zeros.  Small pages make
// many boxes, and what one warp can issue bounds them, so a bf16 box holds all columns of its
// rows: the tensor map splits a page into groups of 8 rows, and a tile lies in shared memory
// as [8-row group][64-column block][8 rows][128 bytes], which the MMA descriptors address by
// their two strides.  The rows of the last box behind the sequence are cleared in shared
// memory before PV reads them.  e4m3 tiles land in staging slots instead, with their
// scale bytes by cp.async; four converter warps widen them to bf16 (exactly, see paged_rows.cuh) into
// the same layout.  (Loading the codes straight into the converters' registers, one tile
// ahead, left them waiting for loads: 476 against 1061 TFLOP/s with the loads taken out, 2048 rows
// on 32768 keys, 32 heads on 8, D 128.)
//
// Every wait is bounded; on expiry the CTA raises the timeout flag, drains and exits.

constexpr int PC_BN = 128;                 // keys per tile
constexpr float PC_RESCALE_LOG2 = 8.0f;

template <int D, bool E4M3>
struct ChunkCfg {
    static constexpr int SW = D >= 64 ? 128 : 64;       // swizzle span in bytes
    static constexpr int BLK = SW / 2;                  // columns per swizzle block
    static constexpr int NBLK = D / BLK;
    static constexpr int QT_BYTES = 128 * D * 2;        // one 128-row tile
    static constexpr int SLOT = PC_BN * D * 2;          // a K or V tile
    static constexpr int CTRL = 1024;
    static constexpr int GROUP = NBLK * 8 * SW;         // one 8-row group of a K or V tile
    // e4m3: staged codes of a tile, and its 128 scale bytes
    static constexpr int STG_BYTES = PC_BN * D + 128;
    static constexpr int NSTG = E4M3 ? (D == 128 ? 4 : 8) : 0;
    static constexpr int NS_FIT = (232448 - 1024 - CTRL - 2 * QT_BYTES - NSTG * STG_BYTES) / SLOT;
    static constexpr int NS = NS_FIT < 12 ? NS_FIT : 12;
    static constexpr int SMEM = 1024 + 2 * QT_BYTES + NS * SLOT + NSTG * STG_BYTES + CTRL;
    static_assert(NS >= 3, "ring depth");
    static constexpr uint32_t LAYOUT = SW == 128 ? 2u : 4u;
    static constexpr uint32_t O_COL = 256;
    // Head dims up to 64 leave TMEM for a P buffer per group beside the scores, so S_g(j+1) is
    // issued as soon as S_g(j) has been read out; at 128 P_g is stored over S_g, S_g(j+1) waits for
    // PV_g(j), and P_g is announced in two halves, so that PV_g starts under the second.
    static constexpr bool AHEAD = D <= 64;
    static constexpr uint32_t P_COL = AHEAD ? O_COL + 128 : 0, P_STEP = AHEAD ? 64 : PC_BN;
    // warps 0-7 softmax; bf16: 8 copies, 9 MMA; e4m3: 8-11 converters, 12 MMA, 13 copies
    static constexpr int WARP_MMA = E4M3 ? 12 : 9;
    static constexpr int WARP_COPY = E4M3 ? 13 : 8;
    static constexpr int THREADS = E4M3 ? 512 : 320;
    // Score columns in a softmax thread's registers at once.  512 threads leave 128 registers
    // each, so the e4m3 kernel reads the second half of a row twice (for its maximum first).
    static constexpr int COLS = E4M3 ? 64 : 128;
    static_assert(O_COL + 2 * D <= 512, "TMEM");
};

enum : int {
    PCB_QFULL = 0, PCB_QEMPTY = 1, PCB_S = 2 /* [2] */, PCB_P = 4 /* [2], then the second halves' */, PCB_O = 8 /* [2] */,
    PCB_READ = 10 /* [2] S_g read out */, PCB_DRAIN = 12,
    PCB_FULL = 13 /* [12] */, PCB_EMPTY = 25 /* [12] */, PCB_SFULL = 37 /* [8] */, PCB_SEMPTY = 45 /* [8] */, PCB_NUM = 53
};

// Keys that query row i of a sequence with n rows and kv keys sees.
__device__ __forceinline__ int keys_seen(int causal, int kv, int n, int i) {
    return causal ? min(kv, max(0, kv - n + i + 1)) : kv;
}

// One (sequence, key head, token tile): `n` units (key tiles, at least one), n_g of them
// for row tile g.
struct ChunkPair {
    int n, ng0, ng1, tok0, ntok0, ntok1, tpt;   // first token (of tile 0), token counts
    __device__ __forceinline__ int tok(int g) const { return tok0 + (g ? tpt : 0); }
    __device__ __forceinline__ int ntok(int g) const { return g ? ntok1 : ntok0; }
};
__device__ __forceinline__ ChunkPair chunk_pair(const PagedParams& p, int n_q, int n_live, int kv, int qt) {
    ChunkPair c;
    c.tpt = p.tpt;
    c.tok0 = qt * 2 * p.tpt;
    c.ntok0 = max(0, min(p.tpt, n_live - c.tok0));
    c.ntok1 = max(0, min(p.tpt, n_live - c.tok0 - p.tpt));
    auto tiles = [&](int tok, int n) { return n > 0 ? (keys_seen(p.causal, kv, n_q, tok + n - 1) + PC_BN - 1) / PC_BN : 0; };
    c.ng0 = tiles(c.tok0, c.ntok0);
    c.ng1 = tiles(c.tok0 + p.tpt, c.ntok1);
    c.n = max(1, max(c.ng0, c.ng1));
    return c;
}
__device__ __forceinline__ int chunk_qtiles(const PagedParams& p, int n_live) { return (n_live + 2 * p.tpt - 1) / (2 * p.tpt); }
// Units of sequence b for one key head.
__device__ __forceinline__ long long chunk_units(const PagedParams& p, int b, bool report) {
    const int n = query_range(p, b, report).n;
    const int kv = paged_kv_len(p.kv_len, b, p.kv_cap, report);
    const int live = min(n, p.max_q), nq = chunk_qtiles(p, live);
    if (!p.causal) return static_cast<long long>(nq) * max(1, (kv + PC_BN - 1) / PC_BN);
    long long sum = 0;
    for (int qt = 0; qt < nq; ++qt)   // what the tile's last row sees
        sum += max(1, (keys_seen(1, kv, n, min((qt + 1) * 2 * p.tpt, live) - 1) + PC_BN - 1) / PC_BN);
    return sum;
}

// Walks a CTA's run of units.  Every role of the CTA walks the same segments.
struct ChunkWalk {
    int b, h, qt, t0, t1;            // key tiles [t0, t1) of the pair
    int n_q, n_live, kv, q0;         // the sequence's rows (all, computed), keys, first row
    long long left;                  // units of the run from t0 on
    ChunkPair c;

    __device__ __forceinline__ void sequence(const PagedParams& p) {
        const QueryRange r = query_range(p, b, false);
        n_q = r.n;
        n_live = min(r.n, p.max_q);
        q0 = r.t0;
        kv = paged_kv_len(p.kv_len, b, p.kv_cap, false);
    }
    __device__ __forceinline__ void segment(const PagedParams& p) {
        c = chunk_pair(p, n_q, n_live, kv, qt);
        t1 = static_cast<int>(min(static_cast<long long>(c.n), t0 + left));
    }
    // At sequence b, `at` units into it, with `left` units to walk.
    __device__ __forceinline__ void begin(const PagedParams& p, int b_, long long at, long long left_) {
        b = b_;
        left = left_;
        sequence(p);
        const long long units = chunk_units(p, b, false);
        h = static_cast<int>(at / units);
        at -= h * units;
        qt = 0;
        c = chunk_pair(p, n_q, n_live, kv, 0);
        while (at >= c.n) {
            at -= c.n;
            c = chunk_pair(p, n_q, n_live, kv, ++qt);
        }
        t0 = static_cast<int>(at);
        segment(p);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == c.n; }
    __device__ __forceinline__ void next(const PagedParams& p) {
        left -= t1 - t0;
        if (left <= 0) return;
        t0 = 0;   // a segment that ends inside its pair ends the run
        if (++qt == chunk_qtiles(p, n_live)) {
            qt = 0;
            if (++h == p.c.Hkv) {
                h = 0;
                do {
                    ++b;
                    sequence(p);
                } while (n_live == 0);   // a later one has rows: left > 0
            }
        }
        segment(p);
    }
    // key tiles of this segment that row tile g takes
    __device__ __forceinline__ int end(int g) const { return min(t1, g ? c.ng1 : c.ng0); }
};

// Block-wide: the run's length, and for CTA blockIdx.x its first sequence and the units into it.
template <int THREADS>
__device__ __forceinline__ long long chunk_deal(const PagedParams& p, int n_ctas, long long first_of, long long* s_scr, bool report,
                                                int* b_out, long long* at_out, long long* all_out) {
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x;
    long long sum = 0;
    for (int b = tid; b < p.B; b += THREADS) sum += chunk_units(p, b, report);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) s_scr[tid >> 5] = sum;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < W; ++w) all += s_scr[w];
    all *= p.c.Hkv;
    const long long per = max(static_cast<long long>(p.min_units), (all + n_ctas - 1) / n_ctas);
    const long long unit = first_of * per;
    __syncthreads();
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + tid;
        const long long n = b < p.B ? chunk_units(p, b, false) : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if ((tid & 31) >= o) incl += t;
        }
        if ((tid & 31) == 31) s_scr[tid >> 5] = incl;
        __syncthreads();
        long long block = 0;
        for (int w = 0; w < W; ++w) {
            if (w < (tid >> 5)) incl += s_scr[w];
            block += s_scr[w];
        }
        incl += base;
        if (n > 0 && (incl - n) * p.c.Hkv <= unit && unit < incl * p.c.Hkv) {
            s_scr[W] = b;
            s_scr[W + 1] = unit - (incl - n) * p.c.Hkv;
        }
        base += block;
        __syncthreads();
    }
    *b_out = static_cast<int>(s_scr[W]);
    *at_out = s_scr[W + 1];
    *all_out = all;
    return per;
}

// Sixteen codes of a row as bf16 values, to two 16-byte chunks (ch, ch + 1 before the swizzle)
// of the row's 128-byte line; lanes with `flip` store the second first, so that a quarter
// warp touches all banks.
__device__ __forceinline__ void store_codes(const uint4& d, uint32_t code, uint8_t* line, int ch, int sw, bool flip) {
    const uint32_t f = scale_factor(code) * 0x10001u;
    const uint32_t wd[4] = {d.x, d.y, d.z, d.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[2 * e] = widen2(__byte_perm(wd[e], 0u, 0x1404), f);
        o[2 * e + 1] = widen2(__byte_perm(wd[e], 0u, 0x3424), f);
    }
    if (code > 134u && code != SCALE_NAN) {   // a scale above 2^7: the rest of it
        const uint32_t f2 = ((code - 7u) << 7) * 0x10001u;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], f2);
    }
    const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
    *reinterpret_cast<uint4*>(line + (((ch + (flip ? 1 : 0)) ^ sw) << 4)) = flip ? hi : lo;
    *reinterpret_cast<uint4*>(line + (((ch + (flip ? 0 : 1)) ^ sw) << 4)) = flip ? lo : hi;
}
// The block table's entry for the keys from `key` on, asked for a tile ahead; nothing looks at
// it (and so waits for the load) before at().
struct PageAsk {
    int entry, key;
    bool wanted;
};
__device__ __forceinline__ PageAsk page_ask(const PagedParams& p, const int32_t* table, int key, bool wanted) {
    PageAsk a = {0, key, wanted};
    if (wanted) a.entry = __ldg(table + page_index(p, key));
    return a;
}
// Its page and row; none: page num_pages (outside the pool), row 0.
struct PageAt {
    int page, row;
};
__device__ __forceinline__ PageAt page_at(const PagedParams& p, const PageAsk& a, bool report) {
    const bool have = a.wanted && a.entry >= 0 && a.entry < p.c.num_pages;
    if (report && a.wanted && !have) atomicOr(&g_paged_status, STATUS_CACHE);
    return {have ? a.entry : p.c.num_pages, have ? a.key - page_index(p, a.key) * p.c.page_size : 0};
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(ChunkCfg<D, E4M3>::THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedParams p, const int n_ctas) {
    using C = ChunkCfg<D, E4M3>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sKV = smem + 2 * C::QT_BYTES;
    uint8_t* sStg = sKV + C::NS * C::SLOT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sStg + C::NSTG * C::STG_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + PCB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    long long* s_scr = reinterpret_cast<long long*>(tmem_holder + 2);   // 18 words of 8 bytes
    const uint32_t bar0 = smem_u32(bars), sQ_addr = smem_u32(smem), sKV_addr = smem_u32(sKV);
#define CBAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    allow_next_kernel();
    int b_first;
    long long at, all;
    const long long per = chunk_deal<C::THREADS>(p, n_ctas, blockIdx.x, s_scr, blockIdx.x == 0, &b_first, &at, &all);
    const long long unit0 = blockIdx.x * per;
    if (unit0 >= all) {
        if (tid == 0) p.shared[blockIdx.x].n = 0;
        return;
    }
    const long long run = min(per, all - unit0);

    if (tid == 0) {
        mbar_init(CBAR(PCB_QFULL), 1);
        mbar_init(CBAR(PCB_QEMPTY), 1);
        mbar_init(CBAR(PCB_DRAIN), 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(CBAR(PCB_S + g), 1);
            mbar_init(CBAR(PCB_P + g), 4);
            mbar_init(CBAR(PCB_P + 2 + g), 4);
            mbar_init(CBAR(PCB_READ + g), 4);
            mbar_init(CBAR(PCB_O + g), 1);
        }
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(CBAR(PCB_FULL + s), E4M3 ? 4 : 1);
            mbar_init(CBAR(PCB_EMPTY + s), 1);
        }
        for (int s = 0; s < C::NSTG; ++s) {
            mbar_init(CBAR(PCB_SFULL + s), 33);    // the byte count's, and every copying lane's scale bytes
            mbar_init(CBAR(PCB_SEMPTY + s), 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const unsigned long long wlim = p.wait_ns;
    ChunkWalk w;
    if (warp < 8) {
        // ================================================================ softmax and epilogue
        const int g = warp >> 2, r = tid & 127;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + static_cast<uint32_t>(g) * PC_BN;
        const uint32_t o_addr = tmem + lane_base + C::O_COL + static_cast<uint32_t>(g) * D;
        const uint32_t p_addr = tmem + lane_base + C::P_COL + static_cast<uint32_t>(g) * C::P_STEP;
        const float sl2 = p.scale_log2;
        const bool pos_scale = sl2 > 0.0f;
        const float mul = pos_scale ? sl2 : 1.0f;
        const int r_tok = r / p.G, r_head = r - r_tok * p.G;
        uint32_t cnt = 0, o_phase = 0;   // tiles of this group, over all segments
        bool ok = true;
        auto arrive = [&](uint32_t bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        for (w.begin(p, b_first, at, run); w.more() && ok; w.next(p)) {
            const bool live = r_tok < w.c.ntok(g) && r_tok < p.tpt;
            const int i = w.c.tok(g) + r_tok;
            const int seen = live ? keys_seen(p.causal, w.kv, w.n_q, i) : 0;
            const int all_seen = keys_seen(p.causal, w.kv, w.n_q, w.c.tok(g));   // by every live row of the tile
            float m_ref = -INFINITY, l_sum = 0.0f;
            const int j1 = w.end(g);
#pragma unroll 1
            for (int j = w.t0; j < j1; ++j) {
                ok = chunk_wait_warp(CBAR(PCB_S + g), cnt & 1u, abort_flag, wlim);
                if (!ok) break;
                tc_fence_after();
                float x[C::COLS];
                // columns [c0, c0 + COLS) of the row, masked by selection
                auto load = [&](int c0) {
                    uint32_t raw[C::COLS];
                    if constexpr (C::COLS == 128) tmem_ld128_wait(s_addr, raw);
                    else tmem_ld64_wait(s_addr + c0, raw);
                    if ((j + 1) * PC_BN > all_seen) {
                        const int lim = seen - j * PC_BN - c0;   // columns this row sees
#pragma unroll
                        for (int c = 0; c < C::COLS; ++c) x[c] = c < lim ? __uint_as_float(raw[c]) * (pos_scale ? 1.0f : sl2) : -INFINITY;
                    } else if (pos_scale) {
#pragma unroll
                        for (int c = 0; c < C::COLS; ++c) x[c] = __uint_as_float(raw[c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < C::COLS; ++c) x[c] = __uint_as_float(raw[c]) * sl2;
                    }
                };
                float mx = -INFINITY;
#pragma unroll
                for (int c0 = PC_BN - C::COLS; c0 >= 0; c0 -= C::COLS) {
                    load(c0);
                    mx = fmaxf(mx, row_max(x));
                }
                mx *= mul;
                if constexpr (C::AHEAD) {
                    if constexpr (C::COLS == PC_BN) arrive(CBAR(PCB_READ + g));
                    // PV of the tile before has read P_g and added to O_g
                    ok = cnt == 0 || chunk_wait_warp(CBAR(PCB_O + g), (cnt - 1) & 1u, abort_flag, wlim);
                    if (!ok) break;
                    tc_fence_after();
                }
                float factor = 1.0f;
                if (j == w.t0) {
                    m_ref = mx;
                } else if (__any_sync(0xffffffffu, mx > m_ref + PC_RESCALE_LOG2)) {
                    const float m_new = fmaxf(m_ref, mx);
                    factor = m_ref == -INFINITY ? 0.0f : exp2_approx(m_ref - m_new);
                    m_ref = m_new;
#pragma unroll 1
                    for (int oc = 0; oc < D / 32; ++oc) {
                        uint32_t o[32];
                        tmem_ld32_wait(o_addr + oc * 32, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                        tmem_st32(o_addr + oc * 32, o);
                    }
                }
                const float neg_m = m_ref == -INFINITY ? 0.0f : -m_ref;   // a row with no key so far: 2^-inf, not NaN
                float2 sp[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) sp[t] = make_float2(0.0f, 0.0f);
                const float2 mul2 = make_float2(mul, mul), neg2 = make_float2(neg_m, neg_m);
#pragma unroll
                for (int cc = 0; cc < PC_BN / 32; ++cc) {
                    constexpr int PER = C::COLS / 32;
                    if (cc != 0 && cc % PER == 0) {
                        load(cc * 32);
                        if constexpr (C::AHEAD) arrive(CBAR(PCB_READ + g));
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = fma2(make_float2(x[cc % PER * 32 + 2 * e], x[cc % PER * 32 + 2 * e + 1]), mul2, neg2);
                        const float p0 = exp2_approx(y.x), p1 = exp2_approx(y.y);
                        sp[e & 3] = add2(sp[e & 3], make_float2(p0, p1));   // the sum takes the weights unrounded
                        pk[e] = pack_bf16(p0, p1);
                    }
                    tmem_st16(p_addr + cc * 16, pk);
                    if (!C::AHEAD && cc == 1) {                             // the first 64 keys' weights
                        tmem_wait_st();
                        arrive(CBAR(PCB_P + g));
                    }
                }
                tmem_wait_st();
                arrive(CBAR(PCB_P + (C::AHEAD ? 0 : 2) + g));
                l_sum = l_sum * factor + (((sp[0].x + sp[1].x) + (sp[2].x + sp[3].x)) + ((sp[0].y + sp[1].y) + (sp[2].y + sp[3].y)));
                ++cnt;
            }
            if (!ok) break;
            const bool has = j1 > w.t0;
            if (has) {
                // D <= 64: one phase per PV; 128: one per segment
                ok = chunk_wait_warp(CBAR(PCB_O + g), C::AHEAD ? (cnt - 1) & 1u : o_phase, abort_flag, wlim);
                if (!ok) break;
                o_phase ^= 1u;
                tc_fence_after();
            }
            const bool some = !(l_sum == 0.0f);   // NaN counts
            const float inv = some ? 1.0f / l_sum : 0.0f;
            const float lse = some ? (m_ref + log2f(l_sum)) * 0.69314718055994530942f : -INFINITY;
            const bool whole = w.whole();
            const long long row = static_cast<long long>(w.q0) + i;
            const int hq = w.h * p.G + r_head;
            const long long part = ((2LL * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * 2 + g) * 128 + r;
#pragma unroll 1
            for (int oc = 0; oc < D / 32; ++oc) {
                uint32_t o[32];
                if (has) {
                    tmem_ld32_wait(o_addr + oc * 32, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (!live) continue;
                if (whole) {
                    __nv_bfloat16* dst = p.out + row * p.out_t + hq * p.out_h + oc * 32;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint4 v;
                        v.x = pack_bf16(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                        v.y = pack_bf16(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                        v.z = pack_bf16(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                        v.w = pack_bf16(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                        *reinterpret_cast<uint4*>(dst + e) = v;
                    }
                } else if (some) {
                    float* dst = p.part_out + part * D + oc * 32;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(dst + e) = make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                                                          __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                }
            }
            if (live) {
                if (!whole) p.part_lse[part] = lse;
                else if (p.lse != nullptr) p.lse[row * p.Hq + hq] = lse;
            }
            tc_fence_before();   // the reads of O_g above, before the next segment's first P
        }
    } else if (warp == C::WARP_MMA) {
        // ================================================================ MMA issuer
        // The whole warp runs converged; its elected lane issues.
        constexpr uint32_t IDESC_S = make_idesc_bf16(128, PC_BN, false);
        constexpr uint32_t IDESC_PV = make_idesc_bf16(128, D, true);
        const uint64_t q_desc0 = make_smem_desc(sQ_addr, 16, 8 * C::SW, C::LAYOUT);
        const uint64_t k_desc0 = make_smem_desc(sKV_addr, 16, C::GROUP, C::LAYOUT);
        const uint64_t v_desc0 = make_smem_desc(sKV_addr, 8 * C::SW, C::GROUP, C::LAYOUT);
        int k_slot = 0, v_slot = 0;
        uint32_t item = 0;                       // ring items consumed: K_t0, then V_j, K_{j+1}
        uint32_t p_phase[2] = {0, 0}, r_phase[2] = {0, 0}, q_phase = 0;
        bool ok = true;
        auto next_item = [&]() -> int {          // waits for the next K or V tile; its slot
            const int slot = static_cast<int>(item % C::NS);
            ok = ok && chunk_wait_warp(CBAR(PCB_FULL + slot), (item / C::NS) & 1u, abort_flag, wlim);
            ++item;
            tc_fence_after();
            return slot;
        };
        auto issue_s = [&](int g) {
            const uint64_t kd = k_desc0 + static_cast<uint64_t>(k_slot) * (C::SLOT >> 4);
            const uint64_t qd = q_desc0 + static_cast<uint64_t>(g) * (C::QT_BYTES >> 4);
            const uint32_t d = tmem + static_cast<uint32_t>(g) * PC_BN;
            if constexpr (C::BLK == 64) {
#pragma unroll
                for (int c = 0; c < C::NBLK; ++c)
                    mma_ss_elect_x4<2, 2>(d, qd + static_cast<uint64_t>((c * 128 * C::SW) >> 4), kd + static_cast<uint64_t>((c * 8 * C::SW) >> 4), IDESC_S, c != 0 ? 1u : 0u);
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) mma_ss_elect(d, qd + 2 * t, kd + 2 * t, IDESC_S, t != 0 ? 1u : 0u);
            }
            tc_commit_elect(CBAR(PCB_S + g));
        };
        auto issue_pv = [&](int g, bool first, int kb0, int kb1) {   // 16-key steps [kb0, kb1)
            const uint64_t vd = v_desc0 + static_cast<uint64_t>(v_slot) * (C::SLOT >> 4);
#pragma unroll
            for (int kb = kb0; kb < kb1; kb += 4)
                mma_ts_elect_x4<8, (2 * C::GROUP) / 16>(tmem + C::O_COL + static_cast<uint32_t>(g) * D, tmem + C::P_COL + static_cast<uint32_t>(g) * C::P_STEP + kb * 8u,
                                                        vd + static_cast<uint64_t>((kb * 2 * C::GROUP) >> 4), IDESC_PV, kb == 0 && first ? 0u : 1u);
        };
        for (w.begin(p, b_first, at, run); w.more() && ok; w.next(p)) {
            const int e0 = w.end(0), e1 = w.end(1), je = max(e0, e1);
            if (je <= w.t0) continue;            // no keys: nothing was loaded
            ok = chunk_wait_warp(CBAR(PCB_QFULL), q_phase, abort_flag, wlim);
            q_phase ^= 1u;
            if (!ok) break;
            k_slot = next_item();
            if (!ok) break;
            if (w.t0 < e0) issue_s(0);
            if (w.t0 < e1) issue_s(1);
            tc_commit_elect(CBAR(PCB_EMPTY + k_slot));
            if (w.t0 + 1 == je) tc_commit_elect(CBAR(PCB_QEMPTY));   // the segment's last S: Q may be replaced
#pragma unroll 1
            for (int j = w.t0; j < je && ok; ++j) {
                v_slot = next_item();
                if (!ok) break;
                if constexpr (!E4M3) {
                    // rows of the last copied box that lie behind the sequence: cleared, since
                    // 0 * NaN would reach every row
                    const int valid = w.kv - j * PC_BN;
                    const int dirty = valid < PC_BN ? (valid + p.box_rows - 1) / p.box_rows * p.box_rows : 0;
                    if (valid < dirty) {
                        constexpr int CH = C::SW / 16;
                        for (int x = lane; x < (dirty - valid) * CH * C::NBLK; x += 32) {
                            const int blk = x / ((dirty - valid) * CH), y = x % ((dirty - valid) * CH);
                            const int r = valid + y / CH;
                            *reinterpret_cast<uint4*>(sKV + v_slot * C::SLOT + (r >> 3) * C::GROUP + blk * (8 * C::SW) + (r & 7) * C::SW + y % CH * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                        __syncwarp();
                    }
                }
                const bool more = j + 1 < je;
                if (more) k_slot = next_item();      // ahead of the waits for P
                if (!ok) break;
                auto arrived = [&](int bar, uint32_t phase) {
                    ok = ok && chunk_wait_warp(CBAR(bar), phase, abort_flag, wlim);
                    tc_fence_after();
                    return ok;
                };
                if constexpr (C::AHEAD) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (j >= (g ? e1 : e0) || !arrived(PCB_READ + g, r_phase[g])) continue;
                        r_phase[g] ^= 1u;
                        if (j + 1 < (g ? e1 : e0)) issue_s(g);
                    }
                    if (!ok) break;
                    if (more) tc_commit_elect(CBAR(PCB_EMPTY + k_slot));
                    if (j + 2 == je) tc_commit_elect(CBAR(PCB_QEMPTY));
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int eg = g ? e1 : e0;
                    if (j < eg) {
                        if (!arrived(PCB_P + g, p_phase[g])) break;
                        if constexpr (C::AHEAD) {
                            issue_pv(g, j == w.t0, 0, PC_BN / 16);
                            tc_commit_elect(CBAR(PCB_O + g));
                        } else {
                            issue_pv(g, j == w.t0, 0, PC_BN / 32);
                            if (!arrived(PCB_P + 2 + g, p_phase[g])) break;
                            issue_pv(g, false, PC_BN / 32, PC_BN / 16);
                            if (j + 1 == eg) tc_commit_elect(CBAR(PCB_O + g));
                        }
                        p_phase[g] ^= 1u;
                    }
                    if (!C::AHEAD && j + 1 < eg) issue_s(g);
                }
                if (!ok) break;
                tc_commit_elect(CBAR(PCB_EMPTY + v_slot));
                if (!C::AHEAD && more) tc_commit_elect(CBAR(PCB_EMPTY + k_slot));
                if (!C::AHEAD && j + 2 == je) tc_commit_elect(CBAR(PCB_QEMPTY));
            }
        }
        // every MMA issued completes before TMEM is released
        tc_commit_elect(CBAR(PCB_DRAIN));
        __syncwarp();
        const uint64_t d0 = global_timer_ns();
        while (!mbar_try_wait(CBAR(PCB_DRAIN), 0)) {
            if (global_timer_ns() - d0 > wlim) {
                atomicOr(&g_paged_status, STATUS_TIMEOUT);
                break;
            }
        }
        __syncwarp();
    } else if (warp == C::WARP_COPY) {
        // ================================================================ copies: Q, K, V
        if (lane == 0) {
            tma_prefetch_map(&tm_q);
            tma_prefetch_map(&tm_k);
            tma_prefetch_map(&tm_v);
        }
        uint32_t item = 0, qe_phase = 0;
        bool ok = true, first = true;
        const int boxes = PC_BN / p.box_rows;
        w.begin(p, b_first, at, run);
        if (lane == 0) p.shared[blockIdx.x] = {w.b, w.h, w.qt, w.t0, w.t0 > 0 ? w.c.n : 0, 0, per};
        constexpr int N = E4M3 ? C::NSTG : C::NS;          // the slots that are filled here
        constexpr int FULL = E4M3 ? PCB_SFULL : PCB_FULL, EMPTY = E4M3 ? PCB_SEMPTY : PCB_EMPTY;
        for (w.begin(p, b_first, at, run); w.more() && ok; w.next(p)) {
            const int je = max(w.end(0), w.end(1));
            if (je <= w.t0) continue;
            if (!first) {
                ok = chunk_wait_warp(CBAR(PCB_QEMPTY), qe_phase, abort_flag, wlim);
                qe_phase ^= 1u;
                if (!ok) break;
            }
            first = false;
            if (lane == 0) {
                const bool both = w.c.ntok1 > 0;
                mbar_arrive_expect_tx(CBAR(PCB_QFULL), (both ? 2 : 1) * p.tpt * p.G * D * 2);
                for (int g = 0; g < (both ? 2 : 1); ++g)
#pragma unroll
                    for (int c = 0; c < C::NBLK; ++c)
                        tma_load_4d(sQ_addr + g * C::QT_BYTES + c * 128 * C::SW, &tm_q, c * C::BLK, 0, w.h, w.q0 + w.c.tok(g), CBAR(PCB_QFULL));
            }
            // lane i < boxes copies box i of a tile (all lanes at once: one lane issuing them in
            // turn took 20 % longer with 16-row pages); its page is looked up one tile ahead
            const int32_t* table = p.table + w.b * p.table_stride;
            auto lookup = [&](int j) {
                const int key = j * PC_BN + lane * p.box_rows;
                return page_ask(p, table, key, lane < boxes && j < je && key < w.kv);
            };
            auto lookup_scale = [&](int j) {               // e4m3: lane's group of 8 rows
                const int key = j * PC_BN + (lane & 15) * 8;
                return page_ask(p, table, key, E4M3 && j < je && key < w.kv);
            };
            PageAsk ask = lookup(w.t0), scale_ask = lookup_scale(w.t0);
            for (int j = w.t0; j < je && ok; ++j) {
                const PageAt a = page_at(p, ask, true), sa = page_at(p, scale_ask, false);
                ask = lookup(j + 1);
                scale_ask = lookup_scale(j + 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = static_cast<int>(item % N);
                    ok = chunk_wait_warp(CBAR(EMPTY + slot), ((item / N) & 1u) ^ 1u, abort_flag, wlim);
                    if (!ok) break;
                    ++item;
                    if (lane == 0) mbar_arrive_expect_tx(CBAR(FULL + slot), E4M3 ? PC_BN * D : C::SLOT);
                    __syncwarp();
                    const bool drop = (p.debug & ATTN_DEBUG_DROP_COPY) && kv == 0 && j == w.t0 && lane == 0;
                    if constexpr (E4M3) {
                        const uint32_t dst = smem_u32(sStg) + slot * C::STG_BYTES;
                        if (lane < boxes && !drop) tma_load_4d(dst + lane * p.box_rows * D, kv ? &tm_v : &tm_k, 0, a.row, w.h, a.page, CBAR(FULL + slot));
                        if (lane < 16) {
                            const bool have = sa.page < p.c.num_pages;
                            const uint8_t* src = p.c.scale[kv];
                            if (have) src += (static_cast<long long>(sa.page) * p.c.Hkv + w.h) * p.c.page_size + sa.row;
                            cp_async8(dst + PC_BN * D + lane * 8, src, have);
                        }
                        cp_async_mbar_arrive_noinc(CBAR(FULL + slot));
                    } else {
                        if (lane < boxes && !drop)
                            tma_load_5d(sKV_addr + slot * C::SLOT + lane * (p.box_rows / 8) * C::GROUP, kv ? &tm_v : &tm_k, 0, 0, w.h * p.head_units[kv],
                                        a.row / 8, a.page, CBAR(FULL + slot));
                    }
                    __syncwarp();
                }
            }
        }
        if (*abort_flag || !ok) {
            // Copies in flight must land before the memory is reused; they have no one to wait for them.
            const uint64_t d0 = global_timer_ns();
            while (global_timer_ns() - d0 < 2000000ull) {
            }
        }
        __syncwarp();
    } else if (E4M3 && warp < 12) {
        // ================================================================ converters: e4m3 K and V
        if constexpr (E4M3) {
            constexpr int CPR = D / 16;          // 16-code chunks per row
            constexpr int X = CPR;               // chunks per thread: 128 rows * CPR / 128 threads
            constexpr int RPX = 128 / CPR;       // rows between a thread's chunks
            const int t = tid - 256;
            const int r0 = t / CPR, c16 = t % CPR;
            const int blk = c16 * 16 / C::BLK, ch = c16 * 16 % C::BLK / 8;
            uint32_t item = 0;
            bool ok = true;
            for (w.begin(p, b_first, at, run); w.more() && ok; w.next(p)) {
                const int je = max(w.end(0), w.end(1));
                for (int j2 = 2 * w.t0; j2 < 2 * je && ok; ++j2) {   // item: tile j2 / 2, K or V
                    const int slot = static_cast<int>(item % C::NS), stg = static_cast<int>(item % C::NSTG);
                    ok = chunk_wait_warp(CBAR(PCB_SFULL + stg), (item / C::NSTG) & 1u, abort_flag, wlim) &&
                         chunk_wait_warp(CBAR(PCB_EMPTY + slot), ((item / C::NS) & 1u) ^ 1u, abort_flag, wlim);
                    if (!ok) break;
                    ++item;
                    const int left = w.kv - (j2 >> 1) * PC_BN;       // rows of the tile that exist
                    const uint8_t* src = sStg + stg * C::STG_BYTES;
                    uint8_t* dst = sKV + slot * C::SLOT + blk * (8 * C::SW);
                    // All of a thread's codes first: a load behind a store to shared memory would wait for it.
                    uint4 d[X];
                    uint32_t code[X];
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        const int r = x * RPX + r0;
                        d[x] = *reinterpret_cast<const uint4*>(src + r * D + c16 * 16);
                        code[x] = src[PC_BN * D + r];
                    }
                    if (left < PC_BN) {                              // a page's rows behind the sequence
#pragma unroll
                        for (int x = 0; x < X; ++x)
                            if (x * RPX + r0 >= left) {
                                d[x] = make_uint4(0u, 0u, 0u, 0u);
                                code[x] = 127u;
                            }
                    }
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        const int r = x * RPX + r0;
                        store_codes(d[x], code[x], dst + (r >> 3) * C::GROUP + (r & 7) * C::SW, ch, C::SW == 128 ? r & 7 : (r >> 1) & 3, blk & 1);
                    }
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(CBAR(PCB_FULL + slot));
                        mbar_arrive(CBAR(PCB_SEMPTY + stg));
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
#undef CBAR
}

// Token tiles that several CTAs of paged_chunk_kernel shared.  Block c (x) looks at the border
// between the runs of CTAs c and c + 1; the first border inside a tile puts the tile together, its
// rows spread over blockIdx.y, one warp a row.  CTA c's part is slot 2c, or 2c + 1 where the
// tile begins in its run.
template <int D>
__global__ void __launch_bounds__(256) paged_chunk_combine_kernel(const PagedParams p) {
    wait_for_main_kernel();                     // every block, so that this grid never ends before that one
    const SharedAt s = p.shared[blockIdx.x + 1];
    if (s.n == 0) return;                       // the border lies between two tiles
    const long long u0 = (blockIdx.x + 1) * s.per - s.t0;   // the tile's first unit
    const long long c0 = u0 / s.per, c1 = (u0 + s.n - 1) / s.per;
    if (c0 != blockIdx.x) return;
    const QueryRange qr = query_range(p, s.b, false);
    const int n_live = min(qr.n, p.max_q), tok0 = s.qt * 2 * p.tpt;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int V = D >= 128 ? 4 : D / 32, NV = D / (32 * V);   // floats per load, loads per lane
    for (int r = blockIdx.y * 8 + warp; r < 256; r += gridDim.y * 8) {
        const int g = r >> 7, rr = r & 127, tok = rr / p.G;
        const int i = tok0 + g * p.tpt + tok;
        if (tok >= p.tpt || i >= n_live) continue;
        auto slot = [&](long long cc) { return ((2 * cc + (cc == c0 ? 1 : 0)) * 2 + g) * 128 + rr; };
        float M = -INFINITY;
#pragma unroll 4
        for (long long cc = c0; cc <= c1; ++cc) M = fmaxf(M, __ldcg(p.part_lse + slot(cc)));
        float sum = 0.0f, acc[NV * V];
#pragma unroll
        for (int e = 0; e < NV * V; ++e) acc[e] = 0.0f;
#pragma unroll 2
        for (long long cc = c0; cc <= c1; ++cc) {
            const float lc = __ldcg(p.part_lse + slot(cc));
            if (lc == -INFINITY) continue;      // nothing was stored
            const float wgt = expf(lc - M);
            sum += wgt;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const float* src = p.part_out + slot(cc) * D + n * 32 * V + lane * V;
                float v[V];
                if constexpr (V == 4) *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(src));
                else if constexpr (V == 2) *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(src));
                else v[0] = __ldcg(src);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[n * V + e] += wgt * v[e];
            }
        }
        const bool some = !(sum == 0.0f);
        const float inv = some ? 1.0f / sum : 0.0f;
        const long long row = static_cast<long long>(qr.t0) + i;
        const int hq = s.h * p.G + rr - tok * p.G;
        __nv_bfloat16* dst = p.out + row * p.out_t + hq * p.out_h;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            __nv_bfloat16* d = dst + n * 32 * V + lane * V;
            if constexpr (V == 4)
                *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16(acc[n * V] * inv, acc[n * V + 1] * inv), pack_bf16(acc[n * V + 2] * inv, acc[n * V + 3] * inv));
            else if constexpr (V == 2)
                *reinterpret_cast<uint32_t*>(d) = pack_bf16(acc[0] * inv, acc[1] * inv);
            else
                *d = __float2bfloat16_rn(acc[0] * inv);
        }
        if (lane == 0 && p.lse != nullptr) p.lse[row * p.Hq + hq] = some ? M + logf(sum) : -INFINITY;
    }
}
