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
// The work is (sequence, key head, token tile) pairs of n key tiles each, dealt to one persistent
// CTA per SM so that every run has the same number of key tiles: run c takes pairs c, c + C,
// c + 2C, ... up to its share; what its pairs have beyond that goes to a pool, in order, which
// the runs whose pairs fall short share out.  So ragged batches and causal triangles leave
// no SM idle, while nearly every pair starts at its first key tile when its neighbours, the other
// token tiles of the same head, do: they read the same K and V at the same time, from L2.
// (Cutting the pairs laid end to end into equal runs balances as well, but each run then
// reads another place of the keys: 1185 against 1670 TFLOP/s at 2368 and 9472 rows on
// 65536 keys, D 256, from L2 misses and the power they cost.)  Pairs worked on by several
// CTAs are put together by paged_chunk_combine_kernel.
//
// K and V are copied by TMA, in boxes of the largest power of two of rows (up to 128) that divides
// the page size, each box from its page; a box behind the sequence or of a page that does
// not exist has its page coordinate outside the pool and reads as zeros.  Small pages make
// many boxes, and what one warp can issue bounds them, so a bf16 box holds all columns of its
// rows: the tensor map splits a page into groups of 8 rows, and a tile lies in shared memory
// as [8-row group][64-column block][8 rows][128 bytes], which the MMA descriptors address by
// their two strides.  The rows of the last box behind the sequence are cleared in shared
// memory before PV reads them.  e4m3 tiles land in staging slots instead, with their
// scale bytes by cp.async; converter warps widen them to bf16 (exactly, see paged_rows.cuh) into
// the same layout.  Softmax, converters, copies and MMAs then run five instruction streams
// on an SM, and their code is kept small, by rolled loops: in its unrolled form the kernel waited for
// instructions (1385 against 1145 us, 2048 causal rows on 32768 keys, 32 heads on 8, D 128).  (Loading the codes straight into the converters' registers, one tile
// ahead, left them waiting for loads: 476 against 1061 TFLOP/s with the loads taken out, 2048 rows
// on 32768 keys, 32 heads on 8, D 128.)
//
// What bounds it, measured.  D 64: the softmax (the exponential unit is 63 % busy; 8192 rows on 16384
// keys, 8 heads: 472 us, 582 TFLOP/s, the dense kernel 424 us, whose softmax, unlike this one, does not spill:
// 168 registers a thread for ten warps).  D 128: the tensor pipe and shared
// memory, and power in long runs (2048 causal rows on 32768 keys, 32 heads on 8: 860 to 873 us, 1.2 PFLOP/s).
// e4m3: the converters' ALU work beside the softmax (the same chunk 1180 us, 3 % of it to find codes
// of NaN; at D 64, 16 sequences of 256 rows on 4096 keys, 167 us against 147 with bf16 pages).  A change of segment costs about 4 us: the
// pipeline of S, softmax and PV drains and fills again.  (Copying a segment's first tiles before its Q
// had room did not shorten that.)
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
    static constexpr int CTRL = 2048;                   // barriers, TMEM address, abort flag, the deal
    static constexpr int GROUP = NBLK * 8 * SW;         // one 8-row group of a K or V tile
    // e4m3: staged codes of a tile, and its 128 scale bytes
    static constexpr int STG_BYTES = PC_BN * D + 128;
    static constexpr int NSTG = E4M3 ? (D == 128 ? 4 : 8) : 0;
    static constexpr int NS_FIT = (232448 - CTRL - 2 * QT_BYTES - NSTG * STG_BYTES) / SLOT;
    static constexpr int NS = NS_FIT < 12 ? NS_FIT : 12;
    static constexpr int SMEM = 2 * QT_BYTES + NS * SLOT + NSTG * STG_BYTES + CTRL;
    static_assert(NS >= 3, "ring depth");
    static constexpr uint32_t LAYOUT = SW == 128 ? 2u : 4u;
    static constexpr uint32_t O_COL = 256;
    // Head dims up to 64 leave TMEM for a P buffer per group beside the scores, so S_g(j+1) is
    // issued as soon as S_g(j) has been read out; at 128 P_g is stored over S_g, S_g(j+1) waits for
    // PV_g(j), and P_g is announced in two halves, so that PV_g starts under the second.
    static constexpr bool AHEAD = D <= 64;
    static constexpr uint32_t P_COL = AHEAD ? O_COL + 128 : 0, P_STEP = AHEAD ? 64 : PC_BN;
    // warps 0-7 softmax; bf16: 8 copies, 9 MMA; e4m3: NCONV converters from 8 on, then MMA and copies
    // (two converters keep up at 32 dims: 305 -> 277 us at 1200 rows on 30000 keys; at 64: 515 -> 604 us)
    static constexpr int NCONV = !E4M3 ? 0 : D == 32 ? 2 : 4;
    static constexpr int WARP_MMA = E4M3 ? 8 + NCONV : 9;
    static constexpr int WARP_COPY = E4M3 ? 9 + NCONV : 8;
    static constexpr int THREADS = !E4M3 ? 320 : D == 32 ? 384 : 512;
    // Score columns in a softmax thread's registers at once.  512 threads leave 128 registers
    // each, so the e4m3 kernels with four converters read the second half of a row twice (for its maximum first).
    static constexpr int COLS = THREADS == 512 ? 64 : 128;
    static_assert(O_COL + 2 * D <= 512, "TMEM");
};

enum : int {
    PCB_QFULL = 0, PCB_QEMPTY = 1, PCB_S = 2 /* [2] */, PCB_P = 4 /* [2], then the second halves' */, PCB_O = 8 /* [2] */,
    PCB_READ = 10 /* [2] S_g read out */, PCB_DRAIN = 12,
    PCB_FULL = 13 /* [12] */, PCB_EMPTY = 25 /* [12] */, PCB_SFULL = 37 /* [8] */, PCB_SEMPTY = 45 /* [8] */,
    PCB_GFULL = 53 /* [4] segments */, PCB_GEMPTY = 57 /* [4] */, PCB_NUM = 61
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
    auto tiles = [&](int tok, int n) { return n > 0 ? tiles_of(keys_seen(p.causal, kv, n_q, tok + n - 1), PC_BN) : 0; };
    c.ng0 = tiles(c.tok0, c.ntok0);
    c.ng1 = tiles(c.tok0 + p.tpt, c.ntok1);
    c.n = max(1, max(c.ng0, c.ng1));
    return c;
}
__device__ __forceinline__ int chunk_qtiles(const PagedParams& p, int n_live) { return (n_live + 2 * p.tpt - 1) / (2 * p.tpt); }

// A pair by its number, counted over sequences, key heads and token tiles (fastest).  Used by a
// converged warp, whose lanes hold 32 sequences at a time: steps inside those read nothing.
struct PairSeek {
    int b, nq;                       // sequence and its token tiles
    int n_q, n_live, kv, q0;         // its rows (all, computed), keys, first row
    long long base;                  // pairs of the sequences before it
    int w_b;                         // first of the 32 sequences
    long long w_base, w_end;         // pairs before them, and with them
    int l_n, l_q0, l_kv, l_nq;       // this lane's sequence
    long long l_base;                // pairs before it
    __device__ __forceinline__ void window(const PagedParams& p, int first, long long pairs_before) {
        const int lane = threadIdx.x & 31, mine = first + lane;
        w_b = first;
        w_base = pairs_before;
        l_n = l_q0 = l_kv = l_nq = 0;
        if (mine < p.B) {
            const QueryRange r = query_range(p, mine, false);
            l_n = r.n;
            l_q0 = r.t0;
            l_kv = paged_kv_len(p.kv_len, mine, p.kv_cap, false);
            l_nq = chunk_qtiles(p, min(r.n, p.max_q));
        }
        const long long pairs = static_cast<long long>(l_nq) * p.c.Hkv;
        long long incl = pairs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        l_base = w_base + incl - pairs;
        w_end = w_base + __shfl_sync(0xffffffffu, incl, 31);
    }
    __device__ __forceinline__ void begin(const PagedParams& p) { window(p, 0, 0); }
    // To pair idx (there is one).
    __device__ __forceinline__ void to(const PagedParams& p, long long idx) {
        bool back = idx < w_base;
        while (back || (idx >= w_end && w_b + 32 < p.B)) {
            window(p, back ? 0 : w_b + 32, back ? 0 : w_end);
            back = false;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, l_base <= idx && idx < l_base + static_cast<long long>(l_nq) * p.c.Hkv);
        const int l = __ffs(hit | 0x80000000u) - 1;
        b = w_b + l;
        base = __shfl_sync(0xffffffffu, l_base, l);
        nq = __shfl_sync(0xffffffffu, l_nq, l);
        n_q = __shfl_sync(0xffffffffu, l_n, l);
        q0 = __shfl_sync(0xffffffffu, l_q0, l);
        kv = __shfl_sync(0xffffffffu, l_kv, l);
        n_live = min(n_q, p.max_q);
    }
};

// The deal (in shared memory): C runs of T units (key tiles); run c's pairs exceed T by E[c+1] - E[c]
// units, which are [E[c], E[c+1]) of the pool, and fall short of it by D[c+1] - D[c]: it takes
// [D[c], D[c+1]) of the pool, as far as there is one.  Pairs and units are counted in 32 bits: work of
// PC_MAX_UNITS or more (seconds of it) is refused, with the range flag.
constexpr int PC_MAX_RUNS = 148;
constexpr unsigned long long PC_MAX_UNITS = 1ull << 31;
struct ChunkDeal {
    uint32_t E[PC_MAX_RUNS + 1], D[PC_MAX_RUNS + 1];
    uint32_t scan[2][8];
    uint32_t T, total, over;         // units per run, all units; too many
};
// Block-wide, at least PC_MAX_RUNS threads.  scratch: shared memory for `cap` sequences at a time,
// {pairs before it, rows, keys, token tiles}.
__device__ __forceinline__ void chunk_deal(const PagedParams& p, int C, ChunkDeal* s, int4* scratch, int cap) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long load = 0;     // key tiles of run tid's pairs
    uint32_t before = 0;             // pairs of the sequences before this batch
    if (tid == 0) s->over = 0u;
    for (int b0 = 0; b0 < p.B; b0 += cap) {
        const int nb = min(cap, p.B - b0);
        for (int i = tid; i < nb; i += blockDim.x) {
            const bool report = blockIdx.x == 0;   // one block reports ranges out of bounds
            const int n = query_range(p, b0 + i, report).n;
            scratch[i] = make_int4(0, n, paged_kv_len(p.kv_len, b0 + i, p.kv_cap, report), chunk_qtiles(p, min(n, p.max_q)));
        }
        __syncthreads();
        if (warp == 0) {
            unsigned long long carry = 0;
            for (int i0 = 0; i0 < nb; i0 += 32) {
                const unsigned long long v = i0 + lane < nb ? static_cast<unsigned long long>(scratch[i0 + lane].w) * p.c.Hkv : 0ull;
                unsigned long long incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += t;
                }
                if (i0 + lane < nb) scratch[i0 + lane].x = static_cast<int>(carry + incl - v);
                carry += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) {
                if (before + carry >= PC_MAX_UNITS) s->over = 1u;
                s->total = static_cast<uint32_t>(carry);
            }
        }
        __syncthreads();
        if (s->over) break;
        const uint32_t pairs = s->total;
        if (tid < C) {
            int i = 0;
            for (uint32_t l = (static_cast<uint32_t>(tid) + C - before % C) % C; l < pairs; l += C) {
                while (l >= static_cast<uint32_t>(scratch[i].x) + static_cast<uint32_t>(scratch[i].w) * p.c.Hkv) ++i;
                const int4 q = scratch[i];
                load += chunk_pair(p, q.y, min(q.y, p.max_q), q.z, static_cast<int>((l - static_cast<uint32_t>(q.x)) % static_cast<uint32_t>(q.w))).n;
            }
        }
        before += pairs;
        __syncthreads();
    }
    const bool mine_over = load >= PC_MAX_UNITS;
    unsigned long long sum = load;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const bool over = __syncthreads_or(s->over || mine_over || sum >= PC_MAX_UNITS) != 0;
    if (lane == 0 && warp < 5) s->scan[0][warp] = static_cast<uint32_t>(sum);
    __syncthreads();
    uint32_t total = 0;
    unsigned long long total64 = 0;
    for (int w = 0; w < 5; ++w) total64 += s->scan[0][w];
    if (over || total64 >= PC_MAX_UNITS) {   // uniform
        if (blockIdx.x == 0 && tid == 0) atomicOr(&g_paged_status, STATUS_CACHE);
        load = 0;                            // nothing is done
    } else {
        total = static_cast<uint32_t>(total64);
    }
    const uint32_t T = max(static_cast<uint32_t>(p.min_units), (total + C - 1) / C);
    __syncthreads();
    const uint32_t mine = static_cast<uint32_t>(load);
    const uint32_t ex = mine > T ? mine - T : 0u, de = tid < C && mine < T ? T - mine : 0u;
    uint32_t ie = ex, id = de;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t e = __shfl_up_sync(0xffffffffu, ie, o), d = __shfl_up_sync(0xffffffffu, id, o);
        if (lane >= o) {
            ie += e;
            id += d;
        }
    }
    if (lane == 31 && warp < 5) {
        s->scan[0][warp] = ie;
        s->scan[1][warp] = id;
    }
    __syncthreads();
    for (int w = 0; w < warp && w < 5; ++w) {
        ie += s->scan[0][w];
        id += s->scan[1][w];
    }
    if (tid < C) {
        s->E[tid + 1] = ie;
        s->D[tid + 1] = id;
    }
    if (tid == 0) {
        s->E[0] = s->D[0] = 0u;
        s->T = T;
        s->total = total;
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // TMA writes where the scratch was
    __syncthreads();
}
// The last run r with table[r] <= x (and so table[r + 1] > x, for x below table[C]).
__device__ __forceinline__ int deal_find(const uint32_t* table, int C, uint32_t x) {
    int lo = 0, hi = C - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Walks a run's segments: key tiles [t0, t1) of a pair.
struct ChunkWalk {
    PairSeek k;
    int h, qt, t0, t1;
    ChunkPair c;
    int run, C, source;              // whose list of pairs this is: the run's own, or one in the pool
    long long idx;                   // pair
    uint32_t left;                   // units to take from this list from t0 on
    uint32_t pool, pool_end;         // next pool unit, and the end of the run's share
    bool own, tail;                  // own list; the first piece of a pair that its own run began

    __device__ __forceinline__ void pair(const PagedParams& p) {
        k.to(p, idx);
        const int i = static_cast<int>(idx - k.base);
        h = i / k.nq;
        qt = i - h * k.nq;
        c = chunk_pair(p, k.n_q, k.n_live, k.kv, qt);
    }
    __device__ __forceinline__ void cut() { t1 = static_cast<int>(min(static_cast<uint32_t>(c.n), t0 + left)); }
    __device__ __forceinline__ void begin(const PagedParams& p, const ChunkDeal* s, int run_, int C_) {
        run = source = run_;
        C = C_;
        own = true;
        tail = false;
        pool = s->D[run];
        pool_end = min(s->D[run + 1], s->E[C]);
        left = s->T - (s->D[run + 1] - s->D[run]);   // its own pairs' units, at most T
        t0 = t1 = 0;
        idx = run;
        k.begin(p);
        if (left > 0) {
            pair(p);
            cut();
        } else {
            from_pool(p, s);
        }
    }
    __device__ __forceinline__ void from_pool(const PagedParams& p, const ChunkDeal* s) {
        own = false;
        left = 0;
        if (pool >= pool_end) return;
        source = deal_find(s->E, C, pool);
        // skip runs without excess that share the table value
        uint32_t off = s->T + (pool - s->E[source]);   // units into that run's list
        idx = source;
        pair(p);
        while (off >= static_cast<uint32_t>(c.n)) {
            off -= c.n;
            idx += C;
            pair(p);
        }
        t0 = static_cast<int>(off);
        tail = t0 > 0 && pool == s->E[source];
        left = min(pool_end, s->E[source + 1]) - pool;
        pool += left;
        cut();
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const PagedParams& p, const ChunkDeal* s) {
        left -= t1 - t0;
        if (left > 0) {
            idx += C;
            t0 = 0;
            tail = false;
            pair(p);
            cut();
        } else {
            from_pool(p, s);
        }
    }
    // key tiles of this segment that row tile g takes
    __device__ __forceinline__ int end(int g) const { return min(t1, g ? c.ng1 : c.ng0); }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == c.n; }
    // Where a part of a pair is kept: the part that the pair's own run began, the first pool piece of
    // such a pair, a piece that a run's share of the pool begins inside of, one that it ends inside of.
    __device__ __forceinline__ int slot() const { return own ? run : tail ? C + source : t0 > 0 ? 2 * C + run : 3 * C + run; }
};
// A segment as the CTA's warps see it.  The copying warp, which is ahead of the others, walks and
// hands the segments round through a short ring in shared memory, so that the walk's state
// takes no registers beside a softmax row's.
constexpr int PC_SEGS = 4;
struct ChunkSeg {
    int b, h, t0, t1;                // key tiles [t0, t1); t1 = 0: no more segments
    int n, ng0, ng1;                 // of the pair, and of each row tile
    int tok0, ntok0, ntok1;
    int kv, n_q, q0, slot;
    __device__ __forceinline__ int end(int g) const { return min(t1, g ? ng1 : ng0); }
};
__device__ __forceinline__ ChunkSeg make_seg(const ChunkWalk& w) {
    return {w.k.b, w.h, w.t0, w.t1, w.c.n, w.c.ng0, w.c.ng1, w.c.tok0, w.c.ntok0, w.c.ntok1, w.k.kv, w.k.n_q, w.k.q0, w.slot()};
}
// Producer (a converged warp whose lane 0 walks) and consumers (one arrival a warp) of the ring.
struct SegRing {
    ChunkSeg* seg;
    uint32_t full, empty;            // barriers, PC_SEGS each
    uint32_t i;
    __device__ __forceinline__ bool put(const ChunkSeg& s, volatile int* abort_flag, unsigned long long limit) {
        const uint32_t at = i % PC_SEGS;
        if (!chunk_wait_warp(empty + 8 * at, ((i / PC_SEGS) & 1u) ^ 1u, abort_flag, limit)) return false;
        if ((threadIdx.x & 31) == 0) {
            seg[at] = s;
            mbar_arrive(full + 8 * at);
        }
        ++i;
        __syncwarp();
        return true;
    }
    __device__ __forceinline__ const ChunkSeg* get(volatile int* abort_flag, unsigned long long limit) {
        const uint32_t at = i % PC_SEGS;
        if (!chunk_wait_warp(full + 8 * at, (i / PC_SEGS) & 1u, abort_flag, limit)) return nullptr;
        return seg + at;
    }
    __device__ __forceinline__ void done() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * (i % PC_SEGS));
        ++i;
    }
};
// The records for the combine kernel: of the pair that the run began and did not finish, and of
// the one that its share of the pool ends inside of.  Written by one lane, segment by segment.
__device__ __forceinline__ void chunk_record_none(const PagedParams& p, int run, int C) {
    p.shared[run].parts = p.shared[C + run].parts = 0;
    p.shared[run].has_s = 0;
}
__device__ __forceinline__ void chunk_record(const PagedParams& p, const ChunkDeal* s, const ChunkWalk& w) {
    if (!w.own && w.t0 > 0 && !w.tail) p.shared[w.run].has_s = 1;
    if (w.t1 == w.c.n || (!w.own && w.t0 > 0)) return;
    SharedPair& r = p.shared[w.own ? w.run : w.C + w.run];
    r.b = w.k.b;
    r.h = w.h;
    r.qt = w.qt;
    r.parts = w.own ? 2 : 1;
    r.part[0] = w.slot();
    r.part[1] = w.C + w.run;
    // own: the rest of the pair is the run's part of the pool; otherwise it lies behind this piece
    const uint32_t x = w.own ? s->E[w.run] : w.pool;
    r.s0 = w.own ? deal_find(s->D, w.C, x) + 1 : w.run + 1;
    r.s1 = deal_find(s->D, w.C, x + (w.c.n - w.t1) - 1);
}

// Sixteen codes of a row as bf16 values, to two 16-byte chunks (ch, ch + 1 before the swizzle)
// of the row's 128-byte line; lanes with `flip` store the second first, so that a quarter
// warp touches all banks.  ODD false: scales up to 2^7 (SCALE_ONE_STEP) and codes of numbers.  What lies
// beyond takes another multiply or becomes NaN, in a second pass, so that only tiles that have it
// pay for it (the multiply alone was 5 % of the kernel at D = 128, 6 % at 256).  `top` collects what tells (see
// needs_odd): the largest scale code, and the largest magnitudes.
constexpr uint32_t SCALE_ONE_STEP = 134;
struct TopCodes {
    uint32_t scale = 0u, magnitudes = 0u;
};
__device__ __forceinline__ bool needs_odd(const TopCodes& t) { return t.scale > SCALE_ONE_STEP || nan_codes(t.magnitudes) != 0u; }
template <bool ODD>
__device__ __forceinline__ void store_codes(const uint4& d, uint32_t code, uint8_t* line, int ch, int sw, bool flip, TopCodes& top) {
    const uint32_t f = scale_factor(code) * 0x10001u;
    const uint32_t wd[4] = {d.x, d.y, d.z, d.w};
    uint32_t o[8];
    if (!ODD) top.scale = max(top.scale, code);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t t0 = __byte_perm(wd[e], 0u, 0x1404), t1 = __byte_perm(wd[e], 0u, 0x3424);
        const uint32_t m0 = code_magnitudes(t0), m1 = code_magnitudes(t1);
        o[2 * e] = mul_bf16x2(code_signs(t0) | m0, f);
        o[2 * e + 1] = mul_bf16x2(code_signs(t1) | m1, f);
        if constexpr (ODD) {
            if (code > SCALE_ONE_STEP && code != SCALE_NAN) {
                const uint32_t f2 = ((code - 7u) << 7) * 0x10001u;
                o[2 * e] = mul_bf16x2(o[2 * e], f2);
                o[2 * e + 1] = mul_bf16x2(o[2 * e + 1], f2);
            }
            o[2 * e] |= nan_codes(m0);
            o[2 * e + 1] |= nan_codes(m1);
        } else {
            top.magnitudes = __vimax3_u16x2(top.magnitudes, m0, m1);
        }
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
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {   // swizzled tiles need it
        if (threadIdx.x == 0) atomicOr(&g_paged_status, STATUS_LAYOUT);
        return;
    }
    uint8_t* sKV = smem + 2 * C::QT_BYTES;
    uint8_t* sStg = sKV + C::NS * C::SLOT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sStg + C::NSTG * C::STG_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + PCB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    ChunkDeal* deal = reinterpret_cast<ChunkDeal*>(tmem_holder + 2);
    SegRing segs = {reinterpret_cast<ChunkSeg*>(deal + 1), 0, 0, 0};
    static_assert(PCB_NUM * 8 + 8 + sizeof(ChunkDeal) + PC_SEGS * sizeof(ChunkSeg) <= C::CTRL, "control area");
    const uint32_t bar0 = smem_u32(bars), sQ_addr = smem_u32(smem), sKV_addr = smem_u32(sKV);
#define CBAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    allow_next_kernel();
    const int run = blockIdx.x;
    segs.full = CBAR(PCB_GFULL);
    segs.empty = CBAR(PCB_GEMPTY);
    chunk_deal(p, n_ctas, deal, reinterpret_cast<int4*>(sKV), 4096);

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
            mbar_init(CBAR(PCB_FULL + s), E4M3 ? C::NCONV : 1);
            mbar_init(CBAR(PCB_EMPTY + s), 1);
        }
        for (int s = 0; s < C::NSTG; ++s) {
            mbar_init(CBAR(PCB_SFULL + s), 33);    // the byte count's, and every copying lane's scale bytes
            mbar_init(CBAR(PCB_SEMPTY + s), C::NCONV);
        }
        for (int i = 0; i < PC_SEGS; ++i) {
            mbar_init(CBAR(PCB_GFULL + i), 1);
            mbar_init(CBAR(PCB_GEMPTY + i), 9 + C::NCONV);   // 8 softmax warps, MMA, converters
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
        while (ok) {
            // (a pair without tokens for this group's tile leaves it waiting for the length of a segment)
            const ChunkSeg* sg = segs.get(abort_flag, wlim < 1ull << 36 ? wlim * (deal->T + 1ull) : wlim);
            ok = sg != nullptr;
            if (!ok || sg->t1 == 0) break;
            const int i = sg->tok0 + g * p.tpt + r_tok;
            // Rows that are not live hold another sequence's queries or what was in shared memory.  When a warp moves
            // its maxima decides how its rows are rounded, so these have no say in it: their reference is infinite.
            const bool live = r_tok < (g ? sg->ntok1 : sg->ntok0) && r_tok < p.tpt;
            const int seen = live ? keys_seen(p.causal, sg->kv, sg->n_q, i) : 0;
            const int all_seen = keys_seen(p.causal, sg->kv, sg->n_q, sg->tok0 + g * p.tpt);   // by every live row of the tile
            const int t0 = sg->t0;
            float m_ref = -INFINITY, l_sum = 0.0f;
            const int j1 = sg->end(g);
#pragma unroll 1
            for (int j = t0; j < j1; ++j) {
                ok = chunk_wait_warp(CBAR(PCB_S + g), cnt & 1u, abort_flag, wlim);
                if (!ok) break;
                tc_fence_after();
                float x[C::COLS];
                // columns [c0, c0 + COLS) of the row, masked by selection
                auto load = [&](int c0) {
                    uint32_t raw[C::COLS];
                    if constexpr (C::COLS == 128) tmem_ld128_wait(s_addr, raw);
                    else tmem_ld64_wait(s_addr + c0, raw);
                    if (all_seen - j * PC_BN < PC_BN || !pos_scale) {
                        const int lim = seen - j * PC_BN - c0;   // columns this row sees
#pragma unroll
                        for (int c = 0; c < C::COLS; ++c) x[c] = c < lim ? __uint_as_float(raw[c]) * (pos_scale ? 1.0f : sl2) : -INFINITY;
                    } else {
#pragma unroll
                        for (int c = 0; c < C::COLS; ++c) x[c] = __uint_as_float(raw[c]);
                    }
                };
                float mx = -INFINITY;
#pragma unroll 1
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
                if (j == t0) {
                    m_ref = live ? mx : INFINITY;
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
                // (rolled where the columns come in halves: with the converters' code beside it, the kernel
                // waits for instructions otherwise)
#pragma unroll 1
                for (int c0 = 0; c0 < PC_BN; c0 += C::COLS) {
                    if (c0 != 0) {
                        load(c0);
                        if constexpr (C::AHEAD) arrive(CBAR(PCB_READ + g));
                    }
#pragma unroll
                    for (int cc = 0; cc < C::COLS / 32; ++cc) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = fma2(make_float2(x[cc * 32 + 2 * e], x[cc * 32 + 2 * e + 1]), mul2, neg2);
                            const float p0 = exp2_approx(y.x), p1 = exp2_approx(y.y);
                            sp[e & 3] = add2(sp[e & 3], make_float2(p0, p1));   // the sum takes the weights unrounded
                            pk[e] = pack_bf16(p0, p1);
                        }
                        tmem_st16(p_addr + c0 / 2 + cc * 16, pk);
                        if (!C::AHEAD && c0 == 0 && cc == 1) {                  // the first 64 keys' weights
                            tmem_wait_st();
                            arrive(CBAR(PCB_P + g));
                        }
                    }
                }
                tmem_wait_st();
                arrive(CBAR(PCB_P + (C::AHEAD ? 0 : 2) + g));
                l_sum = l_sum * factor + (((sp[0].x + sp[1].x) + (sp[2].x + sp[3].x)) + ((sp[0].y + sp[1].y) + (sp[2].y + sp[3].y)));
                ++cnt;
            }
            if (!ok) break;
            const bool has = j1 > t0;
            if (has) {
                if ((p.debug & ATTN_DEBUG_LATE_SOFTMAX) && (warp & 1)) debug_pause();
                // D <= 64: one phase per PV; 128: one per segment
                ok = chunk_wait_warp(CBAR(PCB_O + g), C::AHEAD ? (cnt - 1) & 1u : o_phase, abort_flag, wlim);
                if (!ok) break;
                o_phase ^= 1u;
                tc_fence_after();
            }
            const bool some = !(l_sum == 0.0f);   // NaN counts
            const float inv = some ? 1.0f / l_sum : 0.0f;
            const float lse = some ? (m_ref + log2f(l_sum)) * 0.69314718055994530942f : -INFINITY;
            const bool whole = t0 == 0 && sg->t1 == sg->n;
            const long long row = static_cast<long long>(sg->q0) + i;
            const int hq = sg->h * p.G + r_head;
            const long long part = (sg->slot * 2LL + g) * 128 + r;
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
            segs.done();
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
        for (; ok; segs.done()) {
            const ChunkSeg* sg = segs.get(abort_flag, wlim);
            ok = sg != nullptr;
            if (!ok || sg->t1 == 0) break;
            const int t0 = sg->t0, kv = sg->kv;
            const int e0 = sg->end(0), e1 = sg->end(1), je = max(e0, e1);
            if (je <= t0) continue;              // no keys: nothing was loaded
            ok = chunk_wait_warp(CBAR(PCB_QFULL), q_phase, abort_flag, wlim);
            q_phase ^= 1u;
            if (!ok) break;
            k_slot = next_item();
            if (!ok) break;
            if (t0 < e0) issue_s(0);
            if (t0 < e1) issue_s(1);
            tc_commit_elect(CBAR(PCB_EMPTY + k_slot));
            if (t0 + 1 == je) tc_commit_elect(CBAR(PCB_QEMPTY));   // the segment's last S: Q may be replaced
#pragma unroll 1
            for (int j = t0; j < je && ok; ++j) {
                v_slot = next_item();
                if (!ok) break;
                if constexpr (!E4M3) {
                    // rows of the last copied box that lie behind the sequence: cleared, since
                    // 0 * NaN would reach every row
                    const int valid = kv - j * PC_BN;
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
                            issue_pv(g, j == t0, 0, PC_BN / 16);
                            tc_commit_elect(CBAR(PCB_O + g));
                        } else {
                            issue_pv(g, j == t0, 0, PC_BN / 32);
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
        constexpr int N = E4M3 ? C::NSTG : C::NS;          // the slots that are filled here
        constexpr int FULL = E4M3 ? PCB_SFULL : PCB_FULL, EMPTY = E4M3 ? PCB_SEMPTY : PCB_EMPTY;
        ChunkWalk w;
        if (lane == 0) chunk_record_none(p, run, n_ctas);
        w.begin(p, deal, run, n_ctas);
        for (; ok; w.next(p, deal)) {
            ok = segs.put(w.more() ? make_seg(w) : ChunkSeg{}, abort_flag, wlim);
            if (!ok || !w.more()) break;
            if (lane == 0) chunk_record(p, deal, w);
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
                        tma_load_4d(sQ_addr + g * C::QT_BYTES + c * 128 * C::SW, &tm_q, c * C::BLK, 0, w.h, w.k.q0 + w.c.tok(g), CBAR(PCB_QFULL));
            }
            // lane i < boxes copies box i of a tile (all lanes at once: one lane issuing them in
            // turn took 20 % longer with 16-row pages); its page is looked up one tile ahead
            const int32_t* table = p.table + w.k.b * p.table_stride;
            auto lookup = [&](int j) {
                const int key = key_at(j, PC_BN, lane * p.box_rows);
                return page_ask(p, table, key, lane < boxes && j < je && key < w.k.kv);
            };
            auto lookup_scale = [&](int j) {               // e4m3: lane's group of 8 rows
                const int key = key_at(j, PC_BN, (lane & 15) * 8);
                return page_ask(p, table, key, E4M3 && j < je && key < w.k.kv);
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
    } else if (E4M3 && warp < 8 + C::NCONV) {
        // ================================================================ converters: e4m3 K and V
        if constexpr (E4M3) {
            constexpr int CPR = D / 16;          // 16-code chunks per row
            constexpr int X = 4 * CPR / C::NCONV;       // chunks per thread: 128 rows * CPR over the converters' threads
            constexpr int RPX = 32 * C::NCONV / CPR;    // rows between a thread's chunks
            const int t = tid - 256;
            const int r0 = t / CPR, c16 = t % CPR;
            const int blk = c16 * 16 / C::BLK, ch = c16 * 16 % C::BLK / 8;
            uint32_t item = 0;
            bool ok = true;
            for (; ok; segs.done()) {
                const ChunkSeg* sg = segs.get(abort_flag, wlim);
                ok = sg != nullptr;
                if (!ok || sg->t1 == 0) break;
                const int je = max(sg->end(0), sg->end(1)), kv = sg->kv;
                for (int j2 = 2 * sg->t0; j2 < 2 * je && ok; ++j2) {   // item: tile j2 / 2, K or V
                    const int slot = static_cast<int>(item % C::NS), stg = static_cast<int>(item % C::NSTG);
                    ok = chunk_wait_warp(CBAR(PCB_SFULL + stg), (item / C::NSTG) & 1u, abort_flag, wlim) &&
                         chunk_wait_warp(CBAR(PCB_EMPTY + slot), ((item / C::NS) & 1u) ^ 1u, abort_flag, wlim);
                    if (!ok) break;
                    ++item;
                    const int left = kv - (j2 >> 1) * PC_BN;       // rows of the tile that exist
                    const uint8_t* src = sStg + stg * C::STG_BYTES;
                    uint8_t* dst = sKV + slot * C::SLOT + blk * (8 * C::SW);
                    // Four loads, then their stores: a load behind a store to shared memory would wait for
                    // it (and eight at once make more code than they save).
                    constexpr int XB = X < 4 ? X : 4;
                    TopCodes top;
#pragma unroll 1
                    for (int xb = r0; xb < PC_BN; xb += XB * RPX) {
                        uint4 d[XB];
                        uint32_t code[XB];
#pragma unroll
                        for (int x = 0; x < XB; ++x) {
                            const int r = x * RPX + xb;
                            d[x] = *reinterpret_cast<const uint4*>(src + r * D + c16 * 16);
                            code[x] = src[PC_BN * D + r];
                        }
                        if (left < PC_BN) {                          // a page's rows behind the sequence
#pragma unroll
                            for (int x = 0; x < XB; ++x)
                                if (x * RPX + xb >= left) {
                                    d[x] = make_uint4(0u, 0u, 0u, 0u);
                                    code[x] = 127u;
                                }
                        }
#pragma unroll
                        for (int x = 0; x < XB; ++x) {
                            const int r = x * RPX + xb;
                            store_codes<false>(d[x], code[x], dst + (r >> 3) * C::GROUP + (r & 7) * C::SW, ch, C::SW == 128 ? r & 7 : (r >> 1) & 3, blk & 1, top);
                        }
                    }
                    if (needs_odd(top)) {
#pragma unroll 1
                        for (int r = r0; r < min(left, PC_BN); r += RPX)
                            store_codes<true>(*reinterpret_cast<const uint4*>(src + r * D + c16 * 16), src[PC_BN * D + r],
                                              dst + (r >> 3) * C::GROUP + (r & 7) * C::SW, ch, C::SW == 128 ? r & 7 : (r >> 1) & 3, blk & 1, top);
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

// Pairs that several CTAs worked on: a SharedPair, as chunk_record wrote it, to a block (x), its rows spread
// over blockIdx.y, one warp a row.
template <int D>
__global__ void __launch_bounds__(256) paged_chunk_combine_kernel(const PagedParams p, const int n_runs) {
    wait_for_main_kernel();                     // every block, so that this grid never ends before that one
    const SharedPair s = p.shared[blockIdx.x];
    if (s.parts == 0) return;
    const QueryRange qr = query_range(p, s.b, false);
    const int n_live = min(qr.n, p.max_q), tok0 = s.qt * 2 * p.tpt;
    // the parts' slots, for all rows
    __shared__ int s_slot[2 + PC_MAX_RUNS];
    __shared__ int s_count[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mine = s.s0 + static_cast<int>(threadIdx.x);        // (at most PC_MAX_RUNS of them, 256 threads)
    const bool has = mine <= s.s1 && __ldcg(&p.shared[mine].has_s) != 0;
    const unsigned bits = __ballot_sync(0xffffffffu, has);
    if (lane == 0) s_count[warp] = __popc(bits);
    __syncthreads();
    int n = s.parts, rank = s.parts + __popc(bits & ((1u << lane) - 1u));
    for (int w = 0; w < 8; ++w) {
        if (w < warp) rank += s_count[w];
        n += s_count[w];
    }
    if (has) s_slot[rank] = 2 * n_runs + mine;
    if (static_cast<int>(threadIdx.x) < s.parts) s_slot[threadIdx.x] = s.part[threadIdx.x];
    __syncthreads();
    constexpr int V = D >= 128 ? 4 : D / 32, NV = D / (32 * V);   // floats per load, loads per lane
    for (int r = blockIdx.y * 8 + warp; r < 256; r += gridDim.y * 8) {
        const int g = r >> 7, rr = r & 127, tok = rr / p.G;
        const int i = tok0 + g * p.tpt + tok;
        if (tok >= p.tpt || i >= n_live) continue;
        auto at = [&](int k) { return (s_slot[k] * 2LL + g) * 128 + rr; };
        const float first = lane < n ? __ldcg(p.part_lse + at(lane)) : -INFINITY;
        float M = first;
        for (int k = lane + 32; k < n; k += 32) M = fmaxf(M, __ldcg(p.part_lse + at(k)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float sum = 0.0f, acc[NV * V];
#pragma unroll
        for (int e = 0; e < NV * V; ++e) acc[e] = 0.0f;
        // weights 32 at a time, one per lane, so that the loads of consecutive parts overlap
        for (int k0 = 0; k0 < n; k0 += 32) {
            const float lc = k0 == 0 ? first : k0 + lane < n ? __ldcg(p.part_lse + at(k0 + lane)) : -INFINITY;
            const float w_l = lc == -INFINITY ? 0.0f : expf(lc - M);
            const unsigned there = __ballot_sync(0xffffffffu, lc != -INFINITY);   // (a part without keys stored no values)
            const int m = min(32, n - k0);
#pragma unroll 4
            for (int k = 0; k < m; ++k) {
                const float wgt = __shfl_sync(0xffffffffu, w_l, k);
                sum += wgt;
                if (!(there >> k & 1u)) continue;
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const float* src = p.part_out + at(k0 + k) * D + q * 32 * V + lane * V;
                    float v[V];
                    if constexpr (V == 4) *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(src));
                    else if constexpr (V == 2) *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(src));
                    else v[0] = __ldcg(src);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[q * V + e] += wgt * v[e];
                }
            }
        }
        const bool some = !(sum == 0.0f);
        const float inv = some ? 1.0f / sum : 0.0f;
        const long long row = static_cast<long long>(qr.t0) + i;
        const int hq = s.h * p.G + rr - tok * p.G;
        __nv_bfloat16* dst = p.out + row * p.out_t + hq * p.out_h;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            __nv_bfloat16* d = dst + q * 32 * V + lane * V;
            if constexpr (V == 4)
                *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16(acc[q * V] * inv, acc[q * V + 1] * inv), pack_bf16(acc[q * V + 2] * inv, acc[q * V + 3] * inv));
            else if constexpr (V == 2)
                *reinterpret_cast<uint32_t*>(d) = pack_bf16(acc[0] * inv, acc[1] * inv);
            else
                *d = __float2bfloat16_rn(acc[0] * inv);
        }
        if (lane == 0 && p.lse != nullptr) p.lse[row * p.Hq + hq] = some ? M + logf(sum) : -INFINITY;
    }
}
