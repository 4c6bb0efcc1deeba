// paged_pair.cuh -- attention over pages for many query rows per key head at head dim 256,
// on CTA pairs (cta_group::2).  Included by paged.cu inside namespace attn, after
// paged_chunk.cuh, whose rows, walk and deal of the work it shares (a run belongs to a pair).
//
// At 256 dims a 128-row tile fills a CTA's TMEM (S twice, O), so each CTA of a pair takes one of
// the two row tiles and half of every K and V tile (keys [64 r, +64) of K, value columns
// [128 r, +128) of V for rank r): M = 256 MMAs issued by the leader read A from each CTA and
// B across both, and each K/V byte brought to an SM still serves 256 rows.
//
// MMA order per segment: S(0), S(1), then PV(j), S(j+2), P(j) stored over S(j).  The
// softmax of tile j runs under the MMAs of its neighbours.  A rescale of O waits for
// PV(j-1), announced by a commit per PV on two barriers in turn: a parity wait tells a phase from
// the next one only, and a warp may come to its wait before or after the PV that it waits for.
//
// The pages behind a sequence: boxes that lie behind it entirely read as zeros (their page
// coordinate is outside the pool); the rows of the last V box are loaded and stored by the
// copying warp itself, zeros behind the sequence, and its arrival orders them before the MMA.
//
// Measured: 2000 rows on 100000 keys (8 heads, bf16) 1.08 to 1.11 ms, 1.5 PFLOP/s, in short runs, 1.28 to 1.31 ms under
// the power cap; 2368 rows on 8192 keys 144 to 154 us, over e4m3 pages 243 to 247 us, where the four converter warps
// of each CTA set the pace.

template <bool E4M3>
struct PagedPairCfg {
    static constexpr int D = 256;
    static constexpr int QT_BYTES = 128 * D * 2;
    static constexpr int KH = 64;                       // keys of a K tile held by one CTA
    static constexpr int KGROUP = 4 * 1024;             // an 8-row group of a K half: four 64-column blocks
    static constexpr int VGROUP = 2 * 1024;             // and of a V half: two
    static constexpr int SLOT = 32768;                  // one CTA's half of a K or V tile
    static constexpr int NS = E4M3 ? 3 : 5;
    static constexpr int STG_BYTES = SLOT / 2 + 128;    // e4m3: staged codes of a half tile, scale bytes
    static constexpr int NSTG = E4M3 ? 4 : 0;
    static constexpr int CTRL = 2048;
    static constexpr int SMEM = QT_BYTES + NS * SLOT + NSTG * STG_BYTES + CTRL;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr uint32_t O_COL = 256;
    // warps 0-3 softmax, 4 copies, 5 MMA (leader) and TMEM; e4m3: 6 and 7 idle, 8-11 converters
    static constexpr int WARP_COPY = 4, WARP_MMA = 5, WARP_CONV = 8;
    static constexpr int THREADS = E4M3 ? 384 : 192;
};
enum : int {
    PPB_QFULL = 0, PPB_QEMPTY = 1, PPB_S = 2 /* [2] */, PPB_P = 4 /* [2] */, PPB_PV = 6 /* [2] */, PPB_DRAIN = 8,
    PPB_FULL = 9 /* [5] */, PPB_EMPTY = 14 /* [5] */, PPB_SFULL = 19 /* [4] */, PPB_SEMPTY = 23 /* [4] */, PPB_GFULL = 27 /* [4] segments */, PPB_GEMPTY = 31 /* [4] */, PPB_NUM = 35
};

// Item i of a segment of n key tiles in the MMA warp's order: K(0), K(1), then V(j), K(j+2).
struct PairItem {
    int j;
    bool k;
};
__device__ __forceinline__ PairItem pair_item(int i, int n) {
    const int ahead = min(2, n), m = i - ahead, mixed = 2 * (n - ahead);
    if (m < 0) return {i, true};
    if (m >= mixed) return {m - (n - ahead), false};
    return {(m >> 1) + ((m & 1) ? 2 : 0), (m & 1) != 0};
}

// Arrival on a barrier of the pair's leader that orders this thread's earlier shared-memory
// stores (after a proxy fence) before the leader's MMAs.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}

template <bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PagedPairCfg<E4M3>::THREADS, 1)
    paged_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedParams p, const int n_pairs) {
    using C = PagedPairCfg<E4M3>;
    constexpr int D = C::D;
    extern __shared__ __align__(1024) uint8_t smem[];
    // swizzled tiles need 1024-byte alignment; both CTAs see the same layout and return together
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_paged_status, STATUS_LAYOUT);
        return;
    }
    uint8_t* sKV = smem + C::QT_BYTES;
    uint8_t* sStg = sKV + C::NS * C::SLOT;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sStg + C::NSTG * C::STG_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + PPB_NUM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    ChunkDeal* deal = reinterpret_cast<ChunkDeal*>(tmem_holder + 2);
    SegRing segs = {reinterpret_cast<ChunkSeg*>(deal + 1), 0, 0, 0};
    static_assert(PPB_NUM * 8 + 8 + sizeof(ChunkDeal) + PC_SEGS * sizeof(ChunkSeg) <= C::CTRL, "control area");
    const uint32_t bar0 = smem_u32(bars), sQ_addr = smem_u32(smem), sKV_addr = smem_u32(sKV);
#define PPBAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int run = static_cast<int>(blockIdx.x >> 1);

    allow_next_kernel();
    segs.full = PPBAR(PPB_GFULL);
    segs.empty = PPBAR(PPB_GEMPTY);
    chunk_deal(p, n_pairs, deal, reinterpret_cast<int4*>(sKV), 4096);

    if (tid == 0) {
        mbar_init(PPBAR(PPB_QFULL), 1);
        mbar_init(PPBAR(PPB_QEMPTY), 1);
        mbar_init(PPBAR(PPB_DRAIN), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(PPBAR(PPB_PV + i), 1);
            mbar_init(PPBAR(PPB_S + i), 1);
            mbar_init(PPBAR(PPB_P + i), 8);
        }
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(PPBAR(PPB_FULL + s), E4M3 ? 8 : 2);
            mbar_init(PPBAR(PPB_EMPTY + s), 1);
        }
        for (int s = 0; s < C::NSTG; ++s) {
            mbar_init(PPBAR(PPB_SFULL + s), 33);   // the byte count's, and every copying lane's scale bytes
            mbar_init(PPBAR(PPB_SEMPTY + s), 4);
        }
        for (int i = 0; i < PC_SEGS; ++i) {
            mbar_init(PPBAR(PPB_GFULL + i), 1);
            mbar_init(PPBAR(PPB_GEMPTY + i), 4 + (leader ? 1 : 0) + (E4M3 ? 4 : 0));   // softmax, MMA, converters
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::WARP_MMA) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const unsigned long long wlim = p.wait_ns;

    if (warp < 4) {
        // ================================================================ softmax and epilogue (both CTAs)
        const int g = rank, r = tid;
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t o_addr = tmem + lane_base + C::O_COL;
        const float sl2 = p.scale_log2;
        const bool pos_scale = sl2 > 0.0f;
        const float mul = pos_scale ? sl2 : 1.0f;
        const int r_tok = r / p.G, r_head = r - r_tok * p.G;
        const uint32_t p_bar[2] = {mapa_shared(PPBAR(PPB_P), 0), mapa_shared(PPBAR(PPB_P + 1), 0)};
        uint32_t cnt = 0;   // key tiles processed, over all segments
        bool ok = true;
        // PV of the tile before tile cnt.  Its barrier's phase before is that of PV two tiles earlier, which
        // "S ready" of its own tile vouched for, and the phase after needs this warp's P(cnt + 1).
        auto wait_pv = [&]() { return chunk_wait_warp(PPBAR(PPB_PV + ((cnt - 1) & 1)), ((cnt - 1) >> 1) & 1, abort_flag, wlim); };
        while (ok) {
            const ChunkSeg* sg = segs.get(abort_flag, wlim);
            ok = sg != nullptr;
            if (!ok || sg->t1 == 0) break;
            const int i = sg->tok0 + g * p.tpt + r_tok;
            const bool live = r_tok < (g ? sg->ntok1 : sg->ntok0) && r_tok < p.tpt;   // (others have no say, as in paged_chunk.cuh)
            const int seen = live ? keys_seen(p.causal, sg->kv, sg->n_q, i) : 0;
            const int all_seen = keys_seen(p.causal, sg->kv, sg->n_q, sg->tok0 + g * p.tpt);
            const int t0 = sg->t0;
            float m_ref = -INFINITY, l_sum = 0.0f;
            const int je = max(sg->end(0), sg->end(1));
#pragma unroll 1
            for (int j = t0; j < je; ++j) {
                ok = chunk_wait_warp(PPBAR(PPB_S + (cnt & 1)), (cnt >> 1) & 1, abort_flag, wlim);
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_addr = tmem + lane_base + (cnt & 1) * PC_BN;
                uint32_t raw[PC_BN];
                tmem_ld128_wait(s_addr, raw);
                float x[PC_BN];
                if (all_seen - j * PC_BN < PC_BN || !pos_scale) {
                    const int lim = seen - j * PC_BN;
#pragma unroll
                    for (int c = 0; c < PC_BN; ++c) x[c] = c < lim ? __uint_as_float(raw[c]) * (pos_scale ? 1.0f : sl2) : -INFINITY;
                } else {
#pragma unroll
                    for (int c = 0; c < PC_BN; ++c) x[c] = __uint_as_float(raw[c]);
                }
                const float mx = row_max(x) * mul;
                float factor = 1.0f;
                bool rescale = false;
                if (j == t0) {
                    m_ref = live ? mx : INFINITY;
                } else if (__any_sync(0xffffffffu, mx > m_ref + PC_RESCALE_LOG2)) {
                    const float m_new = fmaxf(m_ref, mx);
                    factor = m_ref == -INFINITY ? 0.0f : exp2_approx(m_ref - m_new);
                    m_ref = m_new;
                    rescale = true;
                }
                const float neg_m = m_ref == -INFINITY ? 0.0f : -m_ref;
                float2 sp[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) sp[t] = make_float2(0.0f, 0.0f);
                const float2 mul2 = make_float2(mul, mul), neg2 = make_float2(neg_m, neg_m);
#pragma unroll
                for (int cc = 0; cc < PC_BN / 32; ++cc) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = fma2(make_float2(x[cc * 32 + 2 * e], x[cc * 32 + 2 * e + 1]), mul2, neg2);
                        const float p0 = exp2_approx(y.x), p1 = exp2_approx(y.y);
                        sp[e & 3] = add2(sp[e & 3], make_float2(p0, p1));
                        pk[e] = pack_bf16(p0, p1);
                    }
                    tmem_st16(s_addr + cc * 16, pk);
                }
                l_sum = l_sum * factor + (((sp[0].x + sp[1].x) + (sp[2].x + sp[3].x)) + ((sp[0].y + sp[1].y) + (sp[2].y + sp[3].y)));
                if (rescale) {
                    ok = wait_pv();
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int oc = 0; oc < D / 32; ++oc) {
                        uint32_t o[32];
                        tmem_ld32_wait(o_addr + oc * 32, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                        tmem_st32(o_addr + oc * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(p_bar[cnt & 1]);
                ++cnt;
            }
            if (!ok) break;
            const bool has = je > t0;
            if (has) {
                if ((p.debug & ATTN_DEBUG_LATE_SOFTMAX) && (warp & 1)) debug_pause();
                ok = wait_pv();
                if (!ok) break;
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
            tc_fence_before();   // the reads of O above, before the next segment's first P
            segs.done();
        }
    } else if (warp == C::WARP_MMA) {
        // ================================================================ MMA issuer (leader)
        if (leader) {
            constexpr uint32_t IDESC_S = make_idesc_bf16(256, PC_BN, false);
            constexpr uint32_t IDESC_PV = make_idesc_bf16(256, D, true);
            const uint64_t q_desc0 = make_smem_desc(sQ_addr, 16, 1024, 2);
            const uint64_t k_desc0 = make_smem_desc(sKV_addr, 16, C::KGROUP, 2);
            const uint64_t v_desc0 = make_smem_desc(sKV_addr, 1024, C::VGROUP, 2);
            uint32_t item = 0, s_cnt = 0, p_cnt = 0, q_phase = 0;
            bool ok = true;
            auto next_item = [&]() -> int {
                const int slot = static_cast<int>(item % C::NS);
                ok = ok && chunk_wait_warp<true>(PPBAR(PPB_FULL + slot), (item / C::NS) & 1u, abort_flag, wlim);
                ++item;
                tc_fence_after();
                return slot;
            };
            auto issue_s = [&]() {
                const int slot = next_item();
                if (!ok) return;
                const uint64_t kd = k_desc0 + static_cast<uint64_t>(slot) * (C::SLOT >> 4);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    mma_ss_pair_elect_x4<2, 2>(tmem + (s_cnt & 1) * PC_BN, q_desc0 + static_cast<uint64_t>((c * 128 * 128) >> 4),
                                               kd + static_cast<uint64_t>((c * 1024) >> 4), IDESC_S, c != 0 ? 1u : 0u);
                tc_commit_pair_elect(PPBAR(PPB_EMPTY + slot), 0x3);
                tc_commit_pair_elect(PPBAR(PPB_S + (s_cnt & 1)), 0x3);
                ++s_cnt;
            };
            for (; ok; segs.done()) {
                const ChunkSeg* sg = segs.get(abort_flag, wlim);
                ok = sg != nullptr;
                if (!ok || sg->t1 == 0) break;
                const int t0 = sg->t0, je = max(sg->end(0), sg->end(1));
                if (je <= t0) continue;
                ok = chunk_wait_warp(PPBAR(PPB_QFULL), q_phase, abort_flag, wlim);
                q_phase ^= 1u;
                if (!ok) break;
                issue_s();
                if (ok && t0 + 1 < je) issue_s();
                if (ok && t0 + 2 >= je) tc_commit_pair_elect(PPBAR(PPB_QEMPTY), 0x3);   // the segment's last S
#pragma unroll 1
                for (int j = t0; j < je && ok; ++j) {
                    const int slot = next_item();   // V
                    ok = ok && chunk_wait_warp(PPBAR(PPB_P + (p_cnt & 1)), (p_cnt >> 1) & 1, abort_flag, wlim);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = v_desc0 + static_cast<uint64_t>(slot) * (C::SLOT >> 4);
#pragma unroll
                    for (int kb = 0; kb < PC_BN / 16; kb += 4)
                        mma_ts_pair_elect_x4<8, (2 * C::VGROUP) / 16>(tmem + C::O_COL, tmem + (p_cnt & 1) * PC_BN + kb * 8u,
                                                                      vd + static_cast<uint64_t>((kb * 2 * C::VGROUP) >> 4), IDESC_PV, kb == 0 && j == t0 ? 0u : 1u);
                    tc_commit_pair_elect(PPBAR(PPB_EMPTY + slot), 0x3);
                    tc_commit_pair_elect(PPBAR(PPB_PV + (p_cnt & 1)), 0x3);
                    ++p_cnt;
                    if (j + 2 < je) {
                        issue_s();
                        if (ok && j + 3 == je) tc_commit_pair_elect(PPBAR(PPB_QEMPTY), 0x3);
                    }
                }
            }
            tc_commit_pair_elect(PPBAR(PPB_DRAIN), 0x1);
            __syncwarp();
            const uint64_t d0 = global_timer_ns();
            while (!mbar_try_wait(PPBAR(PPB_DRAIN), 0)) {
                if (global_timer_ns() - d0 > wlim) {
                    atomicOr(&g_paged_status, STATUS_TIMEOUT);
                    break;
                }
            }
        }
        __syncwarp();
    } else if (warp == C::WARP_COPY) {
        // ================================================================ copies (both CTAs): Q, and K and V halves
        if (lane == 0) {
            tma_prefetch_map(&tm_q);
            tma_prefetch_map(&tm_k);
            tma_prefetch_map(&tm_v);
        }
        // Q is read once; half of the K/V lines are kept in L2 ahead of it and of the output
        const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last_half();
        const uint32_t l_q = mapa_shared(PPBAR(PPB_QFULL), 0);
        uint32_t item = 0, qe_phase = 0;
        bool ok = true, first = true;
        const int k_boxes = C::KH >> p.box_shift, v_boxes = PC_BN >> p.box_shift;   // box_rows <= 64
        ChunkWalk w;
        if (leader && lane == 0) chunk_record_none(p, run, n_pairs);
        w.begin(p, deal, run, n_pairs);
        for (; ok; w.next(p, deal)) {
            ok = segs.put(w.more() ? make_seg(w) : ChunkSeg{}, abort_flag, wlim);
            if (!ok || !w.more()) break;
            if (leader && lane == 0) chunk_record(p, deal, w);
            const int je = max(w.end(0), w.end(1));
            if (je <= w.t0) continue;
            if (!first) {
                ok = chunk_wait_warp(PPBAR(PPB_QEMPTY), qe_phase, abort_flag, wlim);
                qe_phase ^= 1u;
                if (!ok) break;
            }
            first = false;
            if (lane == 0) {
                if (leader) mbar_arrive_expect_tx(PPBAR(PPB_QFULL), (w.c.ntok1 > 0 ? 2 : 1) * p.tpt * p.G * D * 2);
                if (w.c.ntok(rank) > 0)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d_pair_hint(sQ_addr + c * 128 * 128, &tm_q, c * 64, 0, w.h, w.k.q0 + w.c.tok(rank), l_q, pol_q);
            }
            const int32_t* table = p.table + w.k.b * p.table_stride;
            // lane i copies box i of this CTA's K half / of V; pages are looked up a tile ahead
            auto lookup = [&](int j, bool k) {
                const int key = key_at(j, PC_BN, (k ? rank * C::KH : 0) + lane * p.box_rows);
                return page_ask(p, table, key, lane < (k ? k_boxes : v_boxes) && j < je && key < w.k.kv);
            };
            auto lookup_scale = [&](int j, bool k) {       // e4m3: the lane's group of 8 rows
                const int key = key_at(j, PC_BN, (k ? rank * C::KH : 0) + lane * 8);
                return page_ask(p, table, key, E4M3 && lane < (k ? 8 : 16) && j < je && key < w.k.kv);
            };
            auto copy = [&](bool k, int j, const PageAsk& ask, const PageAsk& scale_ask) {
                const PageAt a = page_at(p, ask, true);
                if constexpr (E4M3) {
                    const PageAt sa = page_at(p, scale_ask, false);
                    // into staging, on this CTA's own barriers
                    const int slot = static_cast<int>(item % C::NSTG);
                    ok = ok && chunk_wait_warp(PPBAR(PPB_SEMPTY + slot), ((item / C::NSTG) & 1u) ^ 1u, abort_flag, wlim);
                    if (!ok) return;
                    ++item;
                    if (lane == 0) mbar_arrive_expect_tx(PPBAR(PPB_SFULL + slot), C::SLOT / 2);
                    __syncwarp();
                    const bool drop = (p.debug & ATTN_DEBUG_DROP_COPY) && leader && k && j == w.t0 && lane == 0;
                    const uint32_t dst = smem_u32(sStg) + slot * C::STG_BYTES;
                    if (lane < (k ? k_boxes : v_boxes) && !drop)
                        tma_load_4d(dst + lane * p.box_rows * (k ? 256 : 128), k ? &tm_k : &tm_v, k ? 0 : rank * 128, a.row, w.h, a.page, PPBAR(PPB_SFULL + slot));
                    if (lane < (k ? 8 : 16)) {
                        const bool have = sa.page < p.c.num_pages;
                        const uint8_t* src = p.c.scale[k ? 0 : 1];
                        if (have) src += (static_cast<long long>(sa.page) * p.c.Hkv + w.h) * p.c.page_size + sa.row;
                        cp_async8(dst + C::SLOT / 2 + lane * 8, src, have);
                    }
                    cp_async_mbar_arrive_noinc(PPBAR(PPB_SFULL + slot));
                    __syncwarp();
                } else {
                    const int slot = static_cast<int>(item % C::NS);
                    ok = ok && chunk_wait_warp(PPBAR(PPB_EMPTY + slot), ((item / C::NS) & 1u) ^ 1u, abort_flag, wlim);
                    if (!ok) return;
                    ++item;
                    const uint32_t l_full = mapa_shared(PPBAR(PPB_FULL + slot), 0);
                    const int valid = w.k.kv - j * PC_BN;      // rows of the tile that exist
                    const int cut = !k && valid < PC_BN && (valid & (p.box_rows - 1)) != 0 ? valid >> p.box_shift : -1;   // the box to fill by hand
                    if (cut >= 0) {
                        const int pg = __shfl_sync(0xffffffffu, a.page, cut), r0 = __shfl_sync(0xffffffffu, a.row, cut);
                        const int n = pg < p.c.num_pages ? valid - cut * p.box_rows : 0;
                        const uint8_t* src = p.c.data[1] + w.h * p.c.sh[1] + rank * 256;
                        if (n > 0) src += pg * p.c.sp[1] + r0 * p.c.st[1];
                        for (int x = lane; x < p.box_rows * 16; x += 32) {
                            const int rr = x >> 4, c = x & 15, r = cut * p.box_rows + rr;
                            uint4 v = make_uint4(0u, 0u, 0u, 0u);
                            if (rr < n) v = __ldg(reinterpret_cast<const uint4*>(src + rr * p.c.st[1]) + c);
                            *reinterpret_cast<uint4*>(sKV + slot * C::SLOT + (r >> 3) * C::VGROUP + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
                        }
                        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                        __syncwarp();
                    }
                    if (lane == 0) {
                        if (leader) mbar_arrive_expect_tx(PPBAR(PPB_FULL + slot), 2 * (C::SLOT - (cut >= 0 ? p.box_rows * 256 : 0)));
                        else if (cut >= 0) mbar_arrive_cluster_release(l_full);
                        else mbar_arrive_remote(l_full);
                    }
                    __syncwarp();
                    const bool drop = (p.debug & ATTN_DEBUG_DROP_COPY) && leader && k && j == w.t0 && lane == 0;
                    const uint32_t dst = sKV_addr + slot * C::SLOT + lane * (p.box_rows / 8) * (k ? C::KGROUP : C::VGROUP);
                    if (lane < (k ? k_boxes : v_boxes) && lane != cut && !drop)
                        tma_load_5d_pair_hint(dst, k ? &tm_k : &tm_v, 0, 0, w.h * p.head_units[k ? 0 : 1] + (k ? 0 : 2 * rank), a.row / 8, a.page, l_full, pol_kv);
                    __syncwarp();
                }
            };
            // items in the MMA warp's order; their pages are looked up two items ahead
            const int n = je - w.t0;
            if constexpr (E4M3) {
                // one copy of the code, as in the converters
                PairItem it0 = pair_item(0, n), it1 = pair_item(1, n);
                PageAsk a0 = lookup(w.t0 + it0.j, it0.k), s0 = lookup_scale(w.t0 + it0.j, it0.k);
                PageAsk a1 = lookup(w.t0 + it1.j, it1.k), s1 = lookup_scale(w.t0 + it1.j, it1.k);
#pragma unroll 1
                for (int i = 0; i < 2 * n && ok; ++i) {
                    const PairItem it2 = i + 2 < 2 * n ? pair_item(i + 2, n) : PairItem{n, false};   // (behind the segment: no lookup)
                    const PageAsk a2 = lookup(w.t0 + it2.j, it2.k), s2 = lookup_scale(w.t0 + it2.j, it2.k);
                    copy(it0.k, w.t0 + it0.j, a0, s0);
                    it0 = it1;
                    a0 = a1;
                    s0 = s1;
                    it1 = it2;
                    a1 = a2;
                    s1 = s2;
                }
            } else {
                // (the loop above costs bf16, which has fewer instructions to wait for, 4 to 10 %)
                PageAsk ka = lookup(w.t0, true), va = lookup(w.t0, false), kn = lookup(w.t0 + 1, true);
                copy(true, w.t0, ka, ka);
                ka = lookup(w.t0 + 2, true);
                if (n > 1) copy(true, w.t0 + 1, kn, kn);
                for (int j = w.t0; j < je && ok; ++j) {
                    kn = lookup(j + 3, true);
                    const PageAsk vn = lookup(j + 1, false);
                    copy(false, j, va, va);
                    if (j + 2 < je) copy(true, j + 2, ka, ka);
                    ka = kn;
                    va = vn;
                }
            }
        }
        if (*abort_flag || !ok) {
            // copies in flight must land before the memory is reused
            const uint64_t d0 = global_timer_ns();
            while (global_timer_ns() - d0 < 2000000ull) {
            }
        }
        __syncwarp();
    } else if (E4M3 && warp >= C::WARP_CONV) {
        // ================================================================ converters (both CTAs): e4m3 K and V halves
        if constexpr (E4M3) {
            constexpr int X = 8;                 // 16-code chunks per thread and item
            const int t = tid - 32 * C::WARP_CONV;
            uint32_t item = 0;
            bool ok = true;
            for (; ok; segs.done()) {
                const ChunkSeg* sg = segs.get(abort_flag, wlim);
                ok = sg != nullptr;
                if (!ok || sg->t1 == 0) break;
                const int t0 = sg->t0, je = max(sg->end(0), sg->end(1)), kv = sg->kv;
                const int n = max(0, je - t0);
                // (one copy of the code for K and V: the kernel waits for instructions otherwise)
#pragma unroll 1
                for (int i = 0; i < 2 * n && ok; ++i) {
                    const PairItem it = pair_item(i, n);
                    const bool k = it.k;
                    const int j = t0 + it.j;
                    const int slot = static_cast<int>(item % C::NS), stg = static_cast<int>(item % C::NSTG);
                    ok = chunk_wait_warp(PPBAR(PPB_SFULL + stg), (item / C::NSTG) & 1u, abort_flag, wlim) &&
                         chunk_wait_warp(PPBAR(PPB_EMPTY + slot), ((item / C::NS) & 1u) ^ 1u, abort_flag, wlim);
                    if (!ok) break;
                    ++item;
                    // K: this rank's 64 rows of 16 chunks; V: 128 rows of this rank's 8 chunks
                    const int lg = k ? 4 : 3, RPX = 128 >> lg, group = k ? C::KGROUP : C::VGROUP;   // log2 of a row's chunks
                    const int r0 = t >> lg, c16 = t & ((1 << lg) - 1), blk = c16 >> 2;
                    const int left = kv - j * PC_BN - (k ? rank * C::KH : 0);   // rows that exist
                    const uint8_t* src = sStg + stg * C::STG_BYTES;
                    uint8_t* dst = sKV + slot * C::SLOT + blk * 1024;
                    constexpr int XB = 4;                // loads before stores, as in paged_chunk.cuh
                    TopCodes top;
#pragma unroll 1
                    for (int xb = 0; xb < X; xb += XB) {
                        uint4 d[XB];
                        uint32_t code[XB];
                        const int rb = r0 + xb * RPX;
#pragma unroll
                        for (int x = 0; x < XB; ++x) {
                            d[x] = *reinterpret_cast<const uint4*>(src + (t + (xb + x) * 128) * 16);
                            code[x] = src[C::SLOT / 2 + rb + x * RPX];
                        }
                        if (left < 128 / (k ? 2 : 1)) {
#pragma unroll
                            for (int x = 0; x < XB; ++x)
                                if (rb + x * RPX >= left) {
                                    d[x] = make_uint4(0u, 0u, 0u, 0u);
                                    code[x] = 127u;
                                }
                        }
#pragma unroll
                        for (int x = 0; x < XB; ++x) {
                            const int r = rb + x * RPX;
                            store_codes<false>(d[x], code[x], dst + (r >> 3) * group + (r & 7) * 128, (c16 & 3) * 2, r & 7, blk & 1, top);
                        }
                    }
                    if (needs_odd(top)) {
#pragma unroll 1
                        for (int r = r0; r < min(left, 128 >> (k ? 1 : 0)); r += RPX)
                            store_codes<true>(*reinterpret_cast<const uint4*>(src + (((r - r0) << lg) + t) * 16), src[C::SLOT / 2 + r],
                                              dst + (r >> 3) * group + (r & 7) * 128, (c16 & 3) * 2, r & 7, blk & 1, top);
                    }
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_cluster_release(mapa_shared(PPBAR(PPB_FULL + slot), 0));
                        mbar_arrive(PPBAR(PPB_SEMPTY + stg));
                    }
                }
            }
        }
    }

    // Neither CTA may release its TMEM or leave while the pair's MMAs, commits or copies may
    // still touch the other one.
    tc_fence_before();
    cluster_sync();
    if (warp == C::WARP_MMA) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
#undef PPBAR
}
