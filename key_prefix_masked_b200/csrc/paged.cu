// paged.cu -- serving operators around the prefix-masked attention: per-head norm and
// rotation of q and k (rope.cuh), a paged key/value cache written and read back
// (cache.cuh), and attention of new tokens over the pages (paged_rows.cuh for
// few query rows per key head, paged_chunk.cuh and paged_pair.cuh for many).  The C ABI is
// in include/attn_prefix.h.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <type_traits>

#include "attn_prefix.h"
#include "host_common.h"
#include "ptx.cuh"
#include "softmax_math.cuh"
#include "tmem_ops.cuh"

namespace attn {

static __device__ unsigned int g_paged_status = 0;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

// kv_len[b] clamped to [0, cap]; `report`: this thread raises the flag.
__device__ __forceinline__ int paged_kv_len(const int32_t* kv_len, int b, int cap, bool report) {
    const int kv = __ldg(kv_len + b);
    if (kv >= 0 && kv <= cap) return kv;
    if (report) atomicOr(&g_paged_status, STATUS_KVLEN);
    return kv < 0 ? 0 : cap;
}

#include "rope.cuh"
#include "cache.cuh"

// What the few-row combine kernel needs of a run that begins inside a (sequence, key head):
// n units, t0 of them in earlier runs of `per` units.  n = 0: the run begins at a border, or there is none.
struct SharedAt {
    int b, h, t0, n;
    long long per;
};

// What the chunk kernels' combine needs of a pair that several runs worked on: `parts` slots by
// number (0: none) and slots 2C + s0 .. 2C + s1, of those runs whose first record says has_s (paged_chunk.cuh).
struct SharedPair {
    int b, h, qt, parts, part[2], s0, s1, has_s;
};

struct PagedParams {
    CacheView c;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    long long q_t, q_h, out_t, out_h;   // element strides
    const int32_t* table;
    long long table_stride;
    const int32_t* kv_len;
    const int32_t* q_start;             // null: one row per sequence
    float* part_out;                    // partial results of sequences shared by several CTAs
    float* part_lse;
    SharedAt* shared_at;                // by run (paged_rows.cuh)
    SharedPair* shared;                 // two by run (paged_chunk.cuh)
    int B, T, Hq, G, max_q, kv_cap, causal;
    int min_units;                      // least tiles that a CTA takes
    int tile_keys;                      // paged_rows.cuh: keys per tile
    int page_shift;                     // log2(page_size), -1 if it is no power of two
    int tpt, box_rows, box_shift;       // paged_chunk.cuh: tokens per row tile, rows per copied box and their log2
    int head_units[2];                  // and a head's distance in column blocks (k, v)
    unsigned debug;
    unsigned long long wait_ns;
    float scale_log2;
};
// Tiles of `size` keys that hold `keys` keys, and key `at` of a tile.  A sequence has up to 2^31 - 1 keys, and
// its last tile may end behind that: the sums are unsigned.
__device__ __forceinline__ int tiles_of(int keys, int size) { return static_cast<int>((static_cast<uint32_t>(keys) + size - 1u) / size); }
__device__ __forceinline__ int key_at(int tile, int size, int at) { return static_cast<int>(static_cast<uint32_t>(tile) * size + at); }
// Index into the block table of the page that holds `key`.
__device__ __forceinline__ int page_index(const PagedParams& p, int key) {
    return p.page_shift >= 0 ? key >> p.page_shift : key / p.c.page_size;
}

// Rows [t0, t0 + n) of q belong to sequence b.
struct QueryRange {
    int t0, n;
};
__device__ __forceinline__ QueryRange query_range(const PagedParams& p, int b, bool report) {
    if (p.q_start == nullptr) return {b, 1};
    const int a = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
    const int t0 = min(max(a, 0), p.T), t1 = min(max(e, t0), p.T);
    if (report && (t0 != a || t1 != e || t1 - t0 > p.max_q)) atomicOr(&g_paged_status, STATUS_CACHE);
    return {t0, t1 - t0};
}
// Bounded waits on an mbarrier phase: false if the CTA's abort flag (where there is one) is set or
// the time limit runs out, which sets it and the device timeout flag.
template <bool CLUSTER>   // acquire at cluster scope
__device__ __forceinline__ bool chunk_poll(uint32_t bar, uint32_t parity) {
    return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}
template <bool CLUSTER>
__device__ __noinline__ bool chunk_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long limit_ns) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (chunk_poll<CLUSTER>(bar, parity)) return true;
        if (abort_flag != nullptr && *abort_flag) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            if (abort_flag != nullptr) *abort_flag = 1;
            atomicOr(&g_paged_status, STATUS_TIMEOUT);
            return false;
        }
    }
}
// Waits of a whole warp, which stays converged: true once every lane has seen the phase complete.
template <bool CLUSTER = false>
__device__ __forceinline__ bool chunk_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long limit_ns) {
    if (__all_sync(0xffffffffu, chunk_poll<CLUSTER>(bar, parity))) return true;
    return __all_sync(0xffffffffu, chunk_wait_slow<CLUSTER>(bar, parity, abort_flag, limit_ns)) != 0;
}

// ATTN_DEBUG_LATE_SOFTMAX: 20 us, in which every MMA that was issued completes.
__device__ __forceinline__ void debug_pause() {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 20000ull) {
    }
}

// A combine kernel's wait for the kernel before it in the stream to be complete (it is launched
// without one); allow_next_kernel, in that kernel, lets it be launched.
__device__ __forceinline__ void wait_for_main_kernel() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void allow_next_kernel() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

#include "paged_rows.cuh"
#include "paged_chunk.cuh"
#include "paged_pair.cuh"

bool read_paged_flags(unsigned* flags) { return cudaMemcpyFromSymbol(flags, g_paged_status, sizeof *flags) == cudaSuccess; }
bool clear_paged_flags() {
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_paged_status, &zero, sizeof zero) == cudaSuccess;
}

}  // namespace attn

// =========================================================================== host side
namespace {

using namespace attn;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides given by value or by pointer; absent or all-zero: contiguous.
bool strides_of(const attn_strides* s, int H, int T, int D, Strides* out) {
    if (s != nullptr && s->b == 0 && s->h == 0 && s->t == 0) s = nullptr;
    return resolve_strides(s, H, T, D, out);
}
// Token-major [T, H, D] rows (b ignored); absent or all-zero: contiguous.
bool token_strides_of(const attn_strides* s, int H, int D, Strides* out) {
    if (s == nullptr || (s->h == 0 && s->t == 0)) {
        *out = {0, D, static_cast<long long>(H) * D};
        return true;
    }
    if (s->h < 0 || s->t < 0 || (s->h & 7) || (s->t & 7)) return false;
    *out = {0, static_cast<long long>(s->h), static_cast<long long>(s->t)};
    return true;
}
// log2 of a page size that is a power of two, -1 otherwise
int page_shift(int page_size) {
    if ((page_size & (page_size - 1)) != 0) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}
bool head_dim_ok(int D) { return D == 32 || D == 64 || D == 128 || D == 256; }

attn_status cache_view(const attn_cache* c, CacheView* v) {
    if (c == nullptr || !c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return ATTN_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->page_size <= 0 || c->Hkv <= 0) return ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(c->num_pages) * c->page_size > 0x7fffffffLL || c->Hkv > 65535) return ATTN_ERR_INVALID_ARG;
    if (c->format != ATTN_CACHE_BF16 && c->format != ATTN_CACHE_E4M3) return ATTN_ERR_UNSUPPORTED;
    if (!head_dim_ok(c->D) || (c->page_size & 7)) return ATTN_ERR_UNSUPPORTED;
    const bool e4m3 = c->format == ATTN_CACHE_E4M3;
    if (e4m3 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 8) || !aligned(c->v_scale, 8))) return ATTN_ERR_INVALID_ARG;
    const int size = e4m3 ? 1 : 2;
    Strides s[2];
    if (!strides_of(&c->k_strides, c->Hkv, c->page_size, c->D, &s[0]) ||
        !strides_of(&c->v_strides, c->Hkv, c->page_size, c->D, &s[1]))
        return ATTN_ERR_INVALID_ARG;
    memset(v, 0, sizeof *v);
    for (int i = 0; i < 2; ++i) {
        if ((s[i].b * size) & 15 || (s[i].h * size) & 15 || (s[i].t * size) & 15) return ATTN_ERR_INVALID_ARG;
        const int blk = c->D < 64 ? c->D : 64;
        if (c->Hkv == 1) s[i].h = c->D;                                       // not used
        if (s[i].h % blk != 0 || s[i].h == 0 || (s[i].b == 0 && c->num_pages > 1)) return ATTN_ERR_INVALID_ARG;
        if (s[i].h / blk > (0x7fffffffLL - c->D) / c->Hkv) return ATTN_ERR_INVALID_ARG;   // the kernels count heads in blocks
        v->data[i] = static_cast<uint8_t*>(i ? c->v : c->k);
        v->scale[i] = e4m3 ? (i ? c->v_scale : c->k_scale) : nullptr;
        v->sp[i] = s[i].b * size;
        v->sh[i] = s[i].h * size;
        v->st[i] = s[i].t * size;
    }
    v->num_pages = c->num_pages;
    v->page_size = c->page_size;
    v->Hkv = c->Hkv;
    v->D = c->D;
    v->e4m3 = e4m3;
    return ATTN_OK;
}

constexpr int SM_COUNT = 148;   // B200

attn_status launched() { return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

template <int D>
attn_status launch_rope(const RopeParams& prm, int mode, long long tokens, cudaStream_t stream) {
    constexpr int RPW = 256 / D;   // rows per step of a warp
    RopeParams p = prm;
    // Few tokens: their heads are spread over warps until there are eight per SM; many: a warp
    // takes a token's heads, but at most 16 steps of them (the sines cost about as much as six).
    const int steps = (p.op[0].H + p.op[1].H + RPW - 1) / RPW;
    long long parts = (8LL * SM_COUNT + tokens - 1) / tokens;
    if (parts < (steps + 15) / 16) parts = (steps + 15) / 16;
    if (parts > steps) parts = steps;
    p.rows_per_part = static_cast<int>((steps + parts - 1) / parts) * RPW;
    p.parts = (p.op[0].H + p.op[1].H + p.rows_per_part - 1) / p.rows_per_part;
    p.tasks = tokens * p.parts;
    const long long grid = (p.tasks + ROPE_THREADS / 32 - 1) / (ROPE_THREADS / 32);
    if (grid > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    const unsigned g = static_cast<unsigned>(grid);
    if (mode == ROPE_INTERLEAVED) qk_norm_rope_kernel<D, ROPE_INTERLEAVED><<<g, ROPE_THREADS, 0, stream>>>(p);
    else if (mode == ROPE_HALF) qk_norm_rope_kernel<D, ROPE_HALF><<<g, ROPE_THREADS, 0, stream>>>(p);
    else qk_norm_rope_kernel<D, ROPE_HALF_SCALAR><<<g, ROPE_THREADS, 0, stream>>>(p);
    return launched();
}

template <int D>
attn_status launch_write(const CacheWriteParams& prm, long long tokens, cudaStream_t stream) {
    constexpr int RPW = 256 / D;   // rows per step of a warp
    CacheWriteParams p = prm;
    p.page_shift = page_shift(p.c.page_size);
    // few tokens: their rows are spread over warps until there are eight per SM
    const int steps = (2 * p.c.Hkv + RPW - 1) / RPW;
    long long parts = (8LL * SM_COUNT + tokens - 1) / tokens;
    if (parts > steps) parts = steps;
    p.rows_per_part = static_cast<int>((steps + parts - 1) / parts) * RPW;
    p.parts = (2 * p.c.Hkv + p.rows_per_part - 1) / p.rows_per_part;
    p.tasks = tokens * p.parts;
    const long long grid = (p.tasks + CACHE_THREADS / 32 - 1) / (CACHE_THREADS / 32);
    if (grid > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    if (p.c.e4m3) cache_write_kernel<D, true><<<static_cast<unsigned>(grid), CACHE_THREADS, 0, stream>>>(p);
    else cache_write_kernel<D, false><<<static_cast<unsigned>(grid), CACHE_THREADS, 0, stream>>>(p);
    return launched();
}

template <int D>
attn_status launch_read(const CacheReadParams& prm, int B, cudaStream_t stream) {
    const int ROWS = CACHE_THREADS / (D / (prm.c.e4m3 ? 16 : 8)) * CACHE_READ_U;
    CacheReadParams p = prm;
    p.page_shift = page_shift(p.c.page_size);
    const long long n_rb = (static_cast<long long>(p.Tk) + ROWS - 1) / ROWS;
    const long long grid = n_rb * B * p.c.Hkv;
    if (grid > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    p.n_rb = static_cast<int>(n_rb);
    if (p.c.e4m3) cache_read_kernel<D, true><<<static_cast<unsigned>(grid), CACHE_THREADS, 0, stream>>>(p);
    else cache_read_kernel<D, false><<<static_cast<unsigned>(grid), CACHE_THREADS, 0, stream>>>(p);
    return launched();
}

// CTAs of the few-row kernel: every resident slot, or fewer where the largest possible work
// (every sequence of kv_cap keys) needs fewer.
constexpr int ROWS_MIN_UNITS = 2;
int rows_ctas(int per_sm, int tile_keys, int B, int Hkv, long long kv_cap) {
    const long long enough = static_cast<long long>(ROWS_MIN_UNITS) * SM_COUNT * per_sm;
    const long long pairs = static_cast<long long>(B) * Hkv, units = pairs < enough ? pairs * ((kv_cap + tile_keys - 1) / tile_keys) : enough;
    const long long most = (units + ROWS_MIN_UNITS - 1) / ROWS_MIN_UNITS;
    return static_cast<int>(most < SM_COUNT * per_sm ? most : SM_COUNT * per_sm);
}
// Few rows per key head: at most one m16 tile of them.  16 rows on the chunk kernels instead (64 heads
// on 4, 32 sequences of 16384 keys, D 128): bf16 231 against 182 us, e4m3 319 against 147.  Beyond the border the
// chunk kernels' two 128-row tiles are mostly empty and a key costs as much as for full ones: 17 rows (4 heads on
// 4, same keys) bf16 238 us, e4m3 325; 64 rows 252 and 322; 128 rows 270 and 341; 256 rows 326 and 407.
bool few_rows(long long max_q, int G) { return max_q * G <= PR_ROWS; }

// A combine kernel behind the main one, launched to overlap it (it waits on the device).
template <typename... Args>
attn_status launch_combine(void (*kern)(Args...), dim3 grid, int threads, cudaStream_t stream, const Args&... args) {
    if (grid.x == 0) return launched();
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    memset(&attr, 0, sizeof attr);
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kern, args...);
    return launched();
}

template <int D, bool E4M3>
attn_status launch_rows(PagedParams p, void* workspace, cudaStream_t stream) {
    using C = RowsCfg<D, E4M3>;
    const int n = rows_ctas(C::PER_SM, C::TK, p.B, p.c.Hkv, p.kv_cap);
    p.min_units = ROWS_MIN_UNITS;
    p.tile_keys = C::TK;
    p.part_out = static_cast<float*>(workspace);
    p.part_lse = p.part_out + 2LL * n * PR_ROWS * D;
    p.shared_at = reinterpret_cast<SharedAt*>(p.part_lse + 2LL * n * PR_ROWS);
    if (cudaFuncSetAttribute(paged_rows_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    CUtensorMap mk, mv;
    memset(&mk, 0, sizeof mk);
    mv = mk;
    p.box_rows = p.c.page_size & -p.c.page_size;
    if (p.box_rows > C::WK) p.box_rows = C::WK;
    for (int i = 0; E4M3 && i < 2; ++i) {
        const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.c.page_size), static_cast<cuuint64_t>(p.c.Hkv),
                                    static_cast<cuuint64_t>(p.c.num_pages)};
        const cuuint64_t str[3] = {static_cast<cuuint64_t>(p.c.st[i]), static_cast<cuuint64_t>(p.c.sh[i]), static_cast<cuuint64_t>(p.c.sp[i])};
        const cuuint32_t box[4] = {C::SW, static_cast<cuuint32_t>(p.box_rows), 1u, 1u};
        if (!encode_map(i ? &mv : &mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.c.data[i], dims, str, box,
                        C::SW == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : C::SW == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B))
            return ATTN_ERR_CUDA;
    }
    paged_rows_kernel<D, E4M3><<<n, PR_THREADS, C::SMEM, stream>>>(mk, mv, p, n);
    return launch_combine(paged_rows_combine_kernel<D>, dim3(n - 1, p.max_q * p.G), PR_THREADS, stream, p);
}

// Runs of the chunk kernels: one per SM (per CTA pair at head dim 256), or fewer where the
// largest possible work needs fewer.
constexpr int CHUNK_MIN_UNITS = 2;
int chunk_runs(int B, int Hkv, int G, int D, long long max_q, long long kv_cap) {
    const int tokens = 2 * (128 / G), all = D == 256 ? SM_COUNT / 2 : SM_COUNT;
    const long long enough = static_cast<long long>(CHUNK_MIN_UNITS) * all;
    long long units = static_cast<long long>(B) * Hkv;   // (each factor is below 2^31)
    for (const long long f : {(max_q + tokens - 1) / tokens, (kv_cap + PC_BN - 1) / PC_BN}) units = units < enough ? units * f : enough;
    const long long most = (units + CHUNK_MIN_UNITS - 1) / CHUNK_MIN_UNITS;
    return static_cast<int>(most < all ? most : all);
}

template <int D, bool E4M3>
attn_status launch_chunk(PagedParams p, void* workspace, cudaStream_t stream) {
    constexpr bool PAIR = D == 256;
    constexpr int BLK = D >= 64 ? 64 : 32;
    const int n = chunk_runs(p.B, p.c.Hkv, p.G, D, p.max_q, p.kv_cap);
    p.min_units = CHUNK_MIN_UNITS;
    p.part_out = static_cast<float*>(workspace);
    p.part_lse = p.part_out + 1024LL * n * D;
    p.shared = reinterpret_cast<SharedPair*>(p.part_lse + 1024LL * n);
    p.tpt = 128 / p.G;
    p.box_rows = p.c.page_size & -p.c.page_size;   // the largest power of two that divides it
    const int most = PAIR ? 64 : PC_BN;
    if (p.box_rows > most) p.box_rows = most;
    p.box_shift = page_shift(p.box_rows);
    const CUtensorMapSwizzle swz = BLK == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, p.q, p.T, p.c.Hkv, p.G, D, {p.q_t, p.G * p.q_h, p.q_h}, BLK, p.G, swz, p.tpt)) return ATTN_ERR_CUDA;
    // K, V.  e4m3: rows of D codes (half of V's at head dim 256), as they lie.  bf16: a page as
    // [8-row group][head and column block][8 rows][block], so that one box takes whole rows
    // into shared memory group by group; heads are counted in column blocks.
    for (int i = 0; i < 2; ++i) {
        const CacheView& c = p.c;
        CUtensorMap* m = i ? &mv : &mk;
        p.head_units[i] = static_cast<int>(c.sh[i] / (2 * BLK));
        const cuuint64_t u = static_cast<cuuint64_t>(c.Hkv - 1) * p.head_units[i] + D / BLK;
        const cuuint64_t sp = c.sp[i], sh = c.sh[i], st = c.st[i], P = c.num_pages, page = c.page_size;
        const cuuint32_t rows = p.box_rows, part = PAIR && i ? 2u : 1u;   // a V box of a pair: half the columns
        if (E4M3) {
            const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), page, static_cast<cuuint64_t>(c.Hkv), P}, str[3] = {st, sh, sp};
            const cuuint32_t box[4] = {D / part, rows, 1u, 1u};
            if (!encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.data[i], dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE)) return ATTN_ERR_CUDA;
        } else {
            const cuuint64_t dims[5] = {static_cast<cuuint64_t>(BLK), 8, u, page / 8, P}, str[4] = {st, 2 * BLK, 8 * st, sp};
            const cuuint32_t box[5] = {static_cast<cuuint32_t>(BLK), 8u, static_cast<cuuint32_t>(D / BLK) / part, rows / 8, 1u};
            if (!encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, c.data[i], dims, str, box, swz)) return ATTN_ERR_CUDA;
        }
    }
    int grid, threads, smem;
    void (*kern)(CUtensorMap, CUtensorMap, CUtensorMap, PagedParams, int);
    if constexpr (PAIR) {
        using C = PagedPairCfg<E4M3>;
        kern = paged_pair_kernel<E4M3>;
        grid = 2 * n;
        threads = C::THREADS;
        smem = C::SMEM;
    } else {
        using C = ChunkCfg<D, E4M3>;
        kern = paged_chunk_kernel<D, E4M3>;
        grid = n;
        threads = C::THREADS;
        smem = C::SMEM;
    }
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    kern<<<grid, threads, smem, stream>>>(mq, mk, mv, p, n);
    return launch_combine(paged_chunk_combine_kernel<D>, dim3(2 * n, 16), 256, stream, p, n);
}

template <int D>
attn_status launch_paged(const PagedParams& p, void* workspace, cudaStream_t stream) {
    if (few_rows(p.max_q, p.G)) return p.c.e4m3 ? launch_rows<D, true>(p, workspace, stream) : launch_rows<D, false>(p, workspace, stream);
    return p.c.e4m3 ? launch_chunk<D, true>(p, workspace, stream) : launch_chunk<D, false>(p, workspace, stream);
}

#define ATTN_BY_HEAD_DIM(D, CALL)          \
    switch (D) {                           \
        case 32: return CALL(32);          \
        case 64: return CALL(64);          \
        case 128: return CALL(128);        \
        default: return CALL(256);         \
    }

}  // namespace

extern "C" {

attn_status attn_qk_norm_rope(const attn_rope_operand* q, const attn_rope_operand* k, const int32_t* positions,
                              const double* inv_freq, int B, int T, int D, int R, int interleaved, float eps,
                              float attn_factor, cudaStream_t stream) {
    if (!q || !q->x || B <= 0 || T <= 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * T > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    if (R < 0 || R > D || (R & 1) || !isfinite(eps) || eps < 0.0f || !isfinite(attn_factor)) return ATTN_ERR_INVALID_ARG;
    if (R > 0 && (!positions || !aligned(positions, 4) || !inv_freq || !aligned(inv_freq, 8))) return ATTN_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return ATTN_ERR_UNSUPPORTED;
    RopeParams p;
    memset(&p, 0, sizeof p);
    const attn_rope_operand* ops[2] = {q, k != nullptr && k->x != nullptr ? k : nullptr};
    for (int i = 0; i < 2; ++i) {
        const attn_rope_operand* o = ops[i];
        if (o == nullptr) continue;
        if (!o->y || !aligned16(o->x) || !aligned16(o->y) || o->H <= 0) return ATTN_ERR_INVALID_ARG;
        if (o->weight && !aligned16(o->weight)) return ATTN_ERR_INVALID_ARG;
        Strides x, y;
        if (!strides_of(&o->x_strides, o->H, T, D, &x) || !strides_of(&o->y_strides, o->H, T, D, &y))
            return ATTN_ERR_INVALID_ARG;
        p.op[i] = {static_cast<const __nv_bfloat16*>(o->x), static_cast<__nv_bfloat16*>(o->y), o->weight, o->H,
                   o->weight_fp32 != 0, x.b, x.h, x.t, y.b, y.h, y.t};
    }
    if (static_cast<long long>(p.op[0].H) + p.op[1].H > 65535) return ATTN_ERR_INVALID_ARG;
    attn_status st = check_device();
    if (st != ATTN_OK) return st;
    p.pos = positions;
    p.inv_freq = inv_freq;
    p.T = T;
    p.R = R;
    p.eps = eps;
    p.factor = attn_factor;
    const int mode = interleaved ? ROPE_INTERLEAVED : (R & 7) == 0 ? ROPE_HALF : ROPE_HALF_SCALAR;
    const long long tokens = static_cast<long long>(B) * T;
#define CALL(DD) launch_rope<DD>(p, mode, tokens, stream)
    ATTN_BY_HEAD_DIM(D, CALL)
#undef CALL
}

attn_status attn_cache_write(const attn_cache* cache, const void* k, const void* v, const attn_strides* k_strides,
                             const attn_strides* v_strides, const int32_t* slots, int T, cudaStream_t stream) {
    CacheWriteParams p;
    memset(&p, 0, sizeof p);
    attn_status st = cache_view(cache, &p.c);
    if (st != ATTN_OK) return st;
    if (!k || !v || !aligned16(k) || !aligned16(v) || !slots || !aligned(slots, 4) || T <= 0) return ATTN_ERR_INVALID_ARG;
    Strides s[2];
    if (!token_strides_of(k_strides, cache->Hkv, cache->D, &s[0]) || !token_strides_of(v_strides, cache->Hkv, cache->D, &s[1]))
        return ATTN_ERR_INVALID_ARG;
    if ((st = check_device()) != ATTN_OK) return st;
    p.src[0] = static_cast<const __nv_bfloat16*>(k);
    p.src[1] = static_cast<const __nv_bfloat16*>(v);
    for (int i = 0; i < 2; ++i) {
        p.st[i] = s[i].t;
        p.sh[i] = 2 * s[i].h;
    }
    p.slots = slots;
#define CALL(DD) launch_write<DD>(p, T, stream)
    ATTN_BY_HEAD_DIM(cache->D, CALL)
#undef CALL
}

attn_status attn_cache_read(const attn_cache* cache, const int32_t* block_table, int64_t table_stride, int max_pages,
                            const int32_t* kv_len, void* k_out, void* v_out, const attn_strides* k_strides,
                            const attn_strides* v_strides, int B, int Tk, cudaStream_t stream) {
    CacheReadParams p;
    memset(&p, 0, sizeof p);
    attn_status st = cache_view(cache, &p.c);
    if (st != ATTN_OK) return st;
    if (!block_table || !aligned(block_table, 4) || !kv_len || !aligned(kv_len, 4)) return ATTN_ERR_INVALID_ARG;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return ATTN_ERR_INVALID_ARG;
    if (B <= 0 || Tk <= 0 || max_pages <= 0 || table_stride < 0) return ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * cache->Hkv > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    Strides s[2];
    if (!strides_of(k_strides, cache->Hkv, Tk, cache->D, &s[0]) || !strides_of(v_strides, cache->Hkv, Tk, cache->D, &s[1]))
        return ATTN_ERR_INVALID_ARG;
    if ((st = check_device()) != ATTN_OK) return st;
    p.dst[0] = static_cast<__nv_bfloat16*>(k_out);
    p.dst[1] = static_cast<__nv_bfloat16*>(v_out);
    for (int i = 0; i < 2; ++i) {
        p.sb[i] = s[i].b;
        p.sh[i] = s[i].h;
        p.st[i] = s[i].t;
    }
    p.table = block_table;
    p.table_stride = table_stride;
    p.kv_len = kv_len;
    p.max_pages = max_pages;
    p.Tk = Tk;
#define CALL(DD) launch_read<DD>(p, B, stream)
    ATTN_BY_HEAD_DIM(cache->D, CALL)
#undef CALL
}

size_t attn_paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int page_size, int max_pages, int max_q) {
    if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > 128 || D <= 0 || page_size <= 0 || max_pages <= 0 || max_q <= 0)
        return 0;
    const long long q = max_q < T ? max_q : T, cap = static_cast<long long>(max_pages) * page_size;
    // per run: its parts (two of 16 rows, four of 256) of D + 1 floats a row, and the records
    if (few_rows(q, Hq / Hkv))
        return rows_ctas(2, RowsCfg<32, false>::TK, B, Hkv, cap) * (2ull * PR_ROWS * (D + 1) * sizeof(float) + sizeof(SharedAt));
    return chunk_runs(B, Hkv, Hq / Hkv, D, q, cap) * (1024ull * (D + 1) * sizeof(float) + 2 * sizeof(SharedPair));
}

attn_status attn_paged_fwd(const attn_cache* cache, const void* q, const attn_strides* q_strides,
                           const int32_t* block_table, int64_t table_stride, int max_pages, const int32_t* kv_len,
                           const int32_t* q_start, void* out, const attn_strides* out_strides, float* lse,
                           void* workspace, int B, int T, int Hq, int max_q, int causal, float scale,
                           cudaStream_t stream) {
    PagedParams p;
    memset(&p, 0, sizeof p);
    attn_status st = cache_view(cache, &p.c);
    if (st != ATTN_OK) return st;
    if (!q || !out || !aligned16(q) || !aligned16(out) || !block_table || !aligned(block_table, 4)) return ATTN_ERR_INVALID_ARG;
    if (!kv_len || !aligned(kv_len, 4) || !aligned(q_start, 4) || !aligned(lse, 4)) return ATTN_ERR_INVALID_ARG;
    if (B <= 0 || T <= 0 || Hq <= 0 || max_q <= 0 || max_pages <= 0 || table_stride < 0) return ATTN_ERR_INVALID_ARG;
    if (Hq % cache->Hkv != 0 || Hq / cache->Hkv > 128 || (q_start == nullptr && B != T)) return ATTN_ERR_INVALID_ARG;
    if (!isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * Hq > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    const long long cap = static_cast<long long>(max_pages) * cache->page_size;
    if (cap > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
    Strides sq, so;
    if (!token_strides_of(q_strides, Hq, cache->D, &sq) || !token_strides_of(out_strides, Hq, cache->D, &so))
        return ATTN_ERR_INVALID_ARG;
    for (const Strides& s : {sq, so})   // rows of their own (no broadcast heads or tokens)
        if ((Hq > 1 && s.h == 0) || (T > 1 && s.t == 0)) return ATTN_ERR_INVALID_ARG;
    const int rows_q = q_start == nullptr ? 1 : max_q < T ? max_q : T;
    const size_t need = attn_paged_workspace_bytes(B, T, Hq, cache->Hkv, cache->D, cache->page_size, max_pages, rows_q);
    if (need != 0 && (!workspace || !aligned16(workspace))) return ATTN_ERR_INVALID_ARG;
    if ((st = check_device()) != ATTN_OK) return st;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.q_t = sq.t;
    p.q_h = sq.h;
    p.out_t = so.t;
    p.out_h = so.h;
    p.table = block_table;
    p.table_stride = table_stride;
    p.kv_len = kv_len;
    p.q_start = q_start;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.G = Hq / cache->Hkv;
    p.max_q = rows_q;
    p.kv_cap = static_cast<int>(cap);
    p.causal = causal != 0;
    p.page_shift = page_shift(cache->page_size);
    p.debug = g_debug.load(std::memory_order_relaxed);
    p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    p.scale_log2 = scale * 1.44269504088896340736f;
#define CALL(DD) launch_paged<DD>(p, workspace, stream)
    ATTN_BY_HEAD_DIM(cache->D, CALL)
#undef CALL
}

}  // extern "C"
