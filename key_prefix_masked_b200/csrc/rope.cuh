// rope.cuh -- per-head RMS norm and rotation by position of queries and keys.
// Included by paged.cu inside namespace attn.
//
//     y = x / sqrt(mean(x^2) + eps) * w,   then on pair i of the first R elements
//     (a, b) -> f (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i]
//
// The kernel reads and writes every element once (2 + 2 bytes against ~8 operations), so
// HBM bounds it.  A warp takes one token (or, where there are few tokens, a part of its heads):
// each lane computes the sines and cosines of its four pairs once, into registers, keeps the
// weights of its eight elements there too, and then streams the heads' rows through, with
// ROPE_U rows in flight.  No shared memory and no barrier, so the warps of an SM cover each
// other's latencies.  Measured at 65536 tokens of 40 heads of 128 (1.34 GB): 255 to 269 us, 5.0 to 5.3 TB/s
// (R = 36 in the half layout, whose pairs lie at no 8-byte border and are moved two bytes at a time: 519 us); one
// block per token, with the sines shared through shared memory, 394 us; one row in flight per lane
// 281 us, three 298, four 284 (fewer warps fit), blocks of 256 threads 282.
//
// Angles: position * inv_freq / 2 pi is formed in fp64 and reduced to a fraction of a turn
// by subtracting its nearest integer (exact), before the fp32 sincospi.  In fp32 the angle
// of position 10^6 would be off by up to 0.06 radians; here its error is below 10^-9.

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_U = 2;            // steps (rows per lane) in flight
enum : int { ROPE_HALF = 0, ROPE_INTERLEAVED = 1, ROPE_HALF_SCALAR = 2 };

struct RopeOperand {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const void* w;
    int H, w_fp32;
    long long xb, xh, xt, yb, yh, yt;   // element strides
};
struct RopeParams {
    RopeOperand op[2];   // q, k (H = 0: absent)
    const int32_t* pos;
    const double* inv_freq;
    int T, R;
    int parts, rows_per_part;   // warps per token, and rows (heads) of each
    long long tasks;            // tokens * parts
    float eps, factor;
};

// The eight elements of a lane's chunk c of a row, as four pairs: the offsets of a pair's
// first (k = 0) and second (k = 1) element.  With R % 8 == 0 they are two runs of four
// (8-byte accesses) in the half layout, one run of eight in the interleaved one.
template <int D, int MODE>
struct RopeChunk {
    static constexpr int LPR = D / 8;   // lanes per row
    int lo, hi, n_rot;                  // run starts; pairs p < n_rot are rotated
    __device__ __forceinline__ RopeChunk(int c, int R) {
        if constexpr (MODE == ROPE_HALF) {
            const bool rot = 8 * c < R;
            lo = rot ? 4 * c : 8 * c;
            hi = rot ? R / 2 + 4 * c : 8 * c + 4;
            n_rot = rot ? 4 : 0;
        } else if constexpr (MODE == ROPE_INTERLEAVED) {
            lo = 8 * c;
            hi = 8 * c + 4;
            n_rot = min(4, max(0, R / 2 - 4 * c));
        } else {
            // pairs c, c + LPR, ...: pair p < R/2 is (p, p + R/2), the others are neighbours behind R
            lo = c;
            hi = R / 2;
            n_rot = min(4, max(0, (R / 2 - c + LPR - 1) / LPR));
        }
    }
    __device__ __forceinline__ int pair(int c, int p) const { return MODE == ROPE_HALF_SCALAR ? c + LPR * p : 4 * c + p; }
    // scalar mode: element offsets of pair p
    __device__ __forceinline__ int first(int p) const {
        const int i = lo + LPR * p;
        return p < n_rot ? i : 2 * i;
    }
    __device__ __forceinline__ int second(int p) const {
        const int i = lo + LPR * p;
        return p < n_rot ? i + hi : 2 * i + 1;
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* row, uint32_t (&v)[4]) const {
        if constexpr (MODE == ROPE_HALF) {
            const uint2 a = *reinterpret_cast<const uint2*>(row + lo);
            const uint2 b = *reinterpret_cast<const uint2*>(row + hi);
            v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
        } else if constexpr (MODE == ROPE_INTERLEAVED) {
            const uint4 a = *reinterpret_cast<const uint4*>(row + lo);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        } else {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p] = static_cast<uint32_t>(r[first(p)]) | static_cast<uint32_t>(r[second(p)]) << 16;
        }
    }
    // a[p], b[p]: first and second element of pair p
    static __device__ __forceinline__ void unpack(const uint32_t (&v)[4], float (&a)[4], float (&b)[4]) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            a[p] = MODE == ROPE_HALF ? f[p] : f[2 * p];
            b[p] = MODE == ROPE_HALF ? f[4 + p] : f[2 * p + 1];
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* row, const float (&a)[4], const float (&b)[4]) const {
        if constexpr (MODE == ROPE_HALF) {
            *reinterpret_cast<uint2*>(row + lo) = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
            *reinterpret_cast<uint2*>(row + hi) = make_uint2(pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]));
        } else if constexpr (MODE == ROPE_INTERLEAVED) {
            *reinterpret_cast<uint4*>(row + lo) = make_uint4(pack_bf16(a[0], b[0]), pack_bf16(a[1], b[1]),
                                                             pack_bf16(a[2], b[2]), pack_bf16(a[3], b[3]));
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                row[first(p)] = __float2bfloat16_rn(a[p]);
                row[second(p)] = __float2bfloat16_rn(b[p]);
            }
        }
    }
    // the weights of the lane's elements, in pair order
    __device__ __forceinline__ void weights(const void* w, int fp32, float (&wa)[4], float (&wb)[4]) const {
        if (fp32) {
            const float* r = static_cast<const float*>(w);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                wa[p] = __ldg(r + (MODE == ROPE_HALF ? lo + p : MODE == ROPE_INTERLEAVED ? lo + 2 * p : first(p)));
                wb[p] = __ldg(r + (MODE == ROPE_HALF ? hi + p : MODE == ROPE_INTERLEAVED ? lo + 2 * p + 1 : second(p)));
            }
        } else {
            uint32_t v[4];
            load(static_cast<const __nv_bfloat16*>(w), v);
            unpack(v, wa, wb);
        }
    }
};

template <int D, int MODE>
__global__ void __launch_bounds__(ROPE_THREADS) qk_norm_rope_kernel(const RopeParams p) {
    using Chunk = RopeChunk<D, MODE>;
    constexpr int LPR = Chunk::LPR;
    constexpr int RPW = 32 / LPR;   // rows per step of the warp
    const int lane = threadIdx.x & 31;
    const long long task = static_cast<long long>(blockIdx.x) * (ROPE_THREADS / 32) + (threadIdx.x >> 5);
    if (task >= p.tasks) return;
    const long long token = task / p.parts;
    const int part = static_cast<int>(task - token * p.parts);
    const long long b = token / p.T;
    const int t = static_cast<int>(token - b * p.T);
    const int c = lane % LPR;
    const Chunk ch(c, p.R);
    const int begin = part * p.rows_per_part, end = min(p.op[0].H + p.op[1].H, begin + p.rows_per_part);

    float2 cs[4];
    bool have_cs = false;
#pragma unroll 1
    for (int o = 0; o < 2; ++o) {
        const RopeOperand& op = p.op[o];
        // this part's heads of the operand
        const int h0 = max(0, begin - (o ? p.op[0].H : 0)), h1 = min(op.H, end - (o ? p.op[0].H : 0));
        if (h0 >= h1) continue;
        const __nv_bfloat16* x = op.x + b * op.xb + t * op.xt;
        __nv_bfloat16* y = op.y + b * op.yb + t * op.yt;
        const int r0 = h0 + lane / LPR;
        const __nv_bfloat16* xr = x + r0 * op.xh;    // the row that is loaded next
        __nv_bfloat16* yr = y + r0 * op.yh;          // and the one that is stored next
        const long long x_step = RPW * op.xh, y_step = RPW * op.yh;
        uint32_t raw[ROPE_U][4];
        auto load = [&](int r, uint32_t (&v)[4]) {   // row r (a head), zeros behind the last
            if (r < h1) {
                ch.load(xr, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = 0u;
            }
            xr += x_step;
        };
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) load(r0 + u * RPW, raw[u]);
        float wa[4], wb[4];
        if (op.w != nullptr) ch.weights(op.w, op.w_fp32, wa, wb);
        if (!have_cs) {
            have_cs = true;
            const double pos = p.R > 0 ? static_cast<double>(__ldg(p.pos + token)) : 0.0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                cs[q] = make_float2(1.0f, 0.0f);
                if (q < ch.n_rot) {
                    double turns = pos * __ldg(p.inv_freq + ch.pair(c, q)) * 0.15915494309189533577;   // 1 / (2 pi)
                    turns -= rint(turns);
                    sincospif(static_cast<float>(2.0 * turns), &cs[q].y, &cs[q].x);
                    cs[q].x *= p.factor;
                    cs[q].y *= p.factor;
                }
            }
        }
#pragma unroll 1
        for (int r = r0; r - lane / LPR < h1; r += ROPE_U * RPW) {
#pragma unroll
            for (int u = 0; u < ROPE_U; ++u) {
                const int row = r + u * RPW;
                float a[4], bb[4];
                Chunk::unpack(raw[u], a, bb);
                load(row + ROPE_U * RPW, raw[u]);
                // packed pairs: elements 0, 1 and 2, 3 of a and of bb
                float2 a2[2] = {make_float2(a[0], a[1]), make_float2(a[2], a[3])};
                float2 b2[2] = {make_float2(bb[0], bb[1]), make_float2(bb[2], bb[3])};
                if (op.w != nullptr) {
                    const float2 zero = make_float2(0.0f, 0.0f);
                    const float2 s2 = fma2(b2[1], b2[1], fma2(a2[1], a2[1], fma2(b2[0], b2[0], fma2(a2[0], a2[0], zero))));
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int k = LPR / 2; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
                    const float rs = rsqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        a2[q] = mul2(mul2(a2[q], make_float2(rs, rs)), make_float2(wa[2 * q], wa[2 * q + 1]));
                        b2[q] = mul2(mul2(b2[q], make_float2(rs, rs)), make_float2(wb[2 * q], wb[2 * q + 1]));
                    }
                }
                __nv_bfloat16* dst = yr;
                yr += y_step;
                if (row >= h1) continue;
                if (ch.n_rot == 4) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 co = make_float2(cs[2 * q].x, cs[2 * q + 1].x), si = make_float2(cs[2 * q].y, cs[2 * q + 1].y);
                        const float2 ni = make_float2(-cs[2 * q].y, -cs[2 * q + 1].y);
                        const float2 z = fma2(a2[q], co, mul2(b2[q], ni));
                        b2[q] = fma2(b2[q], co, mul2(a2[q], si));
                        a2[q] = z;
                    }
                }
                a[0] = a2[0].x; a[1] = a2[0].y; a[2] = a2[1].x; a[3] = a2[1].y;
                bb[0] = b2[0].x; bb[1] = b2[0].y; bb[2] = b2[1].x; bb[3] = b2[1].y;
                if (MODE != ROPE_HALF && ch.n_rot < 4) {   // the chunk in which the rotated part ends
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        if (q < ch.n_rot) {
                            const float z = a[q] * cs[q].x - bb[q] * cs[q].y;
                            bb[q] = bb[q] * cs[q].x + a[q] * cs[q].y;
                            a[q] = z;
                        }
                    }
                }
                ch.store(dst, a, bb);
            }
        }
    }
}
