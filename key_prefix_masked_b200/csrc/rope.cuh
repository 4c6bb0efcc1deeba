// rope.cuh -- per-head RMS norm and rotation by position of queries and keys.
// Included by paged.cu inside namespace attn.
//
//     y = x / sqrt(mean(x^2) + eps) * w,   then on pair i of the first R elements
//     (a, b) -> f (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i]
//
// The kernel reads and writes every element once (2 + 2 bytes against ~8 operations), so
// HBM bounds it.  One block takes one token's heads: the R/2 sines and cosines are computed
// once into shared memory and used by all heads of q and k; each lane keeps its four
// pairs' values in registers.  The first rows are loaded before the sines, so that the
// loads are in flight meanwhile.
//
// Angles: position * inv_freq / 2 pi is formed in fp64 and reduced to a fraction of a turn
// by subtracting its nearest integer (exact), before the fp32 sincospi.  In fp32 the angle
// of position 10^6 would be off by up to 0.06 radians; here its error is below 10^-9.

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_U = 4;            // rows that one thread has in flight
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
    int T, R, rows_per_y;
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
    constexpr int RPI = ROPE_THREADS / LPR;   // rows per step of the block
    __shared__ float2 s_cs[D / 2];
    const int tid = threadIdx.x;
    const int c = tid % LPR;
    const Chunk ch(c, p.R);
    const int rows = p.op[0].H + p.op[1].H;
    const int b = static_cast<int>(blockIdx.x / p.T), t = static_cast<int>(blockIdx.x % p.T);
    const int begin = blockIdx.y * p.rows_per_y;
    const int end = min(rows, begin + p.rows_per_y);

    const __nv_bfloat16* base[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) base[o] = p.op[o].x + b * p.op[o].xb + t * p.op[o].xt;
    uint32_t raw[ROPE_U][4];
    auto load_rows = [&](int r0) {
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int r = r0 + u * RPI + tid / LPR;
            if (r < end) {
                const int o = r >= p.op[0].H;
                ch.load(base[o] + (o ? r - p.op[0].H : r) * p.op[o].xh, raw[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[u][i] = 0u;
            }
        }
    };
    load_rows(begin);
    const double pos = p.R > 0 ? static_cast<double>(__ldg(p.pos + blockIdx.x)) : 0.0;
    for (int i = tid; i < p.R / 2; i += ROPE_THREADS) {
        double turns = pos * __ldg(p.inv_freq + i) * 0.15915494309189533577;   // 1 / (2 pi)
        turns -= rint(turns);
        float s, co;
        sincospif(static_cast<float>(2.0 * turns), &s, &co);
        s_cs[i] = make_float2(co * p.factor, s * p.factor);
    }
    __syncthreads();
    float2 cs[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) cs[q] = q < ch.n_rot ? s_cs[ch.pair(c, q)] : make_float2(1.0f, 0.0f);

    for (int r0 = begin; r0 < end; r0 += ROPE_U * RPI) {
        if (r0 != begin) load_rows(r0);
#pragma unroll
        for (int u = 0; u < ROPE_U; ++u) {
            const int r = r0 + u * RPI + tid / LPR;
            const int o = r >= p.op[0].H;
            const RopeOperand& op = p.op[o];
            float a[4], bb[4];
            Chunk::unpack(raw[u], a, bb);
            if (op.w != nullptr || p.op[o ^ 1].w != nullptr) {   // uniform over the block: the shuffles need whole warps
                float ss = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) ss += a[q] * a[q] + bb[q] * bb[q];
#pragma unroll
                for (int k = LPR / 2; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
                if (op.w != nullptr) {
                    const float rs = rsqrtf(ss * (1.0f / D) + p.eps);
                    float wa[4], wb[4];
                    ch.weights(op.w, op.w_fp32, wa, wb);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        a[q] = a[q] * rs * wa[q];
                        bb[q] = bb[q] * rs * wb[q];
                    }
                }
            }
            if (r >= end) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q < ch.n_rot) {
                    const float x = a[q] * cs[q].x - bb[q] * cs[q].y;
                    bb[q] = bb[q] * cs[q].x + a[q] * cs[q].y;
                    a[q] = x;
                }
            }
            ch.store(op.y + b * op.yb + t * op.yt + (o ? r - p.op[0].H : r) * op.yh, a, bb);
        }
    }
}
