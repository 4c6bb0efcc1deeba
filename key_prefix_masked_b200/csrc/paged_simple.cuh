// paged_simple.cuh -- attention over pages, one warp per (query row, head).
// Included by paged.cu inside namespace attn.
//
// The definition, key by key, with the online softmax: the running maximum m and sum l,
// o <- o 2^(m - m') + p v.  Correct for every case; neither the loads nor the arithmetic are tiled.

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) paged_simple_kernel(const PagedParams p) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int hq = static_cast<int>(w % p.Hq);
    const int i = static_cast<int>((w / p.Hq) % p.max_q);
    const int b = static_cast<int>(w / p.Hq / p.max_q);
    if (b >= p.B) return;
    const QueryRange qr = query_range(p, b, i == 0 && hq == 0 && lane == 0);
    if (i >= min(qr.n, p.max_q)) return;
    const int kv = paged_kv_len(p.kv_len, b, p.kv_cap, i == 0 && hq == 0 && lane == 0);
    const int seen = p.causal ? min(kv, max(0, kv - qr.n + i + 1)) : kv;
    const int h = hq / p.G;
    float q[PER], o[PER];
    const __nv_bfloat16* qp = p.q + (qr.t0 + i) * p.q_t + hq * p.q_h + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        q[e] = __bfloat162float(qp[e]) * p.scale_log2;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    auto row = [&](int w_, int page, int r, float (&x)[PER]) {
        if (page < 0) {
#pragma unroll
            for (int e = 0; e < PER; ++e) x[e] = 0.0f;
            return;
        }
        const uint8_t* src = p.c.data[w_] + page * p.c.sp[w_] + h * p.c.sh[w_] + r * p.c.st[w_];
        if constexpr (E4M3) {
            const float s = scale_value(p.c.scale[w_][(static_cast<long long>(page) * p.c.Hkv + h) * p.c.page_size + r]);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(src[lane * PER + e], __NV_E4M3))) * s;
        } else {
#pragma unroll
            for (int e = 0; e < PER; ++e) x[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[lane * PER + e]);
        }
    };
    for (int j = 0; j < seen; ++j) {
        const int pj = j / p.c.page_size, r = j - pj * p.c.page_size;
        const int page = checked_page(p, b, pj, lane == 0);
        float x[PER], s = 0.0f;
        row(0, page, r, x);
#pragma unroll
        for (int e = 0; e < PER; ++e) s += q[e] * x[e];
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        const float m_new = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.0f : exp2f(m - m_new), pr = exp2f(s - m_new);
        m = m_new;
        l = l * f + pr;
        row(1, page, r, x);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = o[e] * f + pr * x[e];
    }
    const float inv = seen > 0 ? 1.0f / l : 0.0f;
    __nv_bfloat16* op = p.out + (qr.t0 + i) * p.out_t + hq * p.out_h + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) op[e] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[static_cast<long long>(qr.t0 + i) * p.Hq + hq] = seen > 0 ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}
