// kv8_decode.cuh -- one generation step over the paged 8-bit cache of kv8.cuh, for requests of
// different lengths: request b has n_b = seq_len[b] tokens, the new one at position n_b - 1.
//   1. kv8_token_kernel: the layer's prologue of the new token, as in decode.cuh (every qhat, khat and
//      v' element the correctly rounded bf16 of its exact value); qhat goes to the workspace, khat and v'
//      into the token's page, whose scale grows where they need it (kv8.cuh).
//   2. the attention of qhat over the cached keys [max(0, n_b - W, min(start_b, n_b - 1)), n_b):
//      out = sum_j softmax_j(qhat . k_j / sqrt(D)) v_j,  lse = ln sum_j exp(qhat . k_j / sqrt(D)).
// Requests with n_b <= 0 are empty rows: out = 0, lse = -inf.
#pragma once

#include "kv8.cuh"

namespace swa {

constexpr int kKv8MaxGroup = 64;  // query heads of one key/value head

struct Kv8TokenParams {
    const __nv_bfloat16* q;       // (B, H, D)
    const __nv_bfloat16* k;       // (B, Hkv, D), or null: the token is in the cache already
    const __nv_bfloat16* v;
    const __nv_bfloat16* ve;      // value-embedding layers, else null
    const __nv_bfloat16* gate_x;
    const __nv_bfloat16* Wg;
    const int* table;             // (B, max_pages)
    const int* seq_len;           // (B)
    __nv_bfloat16* qh;            // (B, H, D), workspace
    __nv_bfloat16* out;           // (B, H, D): the empty rows are written here
    float* lse;                   // (B, H) or null
    Kv8Store c;
    int H, max_pages;
    double base, eps;
};

// Number of cached keys of request b: its sequence length, 0 where that is not positive or (recorded)
// does not fit in the block table.
__device__ __forceinline__ int kv8_length(const int* seq_len, int b, int max_pages, int log_p) {
    const int n = __ldg(seq_len + b);
    return n <= 0 || (long long)n > ((long long)max_pages << log_p) ? 0 : n;
}

// Rows of request b = blockIdx.x: its H query rows, then its Hkv key/value rows (when the token is to be
// appended), D/8 lanes a row; blockIdx.y takes one group of 256 / (D/8) rows.  The RoPE row of the
// token's position is built in shared memory by every block, in the split of the prefill table.
template <int D>
__global__ void __launch_bounds__(256) kv8_token_kernel(const Kv8TokenParams p) {
    constexpr int TPR = D / 8, HALF = D / 2, RPB = 256 / TPR;
    __shared__ float4 s_tab32[HALF];
    __shared__ double2 s_tab64[HALF];
    const int b = (int)blockIdx.x;
    const int Hkv = p.c.Hkv;
    const int n = kv8_length(p.seq_len, b, p.max_pages, p.c.log_p);
    const bool append = p.k != nullptr;
    if (n == 0) {
        if (blockIdx.y == 0) {
            if (threadIdx.x == 0 && p.seq_len[b] > 0) record_error(kErrIndex, kSiteKvLen);
            for (int i = threadIdx.x; i < p.H * TPR; i += 256)
                reinterpret_cast<uint4*>(p.out + (long long)b * p.H * D)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse != nullptr)
                for (int i = threadIdx.x; i < p.H; i += 256) p.lse[(long long)b * p.H + i] = -INFINITY;
        }
        return;
    }
    const int pos = n - 1;
    if ((int)threadIdx.x < HALF) {
        const int i = (int)threadIdx.x;
        const double theta = pow(p.base, -2.0 * (double)i / (double)D);
        double sn, cs;
        sincos((double)pos * theta, &sn, &cs);
        float c_hi, c_lo, s_hi, s_lo;
        rope_split(cs, c_hi, c_lo);
        rope_split(sn, s_hi, s_lo);
        s_tab32[i] = make_float4(c_hi, c_lo, s_hi, s_lo);
        s_tab64[i] = make_double2(cs, sn);
    }
    // this thread's row, its inputs loaded before the barrier
    const int row = (int)blockIdx.y * RPB + (int)threadIdx.x / TPR;
    const int c = (int)threadIdx.x % TPR, i0 = 4 * c;
    const bool is_q = row < p.H;
    const int hk = row - p.H;
    const bool is_kv = !is_q && append && hk < Hkv;
    uint2 x0 = make_uint2(0u, 0u), x1 = x0, v0 = x0, v1 = x0, e0 = x0, e1 = x0;
    float2 gw = make_float2(0.f, 0.f);
    int page = -1;
    float old_scale[2] = {1.f, 1.f};
    if (is_q || is_kv) {
        const __nv_bfloat16* src = is_q ? p.q + ((long long)b * p.H + row) * D : p.k + ((long long)b * Hkv + hk) * D;
        x0 = ldg_stream8(src + i0);
        x1 = ldg_stream8(src + HALF + i0);
    }
    if (is_kv) {
        const __nv_bfloat16* vr = p.v + ((long long)b * Hkv + hk) * D;
        v0 = ldg_stream8(vr + i0);
        v1 = ldg_stream8(vr + HALF + i0);
        page = __ldg(p.table + (long long)b * p.max_pages + (pos >> p.c.log_p));
        if (page < 0 || page >= p.c.n_pages) {
            if (c == 0) record_error(kErrIndex, kSiteKvPage);
            page = -1;
        } else {
            old_scale[0] = p.c.k_scale[(long long)page * Hkv + hk];
            old_scale[1] = p.c.v_scale[(long long)page * Hkv + hk];
        }
        if (p.ve != nullptr) {
            const __nv_bfloat16* er = p.ve + ((long long)b * Hkv + hk) * D;
            e0 = ldg_stream8(er + i0);
            e1 = ldg_stream8(er + HALF + i0);
            // 2 sigmoid(x . Wg[:, h]) in fp64, the 32 channels in order (the prefill gate's order)
            const __nv_bfloat16* xr = p.gate_x + (long long)b * 32;
            double z = 0.0;
#pragma unroll
            for (int cc = 0; cc < 32; ++cc)
                z = fma((double)__bfloat162float(xr[cc]), (double)__bfloat162float(p.Wg[cc * Hkv + hk]), z);
            const double g = 2.0 / (1.0 + exp(-z));
            gw.x = (float)g;
            gw.y = (float)(g - (double)gw.x);
        }
    }
    __syncthreads();
    float4 cs4[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) cs4[e] = s_tab32[i0 + e];
    uint2 o0, o1;
    rope_rms_exact4<D>(x0, x1, cs4, s_tab64 + i0, p.eps, o0, o1);
    if (is_q) {
        __nv_bfloat16* dst = p.qh + ((long long)b * p.H + row) * D;
        *reinterpret_cast<uint2*>(dst + i0) = o0;
        *reinterpret_cast<uint2*>(dst + HALF + i0) = o1;
    }
    if (is_kv && p.ve != nullptr) {
        const double g64 = (double)gw.x + (double)gw.y;
        v0 = gated_add4(v0, e0, gw.x, gw.y, g64);
        v1 = gated_add4(v1, e1, gw.x, gw.y, g64);
    }
    const int off = pos & ((1 << p.c.log_p) - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint2 y0 = u == 0 ? o0 : v0, y1 = u == 0 ? o1 : v1;
        uint32_t a = max_half(max_abs2(max_abs2(max_abs2(max_abs2(0u, y0.x), y0.y), y1.x), y1.y));
#pragma unroll
        for (int d = TPR / 2; d >= 1; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
        __syncwarp();
        if (!is_kv || page < 0) continue;
        int e = scale_exponent(a);
        const long long ph = (long long)page * Hkv + hk;
        uint8_t* blk = (u == 0 ? p.c.k_cache : p.c.v_cache) + (ph << p.c.log_p) * D;
        if (off > 0) {
            const int old = exponent_of(old_scale[u]);
            if (e > old) recode_rows<D>(blk, off, scale_of(max(old - e, -126)), 0, 1, c);
            e = max(e, old);
        }
        const float inv = scale_of(-e);
        *reinterpret_cast<uint32_t*>(blk + (long long)off * D + i0) = encode4(y0.x, y0.y, inv);
        *reinterpret_cast<uint32_t*>(blk + (long long)off * D + HALF + i0) = encode4(y1.x, y1.y, inv);
        if (c == 0) (u == 0 ? p.c.k_scale : p.c.v_scale)[ph] = scale_of(e);
    }
}

struct Kv8AttnParams {
    const __nv_bfloat16* qh;      // (B, H, D)
    const int* table;
    const int* seq_len;
    const int* doc_start;         // (B) or null
    __nv_bfloat16* out;
    float* lse;
    Kv8Store c;
    int H, G, max_pages, W;       // W = 0: no window
    float c1;                     // log2(e) / sqrt(D)
};

// First visible key of a request of n tokens.
__device__ __forceinline__ int kv8_first_key(const Kv8AttnParams& p, int b, int n) {
    int lo = p.W > 0 ? max(0, n - p.W) : 0;
    if (p.doc_start != nullptr) lo = max(lo, min(__ldg(p.doc_start + b), n - 1));
    return lo;
}

// One block of four warps per (request, query head); warp w takes keys lo + w, lo + w + 4, ... and a
// lane D/32 features of each, with the running maximum and sum of the softmax per warp.
template <int D>
__global__ void __launch_bounds__(128) kv8_attn_kernel(const Kv8AttnParams p) {
    constexpr int DPL = D / 32;
    __shared__ float s_o[4][D], s_m[4], s_l[4];
    const int row = (int)blockIdx.x, b = row / p.H, h = row - b * p.H, hk = h / p.G;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int n = kv8_length(p.seq_len, b, p.max_pages, p.c.log_p);
    if (n == 0) return;           // written by the token kernel
    const int lo = kv8_first_key(p, b, n);
    float q[DPL], o[DPL];
#pragma unroll
    for (int e = 0; e < DPL; ++e) {
        q[e] = __bfloat162float(p.qh[(long long)row * D + lane * DPL + e]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = lo + warp; j < n; j += 4) {
        const int page = __ldg(p.table + (long long)b * p.max_pages + (j >> p.c.log_p));
        if (page < 0 || page >= p.c.n_pages) {
            if (lane == 0) record_error(kErrIndex, kSiteKvPage);
            continue;
        }
        const long long ph = (long long)page * p.c.Hkv + hk;
        const long long at = ((ph << p.c.log_p) + (j & ((1 << p.c.log_p) - 1))) * D + lane * DPL;
        const float ks = p.c.k_scale[ph], vs = p.c.v_scale[ph];
        float s = 0.f, vf[DPL];
#pragma unroll
        for (int e = 0; e < DPL; e += 2) {
            const float2 kk = decode2(*reinterpret_cast<const uint16_t*>(p.c.k_cache + at + e));
            const float2 vv = decode2(*reinterpret_cast<const uint16_t*>(p.c.v_cache + at + e));
            s = fmaf(q[e], kk.x, fmaf(q[e + 1], kk.y, s));
            vf[e] = vv.x * vs;
            vf[e + 1] = vv.y * vs;
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= ks * p.c1;
        const float m2 = fmaxf(m, s);
        const float f = exp2f(m - m2), w = exp2f(s - m2);
        l = fmaf(l, f, w);
        m = m2;
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[e] = fmaf(o[e], f, w * vf[e]);
    }
#pragma unroll
    for (int e = 0; e < DPL; ++e) s_o[warp][lane * DPL + e] = o[e];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    if ((int)threadIdx.x < D) {
        const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
            L = fmaf(s_l[w], f, L);
            O = fmaf(s_o[w][threadIdx.x], f, O);
        }
        p.out[(long long)row * D + threadIdx.x] = __float2bfloat16_rn(L > 0.f ? O / L : (L == L ? 0.f : L));
        if (threadIdx.x == 0 && p.lse != nullptr)
            p.lse[row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : (L == L ? -INFINITY : L);
    }
}

}  // namespace swa
