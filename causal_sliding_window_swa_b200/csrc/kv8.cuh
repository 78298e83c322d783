// kv8.cuh -- a paged key/value cache held in 8 bits, for decoding requests of different lengths (the
// pages list a KV cache among the missing pieces: "Let's reproduce GPT-2 (124M)" notes, section 19).
//
// Layout.  A page holds P tokens of every key/value head: codes e4m3 (n_pages, Hkv, P, D), so that one
// page of one head is P * D consecutive bytes, and one scale for each page and head, fp32 (n_pages,
// Hkv).  A cached value is code * scale.
//
// Scale.  scale = 2^e with e the smallest integer (at least kEMin) for which every value of the block
// fits, amax <= 448 * 2^e.  A power of two costs a floating-point code no precision (the relative
// step of a normal code does not depend on the scale), makes every cached value an exact bf16, and
// lets the scale of a page that is still being filled grow without loss: dividing a code by a power
// of two is exact unless it falls below 2^-6, where it is off by at most half of 2^-9.  So a page
// filled token by token holds what one write of all its tokens leaves, except for elements smaller
// than amax * 2^-14, which may be rounded twice.
//
// Operations here: kv_pages_* (which pages a request's tokens live in), kv8_write_kernel (bf16 khat
// and v' rows into the pages), kv8_read_kernel (the reverse).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "prologue.cuh"
#include "ptx.cuh"

namespace swa {

constexpr int kEMin = -60;    // smaller blocks keep the scale 2^-60 (their values become 0 below 2^-70)
constexpr int kEMax = 120;    // 448 * 2^120 is above every finite bf16

// ------------------------------------------------------------------------------------ codes, scales

// The exponent of a block from the bits of its largest magnitude (bf16, sign cleared):
// amax = 2^(E - 127) (1 + M / 128) <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
    const int E = (int)(amax_bits >> 7), M = (int)(amax_bits & 127u);
    const int e = E == 0 ? kEMin : E - 127 - 8 + (M > 96 ? 1 : 0);
    return max(kEMin, min(kEMax, e));
}
__device__ __forceinline__ float scale_of(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The exponent of a stored scale (clamped, so that any stored bits give a usable one).
__device__ __forceinline__ int exponent_of(float scale) {
    return max(kEMin, min(kEMax, (int)((__float_as_uint(scale) >> 23) & 255u) - 127));
}

// Larger magnitude of two bf16 pairs, elementwise; a NaN does not count.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
    const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&m);
    const __nv_bfloat162 b = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x));
    const __nv_bfloat162 r = __hmax2(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_half(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// Four bf16 (two words) times `inv` -> four e4m3 codes, round to nearest even, clamped at 448.
__device__ __forceinline__ uint32_t encode4(uint32_t w0, uint32_t w1, float inv) {
    const float2 a = make_float2(__uint_as_float(w0 << 16) * inv, __uint_as_float(w0 & 0xffff0000u) * inv);
    const float2 b = make_float2(__uint_as_float(w1 << 16) * inv, __uint_as_float(w1 & 0xffff0000u) * inv);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ float2 decode2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes moved to a scale 2^d times as large (d >= 1): divided by 2^d and rounded once more.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float down) {
    const float2 a = decode2(c), b = decode2(c >> 16);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * down, a.y * down), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * down, b.y * down), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// ------------------------------------------------------------------------------------------- write

// The tokens of one call are consecutive rows; a run is a stretch of them that goes into consecutive
// slots of one page.  One block per (window of `win` tokens, head) takes the runs that begin in its
// window: a run of one token by the D/8 lanes of a row group, a longer one by the whole block, its
// rows kept in registers between the maximum and the encoding, so that khat and v' are read once.
struct Kv8Store {
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scale;
    float* v_scale;
    int n_pages, Hkv, log_p;
};

template <int D>
__device__ __forceinline__ void recode_rows(uint8_t* block, int rows, float down, int first, int step, int lane8) {
    for (int r = first; r < rows; r += step) {
        uint2* p = reinterpret_cast<uint2*>(block + (long long)r * D + 8 * lane8);
        const uint2 c = *p;
        *p = make_uint2(recode4(c.x, down), recode4(c.y, down));
    }
}

template <int D, int IT>
__global__ void __launch_bounds__(256) kv8_write_kernel(const __nv_bfloat16* __restrict__ kh,
                                                        const __nv_bfloat16* __restrict__ vp,
                                                        const int* __restrict__ slots, const Kv8Store c, int n_tokens,
                                                        int win) {
    constexpr int TPR = D / 8, RPB = 256 / TPR;
    const int P = 1 << c.log_p;
    const int h = (int)blockIdx.y;
    const long long t0 = (long long)blockIdx.x * win;
    const int group = (int)threadIdx.x / TPR, l8 = (int)threadIdx.x % TPR;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int n_slots = c.n_pages << c.log_p;
    __shared__ int s_run[128], s_n, s_len;
    __shared__ uint32_t s_max[2][8];
    __shared__ int s_old[2];

    auto slot_at = [&](long long t) -> int { return t < n_tokens ? __ldg(slots + t) : -1; };
    // token t goes on where token t - 1 ended
    auto goes_on = [&](long long t) -> bool {
        const int s = slot_at(t);
        return t > 0 && s > 0 && (s & (P - 1)) != 0 && slot_at(t - 1) == s - 1;
    };
    auto block_of = [&](uint8_t* cache, int slot) -> uint8_t* {
        return cache + (((long long)(slot >> c.log_p) * c.Hkv + h) << c.log_p) * D;
    };

    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    if ((int)threadIdx.x < win) {
        const long long t = t0 + threadIdx.x;
        const int s = slot_at(t);
        if (s >= n_slots) record_error(kErrIndex, kSiteKvSlot);
        if (s >= 0 && s < n_slots && !goes_on(t) && goes_on(t + 1)) s_run[atomicAdd(&s_n, 1)] = (int)threadIdx.x;
    }
    __syncthreads();
    const int n_runs = s_n;
    for (int i = 0; i < n_runs; ++i) {
        const long long t = t0 + s_run[i];
        if (threadIdx.x == 0) s_len = P;
        __syncthreads();
        if (threadIdx.x >= 1 && (int)threadIdx.x < P && !goes_on(t + threadIdx.x)) atomicMin(&s_len, (int)threadIdx.x);
        const int slot = slot_at(t);
        const int page = slot >> c.log_p, off = slot & (P - 1);
        float* sc[2] = {c.k_scale + (long long)page * c.Hkv + h, c.v_scale + (long long)page * c.Hkv + h};
        if (threadIdx.x < 2) s_old[threadIdx.x] = exponent_of(*sc[threadIdx.x]);
        __syncthreads();
        const int len = min(s_len, P - off);
        uint4 x[2][IT];
        uint32_t m[2] = {0u, 0u};
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int r = group + it * RPB;
            if (r < len) {
                const long long at = ((t + r) * c.Hkv + h) * D + 8 * l8;
                x[0][it] = *reinterpret_cast<const uint4*>(kh + at);
                x[1][it] = *reinterpret_cast<const uint4*>(vp + at);
            } else {
                x[0][it] = x[1][it] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int it = 0; it < IT; ++it)
                m[u] = max_abs2(max_abs2(max_abs2(max_abs2(m[u], x[u][it].x), x[u][it].y), x[u][it].z), x[u][it].w);
            uint32_t a = max_half(m[u]);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
            if (lane == 0) s_max[u][warp] = a;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t a = s_max[u][0];
#pragma unroll
            for (int w = 1; w < 8; ++w) a = max(a, s_max[u][w]);
            int e = scale_exponent(a);
            uint8_t* blk = block_of(u == 0 ? c.k_cache : c.v_cache, slot);
            if (off > 0) {
                const int old = s_old[u];
                if (e > old) recode_rows<D>(blk, off, scale_of(max(old - e, -126)), group, RPB, l8);
                e = max(e, old);
            }
            const float inv = scale_of(-e);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int r = group + it * RPB;
                if (r < len)
                    *reinterpret_cast<uint2*>(blk + (long long)(off + r) * D + 8 * l8) =
                        make_uint2(encode4(x[u][it].x, x[u][it].y, inv), encode4(x[u][it].z, x[u][it].w, inv));
            }
            if (threadIdx.x == 0) *sc[u] = scale_of(e);
        }
        __syncthreads();
    }
    // runs of one token
    for (int g0 = 0; g0 < win; g0 += RPB) {
        const long long t = t0 + g0 + group;
        const int slot = g0 + group < win ? slot_at(t) : -1;
        const bool mine = slot >= 0 && slot < n_slots && !goes_on(t) && !goes_on(t + 1);
        const int off = slot & (P - 1), page = slot >> c.log_p;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            float* sc = (u == 0 ? c.k_scale : c.v_scale) + (mine ? (long long)page * c.Hkv + h : 0ll);
            float old_scale = 1.f;
            if (mine) {
                x = *reinterpret_cast<const uint4*>((u == 0 ? kh : vp) + (t * c.Hkv + h) * D + 8 * l8);
                old_scale = *sc;
            }
            uint32_t a = max_half(max_abs2(max_abs2(max_abs2(max_abs2(0u, x.x), x.y), x.z), x.w));
#pragma unroll
            for (int d = TPR / 2; d >= 1; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
            __syncwarp();   // every lane has read the old scale
            if (!mine) continue;
            int e = scale_exponent(a);
            uint8_t* blk = block_of(u == 0 ? c.k_cache : c.v_cache, slot);
            if (off > 0) {
                const int old = exponent_of(old_scale);
                if (e > old) recode_rows<D>(blk, off, scale_of(max(old - e, -126)), 0, 1, l8);
                e = max(e, old);
            }
            const float inv = scale_of(-e);
            *reinterpret_cast<uint2*>(blk + (long long)off * D + 8 * l8) =
                make_uint2(encode4(x.x, x.y, inv), encode4(x.z, x.w, inv));
            if (l8 == 0) *sc = scale_of(e);
        }
    }
}

// -------------------------------------------------------------------------------------------- read

// Row r = token * Hkv + h of the results: D/8 lanes, 8 features each.  Slots below 0 (and past the
// cache, which is recorded) give zero rows.
template <int D>
__global__ void __launch_bounds__(256) kv8_read_kernel(const int* __restrict__ slots, const Kv8Store c,
                                                       __nv_bfloat16* __restrict__ kh, __nv_bfloat16* __restrict__ vp,
                                                       int n_rows, FastDiv divH) {
    constexpr int TPR = D / 8;
    const int l8 = (int)threadIdx.x % TPR;
    const int n_slots = c.n_pages << c.log_p;
    for (long long r0 = (blockIdx.x * 256ll + threadIdx.x) / TPR; r0 < n_rows; r0 += gridDim.x * 256ll / TPR) {
        const int r = (int)r0;
        const int t = fdiv(r, divH), h = r - t * c.Hkv;
        const int slot = __ldg(slots + t);
        uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (slot >= 0 && slot < n_slots) {
            const long long ph = (long long)(slot >> c.log_p) * c.Hkv + h;
            const long long at = ((ph << c.log_p) + (slot & ((1 << c.log_p) - 1))) * D + 8 * l8;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint2 w = *reinterpret_cast<const uint2*>((u == 0 ? c.k_cache : c.v_cache) + at);
                const float s = __ldg((u == 0 ? c.k_scale : c.v_scale) + ph);
                const float2 a = decode2(w.x), b = decode2(w.x >> 16), d = decode2(w.y), e = decode2(w.y >> 16);
                o[u] = make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s),
                                  pack_bf16x2(d.x * s, d.y * s), pack_bf16x2(e.x * s, e.y * s));
            }
        } else if (slot >= n_slots) {
            record_error(kErrIndex, kSiteKvSlot);
        }
        *reinterpret_cast<uint4*>(kh + (long long)r * D + 8 * l8) = o[0];
        *reinterpret_cast<uint4*>(vp + (long long)r * D + 8 * l8) = o[1];
    }
}

// ------------------------------------------------------------------------------------------- pages

// One allocator step.  Per request b: L = kv_len, n = n_new, F = first_page (pages before it were
// given back), have = ceil(L / P).
//   n < 0: the request has ended: pages [F, have) go back, L' = 0, F' = 0.
//   else:  pages [F, f) go back, f = max(F, floor(max(0, L - W + 1) / P)): the next query is at
//          position L or later and sees no key before L - W + 1.  (W = 0: none.)
//          need = ceil((L + n) / P) - have, 0 where the request cannot be served at all (n > T, more
//          than max_pages pages, L < 0); S = inclusive sum of need in request order; the request is served
//          iff n > 0 and (need = 0 or S <= free).
// A request that finds no page therefore holds back later ones that need one (their order is kept),
// and since S only grows the served requests' pages are the first taken ones of the ring.
// The free pages are ring[(head + i) mod n_pages], i < free; pages given back are appended behind
// them and are free in the next step.  Only entries outside the free stretch are written, so the
// same inputs give the same results however often the step is repeated.
struct PagesParams {
    const int* table;
    const int* kv_len;
    const int* first;
    const int* pool;       // {head, free}
    const int* n_new;
    int* ring;
    int* table_out;
    int* kv_len_out;
    int* first_out;
    int* pool_out;
    int* slots;
    int* step_len;
    int B, T, max_pages, n_pages, log_p, W;
};

struct PageRecord {
    int L, n;              // tokens before the step, tokens served (0: none)
    int have, take;        // pages before the step, pages taken
    int from, upto;        // pages [from, upto) go back
    int ring_take, ring_give;   // where in the ring the first taken page is, and the first returned one goes
};

__device__ __forceinline__ int ring_at(long long i, int n_pages) { return (int)(i % n_pages); }

// Row b of the table and of the slots, by the lanes first, first + step, ...
__device__ __forceinline__ void pages_fill_row(const PagesParams& p, const PageRecord& r, int b, int first, int step) {
    const int* in = p.table + (long long)b * p.max_pages;
    int* out = p.table_out + (long long)b * p.max_pages;
    const bool copy = in != out;
    auto taken = [&](int j) { return p.ring[ring_at((long long)r.ring_take + (j - r.have), p.n_pages)]; };
    if (copy) {
        for (int j = first; j < p.max_pages; j += step) {
            int v = in[j];
            if (j >= r.from && j < r.upto) {
                p.ring[ring_at((long long)r.ring_give + (j - r.from), p.n_pages)] = v;
                v = -1;
            }
            if (j >= r.have && j < r.have + r.take) v = taken(j);
            out[j] = v;
        }
    } else {
        for (int j = r.from + first; j < r.upto; j += step) {
            p.ring[ring_at((long long)r.ring_give + (j - r.from), p.n_pages)] = in[j];
            out[j] = -1;
        }
        for (int j = r.have + first; j < r.have + r.take; j += step) out[j] = taken(j);
    }
    int* sl = p.slots + (long long)b * p.T;
    const int P = 1 << p.log_p;
    for (int t = first; t < p.T; t += step) {
        int s = -1;
        if (t < r.n) {
            const int pos = r.L + t, j = pos >> p.log_p;
            const int page = j >= r.have ? taken(j) : in[j];
            if (page >= 0 && page < p.n_pages) s = page * P + (pos & (P - 1));
        }
        sl[t] = s;
    }
}

__global__ void __launch_bounds__(1024) kv_pages_kernel(const PagesParams p) {
    __shared__ PageRecord s_rec[1024];
    __shared__ long long s_warp[2][32];
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int P = 1 << p.log_p;
    const int head = min(max(p.pool[0], 0), p.n_pages - 1), free = min(max(p.pool[1], 0), p.n_pages);
    long long base[2] = {0, 0};     // pages wanted and returned by earlier chunks of requests
    long long taken = 0;
    for (int b0 = 0; b0 < p.B; b0 += 1024) {
        const int b = b0 + (int)threadIdx.x;
        PageRecord r{};
        long long need = 0;
        int F = 0, n = 0, give = 0;
        bool ended = false, fits = false;
        if (b < p.B) {
            const long long cap = (long long)p.max_pages << p.log_p;
            r.L = p.kv_len[b];
            n = p.n_new[b];
            F = p.first[b];
            const bool sane = r.L >= 0 && r.L <= cap && F >= 0;
            if (!sane) r.L = max(0, (int)min((long long)r.L, cap));
            r.have = (int)(((long long)r.L + P - 1) >> p.log_p);
            F = min(max(F, 0), r.have);
            ended = n < 0;
            const int low = p.W > 0 ? max(0, r.L - p.W + 1) >> p.log_p : 0;
            r.from = F;
            r.upto = ended ? r.have : max(F, low);
            give = r.upto - r.from;
            fits = sane && n >= 0 && n <= p.T && (long long)r.L + n <= cap;
            if (fits) need = (((long long)r.L + n + P - 1) >> p.log_p) - r.have;
        }
        // inclusive sums over the chunk
        long long v[2] = {need, give};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, v[u], d);
                if (lane >= d) v[u] += o;
            }
            if (lane == 31) s_warp[u][warp] = v[u];
        }
        __syncthreads();
        if (warp < 2) {
            long long w = s_warp[warp][lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, w, d);
                if (lane >= d) w += o;
            }
            s_warp[warp][lane] = w;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) v[u] += base[u] + (warp > 0 ? s_warp[u][warp - 1] : 0ll);
        base[0] += s_warp[0][31];
        base[1] += s_warp[1][31];
        const bool ok = fits && n > 0 && (need == 0 || v[0] <= free);
        r.take = ok ? (int)need : 0;
        r.n = ok ? n : 0;
        r.ring_take = ring_at(head + (v[0] - need), p.n_pages);
        r.ring_give = ring_at((long long)head + free + (v[1] - give), p.n_pages);
        s_rec[threadIdx.x] = r;
        if (b < p.B) {
            const int after = ended ? 0 : r.L + r.n;
            p.kv_len_out[b] = after;
            p.first_out[b] = ended ? 0 : r.upto;
            p.step_len[b] = ok ? after : 0;
        }
        // the last served request that takes pages has the largest sum among them
        long long mine = r.take > 0 ? v[0] : 0ll;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, d));
        __syncthreads();
        if (lane == 0) s_warp[0][warp] = mine;
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < 32; ++w) taken = max(taken, s_warp[0][w]);
        const int n_here = min(1024, p.B - b0);
        for (int i = warp; i < n_here; i += 32) pages_fill_row(p, s_rec[i], b0 + i, lane, 32);
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.pool_out[0] = ring_at((long long)head + taken, p.n_pages);
        p.pool_out[1] = (int)min((long long)p.n_pages, (long long)free - taken + base[1]);
    }
}

}  // namespace swa
