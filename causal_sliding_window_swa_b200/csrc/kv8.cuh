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
// filled token by token holds what one write of all its tokens leaves, except for elements that fall there, which
// may be rounded more than once: amax is above 224 * 2^e, so they are smaller than amax * 2^-6 / 224, or 2^-13.8 of it.
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
    float2 a = make_float2(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u));
    float2 b = make_float2(__uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u));
    a = make_float2(a.x * inv, a.y * inv);
    b = make_float2(b.x * inv, b.y * inv);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
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
// slots of one page.  A group of W warps per (window of `win` tokens, head) takes the runs that begin in its
// window: a run of one token by the D/8 lanes of a row, a longer one by the whole group, its
// rows kept in registers between the maximum and the encoding, so that khat and v' are read once.
// HBM-bound on prompts, where windows are pages long: the first slot says where the window's next page
// begins, and the rows from there on are loaded before the other slots are looked at.  W gives each thread
// four rows of a page (eight of the largest): with fewer, small pages leave too little in flight (16 x 2000 tokens of 12
// heads, D = 128, pages of 16: 88 us by whole blocks, 48 us so).  16 prompts of 1024 to 2048 tokens, 12 heads, D = 128, pages
// of 64: 44 us, 34.5 at 6565 GB/s; where they begin inside a page 50 us.  Single tokens are latency-bound: 64 of 12 heads 3.2 us.
struct Kv8Store {
    uint8_t* k_cache;
    uint8_t* v_cache;
    float* k_scale;
    float* v_scale;
    int n_pages, Hkv, log_p;
};

// Rows first, first + step, ... < rows of a page moved to its new scale, by D/8 lanes.  A single token does this row after row: 16, 32,
// 64 or 128 rows add 3, 7, 12 or 24 us to a decode step in which every token's page grows.
template <int D>
__device__ __forceinline__ void recode_rows(uint8_t* block, int rows, float down, int first, int step, int lane8) {
    for (int r = first; r < rows; r += step) {
        uint2* p = reinterpret_cast<uint2*>(block + (long long)r * D + 8 * lane8);
        const uint2 c = *p;
        *p = make_uint2(recode4(c.x, down), recode4(c.y, down));
    }
}

template <int D, int W, int IT>
__global__ void __launch_bounds__(256, IT == 4 ? 4 : 2) kv8_write_kernel(const __nv_bfloat16* __restrict__ kh,
                                                        const __nv_bfloat16* __restrict__ vp,
                                                        const int* __restrict__ slots, const Kv8Store c, int n_tokens,
                                                        int row_tokens, int win, int windows) {
    constexpr int TPR = D / 8, THREADS = 32 * W, GROUPS = 8 / W, RPG = THREADS / TPR;
    const int P = 1 << c.log_p;
    const int h = (int)blockIdx.y;
    const int grp = (int)threadIdx.x / THREADS, tid = (int)threadIdx.x % THREADS;
    // rows of row_tokens tokens, each of `windows` windows
    const int window = (int)blockIdx.x * GROUPS + grp, row = window / windows, in_row = window - row * windows;
    const long long t0 = (long long)row * row_tokens + (long long)in_row * win;
    if (t0 >= n_tokens) return;
    const int group = tid / TPR, l8 = tid % TPR;
    const int lane = tid & 31, warp = tid >> 5;
    const int n_slots = c.n_pages << c.log_p;
    __shared__ int s_runs[128], s_n[GROUPS], s_len[GROUPS], s_single[GROUPS];     // GROUPS * P <= 128
    __shared__ uint32_t s_max[GROUPS][2][W];
    int* s_run = s_runs + grp * P;
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(THREADS) : "memory"); };

    auto slot_at = [&](long long t) -> int { return t < n_tokens ? __ldg(slots + t) : -1; };
    // token t goes on where token t - 1 ended
    auto goes_on = [&](long long t) -> bool {
        const int s = slot_at(t);
        return t > 0 && s > 0 && (s & (P - 1)) != 0 && slot_at(t - 1) == s - 1;
    };
    auto block_of = [&](uint8_t* cache, int slot) -> uint8_t* {
        return cache + (((long long)(slot >> c.log_p) * c.Hkv + h) << c.log_p) * D;
    };

    // the rows of this block's threads from token t on, `len` of them
    uint4 x[2][IT];
    auto load_rows = [&](long long t, int len) {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int r = group + it * RPG;
            if (r < len) {
                const long long at = ((t + r) * c.Hkv + h) * D + 8 * l8;
                x[0][it] = ldg_stream16(kh + at);
                x[1][it] = ldg_stream16(vp + at);
            }
        }
    };
    // Rows x of a run of `len` tokens whose first slot is `slot`.
    auto store_run = [&](int slot, int len) {
        const int page = slot >> c.log_p, off = slot & (P - 1);
        float* sc[2] = {c.k_scale + (long long)page * c.Hkv + h, c.v_scale + (long long)page * c.Hkv + h};
        int old[2] = {kEMin, kEMin};
        if (off > 0)
#pragma unroll
            for (int u = 0; u < 2; ++u) old[u] = exponent_of(*sc[u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t m = 0u;
#pragma unroll
            for (int it = 0; it < IT; ++it)
                if (group + it * RPG < len)
                    m = max_abs2(max_abs2(max_abs2(max_abs2(m, x[u][it].x), x[u][it].y), x[u][it].z), x[u][it].w);
            uint32_t a = max_half(m);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
            if (lane == 0) s_max[grp][u][warp] = a;
        }
        sync();                   // (and every thread has read the old scales)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t a = s_max[grp][u][0];
#pragma unroll
            for (int w = 1; w < W; ++w) a = max(a, s_max[grp][u][w]);
            int e = scale_exponent(a);
            uint8_t* blk = block_of(u == 0 ? c.k_cache : c.v_cache, slot);
            if (off > 0) {
                if (e > old[u]) recode_rows<D>(blk, off, scale_of(max(old[u] - e, -126)), group, RPG, l8);
                e = max(e, old[u]);
            }
            const float inv = scale_of(-e);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int r = group + it * RPG;
                if (r < len)
                    *reinterpret_cast<uint2*>(blk + (long long)(off + r) * D + 8 * l8) =
                        make_uint2(encode4(x[u][it].x, x[u][it].y, inv), encode4(x[u][it].z, x[u][it].w, inv));
            }
            if (tid == 0) *sc[u] = scale_of(e);
        }
        sync();
    };

    const int here = min(win, row_tokens - in_row * win);          // tokens of the window
    // the page that begins in the window, where its tokens are consecutive: at token `next`
    const int slot0 = slot_at(t0), next = win == P && slot0 >= 0 ? -slot0 & (P - 1) : here;
    if (next < here) load_rows(t0 + next, (int)min((long long)P, n_tokens - t0 - next));
    if (tid == 0) {
        s_n[grp] = 0;
        s_len[grp] = P;
        s_single[grp] = 0;
    }
    sync();
    const int slot1 = next < here ? slot_at(t0 + next) : -1;
    const bool whole = slot1 >= 0 && slot1 < n_slots && !goes_on(t0 + next);      // a run begins there
    if (tid < here) {
        const long long t = t0 + tid;
        const int s = slot_at(t);
        if (s >= n_slots) record_error(kErrIndex, kSiteKvSlot);
        if (s >= 0 && s < n_slots && !goes_on(t)) {
            if (!goes_on(t + 1)) s_single[grp] = 1;
            else if (tid != next) s_run[atomicAdd(&s_n[grp], 1)] = tid;
        }
    }
    if (whole && tid > 0 && tid < P && !goes_on(t0 + next + tid)) atomicMin(&s_len[grp], tid);
    sync();
    if (whole && s_len[grp] > 1) store_run(slot1, s_len[grp]);
    const int n_runs = s_n[grp];
    for (int i = 0; i < n_runs; ++i) {
        const long long t = t0 + s_run[i];
        sync();                            // the length before it has been read
        if (tid == 0) s_len[grp] = P;
        sync();
        if (tid >= 1 && tid < P && !goes_on(t + tid)) atomicMin(&s_len[grp], tid);
        sync();
        const int len = s_len[grp];
        load_rows(t, len);
        store_run(slot_at(t), len);
    }
    // runs of one token
    if (s_single[grp] == 0) return;
    for (int g0 = 0; g0 < here; g0 += RPG) {
        const long long t = t0 + g0 + group;
        const int slot = g0 + group < here ? slot_at(t) : -1;
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

// HBM-bound: 32768 rows of 12 heads, D = 128, of which 24902 are read and the others zeros, 278 MB in 45.5 us, 6.1 TB/s.
// (Stores of 32 bytes a thread and streaming stores measured the same.)
// Row r = token * Hkv + h of the results: D/8 lanes, 8 features each; a thread has NR rows in flight.  Slots
// below 0 (and past the cache, which is recorded) give zero rows.
__device__ __forceinline__ uint2 decode4(uint32_t c, float s) {
    const float2 a = decode2(c), b = decode2(c >> 16);
    return make_uint2(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s));
}
template <int D, int NR>
__global__ void __launch_bounds__(256) kv8_read_kernel(const int* __restrict__ slots, const Kv8Store c,
                                                       __nv_bfloat16* __restrict__ kh, __nv_bfloat16* __restrict__ vp,
                                                       int n_rows, FastDiv divH) {
    constexpr int TPR = D / 8, STEP = 256 / TPR;
    const int l8 = 8 * ((int)threadIdx.x % TPR);
    const int n_slots = c.n_pages << c.log_p;
    const long long r0 = (long long)blockIdx.x * STEP * NR + (int)threadIdx.x / TPR;
    int slot[NR], h[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
        const long long r = r0 + x * STEP;
        slot[x] = -1;
        if (r < n_rows) {
            const int t = fdiv((int)r, divH);
            h[x] = (int)r - t * c.Hkv;
            slot[x] = __ldg(slots + t);
            if (slot[x] >= n_slots) {
                record_error(kErrIndex, kSiteKvSlot);
                slot[x] = -1;
            }
        }
    }
    uint2 w[NR][2];
    float s[NR][2];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
        w[x][0] = w[x][1] = make_uint2(0u, 0u);
        s[x][0] = s[x][1] = 0.f;
        if (slot[x] < 0) continue;
        const long long ph = (long long)(slot[x] >> c.log_p) * c.Hkv + h[x];
        const long long at = ((ph << c.log_p) + (slot[x] & ((1 << c.log_p) - 1))) * D + l8;
        w[x][0] = *reinterpret_cast<const uint2*>(c.k_cache + at);
        w[x][1] = *reinterpret_cast<const uint2*>(c.v_cache + at);
        s[x][0] = c.k_scale[ph];
        s[x][1] = c.v_scale[ph];
    }
#pragma unroll
    for (int x = 0; x < NR; ++x) {
        const long long r = r0 + x * STEP;
        if (r >= n_rows) continue;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint2 a = decode4(w[x][u].x, s[x][u]), b = decode4(w[x][u].y, s[x][u]);
            *reinterpret_cast<uint4*>((u == 0 ? kh : vp) + r * D + l8) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
}

// ------------------------------------------------------------------------------------------- pages

// One allocator step.  Per request b: L = kv_len, n = n_new, F = first_page (pages before it were
// given back), have = ceil(L / P).
//   n < 0: the request has ended: pages [F, have) go back, L' = 0, F' = 0.
//   else:  pages [F, f) go back, f = max(F, floor(max(0, L - W + 1) / P)): the next query is at
//          position L or later and sees no key before L - W + 1.  (W = 0: none.)
//          need = ceil((L + n) / P) - have, 0 where the request cannot be served at all (n > T, more
//          than max_pages pages); S = inclusive sum of need in request order; the request is served
//          iff n > 0 and (need = 0 or S <= free).
//   L < 0, L > max_pages * P, F < 0 or F > have: nothing of the request changes, whatever n is.
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

constexpr int kPagesSegment = 128;         // entries of a table row, or slots, that a warp has at a time

// A row that changes little, in place, by one thread: at most kPagesFew pages either way, and T <= kPagesFew.
constexpr int kPagesFew = 4;
__device__ __forceinline__ bool pages_few(const PageRecord& r) { return r.take <= kPagesFew && r.upto - r.from <= kPagesFew; }
__device__ __forceinline__ void pages_fill_few(const PagesParams& p, const PageRecord& r, int b) {
    int* row = p.table_out + (long long)b * p.max_pages;
    const int P = 1 << p.log_p;
    const int at = r.L >> p.log_p, partial = r.n > 0 && at < r.have ? row[at] : -1;      // a partly filled page
    int back[kPagesFew], got[kPagesFew];
#pragma unroll
    for (int k = 0; k < kPagesFew; ++k) {
        if (k < r.upto - r.from) back[k] = row[r.from + k];
        if (k < r.take) got[k] = p.ring[((unsigned)r.ring_take + (unsigned)k) % (unsigned)p.n_pages];
    }
#pragma unroll
    for (int k = 0; k < kPagesFew; ++k) {
        if (k < r.upto - r.from) {
            p.ring[((unsigned)r.ring_give + (unsigned)k) % (unsigned)p.n_pages] = back[k];
            row[r.from + k] = -1;
        }
        if (k < r.take) row[r.have + k] = got[k];
        if (k < p.T) {
            int page = -1;
            if (k < r.n) {
                const int x = ((r.L + k) >> p.log_p) - r.have;
                page = partial;
#pragma unroll
                for (int y = 0; y < kPagesFew; ++y)
                    if (x == y) page = got[y];
            }
            p.slots[(long long)b * p.T + k] = page >= 0 && page < p.n_pages ? page * P + ((r.L + k) & (P - 1)) : -1;
        }
    }
}

// One segment of row b: entries of the table (seg < table_segs) or slots.
__device__ __forceinline__ void pages_fill(const PagesParams& p, const PageRecord& r, int b, int seg, int table_segs,
                                           int lane) {
    const int* in = p.table + (long long)b * p.max_pages;
    auto taken = [&](int j) {              // entry j >= have; at most n_pages pages are taken
        const unsigned x = (unsigned)r.ring_take + (unsigned)(j - r.have);
        return p.ring[x >= (unsigned)p.n_pages ? x - (unsigned)p.n_pages : x];
    };
    if (seg < table_segs) {
        int* out = p.table_out + (long long)b * p.max_pages;
        const int first = seg * kPagesSegment;
        // in place, only what changes is touched
        if (in == out && first + kPagesSegment <= r.have && (first >= r.upto || first + kPagesSegment <= r.from)) return;
        if (in == out && first >= r.have + r.take) return;
        int v[kPagesSegment / 32];
#pragma unroll
        for (int x = 0; x < kPagesSegment / 32; ++x) {
            const int j = first + 32 * x + lane;
            if (j < p.max_pages) v[x] = j >= r.have && j < r.have + r.take ? taken(j) : in[j];
        }
#pragma unroll
        for (int x = 0; x < kPagesSegment / 32; ++x) {
            const int j = first + 32 * x + lane;
            if (j >= p.max_pages) continue;
            if (j >= r.from && j < r.upto) {
                p.ring[((unsigned)r.ring_give + (unsigned)(j - r.from)) % (unsigned)p.n_pages] = v[x];
                v[x] = -1;
            }
            out[j] = v[x];
        }
        return;
    }
    int* sl = p.slots + (long long)b * p.T;
    const int P = 1 << p.log_p, first = (seg - table_segs) * kPagesSegment;
    int v[kPagesSegment / 32];
#pragma unroll
    for (int x = 0; x < kPagesSegment / 32; ++x) {
        const int t = first + 32 * x + lane;
        v[x] = -1;
        if (t < r.n) {
            const int j = (r.L + t) >> p.log_p;
            v[x] = j >= r.have ? taken(j) : in[j];
        }
    }
#pragma unroll
    for (int x = 0; x < kPagesSegment / 32; ++x) {
        const int t = first + 32 * x + lane;
        if (t < p.T) sl[t] = v[x] >= 0 && v[x] < p.n_pages ? v[x] * P + ((r.L + t) & (P - 1)) : -1;
    }
}

// Every block goes through all requests (1024 at a time) and finds every record, and the blocks share the rows'
// segments.  In place, the blocks are one cluster: a request's state is written only after every block has read it; a row's
// segments neither read nor write what another one of them changes (the slots read the table entry of a
// partly filled page, which a step leaves alone; pages are taken from the free stretch of the ring and go back outside it).
// Latency-bound (lengths, two sums, a table or ring entry, the stores): 16 requests 3.5 us.  1000 requests of up to 4096
// tokens in pages of 16, T = 1: in place 4.8 us, where one thread has a row (18.9 by segments); into another state 4.4 us
// by 125 blocks (16.6 by a cluster of eight, whose instructions for 256512 table entries bound it).
__global__ void __launch_bounds__(1024, 1) kv_pages_kernel(const PagesParams p) {
    __shared__ PageRecord s_rec[1024];
    __shared__ int s_warp[2][32];
    __shared__ int s_taken;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;
    const int P = 1 << p.log_p;
    const int head = min(max(p.pool[0], 0), p.n_pages - 1), free = min(max(p.pool[1], 0), p.n_pages);
    const int table_segs = (p.max_pages + kPagesSegment - 1) / kPagesSegment;
    const int segs = table_segs + (p.T + kPagesSegment - 1) / kPagesSegment;
    int base[2] = {0, 0};           // pages wanted and returned by earlier chunks of requests (B * max_pages < 2^31)
    if (threadIdx.x == 0) s_taken = 0;
    for (int b0 = 0; b0 < p.B; b0 += 1024) {
        const int b = b0 + (int)threadIdx.x;
        PageRecord r{};
        int need = 0, F = 0, n = 0, give = 0;
        bool ended = false, fits = false;
        if (b < p.B) {
            const int cap = p.max_pages << p.log_p;
            r.L = p.kv_len[b];
            n = p.n_new[b];
            F = p.first[b];
            // a state that cannot be stays as it is
            bool sane = r.L >= 0 && r.L <= cap;
            r.have = sane ? (int)(((unsigned)r.L + P - 1) >> p.log_p) : 0;
            sane = sane && F >= 0 && F <= r.have;
            ended = n < 0 && sane;
            const int low = p.W > 0 ? max(0, r.L - p.W + 1) >> p.log_p : 0;
            r.from = F;
            r.upto = !sane ? F : ended ? r.have : max(F, low);
            give = r.upto - r.from;
            fits = sane && n >= 0 && n <= p.T && n <= cap - r.L;
            if (fits) need = (int)(((unsigned)(r.L + n) + P - 1) >> p.log_p) - r.have;
        }
        // inclusive sums over the chunk
        int v[2] = {need, give};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o0 = __shfl_up_sync(0xffffffffu, v[0], d), o1 = __shfl_up_sync(0xffffffffu, v[1], d);
            if (lane >= d) {
                v[0] += o0;
                v[1] += o1;
            }
        }
        if (lane == 31) {
            s_warp[0][warp] = v[0];
            s_warp[1][warp] = v[1];
        }
        __syncthreads();
        if (warp < 2) {
            int w = s_warp[warp][lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, w, d);
                if (lane >= d) w += o;
            }
            s_warp[warp][lane] = w;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            v[u] += base[u] + (warp > 0 ? s_warp[u][warp - 1] : 0);
            base[u] += s_warp[u][31];
        }
        const bool ok = fits && n > 0 && (need == 0 || v[0] <= free);
        r.take = ok ? need : 0;
        r.n = ok ? n : 0;
        r.ring_take = (int)(((unsigned)head + (unsigned)(v[0] - need)) % (unsigned)p.n_pages);
        r.ring_give = (int)((unsigned)(head + (long long)free) % (unsigned)p.n_pages);
        r.ring_give = (int)(((unsigned)r.ring_give + (unsigned)(v[1] - give)) % (unsigned)p.n_pages);
        s_rec[threadIdx.x] = r;
        // the sums only grow: the last served request that takes pages has the largest of theirs
        const unsigned takers = __ballot_sync(0xffffffffu, r.take > 0);
        if (takers != 0u && lane == 31 - __clz(takers)) atomicMax(&s_taken, v[0]);
        if (cluster_nctarank() > 1) cluster_sync_all();
        else __syncthreads();
        if (rank == 0 && b < p.B) {
            const int after = ended ? 0 : r.L + r.n;
            p.kv_len_out[b] = after;
            p.first_out[b] = ended ? 0 : r.upto;
            p.step_len[b] = ok ? after : 0;
        }
        const bool few = p.table == p.table_out && p.T <= kPagesFew;
        if (few) {
            if (b < p.B && (int)threadIdx.x % ranks == rank && pages_few(r)) pages_fill_few(p, r, b);
            if (!__syncthreads_or(b < p.B && !pages_few(r))) continue;
        }
        const int work = min(1024, p.B - b0) * segs;
        for (int x = rank * 32 + warp; x < work; x += ranks * 32) {
            const int row = x / segs;
            if (few && pages_few(s_rec[row])) continue;
            pages_fill(p, s_rec[row], b0 + row, x - row * segs, table_segs, lane);
        }
        __syncthreads();
    }
    if (rank == 0 && threadIdx.x == 0) {
        p.pool_out[0] = (int)(((unsigned)head + (unsigned)s_taken) % (unsigned)p.n_pages);
        p.pool_out[1] = (int)min((long long)p.n_pages, (long long)free - s_taken + base[1]);
    }
}

}  // namespace swa
