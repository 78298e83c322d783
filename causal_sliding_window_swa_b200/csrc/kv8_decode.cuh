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
    int* counters;                // the attention's arrival counters, zeroed here
    int n_counters;
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
    grid_dependents_launch();     // the attention kernel may start: it waits before it reads what is written here
    if (b == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < p.n_counters; i += 256) p.counters[i] = 0;
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

// ------------------------------------------------------------------------------------- attention
//
// HBM-bound: every visible key's and value's code is read once for all query heads of its key/value
// head.  At 6.5 TB/s an SM has to take in 23 codes a clock, each of which is converted and multiplied with
// up to 64 query heads: too much for fp32 lanes, little for the tensor cores, so both products are
// mma.sync m16n8k16 on fp16 operands (a code is exact in fp16, qhat as well down to 2^-17), fp32 sums.
// (tcgen05 would need 128-row tiles of one type: the codes converted into shared memory first, or
// qhat and the weights split into e4m3 parts, for products that are a few percent of the time here.)
//
// Units.  A unit is a chunk of 128 key positions (aligned) of one request and key/value head.  Units are
// numbered request by request, head by head, chunk by chunk, and the blocks (one per SM) take equal
// stretches of them, whatever the requests' lengths: every block finds its first unit from the
// sequence lengths alone, so the host needs no lengths and a captured launch stays valid.  A
// (request, head) item that one block has whole is finished there; the pieces of one that several
// blocks share go to the workspace, and the block that arrives last adds them in order (the result
// does not depend on which one that is).
//
// Pipeline.  A producer warp looks up 32 pages at a time and brings each page's codes into a ring of
// chunk-sized stages by TMA, with the two scales of each 16 keys; eight consumer warps take 16 keys and
// eight query heads at a time: with G <= 8 heads in a group each warp has one 16-key tile of a chunk,
// with more the warps are split over the groups of eight heads (NRT of them) and take NRT tiles.
//   S^T (16 keys x 8 heads) = K qhat^T: a lane's A operand is 16 (or 32) consecutive bytes of key rows g and
//   g + 8 (lane = 4 g + t); the features are taken in the order that this gives, qhat's likewise.
//   O^T (features x 8 heads) += V^T W^T: the bytes of a lane's key pairs are interleaved before the
//   conversion; W^T is the transpose of S^T's layout, which movmatrix makes.
// The TMA swizzle (128 bytes; 64 for D = 64) keeps both reads free of bank conflicts (D = 64: two-way).
//
// Softmax.  With x_j = log2(e) qhat . k_j / sqrt(D) and a running reference m, p_j = 2^(x_j - m) is summed in
// fp32 and w_j = p_j * (value scale) enters the product as fp16 (rounded to 11 bits: off by 2^-12 of each
// weight, an eighth of the output's own rounding).  m is raised, with one rescaling, only when some
// x_j + log2(value scale) passes it by more than 2^kSlack: it is at least the first tile's maximum, so
// weights stay below 2^kSlack and those that fp16 loses are below 2^-24 of the largest.
constexpr int kKv8Chunk = 128;          // key positions of a unit
constexpr int kKv8MaxBlocks = 148;      // blocks of the attention kernel, at most
constexpr float kSlack = 10.f;          // fp16 holds 2^15

enum : unsigned int { kSiteKv8Full = 83, kSiteKv8Empty = 84 };

struct Kv8AttnParams {
    const __nv_bfloat16* qh;      // (B, H, D)
    const int* table;
    const int* seq_len;
    const int* doc_start;         // (B) or null
    __nv_bfloat16* out;
    float* lse;
    Kv8Store c;
    int* counters;                // zero at the start
    float* part;                  // [2 * blocks][G][D + 4]: O, then m and l
    int B, H, G, max_pages, W;    // W = 0: no window
    float c1;                     // log2(e) / sqrt(D)
    unsigned long long wait_limit_ns;
};

template <int D>
struct Kv8Cfg {
    static constexpr int CONSUMERS = 8;
    static constexpr int THREADS = 32 * (CONSUMERS + 1);
    static constexpr int TENSOR = kKv8Chunk * D;                 // bytes of a chunk's K (and V)
    static constexpr int NS = D == 128 ? 5 : 8;                  // ring stages
    static constexpr int OFF_O = NS * 2 * TENSOR;                // warp results [8][8][D]
    static constexpr int OFF_ML = OFF_O + CONSUMERS * 8 * D * 4; // m [8][8], l [8][8]
    static constexpr int OFF_META = OFF_ML + 2 * CONSUMERS * 8 * 4;   // per stage and tile: ks c1, vs, log2 vs, pad
    static constexpr int OFF_BAR = OFF_META + NS * 8 * 16;
    static constexpr int SMEM = OFF_BAR + 2 * NS * 8 + 1024;     // + alignment slack
};

// First visible key of a request of n tokens.
__device__ __forceinline__ int kv8_first_key(const Kv8AttnParams& p, int b, int n) {
    int lo = p.W > 0 ? max(0, n - p.W) : 0;
    if (p.doc_start != nullptr) lo = max(lo, min(__ldg(p.doc_start + b), n - 1));
    return lo;
}

// Position of a block's walk through its units.
struct Kv8Walk {
    int b, hk;             // item
    int n, lo;             // its visible keys [lo, n)
    int ch0, nch;          // its chunks [ch0, ch0 + nch)
    long long begin;       // its first unit

    __device__ __forceinline__ void load(const Kv8AttnParams& p) {
        n = kv8_length(p.seq_len, b, p.max_pages, p.c.log_p);
        lo = n > 0 ? kv8_first_key(p, b, n) : 0;
        ch0 = lo / kKv8Chunk;
        nch = n > 0 ? (n - 1) / kKv8Chunk - ch0 + 1 : 0;
    }
    // to the item after this one
    __device__ __forceinline__ void next(const Kv8AttnParams& p) {
        begin += nch;
        if (++hk < p.c.Hkv) return;
        hk = 0;
        do {
            ++b;
            load(p);
        } while (nch == 0);
    }
};

// The block that has unit u of n units shared by m blocks: block c has [n c / m, n (c + 1) / m).
__device__ __forceinline__ int kv8_owner(long long u, long long n, int m) { return (int)(((u + 1) * m - 1) / n); }

__device__ __forceinline__ uint32_t fp8x2_to_half2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 8x8 matrix of 16-bit elements held two to a lane (row lane / 4), transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void kv8_consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// tm_k, tm_v: the caches as {D, n_pages * Hkv * P} bytes, box {D, P}.  NRT: groups of eight query heads (a
// power of two).
template <int D, int NRT>
__global__ void __launch_bounds__(Kv8Cfg<D>::THREADS, 1) kv8_attn_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                        const __grid_constant__ CUtensorMap tm_v,
                                                                        const Kv8AttnParams p) {
    using C = Kv8Cfg<D>;
    constexpr int KS = C::CONSUMERS / NRT;        // warps that share the keys of a group of heads
    constexpr int NSTEP = D / 16;                 // mma steps along the features
    constexpr int VW = D / 32;                    // 32-bit words of a lane's features of one value row
    extern __shared__ __align__(1024) uint8_t dsmem[];
    uint8_t* smem = dsmem + ((1024u - (smem_u32(dsmem) & 1023u)) & 1023u);
    float* s_o = reinterpret_cast<float*>(smem + C::OFF_O);
    float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);
    float* s_l = s_m + C::CONSUMERS * 8;
    float4* s_meta = reinterpret_cast<float4*>(smem + C::OFF_META);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::NS;
    __shared__ long long s_warp_sum[C::CONSUMERS + 1];
    __shared__ long long s_before;
    __shared__ int s_first, s_last;

    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31u);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(full + s), 1);
            mbar_init(smem_u32(empty + s), C::CONSUMERS);
        }
        fence_barrier_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // this block's units: chunks before each request, summed over a slice of the requests per thread
    Kv8Walk w;
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    const int b_lo = min(p.B, (int)threadIdx.x * per), b_hi = min(p.B, b_lo + per);
    long long mine = 0;
    for (w.b = b_lo; w.b < b_hi; ++w.b) {
        w.load(p);
        mine += w.nch;
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) s_warp_sum[warp] = incl;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i <= C::CONSUMERS; ++i) {
        if (i == warp) incl += total;
        total += s_warp_sum[i];
    }
    const long long n_units = total * p.c.Hkv;
    const int n_blocks = (int)min((long long)gridDim.x, n_units);
    if ((int)blockIdx.x >= n_blocks) return;
    const long long u0 = n_units * blockIdx.x / n_blocks, u1 = n_units * (blockIdx.x + 1) / n_blocks;
    if (u0 >= (incl - mine) * p.c.Hkv && u0 < incl * p.c.Hkv) {
        long long before = incl - mine;
        for (w.b = b_lo;; ++w.b) {
            w.load(p);
            if (u0 < (before + w.nch) * p.c.Hkv) break;
            before += w.nch;
        }
        s_first = w.b;
        s_before = before;
    }
    __syncthreads();
    w.b = s_first;
    w.load(p);
    {
        const long long r = u0 - s_before * p.c.Hkv;
        w.hk = (int)(r / w.nch);
        w.begin = s_before * p.c.Hkv + (long long)w.hk * w.nch;
    }

    if (warp == C::CONSUMERS) {
        // ------------------------------------------------------------------------------- producer
        const int np_log = 7 - p.c.log_p;                  // pages of a chunk
        const int P = 1 << p.c.log_p, tiles = P / 16;
        const uint32_t page_bytes = (uint32_t)(P * D);
        bool waited = false, ok = true;
        int i = 0;
        for (long long u = u0; u < u1 && ok; w.next(p)) {
            const long long end = min(u1, w.begin + w.nch);
            const int c_end = w.ch0 + (int)(end - w.begin);
            int c = w.ch0 + (int)(u - w.begin);
            u = end;
            int base = 0, page = -1;                       // chunk of lane 0's page; this lane's page
            float ks = 0.f, vs = 0.f;
            for (int left = 0; c < c_end; ++c, --left) {
                if (left == 0) {
                    // the pages of the next 32 >> np_log chunks
                    left = 32 >> np_log;
                    base = c;
                    const int j = (c << np_log) + lane;
                    const int c_stop = min(c_end, c + left);
                    page = -1;
                    if ((long long)j * P < min((long long)w.n, (long long)c_stop * kKv8Chunk) && (j + 1) * (long long)P > w.lo) {
                        page = __ldg(p.table + (long long)w.b * p.max_pages + j);
                        if (page < 0 || page >= p.c.n_pages) {
                            record_error(kErrIndex, kSiteKvPage);
                            page = -1;
                        }
                    }
                    // the last chunk holds the new token, which the token kernel writes
                    if (!waited && (long long)c_stop * kKv8Chunk >= w.n) {
                        grid_dependency_wait();
                        asm volatile("fence.proxy.async.global;" ::: "memory");
                        waited = true;
                    }
                    if (page >= 0) {
                        ks = p.c.k_scale[(long long)page * p.c.Hkv + w.hk];
                        vs = p.c.v_scale[(long long)page * p.c.Hkv + w.hk];
                    }
                }
                const int s = i % C::NS;
                if (i >= C::NS && !__all_sync(0xffffffffu, mbar_wait(smem_u32(empty + s), (uint32_t)((i / C::NS) - 1) & 1u,
                                                                     p.wait_limit_ns, kSiteKv8Empty))) {
                    ok = false;
                    break;
                }
                const int rel = lane - ((c - base) << np_log);         // this lane's page within the chunk
                const bool here = rel >= 0 && rel < (1 << np_log);
                const bool load = here && page >= 0;
                if (here)
                    for (int k = 0; k < tiles; ++k)
                        s_meta[s * 8 + rel * tiles + k] =
                            make_float4(ks * p.c1, page >= 0 ? vs : -1.f, log2f(vs), 0.f);
                const uint32_t n_load = (uint32_t)__popc(__ballot_sync(0xffffffffu, load));
                const uint32_t bar = smem_u32(full + s);
                if (lane == 0) mbar_arrive_expect_tx(bar, n_load * 2u * page_bytes);
                __syncwarp();
                if (load) {
                    const uint32_t dst = smem_u32(smem) + (uint32_t)(2 * s) * C::TENSOR + (uint32_t)rel * page_bytes;
                    const int y = (page * p.c.Hkv + w.hk) << p.c.log_p;
                    tma_load_2d(dst, &tm_k, bar, 0, y);
                    tma_load_2d(dst + C::TENSOR, &tm_v, bar, 0, y);
                }
                ++i;
            }
            if (u >= u1) break;
        }
        if (!ok)   // the copies in flight end before the block does
            for (int k = max(0, i - C::NS); k < i; ++k)
                mbar_wait(smem_u32(full + k % C::NS), (uint32_t)(k / C::NS) & 1u, p.wait_limit_ns, kSiteKv8Full);
        return;
    }

    // ----------------------------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const int rt = warp % NRT, sub = warp / NRT;
    grid_dependency_wait();
    bool ok = true;
    int i = 0;
    for (long long u = u0; u < u1;) {
        const long long end = min(u1, w.begin + w.nch);
        const int c_begin = w.ch0 + (int)(u - w.begin), c_end = w.ch0 + (int)(end - w.begin);
        // qhat of heads rt * 8 + g: features in the order of the key rows' bytes
        uint32_t q[NSTEP][2];
        {
            const int hg = rt * 8 + g;
            const __nv_bfloat16* qr = p.qh + ((long long)w.b * p.H + (long long)w.hk * p.G + hg) * D;
#pragma unroll
            for (int st = 0; st < NSTEP; ++st) {
                const int f = D == 128 ? 32 * t + 4 * st : 16 * t + 4 * st;
                uint2 raw = make_uint2(0u, 0u);
                if (hg < p.G) raw = *reinterpret_cast<const uint2*>(qr + f);
                q[st][0] = pack_half2(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u));
                q[st][1] = pack_half2(__uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u));
            }
        }
        float o[2 * VW][4];
#pragma unroll
        for (int k = 0; k < 2 * VW; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;      // heads 2 t and 2 t + 1

        for (int c = c_begin; c < c_end; ++c, ++i) {
            const int s = i % C::NS;
            if (ok && !__all_sync(0xffffffffu, mbar_wait(smem_u32(full + s), (uint32_t)(i / C::NS) & 1u, p.wait_limit_ns,
                                                         kSiteKv8Full)))
                ok = false;
            if (!ok) break;
            const uint8_t* kt = smem + (2 * s) * C::TENSOR;
#pragma unroll 1
            for (int tile = sub; tile < 8; tile += KS) {
                const int pos0 = c * kKv8Chunk + 16 * tile;
                if (pos0 + 16 <= w.lo || pos0 >= w.n) continue;
                const float4 meta = s_meta[s * 8 + tile];
                if (meta.y < 0.f) continue;                            // a page that is not there
                const bool whole = pos0 >= w.lo && pos0 + 16 <= w.n;
                const uint8_t* kr = kt + tile * 16 * D;
                const uint8_t* vr = kr + C::TENSOR;
                uint32_t a[2][VW * 2];                                 // rows g, g + 8
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        const int row = g + 8 * r;
                        const int at = D == 128 ? row * 128 + (((2 * t + x) ^ (row & 7)) << 4)
                                                : row * 64 + ((t ^ ((row >> 1) & 3)) << 4);
                        const uint4 v4 = *reinterpret_cast<const uint4*>(kr + at);
                        a[r][4 * x] = v4.x;
                        a[r][4 * x + 1] = v4.y;
                        a[r][4 * x + 2] = v4.z;
                        a[r][4 * x + 3] = v4.w;
                    }
                uint32_t v[4][VW];                                     // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = 2 * t + (x & 1) + 8 * (x >> 1);
                    if (D == 128) {
                        const uint4 v4 = *reinterpret_cast<const uint4*>(vr + row * 128 + ((g ^ (row & 7)) << 4));
                        v[x][0] = v4.x;
                        v[x][1] = v4.y;
                        v[x][VW - 2] = v4.z;
                        v[x][VW - 1] = v4.w;
                    } else {
                        const uint2 v2 = *reinterpret_cast<const uint2*>(vr + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) +
                                                                         8 * (g & 1));
                        v[x][0] = v2.x;
                        v[x][1] = v2.y;
                    }
                }
                // S^T, two chains
                float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int st = 0; st < NSTEP; ++st) {
                    const uint32_t a0 = fp8x2_to_half2(a[0][st]), a1 = fp8x2_to_half2(a[1][st]);
                    const uint32_t a2 = fp8x2_to_half2(a[0][st] >> 16), a3 = fp8x2_to_half2(a[1][st] >> 16);
                    mma_16816((st & 1) ? s1 : s0, a0, a1, a2, a3, q[st][0], q[st][1]);
                }
                float x0 = (s0[0] + s1[0]) * meta.x, x1 = (s0[1] + s1[1]) * meta.x;    // key g
                float x2 = (s0[2] + s1[2]) * meta.x, x3 = (s0[3] + s1[3]) * meta.x;    // key g + 8
                if (!whole) {
                    // keys outside [lo, n): weight 0 whatever the page holds there
                    if (pos0 + g < w.lo || pos0 + g >= w.n) x0 = x1 = -INFINITY;
                    if (pos0 + g + 8 < w.lo || pos0 + g + 8 >= w.n) x2 = x3 = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int key = pos0 + 2 * t + (x & 1) + 8 * (x >> 1);
                        if (key < w.lo || key >= w.n)
#pragma unroll
                            for (int k = 0; k < VW; ++k) v[x][k] = 0u;
                    }
                }
                float t0 = fmaxf(x0, x2) + meta.z, t1 = fmaxf(x1, x3) + meta.z;
                if (__any_sync(0xffffffffu, t0 > m0 + kSlack || t1 > m1 + kSlack)) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
                        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
                    }
                    t0 = fmaxf(t0, m0);
                    t1 = fmaxf(t1, m1);
                    const float f0 = ex2_approx(m0 - t0), f1 = ex2_approx(m1 - t1);
                    m0 = t0;
                    m1 = t1;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int k = 0; k < 2 * VW; ++k) {
                        o[k][0] *= f0;
                        o[k][1] *= f1;
                        o[k][2] *= f0;
                        o[k][3] *= f1;
                    }
                }
                x0 = ex2_approx(x0 - m0);
                x1 = ex2_approx(x1 - m1);
                x2 = ex2_approx(x2 - m0);
                x3 = ex2_approx(x3 - m1);
                l0 += x0 + x2;
                l1 += x1 + x3;
                const uint32_t b0 = movmatrix_trans(pack_half2(x0 * meta.y, x1 * meta.y));
                const uint32_t b1 = movmatrix_trans(pack_half2(x2 * meta.y, x3 * meta.y));
#pragma unroll
                for (int k = 0; k < VW; ++k) {
                    // features 4 k .. 4 k + 3 of this lane, keys (2 t, 2 t + 1) and (2 t + 8, 2 t + 9)
                    const uint32_t p0 = __byte_perm(v[0][k], v[1][k], 0x5140), p1 = __byte_perm(v[2][k], v[3][k], 0x5140);
                    const uint32_t r0 = __byte_perm(v[0][k], v[1][k], 0x7362), r1 = __byte_perm(v[2][k], v[3][k], 0x7362);
                    mma_16816(o[2 * k], fp8x2_to_half2(p0), fp8x2_to_half2(p0 >> 16), fp8x2_to_half2(p1),
                              fp8x2_to_half2(p1 >> 16), b0, b1);
                    mma_16816(o[2 * k + 1], fp8x2_to_half2(r0), fp8x2_to_half2(r0 >> 16), fp8x2_to_half2(r1),
                              fp8x2_to_half2(r1 >> 16), b0, b1);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(empty + s));
        }

        // The piece's result: the warps' sums joined.
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        kv8_consumers_sync();              // the last piece's results have been read
        if (g == 0) {
            s_m[warp * 8 + 2 * t] = m0;
            s_m[warp * 8 + 2 * t + 1] = m1;
            s_l[warp * 8 + 2 * t] = l0;
            s_l[warp * 8 + 2 * t + 1] = l1;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (rt * 8 + 2 * t + e < p.G)
#pragma unroll
                for (int k = 0; k < 2 * VW; ++k)
                    *reinterpret_cast<float2*>(s_o + (warp * 8 + 2 * t + e) * D + 4 * VW * g + 2 * k) =
                        make_float2(o[k][e], o[k][2 + e]);
        kv8_consumers_sync();
        const bool alone = u == w.begin && end == w.begin + w.nch;
        const int slot = 2 * (int)blockIdx.x + (u0 < w.begin ? 1 : 0);
        for (int x = (int)threadIdx.x; x < p.G * D; x += 256) {
            const int h = x / D, d = x % D;
            const int hr = h >> 3, hc = h & 7;
            float M = -INFINITY;
#pragma unroll
            for (int k = 0; k < KS; ++k) M = fmaxf(M, s_m[(k * NRT + hr) * 8 + hc]);
            float L = 0.f, O = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int at = (k * NRT + hr) * 8 + hc;
                const float f = s_m[at] == -INFINITY && s_l[at] == 0.f ? 0.f : ex2_approx(s_m[at] - M);
                L = fmaf(s_l[at], f, L);
                O = fmaf(s_o[at * D + d], f, O);
            }
            if (alone) {
                const long long row = (long long)w.b * p.H + (long long)w.hk * p.G + h;
                // no visible key (pages outside the cache only): an empty row; a NaN stays one
                p.out[row * D + d] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
                if (d == 0 && p.lse != nullptr) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
            } else {
                float* pt = p.part + ((long long)slot * p.G + h) * (D + 4);
                pt[d] = O;
                if (d == 0) {
                    pt[D] = M;
                    pt[D + 1] = L;
                }
            }
        }
        if (!alone) {
            const int c_first = kv8_owner(w.begin, n_units, n_blocks);
            const int pieces = kv8_owner(w.begin + w.nch - 1, n_units, n_blocks) - c_first + 1;
            __threadfence();
            kv8_consumers_sync();
            if (threadIdx.x == 0) s_last = atomicAdd(p.counters + c_first, 1) == pieces - 1;
            kv8_consumers_sync();
            if (s_last) {
                __threadfence();
                const int first_slot = 2 * c_first + (n_units * c_first / n_blocks < w.begin ? 1 : 0);
                for (int x = (int)threadIdx.x; x < p.G * D; x += 256) {
                    const int h = x / D, d = x % D;
                    auto at = [&](int k) {
                        return p.part + ((long long)(k == 0 ? first_slot : 2 * (c_first + k)) * p.G + h) * (D + 4);
                    };
                    float M = -INFINITY, L = 0.f, O = 0.f;
                    for (int k = 0; k < pieces; ++k) M = fmaxf(M, __ldcg(at(k) + D));
                    for (int k = 0; k < pieces; ++k) {
                        const float mk = __ldcg(at(k) + D), lk = __ldcg(at(k) + D + 1);
                        const float f = mk == -INFINITY && lk == 0.f ? 0.f : ex2_approx(mk - M);
                        L = fmaf(lk, f, L);
                        O = fmaf(__ldcg(at(k) + d), f, O);
                    }
                    const long long row = (long long)w.b * p.H + (long long)w.hk * p.G + h;
                    p.out[row * D + d] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
                    if (d == 0 && p.lse != nullptr)
                        p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
                }
            }
        }
        u = end;
        if (u < u1) w.next(p);
    }
}

}  // namespace swa
