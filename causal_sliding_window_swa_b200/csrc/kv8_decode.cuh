// kv8_decode.cuh -- one generation step over the paged 8-bit cache of kv8.cuh, for requests of
// different lengths: request b has n_b = seq_len[b] tokens, the new one at position n_b - 1.
//   1. kv8_token_kernel: the layer's prologue of the new token, as in decode.cuh (every qhat, khat and
//      v' element the correctly rounded bf16 of its exact value); qhat goes to the workspace, khat and v'
//      into the token's page, whose scale grows where they need it (kv8.cuh).
//   2. the attention of qhat over the cached keys [max(0, n_b - W, min(start_b, n_b - 1)), n_b):
//      out = sum_j softmax_j(qhat . k_j / sqrt(D)) v_j,  lse = ln sum_j exp(qhat . k_j / sqrt(D)).
// Requests with n_b <= 0 are empty rows: out = 0, lse = -inf.
#pragma once

#include <climits>
#include <type_traits>

#include "decode.cuh"
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
    uint2* qh;                    // (B, Hkv) items of qhat as operands (kv8_q_place), workspace
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

// Entry i of the RoPE row of `pos`, in the split of the prefill table.
template <int D>
__device__ __forceinline__ void kv8_rope_entry(double base, int pos, int i, float4* s_tab32, double2* s_tab64) {
    const double theta = pow(base, -2.0 * (double)i / (double)D);
    double sn, cs;
    sincos((double)pos * theta, &sn, &cs);
    float c_hi, c_lo, s_hi, s_lo;
    rope_split(cs, c_hi, c_lo);
    rope_split(sn, s_hi, s_lo);
    s_tab32[i] = make_float4(c_hi, c_lo, s_hi, s_lo);
    s_tab64[i] = make_double2(cs, sn);
}

// The empty row of heads [h0, h0 + heads) of request b, by all threads of the block.
template <int D>
__device__ __forceinline__ void kv8_empty_row(__nv_bfloat16* out, float* lse, long long row0, int heads) {
    for (int i = threadIdx.x; i < heads * (D / 8); i += blockDim.x)
        reinterpret_cast<uint4*>(out + row0 * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (lse != nullptr)
        for (int i = threadIdx.x; i < heads; i += blockDim.x) lse[row0 + i] = -INFINITY;
}

// One row of request b's new token, D/8 lanes (this one is lane c): query head `h` (kQuery), or key/value head `h`
// (kKeyValue), whose khat and v' go into the cache.  load() issues the loads; finish(), once the RoPE row is
// there, is called by whole warps.
enum { kNoRow = 0, kQuery = 1, kKeyValue = 2 };
template <int D>
struct Kv8Row {
    int kind, h, page;
    uint2 x0, x1, v0, v1, e0, e1;
    float2 gw;
    float old_scale[2];

    __device__ __forceinline__ void load(const Kv8TokenParams& p, int b, int pos, int kind_, int h_, int c) {
        constexpr int HALF = D / 2;
        const int i0 = 4 * c, Hkv = p.c.Hkv;
        kind = kind_;
        h = h_;
        page = -1;
        x0 = x1 = v0 = v1 = e0 = e1 = make_uint2(0u, 0u);
        gw = make_float2(0.f, 0.f);
        old_scale[0] = old_scale[1] = 1.f;
        if (kind != kNoRow) {
            const __nv_bfloat16* src =
                kind == kQuery ? p.q + ((long long)b * p.H + h) * D : p.k + ((long long)b * Hkv + h) * D;
            x0 = ldg_stream8(src + i0);
            x1 = ldg_stream8(src + HALF + i0);
        }
        if (kind == kKeyValue) {
            const __nv_bfloat16* vr = p.v + ((long long)b * Hkv + h) * D;
            v0 = ldg_stream8(vr + i0);
            v1 = ldg_stream8(vr + HALF + i0);
            page = __ldg(p.table + (long long)b * p.max_pages + (pos >> p.c.log_p));
            if (page < 0 || page >= p.c.n_pages) {
                if (c == 0) record_error(kErrIndex, kSiteKvPage);
                page = -1;
            } else {
                old_scale[0] = p.c.k_scale[(long long)page * Hkv + h];
                old_scale[1] = p.c.v_scale[(long long)page * Hkv + h];
            }
            if (p.ve != nullptr) {
                const __nv_bfloat16* er = p.ve + ((long long)b * Hkv + h) * D;
                e0 = ldg_stream8(er + i0);
                e1 = ldg_stream8(er + HALF + i0);
                // 2 sigmoid(x . Wg[:, h]) in fp64, the 32 channels in order (the prefill gate's order)
                const __nv_bfloat16* xr = p.gate_x + (long long)b * 32;
                double z = 0.0;
#pragma unroll
                for (int cc = 0; cc < 32; ++cc)
                    z = fma((double)__bfloat162float(xr[cc]), (double)__bfloat162float(p.Wg[cc * Hkv + h]), z);
                const double g = 2.0 / (1.0 + exp(-z));
                gw.x = (float)g;
                gw.y = (float)(g - (double)gw.x);
            }
        }
    }

    // qhat's (or khat's) features 4 c .. and D/2 + 4 c .. in o0, o1.
    __device__ __forceinline__ void finish(const Kv8TokenParams& p, int pos, int c, const float4* s_tab32,
                                           const double2* s_tab64, uint2& o0, uint2& o1) {
        constexpr int TPR = D / 8, HALF = D / 2;
        const int i0 = 4 * c;
        float4 cs4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cs4[e] = s_tab32[i0 + e];
        rope_rms_exact4<D>(x0, x1, cs4, s_tab64 + i0, p.eps, o0, o1);
        if (kind == kKeyValue && p.ve != nullptr) {
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
            if (kind != kKeyValue || page < 0) continue;
            int e = scale_exponent(a);
            const long long ph = (long long)page * p.c.Hkv + h;
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
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Place, in groups of four, of features f .. f + 3 (f a multiple of 4) of head h among an item's heads of qhat as the
// products' B operands, fp16: lane t of a quad takes D/4 consecutive features (kv8_tile), eight of them from each 16 bytes;
// [head][eights][t], a head's eights exchanged in pairs where it is odd: a quad's 64 bytes and the next head's then lie in
// different banks.
template <int D>
__device__ __forceinline__ int kv8_q_place(int h, int f) {
    constexpr int EIGHTS = D / 32;                              // of a lane
    const int eight = f / 8;
    return ((h * EIGHTS + (eight % EIGHTS ^ (h & 1))) * 4 + eight / EIGHTS) * 2 + (f & 4) / 4;
}
__device__ __forceinline__ uint2 bf16x4_to_half4(uint2 raw) {
    return make_uint2(pack_half2(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u)),
                      pack_half2(__uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)));
}

// Rows of request b = blockIdx.x: its H query rows, then its Hkv key/value rows (when the token is to be
// appended); blockIdx.y takes one group of 256 / (D/8) rows.  Every block builds the RoPE row of the token's
// position in shared memory.
template <int D>
__global__ void __launch_bounds__(256) kv8_token_kernel(const Kv8TokenParams p) {
    constexpr int TPR = D / 8, HALF = D / 2, RPB = 256 / TPR;
    __shared__ float4 s_tab32[HALF];
    __shared__ double2 s_tab64[HALF];
    grid_dependents_launch();     // the attention kernel may start: it waits before it reads what is written here
    const int b = (int)blockIdx.x;
    if (b == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < p.n_counters; i += 256) p.counters[i] = 0;
    const int n = kv8_length(p.seq_len, b, p.max_pages, p.c.log_p);
    if (n == 0) {
        if (blockIdx.y == 0) {
            if (threadIdx.x == 0 && p.seq_len[b] > 0) record_error(kErrIndex, kSiteKvLen);
            kv8_empty_row<D>(p.out, p.lse, (long long)b * p.H, p.H);
        }
        return;
    }
    const int row = (int)blockIdx.y * RPB + (int)threadIdx.x / TPR, c = (int)threadIdx.x % TPR;
    const bool is_q = row < p.H, is_kv = !is_q && p.k != nullptr && row - p.H < p.c.Hkv;
    Kv8Row<D> r;
    r.load(p, b, n - 1, is_q ? kQuery : is_kv ? kKeyValue : kNoRow, is_q ? row : row - p.H, c);
    if ((int)threadIdx.x < HALF) kv8_rope_entry<D>(p.base, n - 1, (int)threadIdx.x, s_tab32, s_tab64);
    __syncthreads();
    uint2 o0, o1;
    r.finish(p, n - 1, c, s_tab32, s_tab64, o0, o1);
    if (is_q) {
        const int G = p.H / p.c.Hkv, item = row / G, h = row - item * G;
        uint2* dst = p.qh + ((long long)b * p.c.Hkv + item) * (G * D / 4);
        dst[kv8_q_place<D>(h, 4 * c)] = bf16x4_to_half4(o0);
        dst[kv8_q_place<D>(h, HALF + 4 * c)] = bf16x4_to_half4(o1);
    }
}

// ------------------------------------------------------------------------------------- attention
//
// HBM-bound by its bytes: every visible key's and value's code is read once for all query heads of its
// key/value head.  At 6.5 TB/s an SM has to take in 23 codes a clock, each of which is converted and multiplied with
// up to 64 query heads: too much for fp32 lanes, little for the tensor cores, so both products are
// mma.sync m16n8k16 on fp16 operands (a code is exact in fp16, qhat as well down to 2^-17), fp32 sums.
// (tcgen05 would need 128-row tiles of one type: the codes converted into shared memory first, or
// qhat and the weights split into three e4m3 parts each.  With up to eight heads the products are a few percent
// of the time; with 32 and more they bound the kernel, see below.)
//
// Units.  A unit is a chunk of 64 key positions (aligned) of one request and key/value head.  Units are
// numbered request by request, head by head, chunk by chunk, with kKv8ItemCost more at the end of each
// (request, head) item for what an item costs beside its keys, and the blocks take equal
// stretches of them, whatever the requests' lengths: every block finds its first unit from the
// sequence lengths alone, so the host needs no lengths and a captured launch stays valid.  An
// item that one block has whole is finished there; the pieces of one that several
// blocks share go to the workspace, and the block that arrives last adds them in order (the result
// does not depend on which one that is).
//
// Pipeline.  A producer warp looks up a batch of pages at a time (32 boxes, one to a lane) and brings their codes
// into a ring of chunk-sized stages by TMA, with the scales of each box; items' qhat comes by bulk copy into a
// ring of its own.  Copies of pages that take no new token do not wait for the token kernel (32 requests of up to
// 4096 tokens 43.2 -> 41.5 us).  Eight consumer warps take 16 keys and NT groups of eight query heads at a time.
// With one set of heads they are two sets of four warps that take chunks in turn, each with its producer (one
// producer took 0.12 us a chunk and bounded D = 64); with more heads than a warp holds, the warps are shared out
// over NRG sets of heads.
//   S^T (16 keys x 8 heads) = K qhat^T: a lane's A operand is 16 (or 32) consecutive bytes of key rows g and
//   g + 8 (lane = 4 g + t); the features are taken in the order that this gives, qhat's likewise.
//   O^T (features x 8 heads) += V^T W^T: the bytes of a lane's key pairs are interleaved before the
//   conversion; W^T is the transpose of S^T's layout, which movmatrix makes.
// The TMA swizzle (128 bytes; 64 for D = 64) keeps both reads free of bank conflicts (D = 64: two-way).
// With up to eight heads a warp fits in 96 registers and two blocks in an SM; the loop has none to spare, so the walk
// through the units lives in shared memory.
//
// Softmax.  With x_j = log2(e) qhat . k_j / sqrt(D) and a running reference m, p_j = 2^(x_j - m) is summed in
// fp32 and w_j = p_j * (value scale) enters the product as fp16 (rounded to 11 bits: off by at most 2^-11 of each
// weight, an eighth of the output's own rounding).  m is raised, with one rescaling, only when some
// x_j + log2(value scale) passes it by more than kSlack: it is at least the first tile's maximum, so the largest
// 2^5 w_j, which is what the product takes, lies between 2^5 and 2^15.  A key that weighs little may still be all that counts (one
// that outweighs it may have values of zero, or values in other features), so weights that fp16 would hold in fewer bits are
// multiplied apart, times 2^15, with the codes times 2^-15 (exact in fp16): 11 bits down to 2^-34 of the largest weight, and
// half a step of 2^-45 of it below.  Scores of rows with unit root mean square lie within 33 binades.  A tile with such a weight
// has twice the products with v: where all have, 32 requests of up to 16384 tokens 178 us against 173, 48 of one key/value head
// with 16 heads 48.4 against 44.7.  The test for it takes about 1% (2 to 3% with few keys or 32 heads).  With a value scale of
// 2^e the largest p_j may be 2^-e, so fp32 keeps those above 2^(e - 126) of the largest: 2^-66 at e = 60.
//
// Measured (D = 128, lengths from a quarter to all of the most, fractions of 6565 GB/s): 32 requests of up to 16384 tokens, 12
// heads 194 us, 0.95; of 8192 93 us, 0.88; 48 requests of up to 8192, two key/value heads, one query head each
// 35 us, eight each 37 us, 0.58.  About 12 us do not depend on the keys: the token kernel and the start behind it 2.4, the
// units 2, the first table entries and copies 3, joining the warps, arriving and adding the pieces 3.4, the rest the uneven
// ends.  Bound by the consumers: one key/value head with 16 heads 45, with 32 72, with 64 114 us for the same bytes.
constexpr int kKv8Chunk = 64;           // key positions of a unit
constexpr int kKv8Tiles = kKv8Chunk / 16;
constexpr int kKv8Sms = 148;
// Blocks of the attention kernel, at most: two per SM where a warp has one group of eight heads, else one.
__host__ __device__ constexpr int kv8_max_blocks(int G) { return G <= 8 ? 2 * kKv8Sms : kKv8Sms; }
// What an item costs beside its units, in units (96 items of up to 8192 tokens, G = 8: 37.4 us, with 2 38.3; 256 requests of 128
// tokens and 12 heads 34.9, 36.4 with 2, 44.2 with 0).
constexpr int kKv8ItemCost = 4;
// Items of at most so many units are not split: adding pieces costs more than the uneven ends (768
// items of up to 512 tokens: 23.8 us, with 4 26.8).
constexpr int kKv8Whole = 16;
// Units of a block, at least, where there are few: the pieces are added by one block, which takes longer with more heads (24
// items of 1000 tokens, G = 1: 10.9 us by 2, 14.1 by 6; one of 4000, G = 16: 21.5 by 2, 16.6 by 6).
__host__ __device__ constexpr int kv8_min_share(int G) { return G <= 8 ? 2 : 6; }
constexpr int kKv8StepChunks = 48;      // chunks of a block in the one-launch form, at most
constexpr float kSlack = 10.f;
constexpr float kWeightUp = 32.f;       // weights enter the products times 2^5: up to 2^15, which fp16 holds
constexpr float kHalfLeast = 0x1p-14f;  // fp16 has 11 bits from here on

enum : unsigned int { kSiteKv8Full = 83, kSiteKv8Empty = 84 };

struct Kv8AttnParams {
    const uint2* qh;              // (B, Hkv) items of qhat as operands (kv8_q_place)
    const int* table;
    const int* seq_len;
    const int* doc_start;         // (B) or null
    __nv_bfloat16* out;
    float* lse;
    Kv8Store c;
    int* counters;                // zero at the start
    float* part;                  // [2 * blocks][G][D + 4]: O, then m and l
    int B, H, G, max_pages, W;    // W = 0: no window
    bool append;                  // the new tokens are written by this step
    float c1;                     // log2(e) / sqrt(D)
    unsigned long long wait_limit_ns;
};

// NT groups of eight query heads per warp; NRG sets of warps that split more groups than that; NSTAGES ring stages.
template <int D, int NT, int NRG, int NSTAGES>
struct Kv8Cfg {
    static constexpr int CONSUMERS = 8;
    static constexpr int BLOCKS_PER_SM = NT == 1 ? 2 : 1;
    static constexpr int KSLOTS = CONSUMERS / NRG;               // warps that share the keys of a group of heads
    static constexpr int SETS = KSLOTS > kKv8Tiles ? KSLOTS / kKv8Tiles : 1;    // chunks in work at a time, each with a producer
    static constexpr int TPW = KSLOTS < kKv8Tiles ? kKv8Tiles / KSLOTS : 1;     // tiles of a chunk for each warp
    static constexpr int THREADS = 32 * (CONSUMERS + SETS);
    static constexpr int TENSOR = kKv8Chunk * D;                 // bytes of a chunk's K (and V)
    static constexpr int HEADS = 8 * NT;                         // query heads of a warp
    static constexpr int NTG = NT * NRG;                         // groups of eight heads
    // Ring stages: a multiple of SETS, so that a set of warps takes every use of its stages and its waits see each
    // phase of their barriers in turn.
    static constexpr int NS = NSTAGES;
    // Results on their way to be joined: one head in two of half of the warps, or two heads of each warp.
    static constexpr int MERGE_PITCH = D + 16;
    static constexpr int MERGE = CONSUMERS / 2 * (HEADS / 2) * MERGE_PITCH * 4;
    static constexpr int OFF_O = NS * 2 * TENSOR;
    static constexpr int OFF_ML = OFF_O + MERGE;                 // m [8][HEADS], l [8][HEADS]
    static constexpr int OFF_Q = OFF_ML + 2 * CONSUMERS * HEADS * 4;      // items' qhat operands: two of the largest, or more
    static constexpr int QBYTES = 2 * NTG * 8 * D * 2;
    static constexpr int MAXQ = 8;                               // items in that ring, at most
    static constexpr int OFF_META = OFF_Q + QBYTES;              // per stage and tile: ks c1, 2^5 vs, log2 vs, pad
    static constexpr int OFF_BAR = OFF_META + NS * kKv8Tiles * 16;
    static constexpr int SMEM = OFF_BAR + 2 * (NS + MAXQ) * 8 + 1024;     // + alignment slack
    static_assert(NS % SETS == 0, "a stage belongs to one set of warps");
    static_assert(MERGE >= 4096, "the sums of a shared item's pieces");
    static_assert(OFF_Q % (2 * D) == 0, "a head's operands lie within a multiple of their size");
    static_assert(BLOCKS_PER_SM * (SMEM + 2048) <= 228 * 1024, "shared memory");
};
// The attention kernel's and, with room for its own tables, the one-launch form's.
template <int D, int NT, int NRG>
using Kv8AttnCfg = Kv8Cfg<D, NT, NRG, D == 128 ? (NT == 1 ? 6 : 8) : 12>;
template <int D>
using Kv8StepCfg = Kv8Cfg<D, 1, 1, D == 128 ? 4 : 8>;

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
    int begin;             // its first unit; it has size() of them, of which the last kKv8ItemCost stand for its cost

    __device__ __forceinline__ int size() const { return nch + kKv8ItemCost; }

    __device__ __forceinline__ void load(const Kv8AttnParams& p) {
        const int len = kv8_length(p.seq_len, b, p.max_pages, p.c.log_p);
        set(len, len > 0 ? kv8_first_key(p, b, len) : 0);
    }
    __device__ __forceinline__ void set(int n_, int lo_) {
        n = n_;
        lo = lo_;
        ch0 = lo / kKv8Chunk;
        nch = n > 0 ? (n - 1) / kKv8Chunk - ch0 + 1 : 0;
    }
    // to the item after this one
    __device__ __forceinline__ void next(const Kv8AttnParams& p) {
        begin += size();
        if (++hk < p.c.Hkv) return;
        hk = 0;
        do {
            ++b;
            load(p);
        } while (nch == 0);
    }
};

// n units in m equal stretches (the first n % m one longer): where stretch c begins, and which has unit u.
struct Kv8Shares {
    int m, q, r;
    __device__ __forceinline__ Kv8Shares(int n, int blocks) : m(blocks), q(n / blocks), r(n % blocks) {}
    __device__ __forceinline__ int begin(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int owner(int u) const {
        return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
    }
};

__device__ __forceinline__ uint4 ld_shared_16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
// Four e4m3 codes -> two pairs of fp16, exact.
__device__ __forceinline__ void fp8x4_to_half4(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
// Two fp16 times 2^-15: exact for codes, whose smallest step is 2^-9.
__device__ __forceinline__ uint32_t half2_down15(uint32_t x) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0x1p-15f));
    return *reinterpret_cast<const uint32_t*>(&r);
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
// What a partial sum (m, l) is multiplied with when the reference becomes M, once for each half of the exponent: 0 where the
// sum is empty.  References contain the value scales, 2^-60 to 2^120, so M - m can pass the 126 binades of one factor while l,
// up to 2^60 for each key, is still to be kept; O is relative to the largest weight, and what one factor h * h takes from it
// is nothing.
__device__ __forceinline__ float kv8_half_factor(float m, float l, float M) {
    return m == -INFINITY && l == 0.f ? 0.f : ex2_approx(0.5f * (m - M));
}
__device__ __forceinline__ float kv8_scale_sum(float l, float half_factor) { return l * half_factor * half_factor; }

// One tile of 16 keys at position pos0, rows at kr (and `tensor` bytes behind it the values), for NT groups of eight
// heads.  meta: key scale times c1, value scale times kWeightUp, log2 of the value scale.  q: shared address of this lane's qhat
// operands, of each group's head: 16-byte words at q ^ 64 i (kv8_q_place).
template <int D, int NT>
__device__ __forceinline__ void kv8_tile(const uint8_t* kr, int tensor, int pos0, int lo, int n, const float4& meta,
                                         const uint32_t (&q)[NT], float (&o)[NT][D / 16][4], float (&m)[NT][2],
                                         float (&l)[NT][2], int g, int t) {
    constexpr int NSTEP = D / 16, VW = D / 32;
    const bool whole = pos0 >= lo && pos0 + 16 <= n;
    const uint8_t* vr = kr + tensor;
    uint32_t a[2][NSTEP];                                  // rows g, g + 8
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
            const int row = g + 8 * r;
            const int at = D == 128 ? row * 128 + (((2 * t + x) ^ (row & 7)) << 4) : row * 64 + ((t ^ ((row >> 1) & 3)) << 4);
            const uint4 v4 = *reinterpret_cast<const uint4*>(kr + at);
            a[r][4 * x] = v4.x;
            a[r][4 * x + 1] = v4.y;
            a[r][4 * x + 2] = v4.z;
            a[r][4 * x + 3] = v4.w;
        }
    // S^T, in two chains where there is one group
    constexpr int NC = NT == 1 ? 2 : 1;
    float sc[NT][NC][4];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4 * NC; ++e) sc[x][e / 4][e % 4] = 0.f;
    uint4 qs[NT];
#pragma unroll
    for (int st = 0; st < NSTEP; ++st) {
        if ((st & 1) == 0)
#pragma unroll
            for (int x = 0; x < NT; ++x) qs[x] = ld_shared_16(q[x] ^ (st / 2 * 64));
        uint32_t a0, a1, a2, a3;
        fp8x4_to_half4(a[0][st], a0, a2);
        fp8x4_to_half4(a[1][st], a1, a3);
#pragma unroll
        for (int x = 0; x < NT; ++x)
            mma_16816(sc[x][st % NC], a0, a1, a2, a3, (st & 1) ? qs[x].z : qs[x].x, (st & 1) ? qs[x].w : qs[x].y);
    }
    float w[NT][4];                                        // the weights: keys g and g + 8, heads 2 t and 2 t + 1
    float least = INFINITY;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        float s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = (NC == 2 ? sc[x][0][e] + sc[x][NC - 1][e] : sc[x][0][e]) * meta.x;
        if (!whole) {
            if (pos0 + g < lo || pos0 + g >= n) s[0] = s[1] = -INFINITY;
            if (pos0 + g + 8 < lo || pos0 + g + 8 >= n) s[2] = s[3] = -INFINITY;
        }
        float t0 = fmaxf(s[0], s[2]) + meta.z, t1 = fmaxf(s[1], s[3]) + meta.z;
        if (__any_sync(0xffffffffu, t0 > m[x][0] + kSlack || t1 > m[x][1] + kSlack)) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
            }
            t0 = fmaxf(t0, m[x][0]);
            t1 = fmaxf(t1, m[x][1]);
            const float h0 = ex2_approx(0.5f * (m[x][0] - t0)), h1 = ex2_approx(0.5f * (m[x][1] - t1));
            const float f0 = h0 * h0, f1 = h1 * h1;
            m[x][0] = t0;
            m[x][1] = t1;
            l[x][0] = kv8_scale_sum(l[x][0], h0);
            l[x][1] = kv8_scale_sum(l[x][1], h1);
#pragma unroll
            for (int k = 0; k < 2 * VW; ++k) {
                o[x][k][0] *= f0;
                o[x][k][1] *= f1;
                o[x][k][2] *= f0;
                o[x][k][3] *= f1;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = ex2_approx(s[e] - m[x][e & 1]);
        l[x][0] += s[0] + s[2];
        l[x][1] += s[1] + s[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[x][e] = s[e] * meta.y;
            least = fminf(least, w[x][e]);
        }
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
            const uint2 v2 = *reinterpret_cast<const uint2*>(vr + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (g & 1));
            v[x][0] = v2.x;
            v[x][1] = v2.y;
        }
    }
    if (!whole) {
        // values of keys outside [lo, n) count for nothing, whatever the page holds there
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int key = pos0 + 2 * t + (x & 1) + 8 * (x >> 1);
            if (key < lo || key >= n)
#pragma unroll
                for (int k = 0; k < VW; ++k) v[x][k] = 0u;
        }
    }
    // O^T, with the small weights apart where there are any
    auto add = [&](auto split) {
        constexpr bool kSplit = decltype(split)::value;
        uint32_t b[NT][2], b_small[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float up[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                up[e] = w[x][e] < kHalfLeast ? w[x][e] * 0x1p15f : 0.f;
                if (kSplit && w[x][e] < kHalfLeast) w[x][e] = 0.f;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                b[x][r] = movmatrix_trans(pack_half2(w[x][2 * r], w[x][2 * r + 1]));
                if (kSplit) b_small[x][r] = movmatrix_trans(pack_half2(up[2 * r], up[2 * r + 1]));
            }
        }
#pragma unroll
        for (int k = 0; k < VW; ++k) {
            // features 4 k .. 4 k + 3 of this lane, keys (2 t, 2 t + 1) and (2 t + 8, 2 t + 9)
            uint32_t a[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int bytes = y == 0 ? 0x5140 : 0x7362;
                fp8x4_to_half4(__byte_perm(v[0][k], v[1][k], bytes), a[y][0], a[y][1]);
                fp8x4_to_half4(__byte_perm(v[2][k], v[3][k], bytes), a[y][2], a[y][3]);
            }
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) mma_16816(o[x][2 * k + y], a[y][0], a[y][1], a[y][2], a[y][3], b[x][0], b[x][1]);
            if (kSplit) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[y][e] = half2_down15(a[y][e]);
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        mma_16816(o[x][2 * k + y], a[y][0], a[y][1], a[y][2], a[y][3], b_small[x][0], b_small[x][1]);
            }
        }
    };
    bool split = __any_sync(0xffffffffu, least < kHalfLeast);
    if (split && !whole) {                                 // not for the keys that are not visible, whose weights are 0
        bool small = false;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) small = small || (w[x][e] > 0.f && w[x][e] < kHalfLeast);
        split = __any_sync(0xffffffffu, small);
    }
    if (split) add(std::true_type{});
    else add(std::false_type{});
}

// Four features of the result, and its log-sum-exp: O / L, or an empty row where no key was visible (all on pages
// outside the cache); a NaN stays one.
template <int D>
__device__ __forceinline__ void kv8_store4(const Kv8AttnParams& p, int b, int hk, int h, int d4, const float4& O, float M,
                                           float L) {
    const long long row = (long long)b * p.H + (long long)hk * p.G + h;
    const float inv = L == 0.f ? 0.f : (1.f / kWeightUp) / L;
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * d4) =
        make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
    if (d4 == 0 && p.lse != nullptr) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

__device__ __forceinline__ void kv8_consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Shared memory of a block.
template <class C>
struct Kv8Shared {
    uint8_t* ring;             // stage s: K at 2 s TENSOR, V behind it
    float* o;
    float* m;
    float* l;
    uint4* q;
    float4* meta;
    uint64_t* full;
    uint64_t* empty;
    uint64_t* q_full;
    uint64_t* q_empty;

    __device__ __forceinline__ explicit Kv8Shared(uint8_t* dsmem) {
        ring = dsmem + ((1024u - (smem_u32(dsmem) & 1023u)) & 1023u);
        o = reinterpret_cast<float*>(ring + C::OFF_O);
        m = reinterpret_cast<float*>(ring + C::OFF_ML);
        l = m + C::CONSUMERS * C::HEADS;
        q = reinterpret_cast<uint4*>(ring + C::OFF_Q);
        meta = reinterpret_cast<float4*>(ring + C::OFF_META);
        full = reinterpret_cast<uint64_t*>(ring + C::OFF_BAR);
        empty = full + C::NS;
        q_full = empty + C::NS;
        q_empty = q_full + C::MAXQ;
    }
    // Items in the ring of qhat operands, each of G * D / 8 16-byte words: a power of two.
    static __device__ __forceinline__ int q_ring_log(int words) {
        return 31 - __clz(min(C::MAXQ, C::QBYTES / (16 * words)));
    }
    __device__ __forceinline__ void init_barriers() const {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(full + s), 1);
            mbar_init(smem_u32(empty + s), C::CONSUMERS / C::SETS);
        }
        for (int s = 0; s < C::MAXQ; ++s) {
            mbar_init(smem_u32(q_full + s), 1);
            mbar_init(smem_u32(q_empty + s), C::CONSUMERS);
        }
        fence_barrier_init();
    }
};

// A producer warp: its set's chunks (every SETS-th, from `part` on) of units [u0, u1) from walk position w into the ring; one
// warp for all chunks would bound a block at D = 64.  Box {D, min(P, 64)}.
// kAppend: the block itself writes the new token (the consumers arrive at barrier 2 when that is done), so the item's last
// chunk waits for that.
template <int D, class C, bool kAppend>
__device__ __forceinline__ void kv8_produce(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Kv8AttnParams& p,
                                            const Kv8Shared<C>& sh, Kv8Walk w, int u0, int u1, int part, int lane,
                                            bool append) {
    // A box is a page, or the half of a 128-token page that a chunk has.
    const int box_log = min(p.c.log_p, 6), nb_log = 6 - box_log;   // 64 >> nb_log keys; boxes of a chunk
    const uint32_t box_bytes = (uint32_t)((1 << box_log) * D);
    // A batch: the boxes, one to a lane, of up to 32 >> nb_log chunks of an item.  Its table entries are loaded two
    // batches ahead, its scales one: what the warp spends on a chunk bounds the rate of its set.
    struct Pages {
        int chunks, hk, page, sub;     // this lane's table entry (kNone: not wanted), its first row in the page
        int item;                      // whose first chunks here these are, else -1
    };
    struct Boxes {
        int chunks, ph, row;           // this lane's page and head, and its first row in the cache (-1: none)
        int item;
        float ks, vs;
    };
    constexpr int kNone = INT_MIN;
    int u = u0, c = w.ch0 + (u0 - w.begin);
    bool fresh = true;
    auto look_up = [&]() {
        Pages f{0, w.hk, kNone, 0, -1};
        if (u >= u1) return f;
        if (fresh) f.item = w.b * p.c.Hkv + w.hk;
        fresh = false;
        const int c_end = w.ch0 + (min(u1, w.begin + w.nch) - w.begin);
        f.chunks = min(32 >> nb_log, c_end - c);
        const long long pos = (long long)c * kKv8Chunk + ((long long)lane << box_log);
        f.sub = (int)pos & ((1 << p.c.log_p) - 1);
        if (lane < (f.chunks << nb_log) && pos < w.n && pos + (1 << box_log) > w.lo) {
            f.page = __ldg(p.table + (long long)w.b * p.max_pages + (int)(pos >> p.c.log_p));
            if (f.page == kNone) f.page = -1;
        }
        u += f.chunks;
        c += f.chunks;
        if (u == w.begin + w.nch) u = w.begin + w.size();
        if (c == c_end && u < u1) {
            w.next(p);
            c = w.ch0;
            fresh = true;
        }
        return f;
    };
    auto load_scales = [&](Boxes& x) {
        if (x.row >= 0) {              // volatile: the token may be written while this block runs
            x.ks = *(const volatile float*)(p.c.k_scale + x.ph);
            x.vs = *(const volatile float*)(p.c.v_scale + x.ph);
        }
    };
    auto find = [&](const Pages& f) {
        Boxes x{f.chunks, 0, -1, f.item, 0.f, -1.f};
        if (f.page >= 0 && f.page < p.c.n_pages) {
            x.ph = f.page * p.c.Hkv + f.hk;
            x.row = (x.ph << p.c.log_p) + f.sub;
            load_scales(x);
        } else if (f.page != kNone) {
            record_error(kErrIndex, kSiteKvPage);
        }
        return x;
    };
    int next = part, s = part, uses = 0;   // the set's next chunk, from the batch's first; its stage; how often round the ring
    auto advance = [&]() {
        next += C::SETS;
        if ((s += C::SETS) >= C::NS) {
            s -= C::NS;
            ++uses;
        }
    };
    // Chunk k's copies into stage st, with its scales where `meta` is given.
    auto copy = [&](const Boxes& x, int k, int st, const float4* meta) {
        const int rel = lane - (k << nb_log);
        const bool here = (unsigned)rel < (1u << nb_log), load = here && x.row >= 0;
        if (meta != nullptr && here) sh.meta[st * kKv8Tiles + rel] = *meta;
        const uint32_t n_load = (uint32_t)__popc(__ballot_sync(0xffffffffu, load));
        const uint32_t bar = smem_u32(sh.full + st);
        __syncwarp();
        if (lane == 0) {
            if (meta != nullptr) mbar_arrive_expect_tx(bar, n_load * 2u * box_bytes);
            else asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar),
                              "r"(n_load * 2u * box_bytes)
                              : "memory");
        }
        __syncwarp();
        if (load) {
            const uint32_t dst = smem_u32(sh.ring) + (uint32_t)(2 * st) * C::TENSOR + (uint32_t)rel * box_bytes;
            tma_load_2d(dst, &tm_k, bar, 0, x.row);
            tma_load_2d(dst + C::TENSOR, &tm_v, bar, 0, x.row);
        }
    };
    // An item's qhat (of the token kernel).
    const int q_words = p.G * D / 8, q_ring = 1 << Kv8Shared<C>::q_ring_log(q_words);
    int qs = 0, q_uses = 0;
    auto copy_q = [&](int item) {
        if (kAppend || part > 0 || item < 0) return true;
        if (q_uses > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(sh.q_empty + qs), (uint32_t)(q_uses - 1) & 1u,
                                                             p.wait_limit_ns, kSiteKv8Empty)))
            return false;
        if (lane == 0) {
            const uint32_t bar = smem_u32(sh.q_full + qs);
            mbar_arrive_expect_tx(bar, (uint32_t)q_words * 16u);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(sh.q + qs * q_words)),
                         "l"(p.qh + (long long)item * (2 * q_words)), "r"(q_words * 16), "r"(bar)
                         : "memory");
        }
        __syncwarp();
        if (++qs == q_ring) {
            qs = 0;
            ++q_uses;
        }
        return true;
    };
    // (a scale of zero, which no write leaves, counts as the smallest in the reference: its keys have values of zero)
    auto meta_of = [&](const Boxes& x) {
        return make_float4(x.ks * p.c1, x.row >= 0 ? kWeightUp * x.vs : -1.f, fmaxf(log2f(x.vs), (float)kEMin), 0.f);
    };

    // Chunks before the first item's last page: the token kernel leaves them alone, so their codes need not wait for it.
    const int early = kAppend ? 0 : p.append ? max(0, (((w.n - 1) >> p.c.log_p) << p.c.log_p) / kKv8Chunk - c) : INT_MAX;
    Pages f = look_up();
    Boxes x = find(f);
    f = look_up();
    // the first copies, into an empty ring, do not wait for the scales
    const bool hold = kAppend && append;                       // the last chunk waits for the block's own token
    const int ahead = min(x.chunks - (hold && f.chunks == 0 ? 1 : 0), C::NS);
    int k0 = part;
    for (; k0 < min(ahead, early); k0 += C::SETS) copy(x, k0, k0, nullptr);
    if (!kAppend) {
        grid_dependency_wait();            // qhat, the new tokens' codes and scales
        asm volatile("fence.proxy.async.global;" ::: "memory");
        load_scales(x);
    }
    copy_q(x.item);
    x.item = -1;
    for (; k0 < ahead; k0 += C::SETS) copy(x, k0, k0, nullptr);
    float4 meta = meta_of(x);
    while (next < ahead) {
        const int rel = lane - (next << nb_log);
        if ((unsigned)rel < (1u << nb_log)) sh.meta[s * kKv8Tiles + rel] = meta;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(sh.full + s));
        advance();
    }
    bool ok = true;
    while (x.chunks > 0) {
        const bool last = f.chunks == 0;
        const Boxes y = find(f);
        f = look_up();
        if (!copy_q(x.item)) {
            ok = false;
            break;
        }
        while (next < x.chunks) {
            if (hold && last && next == x.chunks - 1) {
                asm volatile("bar.sync 2, %0;" ::"n"(32 * (C::CONSUMERS + 1)) : "memory");
                asm volatile("fence.proxy.async.global;" ::: "memory");
                load_scales(x);
                meta = meta_of(x);
            }
            if (uses > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(sh.empty + s), (uint32_t)(uses - 1) & 1u,
                                                               p.wait_limit_ns, kSiteKv8Empty))) {
                ok = false;
                break;
            }
            copy(x, next, s, &meta);
            advance();
        }
        if (!ok) break;
        next -= x.chunks;
        x = y;
        meta = meta_of(x);
    }
    if (!ok)   // the copies in flight end before the block does: the stages' latest uses
        for (int k = part; k < C::NS; k += C::SETS)
            if (uses > 0 || k < s)
                mbar_wait(smem_u32(sh.full + k), (uint32_t)(k < s ? uses : uses - 1) & 1u, p.wait_limit_ns, kSiteKv8Full);
    if (!ok && !kAppend && part == 0)
        for (int k = 0; k < q_ring; ++k)
            if (q_uses > 0 || k < qs)
                mbar_wait(smem_u32(sh.q_full + k), (uint32_t)(k < qs ? q_uses : q_uses - 1) & 1u, p.wait_limit_ns, kSiteKv8Full);
}

// Where a warp is in the ring: the next chunk of its set, counted from the piece's first, its stage and phase.
struct Kv8Place {
    int next, s;
    uint32_t phase;
    bool ok;
};

// The consumer warps' work on chunks [c_begin, c_end) of w's item; then the warps' sums are
// joined, and emit(h, d4, O, M, L) gets features 4 d4 .. of each head's sum, its reference and weight.
template <int D, int NT, int NRG, class C, class Emit>
__device__ __forceinline__ void kv8_piece(const Kv8AttnParams& p, const Kv8Shared<C>& sh, const Kv8Walk& w, int c_begin,
                                          int c_end, Kv8Place& at_ring, volatile int* turn, int q_log, int warp, int lane,
                                          Emit emit) {
    constexpr int VW = D / 32;
    const int g = lane >> 2, t = lane & 3;
    const int rg = warp % NRG, kslot = warp / NRG;             // set of heads, share of the keys
    const int h_base = rg * C::HEADS;                          // this warp's first head in the group
    uint32_t q[NT];                                            // heads past the group repeat its last one
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const int h = min(h_base + 8 * x + g, p.G - 1);
        q[x] = smem_u32(sh.q + ((*turn & ((1 << q_log) - 1)) * p.G + h) * (D / 8) + t) ^ (uint32_t)((h & 1) * 64);
    }
    float o[NT][2 * VW][4];
    float m[NT][2], l[NT][2];                                  // heads 2 t and 2 t + 1 of each group
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        m[x][0] = m[x][1] = -INFINITY;
        l[x][0] = l[x][1] = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * VW; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][k][e] = 0.f;
    }
    const int tile0 = kslot * C::TPW % kKv8Tiles, box_tiles = min(p.c.log_p, 6) - 4;
    const int n_chunks = c_end - c_begin, first_pos = c_begin * kKv8Chunk + 16 * tile0;
    for (; at_ring.next < n_chunks; at_ring.next += C::SETS) {
        const int s = at_ring.s;
        if (at_ring.ok && !__all_sync(0xffffffffu, mbar_wait(smem_u32(sh.full + s), at_ring.phase, p.wait_limit_ns, kSiteKv8Full)))
            at_ring.ok = false;
        if (!at_ring.ok) break;
#pragma unroll
        for (int k = 0; k < C::TPW; ++k) {
            const int pos0 = first_pos + at_ring.next * kKv8Chunk + 16 * k;
            const float4 meta = sh.meta[s * kKv8Tiles + ((tile0 + k) >> box_tiles)];
            // not wanted: outside the visible keys, or on a page that is not there
            if (pos0 + 16 > w.lo && pos0 < w.n && meta.y >= 0.f)
                kv8_tile<D, NT>(sh.ring + (2 * s) * C::TENSOR + (tile0 + k) * 16 * D, C::TENSOR, pos0, w.lo, w.n, meta, q, o, m,
                                l, g, t);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(sh.empty + s));
        if ((at_ring.s += C::SETS) >= C::NS) {
            at_ring.s -= C::NS;
            at_ring.phase ^= 1u;
        }
    }
    at_ring.next -= n_chunks;
    const int piece = *turn;                                   // pieces before this one
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(sh.q_empty + (piece & ((1 << q_log) - 1))));
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], d);
    // The warps' sums, the heads of one parity at a time (the buffer holds no more).  With at most four heads every warp
    // puts its own down; with more, half of the warps do, and the others add them to theirs and put those down.  One head
    // takes half of the buffer, in turn, so that warps need not wait for those that read the last piece's.
    // A head's features lie in the buffer as [pair][g][2], so that a warp's stores meet no bank twice.
    constexpr int HH = C::HEADS / 2, PITCH = C::MERGE_PITCH;
    const bool direct = NT == 1 && p.G <= 4, one = NT == 1 && p.G == 1;
    const bool upper = !direct && warp >= C::CONSUMERS / 2;
    const int first = one ? (piece & 1) * C::CONSUMERS : 0;
    const int place = first + (upper ? warp - C::CONSUMERS / 2 : warp) * (one ? 1 : direct ? 2 : HH);
    const int reader = one ? ((int)threadIdx.x + 32 * piece) & 255 : (int)threadIdx.x;    // another warp each time
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (e == 1 && p.G == 1) break;
        auto put = [&]() {                 // heads past the group are left out
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                if (h_base + 8 * x + 2 * t + e >= p.G) continue;
                const int at = place + 4 * x + t;
                if (g == 0) {
                    sh.m[at] = m[x][e];
                    sh.l[at] = l[x][e];
                }
#pragma unroll
                for (int k = 0; k < 2 * VW; ++k)
                    *reinterpret_cast<float2*>(sh.o + at * PITCH + 16 * k + 2 * g) = make_float2(o[x][k][e], o[x][k][2 + e]);
            }
        };
        if (!one) kv8_consumers_sync();    // what the buffer held has been read
        if (direct || upper) put();
        kv8_consumers_sync();
        if (!direct) {
            if (!upper) {
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    if (h_base + 8 * x + 2 * t + e >= p.G) continue;
                    const int at = place + 4 * x + t;
                    const float m2 = sh.m[at], l2 = sh.l[at];
                    const float M = fmaxf(m[x][e], m2);
                    const float h1 = kv8_half_factor(m[x][e], l[x][e], M), h2 = kv8_half_factor(m2, l2, M);
                    const float f1 = h1 * h1, f2 = h2 * h2;
#pragma unroll
                    for (int k = 0; k < 2 * VW; ++k) {
                        const float2 o2 = *reinterpret_cast<const float2*>(sh.o + at * PITCH + 16 * k + 2 * g);
                        o[x][k][e] = o[x][k][e] * f1 + o2.x * f2;
                        o[x][k][2 + e] = o[x][k][2 + e] * f1 + o2.y * f2;
                    }
                    m[x][e] = M;
                    l[x][e] = kv8_scale_sum(l[x][e], h1) + kv8_scale_sum(l2, h2);
                }
                __syncwarp();
                put();                     // where it has just read
            }
            kv8_consumers_sync();
        }
        // SLOTS results of each head, STEP places apart
        auto join = [&](auto slots, auto stride) {
            constexpr int SLOTS = decltype(slots)::value, STEP = decltype(stride)::value;
            const int n_heads = (p.G + 1 - e) / 2;              // heads 2 y + e
            for (int x = reader; x < n_heads * (D / 4); x += 256) {
                const int head = x / (D / 4), d4 = x % (D / 4), y = first + head;
                float mk[SLOTS], M = -INFINITY, L = 0.f;
#pragma unroll
                for (int k = 0; k < SLOTS; ++k) {
                    mk[k] = sh.m[y + k * STEP];
                    M = fmaxf(M, mk[k]);
                }
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                const float* src = sh.o + y * PITCH + 16 * (2 * (d4 % VW)) + 2 * (d4 / VW);
#pragma unroll
                for (int k = 0; k < SLOTS; ++k) {
                    const float lk = sh.l[y + k * STEP], h = kv8_half_factor(mk[k], lk, M), f = h * h;
                    const float2 a = *reinterpret_cast<const float2*>(src + k * STEP * PITCH);
                    const float2 b = *reinterpret_cast<const float2*>(src + k * STEP * PITCH + 16);
                    L += kv8_scale_sum(lk, h);
                    O.x = fmaf(a.x, f, O.x);
                    O.y = fmaf(a.y, f, O.y);
                    O.z = fmaf(b.x, f, O.z);
                    O.w = fmaf(b.y, f, O.w);
                }
                emit(2 * head + e, d4, O, M, L);
            }
        };
        if (one) join(std::integral_constant<int, C::CONSUMERS>{}, std::integral_constant<int, 1>{});
        else if (direct) join(std::integral_constant<int, C::CONSUMERS>{}, std::integral_constant<int, 2>{});
        else join(std::integral_constant<int, C::KSLOTS / 2>{}, std::integral_constant<int, NRG * HH>{});
    }
}

// tm_k, tm_v: the caches as {D, n_pages * Hkv * P} bytes.
template <int D, int NT, int NRG>
__global__ void __launch_bounds__(Kv8AttnCfg<D, NT, NRG>::THREADS, Kv8AttnCfg<D, NT, NRG>::BLOCKS_PER_SM)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const Kv8AttnParams p) {
    using C = Kv8AttnCfg<D, NT, NRG>;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    const Kv8Shared<C> sh(dsmem);
    __shared__ int s_warp_sum[C::CONSUMERS + C::SETS];
    __shared__ int s_from[6], s_to, s_last;
    __shared__ volatile int s_walk[C::CONSUMERS][8], s_units[2];

    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31u);
    // this block's units: chunks before each request, summed over a slice of the requests per thread
    Kv8Walk w;
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    const int b_lo = min(p.B, (int)threadIdx.x * per), b_hi = min(p.B, b_lo + per);
    int mine = 0;
    for (w.b = b_lo; w.b < b_hi; ++w.b) {
        w.load(p);
        if (w.nch > 0) mine += w.size();
    }
    if (threadIdx.x == 32 * C::CONSUMERS) {
        sh.init_barriers();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) s_warp_sum[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < C::CONSUMERS + C::SETS; ++i) {
        if (i == warp) incl += total;
        total += s_warp_sum[i];
    }
    const int n_units = total * p.c.Hkv;
    const int n_blocks = min((int)gridDim.x, (n_units + kv8_min_share(p.G) - 1) / kv8_min_share(p.G));
    if ((int)blockIdx.x >= n_blocks) {
        grid_dependency_wait();        // this grid does not end before the token kernel, even where it has no units
        return;
    }
    if (threadIdx.x == 0) {
        s_units[0] = n_units;
        s_units[1] = n_blocks;
    }
    const Kv8Shares shares(n_units, n_blocks);
    // Where this block's stretch begins and ends: a boundary inside a small item, or among the units of an item's
    // cost, moves to that item's end.
    const int r0 = shares.begin(blockIdx.x), r1 = shares.begin(blockIdx.x + 1);
    if (blockIdx.x + 1 == n_blocks && threadIdx.x == 0) s_to = n_units;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int r = side == 0 ? r0 : r1;
        if (r >= incl * p.c.Hkv || r < (incl - mine) * p.c.Hkv) continue;
        int before = incl - mine;
        for (w.b = b_lo;; ++w.b) {
            if (per > 1) w.load(p);
            if (w.nch == 0) continue;
            if (r < (before + w.size()) * p.c.Hkv) break;
            before += w.size();
        }
        const int hk = (r - before * p.c.Hkv) / w.size(), begin = before * p.c.Hkv + hk * w.size();
        const int at = r > begin && (w.nch <= kKv8Whole || r >= begin + w.nch) ? begin + w.size() : r;
        if (side == 0) {
            s_from[0] = w.b;
            s_from[1] = hk;
            s_from[2] = begin;
            s_from[3] = at;
            s_from[4] = w.n;
            s_from[5] = w.lo;
        } else {
            s_to = at;
        }
    }
    __syncthreads();
    const int u0 = s_from[3], u1 = s_to;
    if (u0 >= u1) return;
    w.b = s_from[0];
    w.hk = s_from[1];
    w.begin = s_from[2];
    w.set(s_from[4], s_from[5]);
    if (u0 == w.begin + w.size()) w.next(p);

    if (warp >= C::CONSUMERS) {
        kv8_produce<D, C, false>(tm_k, tm_v, p, sh, w, u0, u1, warp - C::CONSUMERS, lane, false);
        return;
    }
    grid_dependency_wait();
    const int set = warp / NRG / kKv8Tiles % C::SETS;
    Kv8Place at_ring{set, set, 0u, true};
    const int q_log = Kv8Shared<C>::q_ring_log(p.G * D / 8);
    volatile int* at = s_walk[warp];
    int turn = 0;                                          // pieces
    for (int u = u0; u < s_to;) {
        const int end = min(s_to, w.begin + w.nch);    // of its units with keys
        // the walk goes through shared memory over the loop on the keys, which needs every register
        __syncwarp();
        if (lane == 0) {
            at[0] = w.b;
            at[1] = w.hk;
            at[2] = w.begin;
            at[3] = end;
            at[4] = u == w.begin && end == w.begin + w.nch;            // the item is this block's alone
            at[5] = 2 * (int)blockIdx.x + (r0 < w.begin ? 1 : 0);      // else: the piece's place
            at[6] = turn;
        }
        __syncwarp();
        const uint32_t q_bar = smem_u32(sh.q_full + (turn & ((1 << q_log) - 1)));
        if (at_ring.ok &&
            !__all_sync(0xffffffffu, mbar_wait(q_bar, (uint32_t)(turn >> q_log) & 1u, p.wait_limit_ns, kSiteKv8Full)))
            at_ring.ok = false;
        kv8_piece<D, NT, NRG, C>(p, sh, w, w.ch0 + (u - w.begin), w.ch0 + (end - w.begin), at_ring, at + 6, q_log, warp, lane,
                                 [&](int h, int d4, const float4& O, float M, float L) {
                                     if (at[4]) {
                                         kv8_store4<D>(p, at[0], at[1], h, d4, O, M, L);
                                     } else {
                                         float* pt = p.part + ((long long)at[5] * p.G + h) * (D + 4);
                                         *reinterpret_cast<float4*>(pt + 4 * d4) = O;
                                         if (d4 == 0) *reinterpret_cast<float2*>(pt + D) = make_float2(M, L);
                                     }
                                 });
        turn = at[6] + 1;
        w.b = at[0];
        w.hk = at[1];
        w.begin = at[2];
        w.set(w.n, w.lo);
        if (!at[4]) {
            const Kv8Shares shares(s_units[0], s_units[1]);
            const int c_first = shares.owner(w.begin);
            const int pieces = shares.owner(w.begin + w.nch - 1) - c_first + 1;
            kv8_consumers_sync();
            if (threadIdx.x == 0) {        // releases the block's piece (the barrier before it), acquires the others'
                int arrived;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                             : "=r"(arrived)
                             : "l"(p.counters + c_first)
                             : "memory");
                s_last = arrived == pieces - 1;
            }
            kv8_consumers_sync();
            if (s_last) {
                const int first_slot = 2 * c_first + (shares.begin(c_first) < w.begin ? 1 : 0);
                auto part = [&](int k, int h) {
                    return p.part + ((long long)(k == 0 ? first_slot : 2 * (c_first + k)) * p.G + h) * (D + 4);
                };
                // four features to a thread; with few heads, several threads share the pieces, four loads at a time
                float4* s_sum = reinterpret_cast<float4*>(sh.o);
                const int n_out = p.G * (D / 4), share = n_out < 256 ? 256 / n_out : 1;
                for (int x = (int)threadIdx.x; x < n_out * share; x += 256) {
                    const int ox = x % n_out, h = ox / (D / 4), d4 = ox % (D / 4);
                    float M = -INFINITY, L = 0.f;
                    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k0 = x / n_out; k0 < pieces; k0 += 4 * share) {
                        float4 v[4];
                        float2 ml[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int k = k0 + y * share;
                            v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                            ml[y] = make_float2(-INFINITY, 0.f);
                            if (k < pieces) {
                                v[y] = __ldcg(reinterpret_cast<const float4*>(part(k, h)) + d4);
                                ml[y] = __ldcg(reinterpret_cast<const float2*>(part(k, h) + D));
                            }
                        }
                        const float M2 = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
                        const float h0 = kv8_half_factor(M, L, M2), f0 = h0 * h0;
                        L = kv8_scale_sum(L, h0);
                        O.x *= f0;
                        O.y *= f0;
                        O.z *= f0;
                        O.w *= f0;
                        M = M2;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float h = kv8_half_factor(ml[y].x, ml[y].y, M), f = h * h;
                            L += kv8_scale_sum(ml[y].y, h);
                            O.x = fmaf(v[y].x, f, O.x);
                            O.y = fmaf(v[y].y, f, O.y);
                            O.z = fmaf(v[y].z, f, O.z);
                            O.w = fmaf(v[y].w, f, O.w);
                        }
                    }
                    if (share == 1) {
                        kv8_store4<D>(p, w.b, w.hk, h, d4, O, M, L);
                    } else {
                        s_sum[x] = O;
                        if (d4 == 0) {     // of (share, head)
                            sh.m[x / (D / 4)] = M;
                            sh.l[x / (D / 4)] = L;
                        }
                    }
                }
                if (share > 1) {
                    kv8_consumers_sync();
                    if ((int)threadIdx.x < n_out) {
                        const int h = (int)threadIdx.x / (D / 4), d4 = (int)threadIdx.x % (D / 4);
                        float M = -INFINITY, L = 0.f;
                        for (int k = 0; k < share; ++k) M = fmaxf(M, sh.m[k * p.G + h]);
                        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int k = 0; k < share; ++k) {
                            const float lk = sh.l[k * p.G + h], hf = kv8_half_factor(sh.m[k * p.G + h], lk, M), f = hf * hf;
                            const float4 v = s_sum[k * n_out + threadIdx.x];
                            L += kv8_scale_sum(lk, hf);
                            O.x = fmaf(v.x, f, O.x);
                            O.y = fmaf(v.y, f, O.y);
                            O.z = fmaf(v.z, f, O.z);
                            O.w = fmaf(v.w, f, O.w);
                        }
                        kv8_store4<D>(p, w.b, w.hk, h, d4, O, M, L);
                    }
                }
                kv8_consumers_sync();      // before the buffer is written again
            }
        }
        u = at[3] == w.begin + w.nch ? w.begin + w.size() : at[3];
        if (u < s_to) w.next(p);
    }
}

// The step in one launch, for calls with few items: a cluster of blocks per (request, key/value head), each taking an
// equal share of the item's chunks (pages of at most a chunk: the new token's page, whose scale it may change, is then
// in the last chunk alone).  While the first codes load, every block forms qhat of its group's heads itself, and the
// one with the last chunk puts the new token into the cache; the blocks' sums are joined through distributed shared memory.
// Against the two kernels: no dependent launch and nothing in global memory between the blocks (48 items of
// 1000 tokens, D = 128, 15.0 -> 10.7 us; 288 of 2040 30.7 -> 25.2 us, 15.5 at 6565 GB/s), but the split follows each
// item alone, so the GPU is not shared evenly by ragged ones.  Latency-bound where items are short (lengths, table, scales and
// codes follow one another, with the prologue beside them), then by a block's rate of 0.37 us a chunk.
template <int D>
__global__ void __launch_bounds__(Kv8StepCfg<D>::THREADS, 2)
    kv8_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Kv8AttnParams p,
                    const Kv8TokenParams tk) {
    using C = Kv8StepCfg<D>;
    constexpr int TPR = D / 8, HALF = D / 2;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    const Kv8Shared<C> sh(dsmem);
    __shared__ float4 s_tab32[HALF];
    __shared__ double2 s_tab64[HALF];
    __shared__ __align__(16) float s_part[8 * (D + 4)];        // this block's sums: [head][O, then M and L]
    __shared__ volatile int s_turn;                            // the only piece's number
    const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31u);
    const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
    const int item = (int)blockIdx.x / ranks;
    Kv8Walk w;
    w.b = item / p.c.Hkv;
    w.hk = item - w.b * p.c.Hkv;
    w.begin = 0;
    w.load(p);
    if (w.n == 0) {                                            // every block of the cluster alike
        if (rank == 0) {
            if (threadIdx.x == 0 && w.hk == 0 && p.seq_len[w.b] > 0) record_error(kErrIndex, kSiteKvLen);
            kv8_empty_row<D>(p.out, p.lse, (long long)w.b * p.H + w.hk * p.G, p.G);
        }
        return;
    }
    if (threadIdx.x == 0) {
        sh.init_barriers();
        s_turn = 0;
    }
    __syncthreads();
    const int share = (w.nch + ranks - 1) / ranks;
    const int u0 = min(w.nch, rank * share), u1 = min(w.nch, u0 + share);
    const bool append = tk.k != nullptr && u0 < u1 && u1 == w.nch;
    if (warp >= C::CONSUMERS) {
        kv8_produce<D, C, true>(tm_k, tm_v, p, sh, w, u0, u1, warp - C::CONSUMERS, lane, append);
    } else {
        const int row = (int)threadIdx.x / TPR, c = (int)threadIdx.x % TPR;
        Kv8Row<D> r;
        r.load(tk, w.b, w.n - 1, row < p.G ? kQuery : row == p.G && append ? kKeyValue : kNoRow,
               row < p.G ? w.hk * p.G + row : w.hk, c);
        if ((int)threadIdx.x < HALF) kv8_rope_entry<D>(tk.base, w.n - 1, (int)threadIdx.x, s_tab32, s_tab64);
        kv8_consumers_sync();
        uint2 o0, o1;
        r.finish(tk, w.n - 1, c, s_tab32, s_tab64, o0, o1);
        if (append) {
            __threadfence();
            asm volatile("fence.proxy.async.global;" ::: "memory");
            asm volatile("bar.arrive 2, %0;" ::"n"(32 * (C::CONSUMERS + 1)) : "memory");
        }
        if (row < p.G) {
            uint2* q = reinterpret_cast<uint2*>(sh.q);
            q[kv8_q_place<D>(row, 4 * c)] = bf16x4_to_half4(o0);
            q[kv8_q_place<D>(row, HALF + 4 * c)] = bf16x4_to_half4(o1);
        }
        kv8_consumers_sync();
        const int set = warp / kKv8Tiles % C::SETS;
        Kv8Place at_ring{set, set, 0u, true};
        kv8_piece<D, 1, 1, C>(p, sh, w, w.ch0 + u0, w.ch0 + u1, at_ring, &s_turn, 0, warp, lane,
                              [&](int h, int d4, const float4& O, float M, float L) {
                                  if (ranks == 1) {
                                      kv8_store4<D>(p, w.b, w.hk, h, d4, O, M, L);
                                  } else {
                                      float* pt = s_part + h * (D + 4);
                                      *reinterpret_cast<float4*>(pt + 4 * d4) = O;
                                      if (d4 == 0) *reinterpret_cast<float2*>(pt + D) = make_float2(M, L);
                                  }
                              });
    }
    if (ranks == 1) return;
    __syncwarp();
    cluster_sync_all();
    // the outputs, dealt over the blocks
    const int n_out = p.G * (D / 4);
    for (int x = rank * C::THREADS + (int)threadIdx.x; x < n_out; x += ranks * C::THREADS) {
        const int h = x / (D / 4), d4 = x % (D / 4);
        const float* pt = s_part + h * (D + 4);
        float mk[kDecodeMaxCluster], lk[kDecodeMaxCluster];
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kDecodeMaxCluster; ++k) {
            if (k >= ranks) break;
            mk[k] = ld_shared_cluster_f32(pt + D, k);
            lk[k] = ld_shared_cluster_f32(pt + D + 1, k);
            M = fmaxf(M, mk[k]);
        }
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kDecodeMaxCluster; ++k) {
            if (k >= ranks) break;
            const float hf = kv8_half_factor(mk[k], lk[k], M), f = hf * hf;
            L += kv8_scale_sum(lk[k], hf);
            O.x = fmaf(ld_shared_cluster_f32(pt + 4 * d4, k), f, O.x);
            O.y = fmaf(ld_shared_cluster_f32(pt + 4 * d4 + 1, k), f, O.y);
            O.z = fmaf(ld_shared_cluster_f32(pt + 4 * d4 + 2, k), f, O.z);
            O.w = fmaf(ld_shared_cluster_f32(pt + 4 * d4 + 3, k), f, O.w);
        }
        kv8_store4<D>(p, w.b, w.hk, h, d4, O, M, L);
    }
    // the blocks keep their shared memory until all have read it
    cluster_sync_all();
}

}  // namespace swa
