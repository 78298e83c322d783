/*
 * swa_attn.h -- C ABI of the B200 (sm_100a) causal sliding-window attention forward.
 *
 * The layer (one call = one attention layer of the nanochat / modded-NanoGPT speedrun model):
 *
 *   qhat = rms(rope(q)),  khat = rms(rope(k))
 *        intelliparadigm "GPT-2 for $73", section 2.2 (q, k = norm(rope(q)), norm(rope(k)));
 *        section 2.1 (parameter-free RMSNorm); kongchang speedrun explainer, "RoPE" paragraph.
 *        rope: pairs (i, i + D/2), theta_i = rope_base^(-2i/D), position t = 0..T-1 rotates
 *        (a, b) -> (a cos(t theta_i) - b sin(t theta_i), a sin(t theta_i) + b cos(t theta_i)).
 *        rms:  x / sqrt(mean_D(x^2) + eps), no learned scale.
 *   v'   = v + 2 sigmoid(gate_x[b,t,:] . Wg[:, h]) * ve        (value-embedding layers only)
 *        PaperWeekly repost of the nanochat write-up, "Value Embeddings" paragraph.
 *   out  = softmax(qhat khat^T / sqrt(D) + mask) v'
 *        "Let's reproduce GPT-2 (124M)" notes, section 3 (scores, lower-triangular mask that
 *        includes the diagonal, softmax over keys, weighted sum of values).
 *        mask: key j is visible to query i iff 0 <= i - j < W, W = window (intelliparadigm
 *        section 3.2: local windows of 1024 tokens, a full window of 2048 every fourth layer);
 *        window <= 0 or window >= T means full causal.
 *   lse  = ln sum_j exp(qhat_i . khat_j / sqrt(D)) over the visible keys (natural log).
 *
 * Layouts (all row-major, contiguous, no strides):
 *   q, k, v, ve, out : bf16 (B, T, H, D)        -- the native layout (intelliparadigm 3.1)
 *   gate_x           : bf16 (B, T, 32)          -- x[..., :32].contiguous()
 *   Wg               : bf16 [32, H]             -- one gate per head, no bias
 *   lse              : fp32 (B, H, T)
 *
 * Ownership: every pointer is a DEVICE pointer owned by the caller, except where stated.
 * The library never frees a caller pointer and never writes q, k, v, ve, gate_x or Wg.
 *
 * Streams: calls are asynchronous on `stream` (NULL = the legacy default stream) and never
 * synchronise the host, except swa_attn_last_device_status().
 *
 * Threads: calls may come from several host threads at once.  The per-device setup of the first
 * call, the library-owned workspace and the backward's side stream are guarded by locks, and a
 * call that reuses the library workspace on another stream first waits, on the device, for the
 * previous call that used it.  Caller-owned workspaces are the caller's to keep apart.
 *
 * Precision: every qhat, khat and v' element the prologue writes is the correctly rounded bf16
 * (nearest, ties to even) of its exact value, so the tensor-core operands do not depend on how the
 * arithmetic is organised.
 *
 * Errors: a negative swa_status.  Arguments are validated before anything is enqueued; a
 * rejected call has no effect.  Waits inside the kernels are bounded: if one expires, the
 * kernel records SWA_ERR_TIMEOUT in a per-device status word and exits cleanly; read it with
 * swa_attn_last_device_status().
 */
#ifndef SWA_ATTN_H_
#define SWA_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SWA_API __attribute__((visibility("default")))
#else
#define SWA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st* swa_stream_t;

typedef enum swa_status {
    SWA_OK = 0,
    SWA_ERR_INVALID_ARG = -1,  /* null pointer, size < 1, bad eps / rope_base, ve/gate_x/Wg partly set, or
                                  (read via last_device_status) a slot, page or length outside a paged cache */
    SWA_ERR_UNSUPPORTED = -2,  /* D not in {64, 128}, sizes beyond int32 indexing, device not sm_100 */
    SWA_ERR_MISALIGNED = -3,   /* a tensor pointer or the workspace is not 16-byte aligned */
    SWA_ERR_CUDA = -4,         /* a CUDA runtime / driver call failed (launch, allocation by CUDA),
                                  or a kernel found its shared memory misaligned and did nothing */
    SWA_ERR_TIMEOUT = -5,      /* a bounded wait inside a kernel expired (read via last_device_status) */
    SWA_ERR_NO_MEMORY = -6,    /* workspace too small (swa_attn_fwd_ws) or allocation failed */
    SWA_ERR_NO_DEVICE = -7     /* no CUDA device is visible */
} swa_status;

/*
 * Full layer forward.  Steps: RoPE + RMS norm of q and k, gate + add of the value embedding,
 * windowed causal attention, bf16 out and fp32 lse.
 *
 * q, k, v      bf16 (B,T,H,D), read only.
 * ve, gate_x, Wg  value-embedding inputs; all three NULL for a layer without value embeddings,
 *              otherwise all three set (else SWA_ERR_INVALID_ARG).
 * out          bf16 (B,T,H,D), written.
 * lse          fp32 (B,H,T), written; NULL skips it.
 * B, T, H      >= 1;  D in {64, 128};  B*T*H*D < 2^31;  B, H <= 65535 (else SWA_ERR_UNSUPPORTED).
 * window       keys visible to a query, counting itself; <= 0 or >= T is full causal.
 * rope_base    > 0 and finite (10000 in the pages' models).
 * eps          >= 0 and finite (1e-6 here).  At eps = 0 an all-zero q or k head row has no
 *              normalised value (0/0 in the definition): such inputs are outside the domain and
 *              their results are unspecified.
 * stream       CUDA stream (NULL = legacy default stream).
 *
 * Scratch: the library keeps one workspace per device (qhat, khat, v', the gates, the RoPE table),
 * grown on demand with stream-ordered allocation on `stream` and kept until the library is
 * unloaded.  Each call records an event after its kernels; a call on another stream first makes
 * its stream wait for that event, so calls on different streams that share the workspace run one
 * after the other on the GPU (callers that want them to overlap use swa_attn_fwd_ws() with
 * separate workspaces).  Launches: the gate kernel (value-embedding layers), the prologue kernel
 * and the attention kernel, plus the RoPE table when T, D or rope_base changes.
 */
SWA_API int swa_attn_fwd(const void* q, const void* k, const void* v,
                 const void* ve, const void* gate_x, const void* Wg,
                 void* out, float* lse,
                 int B, int T, int H, int D, int window,
                 float rope_base, float eps, swa_stream_t stream);

/*
 * Grouped-query attention (the pages size the key/value projection separately, as kv_dim:
 * intelliparadigm "GPT-2 for $73", model section): as swa_attn_fwd, with q (B,T,H,D) and k, v, ve
 * (B,T,Hkv,D), gate_x
 * (B,T,32), Wg [32,Hkv]; Hkv divides H and query head h attends with key/value head h / (H/Hkv).
 * The prologue runs on the Hkv key/value heads once (not per query head).  Hkv == H is exactly
 * swa_attn_fwd.  Errors as swa_attn_fwd; SWA_ERR_INVALID_ARG if Hkv does not divide H.
 */
SWA_API int swa_attn_fwd_gqa(const void* q, const void* k, const void* v,
                             const void* ve, const void* gate_x, const void* Wg,
                             void* out, float* lse,
                             int B, int T, int H, int Hkv, int D, int window,
                             float rope_base, float eps, swa_stream_t stream);

/*
 * Document-boundary mask (packed documents; the pages list variable-length attention among the
 * changes that were tried: intelliparadigm "GPT-2 for $73", section 7).  As swa_attn_fwd_gqa, plus
 * doc: int32 (B, T) device array of document ids.  A document is a maximal run of equal ids along
 * a sequence (number packed documents in order: ids that never repeat across runs); key j is
 * visible to query i iff 0 <= i - j < window and j is in i's document.  RoPE positions stay the
 * sequence positions 0..T-1.  Key tiles before the first query row's document start are skipped.
 * Uses the library-owned workspace (plus B*T int32 document starts), with its stream ordering.
 * Errors as swa_attn_fwd_gqa; SWA_ERR_INVALID_ARG if doc is NULL, SWA_ERR_MISALIGNED if it is
 * not 4-byte aligned.
 */
SWA_API int swa_attn_fwd_doc(const void* q, const void* k, const void* v,
                             const void* ve, const void* gate_x, const void* Wg, const int* doc,
                             void* out, float* lse,
                             int B, int T, int H, int Hkv, int D, int window,
                             float rope_base, float eps, swa_stream_t stream);

/* Bytes of caller workspace swa_attn_fwd_ws() needs for these sizes (0 on invalid sizes). */
SWA_API size_t swa_attn_workspace_bytes(int B, int T, int H, int D, int has_ve);

/*
 * Byte offset of one section of the workspace, for callers that read the prologue's results
 * (e.g. to keep them for a backward pass) after swa_attn_prologue():
 *   SWA_WS_QHAT, SWA_WS_KHAT   bf16 (B,T,H,D): rms(rope(q)), rms(rope(k)), each element the
 *                              correctly rounded bf16 (nearest, ties to even) of its exact value;
 *   SWA_WS_VPRIME              bf16 (B,T,H,D): v + 2 sigmoid(gate_x . Wg) ve, same rounding
 *                              (value-embedding layers only);
 *   SWA_WS_ROPE_TABLE          the RoPE table (internal format).
 * Returns (size_t)-1 for invalid sizes or a section that does not exist.
 */
enum swa_ws_section { SWA_WS_QHAT = 0, SWA_WS_KHAT = 1, SWA_WS_VPRIME = 2, SWA_WS_ROPE_TABLE = 3 };
SWA_API size_t swa_attn_workspace_offset(int B, int T, int H, int D, int has_ve, int section);

/*
 * Same as swa_attn_fwd() with caller-owned device scratch: `workspace` (16-byte aligned,
 * at least swa_attn_workspace_bytes() bytes) holds qhat, khat, v', the gates and the RoPE table, which
 * is rebuilt on every call (one small extra kernel).  It runs swa_attn_rope_table(),
 * swa_attn_prologue() and swa_attn_attention().  Nothing is allocated.
 * SWA_ERR_NO_MEMORY if ws_bytes is too small.
 */
SWA_API int swa_attn_fwd_ws(const void* q, const void* k, const void* v,
                    const void* ve, const void* gate_x, const void* Wg,
                    void* out, float* lse,
                    int B, int T, int H, int D, int window,
                    float rope_base, float eps,
                    void* workspace, size_t ws_bytes, swa_stream_t stream);

/*
 * The steps of swa_attn_fwd_ws(), exposed for per-stage timing and tests.
 *
 * swa_attn_rope_table: fill the workspace's RoPE table, cos/sin(t * rope_base^(-2i/D)) for
 *   t < T, i < D/2, evaluated in fp64 and stored as fp32.  It depends only on T, D and
 *   rope_base, so a caller that keeps one workspace for many calls of the same T, D and base
 *   builds it once (swa_attn_fwd does that with its own workspace).
 * swa_attn_prologue: RoPE + RMS norm of q and k, gate + add of the value embedding, into the
 *   workspace (same sizes and rules as swa_attn_fwd_ws).  Uses the table already in the
 *   workspace; it does not rebuild it.  It also resets the scheduler counters the attention kernel
 *   takes its work from.
 * swa_attn_attention: the windowed attention on a workspace that swa_attn_prologue() filled
 *   for the same B, T, H, D and value-embedding setting (`v` is read directly when has_ve == 0).
 * All of them: asynchronous on `stream`, validation before any launch, errors as swa_attn_fwd_ws.
 */
SWA_API int swa_attn_rope_table(int B, int T, int H, int D, int has_ve, float rope_base,
                                void* workspace, size_t ws_bytes, swa_stream_t stream);

SWA_API int swa_attn_prologue(const void* q, const void* k, const void* v,
                      const void* ve, const void* gate_x, const void* Wg,
                      int B, int T, int H, int D, float rope_base, float eps,
                      void* workspace, size_t ws_bytes, swa_stream_t stream);

SWA_API int swa_attn_attention(const void* v, int has_ve, void* out, float* lse,
                       int B, int T, int H, int D, int window,
                       void* workspace, size_t ws_bytes, swa_stream_t stream);


/*
 * swa_attn_fwd_noalloc: swa_attn_fwd() for callers that cannot allocate device memory on the
 * call path -- a plugin whose host framework owns all device memory and forbids allocation
 * inside its execute call, or a latency-critical loop where an allocation (which may
 * synchronise the device) is not allowed.  The pages have no counterpart of this entry point.
 *
 * The caller passes inputs and outputs exactly as for swa_attn_fwd(), and the call computes the
 * same result with the same kernels; the scratch (qhat, khat, v', the gates and the RoPE table) lives in
 * a fixed device array compiled into the library, swa_attn_noalloc_scratch_bytes() bytes (64 MiB).
 * Nothing is allocated or freed by the call itself.
 *   - CUDA loads the library's device code, and with it the array, on a device when the library
 *     is first used there (lazy module loading): from then on that device holds the 64 MiB until
 *     the process exits, and that first use may itself allocate.  The first call of
 *     swa_attn_fwd_noalloc() on a device also looks up the array's device address (a runtime query,
 *     once per device, with that device current).  Callers that must not allocate make one warm-up
 *     call on each device outside their no-allocation region and before any stream capture.
 *   - Sizes whose workspace (swa_attn_workspace_bytes()) exceeds that array are rejected with
 *     SWA_ERR_NO_MEMORY before anything is enqueued.
 *   - All calls on a device share the one array and it keeps the last call's contents; every
 *     byte a call reads is written earlier in that call.  Calls that overlap on the GPU (other
 *     streams, other host threads) race on it: serialise them.
 */
SWA_API int swa_attn_fwd_noalloc(const void* q, const void* k, const void* v,
                                 const void* ve, const void* gate_x, const void* Wg,
                                 void* out, float* lse,
                                 int B, int T, int H, int D, int window,
                                 float rope_base, float eps, swa_stream_t stream);

/* Size in bytes of the fixed scratch array behind swa_attn_fwd_noalloc(). */
SWA_API size_t swa_attn_noalloc_scratch_bytes(void);

/* Static description of a status code (never NULL). */
SWA_API const char* swa_attn_strerror(int status);

/*
 * Synchronises `stream`, then returns and clears the current device's status word:
 * SWA_OK, SWA_ERR_TIMEOUT (a bounded wait expired in some kernel since the last read),
 * SWA_ERR_INVALID_ARG (a kernel of the paged cache met a slot, page or length outside it and skipped
 * it) or SWA_ERR_CUDA (the stream reported an error).  If `detail` is not NULL it receives the raw
 * word (bits 0-7 kind, 8-15 wait site, 16-31 block index).
 */
SWA_API int swa_attn_last_device_status(swa_stream_t stream, unsigned int* detail);

/*
 * One generation step with a key/value cache (the pages list a KV cache among the missing
 * pieces: "Let's reproduce GPT-2 (124M)" notes, section 19).  For the new token of every
 * sequence, at position `pos` (the same for all b):
 *   1. the prologue of swa_attn_fwd at position pos: qhat = RMS(RoPE(q, pos)),
 *      khat = RMS(RoPE(k, pos)), v' = v + 2 sigmoid(gate_x . Wg[:, h]) ve (value-embedding
 *      layers) or v; khat and v' are written to k_cache[b, pos, h, :] and v_cache[b, pos, h, :],
 *      bit-identical to what the prefill path computes for that token;
 *   2. attention of qhat over the cached keys j in [max(0, pos - W + 1), pos] (W = Tmax if
 *      window <= 0 or window >= Tmax): out[b,h,:] = sum_j softmax_j(qhat . khat_j / sqrt(D)) v'_j,
 *      lse[b,h] = ln sum_j exp(qhat . khat_j / sqrt(D)).
 * Arguments:
 *   q, k, v      bf16 (B, H, D): the new token's raw projections.
 *   ve, gate_x, Wg  bf16 (B, H, D) / (B, 32) / (32, H), all set (value-embedding layer) or all NULL.
 *   k_cache, v_cache  bf16 (B, Tmax, H, D), caller-owned: entries j < pos (inside the window) must
 *                hold khat / v' of earlier positions (as written by earlier calls or by the prefill
 *                path); entry pos is written.
 *   out          bf16 (B, H, D), written.   lse  fp32 (B, H) or NULL.
 *   workspace    device memory of at least swa_attn_decode_workspace_bytes(B, Tmax, H, D, has_ve,
 *                window) bytes, 16-byte aligned, caller-owned and not retained.
 * Scores, exponentials and weighted sums are fp32 (no bf16 rounding of the weights).  The call is
 * asynchronous on `stream` (two kernels: the token's key/value prologue, then one cluster of CTAs
 * per row for the attention, which also forms qhat); arguments are validated before anything is
 * enqueued.  Errors: SWA_ERR_INVALID_ARG (null pointer, pos outside [0, Tmax), bad rope_base /
 * eps, partial value-embedding set), SWA_ERR_UNSUPPORTED (D not 64/128, sizes beyond int32),
 * SWA_ERR_MISALIGNED, SWA_ERR_NO_MEMORY (workspace too small), SWA_ERR_CUDA.
 */
SWA_API size_t swa_attn_decode_workspace_bytes(int B, int Tmax, int H, int D, int has_ve, int window);
SWA_API int swa_attn_decode(const void* q, const void* k, const void* v, const void* ve,
                            const void* gate_x, const void* Wg, void* k_cache, void* v_cache,
                            int pos, void* out, float* lse, int B, int Tmax, int H, int D,
                            int window, float rope_base, float eps, void* workspace,
                            size_t ws_bytes, swa_stream_t stream);
/* Grouped-query decode step: as swa_attn_decode with q (B, H, D) and k, v, ve (B, Hkv, D),
 * gate_x (B, 32), Wg (32, Hkv), caches (B, Tmax, Hkv, D); Hkv divides H and query head h attends
 * with key/value head h / (H / Hkv).  The workspace size is that of swa_attn_decode for (B, Tmax,
 * H, D).  SWA_ERR_INVALID_ARG if Hkv does not divide H. */
SWA_API int swa_attn_decode_gqa(const void* q, const void* k, const void* v, const void* ve,
                                const void* gate_x, const void* Wg, void* k_cache, void* v_cache,
                                int pos, void* out, float* lse, int B, int Tmax, int H, int Hkv,
                                int D, int window, float rope_base, float eps, void* workspace,
                                size_t ws_bytes, swa_stream_t stream);

/*
 * One generation step of the document-masked layer: as swa_attn_decode_gqa, plus doc_start, an
 * int32 (B,) device array with the first position of each sequence's current document (the
 * document the new token at `pos` belongs to; values above pos are read as pos).  The new token
 * attends to the cached keys [max(pos - W + 1, doc_start[b]), pos] (the document-boundary mask of
 * swa_attn_fwd_doc, row pos).  doc_start = NULL is swa_attn_decode_gqa.  SWA_ERR_MISALIGNED if
 * doc_start is not 4-byte aligned.
 */
SWA_API int swa_attn_decode_doc(const void* q, const void* k, const void* v,
                                const void* ve, const void* gate_x, const void* Wg,
                                void* k_cache, void* v_cache, int pos, const int* doc_start,
                                void* out, float* lse,
                                int B, int Tmax, int H, int Hkv, int D, int window,
                                float rope_base, float eps,
                                void* workspace, size_t ws_bytes, swa_stream_t stream);

/*
 * The layer from its input x: the bias-free q, k, v projection fused with the prologue, then the
 * attention of swa_attn_fwd_gqa.  The pages form q, k, v of each layer as linear maps of the
 * layer input ("Let's reproduce GPT-2 (124M)" notes, section 3, the attention listing;
 * intelliparadigm "GPT-2 for $73", section 2: separate bias-free maps, key/value width kv_dim):
 *   y = x Wqkv^T (fp32 tensor-core accumulation, never rounded or stored), then
 *   qhat = RMS(RoPE(y_q)), khat = RMS(RoPE(y_k)), v' = y_v + 2 sigmoid(x[..., :32] . Wg[:, h]) ve.
 * Arguments (device pointers, caller-owned):
 *   x        bf16 (B, T, C) contiguous, C a multiple of 8 (at least 32 with the value embedding).
 *   Wqkv     bf16 [(H + 2 Hkv) D, C], the linear layer's layout: rows 0 .. H D - 1 give q (head h at
 *            rows h D ..), then Hkv D rows of k, then Hkv D rows of v.
 *   ve, Wg   bf16 (B, T, Hkv, D) gathered value-embedding rows and [32, Hkv], both set or both NULL.
 * swa_attn_qkv_prologue writes qh bf16 (B, T, H, D), kh and vp bf16 (B, T, Hkv, D) (caller buffers);
 * swa_attn_fwd_x writes out bf16 (B, T, H, D) and lse fp32 (B, H, T) (NULL = skip) with qhat, khat,
 * v' kept in the workspace.  workspace: at least swa_attn_fwd_x_workspace_bytes(B, T, H, Hkv, D)
 * bytes, 16-byte aligned, nothing kept between calls.  Both calls leave the workspace's RoPE table
 * in their own form (fp32 cos and sin, no fp64 copy): on a workspace they used, call
 * swa_attn_rope_table() again before swa_attn_prologue().  Asynchronous on `stream`; arguments are
 * validated before anything is enqueued.  Errors: SWA_ERR_INVALID_ARG (null pointer, ve / Wg not
 * both set, C < 32 with the value embedding, Hkv not dividing H, bad rope_base / eps),
 * SWA_ERR_UNSUPPORTED (D not 64 / 128, C not a multiple of 8, B T H D or B T C at least 2^31),
 * SWA_ERR_MISALIGNED, SWA_ERR_NO_MEMORY, SWA_ERR_CUDA.
 */
SWA_API size_t swa_attn_fwd_x_workspace_bytes(int B, int T, int H, int Hkv, int D);
SWA_API int swa_attn_qkv_prologue(const void* x, const void* Wqkv, const void* ve, const void* Wg,
                                  void* qh, void* kh, void* vp, int B, int T, int C, int H, int Hkv,
                                  int D, float rope_base, float eps, void* workspace, size_t ws_bytes,
                                  swa_stream_t stream);
SWA_API int swa_attn_fwd_x(const void* x, const void* Wqkv, const void* ve, const void* Wg, void* out,
                           float* lse, int B, int T, int C, int H, int Hkv, int D, int window,
                           float rope_base, float eps, void* workspace, size_t ws_bytes,
                           swa_stream_t stream);

/*
 * Backward of the layer: the gradient of loss = sum(dout * out) + sum(dlse * lse) for the layer of
 * swa_attn_fwd / swa_attn_fwd_gqa (the pages train it end to end; the log-sum-exp the forward
 * writes lets the backward rebuild the softmax: "Let's reproduce GPT-2 (124M)" notes, the
 * attention-kernel discussion in section 19).  Per visible pair (i, j) with P_ij = exp(s_ij - lse_i):
 *   dP_ij = dout_i . v'_j,  delta_i = dout_i . out_i,  dS_ij = P_ij (dP_ij - delta_i + dlse_i),
 *   dqhat_i = sum_j dS_ij khat_j / sqrt(D),  dkhat_j = sum_i dS_ij qhat_i / sqrt(D),
 *   dv'_j = sum_i P_ij dout_i  (summed over the query heads of a key/value head's group),
 * then the prologue in reverse: dq = RoPE^T(r dqhat - (r^3/D)(x . dqhat) x) per row (likewise dk),
 * dv = dv', dve = g dv', dz = (dv' . ve) 2 sigmoid(z)(1 - sigmoid(z)), dgate_x = dz Wg^T,
 * dWg = gate_x^T dz.
 * Arguments (device pointers, caller-owned, all read-only except the gradients and workspace):
 *   q, k, v, ve, gate_x, Wg   the forward's inputs, shapes as swa_attn_fwd_gqa.
 *   out, lse                  the forward's outputs for these inputs: bf16 (B,T,H,D), fp32 (B,H,T).
 *   dout                      bf16 (B,T,H,D).   dlse  fp32 (B,H,T), or NULL for zero.
 *   dq                        bf16 (B,T,H,D), written.   dk, dv  bf16 (B,T,Hkv,D), written.
 *   dve                       bf16 (B,T,Hkv,D): gradient of the looked-up value-embedding rows.
 *   dgate_x                   fp32 (B,T,32).   dWg  fp32 (32,Hkv).
 *                             These three are set on value-embedding layers and NULL otherwise.
 *   workspace                 at least swa_attn_bwd_workspace_bytes(B,T,H,Hkv,D,has_ve) bytes,
 *                             16-byte aligned; nothing in it is kept between calls.
 * qhat, khat and v' are recomputed by the forward's prologue (bit-identical to the forward's);
 * P and dS enter the tensor-core products as bf16 (round to nearest), accumulation is fp32.
 * Asynchronous on `stream` (about ten kernels); arguments are validated before anything is
 * enqueued.  Errors: SWA_ERR_INVALID_ARG (null pointer, value-embedding gradients not matching the
 * inputs, Hkv not dividing H, bad rope_base / eps), SWA_ERR_UNSUPPORTED, SWA_ERR_MISALIGNED,
 * SWA_ERR_NO_MEMORY (workspace too small), SWA_ERR_CUDA; bounded-wait timeouts inside the kernels
 * are reported by swa_attn_last_device_status().
 */
SWA_API size_t swa_attn_bwd_workspace_bytes(int B, int T, int H, int Hkv, int D, int has_ve);
SWA_API int swa_attn_bwd_gqa(const void* q, const void* k, const void* v, const void* ve,
                             const void* gate_x, const void* Wg, const void* out, const float* lse,
                             const void* dout, const float* dlse, void* dq, void* dk, void* dv,
                             void* dve, float* dgate_x, float* dWg, int B, int T, int H, int Hkv,
                             int D, int window, float rope_base, float eps, void* workspace,
                             size_t ws_bytes, swa_stream_t stream);

/*
 * The backward of the document-masked layer (swa_attn_fwd_doc): as swa_attn_bwd_gqa, plus doc, the
 * same int32 (B, T) document ids the forward took (documents are maximal runs of equal ids).  The
 * query-tile kernel skips key tiles before the tile's first document start and masks keys before
 * each row's document start; the key-tile kernel skips query tiles past the tile's last document end
 * and masks queries past each key's document end.  Workspace: swa_attn_bwd_workspace_bytes() (it
 * reserves the document starts and ends).  doc = NULL is swa_attn_bwd_gqa.  SWA_ERR_MISALIGNED if
 * doc is not 4-byte aligned.
 */
SWA_API int swa_attn_bwd_doc(const void* q, const void* k, const void* v, const void* ve, const void* gate_x,
                             const void* Wg, const int* doc, const void* out, const float* lse,
                             const void* dout, const float* dlse, void* dq, void* dk, void* dv, void* dve,
                             float* dgate_x, float* dWg, int B, int T, int H, int Hkv, int D, int window,
                             float rope_base, float eps, void* workspace, size_t ws_bytes,
                             swa_stream_t stream);
/*
 * swa_attn_bwd_saved: the multi-head backward (as swa_attn_bwd) for a caller that keeps the
 * forward's activations.  Use it when `workspace` (swa_attn_bwd_workspace_bytes() bytes, which
 * covers swa_attn_workspace_bytes()) was passed to the swa_attn_fwd_ws() call that produced `out`
 * and `lse`, with the same q, k, v, ve, gate_x, Wg, sizes, rope_base and eps, and nothing has
 * written to it since.  That call left qhat, khat, v', the gates and the RoPE tables at the
 * offsets this backward reads, so the prologue is not recomputed.  The gradients are bit-identical
 * to swa_attn_bwd's.  The call cannot check that the workspace holds this layer's forward state:
 * any other content gives wrong gradients (every access stays inside the workspace).
 */
SWA_API int swa_attn_bwd_saved(const void* q, const void* k, const void* v, const void* ve,
                               const void* gate_x, const void* Wg, const void* out, const float* lse,
                               const void* dout, const float* dlse, void* dq, void* dk, void* dv,
                               void* dve, float* dgate_x, float* dWg, int B, int T, int H, int D,
                               int window, float rope_base, float eps, void* workspace, size_t ws_bytes,
                               swa_stream_t stream);

/* The multi-head layer: swa_attn_bwd_gqa with Hkv = H. */
SWA_API int swa_attn_bwd(const void* q, const void* k, const void* v, const void* ve,
                         const void* gate_x, const void* Wg, const void* out, const float* lse,
                         const void* dout, const float* dlse, void* dq, void* dk, void* dv, void* dve,
                         float* dgate_x, float* dWg, int B, int T, int H, int D, int window,
                         float rope_base, float eps, void* workspace, size_t ws_bytes,
                         swa_stream_t stream);

/*
 * A paged key/value cache in 8 bits, for decoding requests of different lengths (the pages list a KV
 * cache among the missing pieces: "Let's reproduce GPT-2 (124M)" notes, section 19).
 *
 * The cache.  P = page_size tokens of every key/value head make a page, P in {16, 32, 64, 128}:
 *   k_cache, v_cache  e4m3 (n_pages, Hkv, P, D): khat and v' as codes; a value is code * scale.
 *   k_scale, v_scale  fp32 (n_pages, Hkv): one scale for each page and head, a power of two 2^e, e the
 *                     smallest integer >= -60 with max |value| <= 448 * 2^e over the page's tokens.
 * Caller-owned, 16-byte (scales: 4-byte) aligned; n_pages * Hkv * P < 2^31.  Slot s of a cache is token
 * s % P of page s / P.  Nothing has to be initialised: a page's scale starts anew with its token 0.
 * While a page fills, its scale grows where a new token needs it, and the codes already there are moved
 * to the new scale: exactly, but for values below 2^-13 of the page's largest, which are rounded again (each time by
 * half of 2^-9 of the scale at most: in all less than 2^-8 of the last one).
 * Caching rounds a value to 4 significant bits (half a step is 2^-4 of it, or 2^-10 of the scale).
 * An infinity becomes the largest code at the largest scale, 2^120; a NaN stays a NaN and does not
 * count towards the scale.
 *
 * Requests.  Row b of block_table, int32 (B, max_pages), lists request b's pages in token order: token
 * at position x is in page block_table[b, x / P].  Entries of pages not held are -1.
 *
 * swa_attn_kv_pages: one step of the page allocator, on the GPU, from the requests' lengths.
 *   kv_len      int32 (B): tokens each request has in the cache.
 *   first_page  int32 (B): its pages before this one were given back (0 for a new request).
 *   n_new       int32 (B): tokens that join it in this step, 0 .. T; 0 leaves it idle; negative: it has
 *               ended, gives back all its pages and is empty afterwards.
 *   pool        int32 (2): {head, free}; ring  int32 (n_pages): the free pages are
 *               ring[(head + i) % n_pages], i < free.  A new cache has ring = 0 .. n_pages - 1, pool = {0, n_pages}.
 * With L = kv_len[b], n = n_new[b]:
 *   window > 0: pages that no later query of that window can see, entries before
 *     max(0, L - window + 1) / P, go back to the ring (a cache for several layers: the largest window;
 *     window <= 0: all pages are kept);
 *   need_b = ceil((L + n) / P) - ceil(L / P) pages are taken.  Request b is served iff n >= 1 and either
 *     need_b = 0 or the sum of need over requests 0 .. b is at most `free`: requests are served in order, one that
 *     finds no page holds back those after it that need one, and pages given back in a step are free from the
 *     next step on.  A request that cannot be served at all (n > T, more than max_pages pages) takes nothing and
 *     holds nobody back; like an idle one it gives back the pages that its window has passed.  One whose kv_len or
 *     first_page is not possible (kv_len outside 0 .. max_pages * page_size, first_page outside 0 .. its number of
 *     pages) is left as it was.
 * Results (each may be the array it follows from, for a step in place; other overlaps are not allowed):
 *   block_table_out, kv_len_out, first_page_out, pool_out   the state after the step (ring is always updated in
 *               place: only entries outside the free stretch change, so a step can be repeated from
 *               the same inputs);
 *   slots       int32 (B, T): slots[b, t] is the slot of request b's t-th new token, -1 for t >= n_new[b] and
 *               for requests that were not served;
 *   step_len    int32 (B): kv_len_out[b] where tokens joined, else 0: the seq_len of swa_attn_kv8_decode.
 *               A request that asked for tokens and has step_len 0 was not served.
 * Errors: SWA_ERR_INVALID_ARG (null pointer, size < 1), SWA_ERR_UNSUPPORTED (page_size, n_pages * page_size,
 * max_pages * page_size, B * T or B * max_pages at least 2^31), SWA_ERR_MISALIGNED (4 bytes), SWA_ERR_CUDA.
 */
SWA_API int swa_attn_kv_pages(const int* block_table, const int* kv_len, const int* first_page, const int* pool,
                              const int* n_new, int* ring, int* block_table_out, int* kv_len_out,
                              int* first_page_out, int* pool_out, int* slots, int* step_len, int B, int T,
                              int max_pages, int n_pages, int page_size, int window, swa_stream_t stream);

/*
 * swa_attn_kv8_write: rows kh, vp bf16 (B, T, Hkv, D) (khat and v', as swa_attn_qkv_prologue or the workspace
 * of swa_attn_fwd_ws gives them for positions 0, 1, ...) into the slots of slots, int32 (B, T).  Rows whose
 * slot is negative are skipped; a slot past the cache is recorded (swa_attn_last_device_status) and
 * skipped.  The rows of one call that go into one page must be consecutive rows with consecutive slots
 * (as swa_attn_kv_pages numbers them; nothing skipped between them): otherwise that page's values are
 * unspecified.  Tokens of a page before the first slot written there must be in the cache already, unless
 * that is the page's token 0.  Nothing but the pages and scales of the slots is written.
 * Errors: SWA_ERR_INVALID_ARG, SWA_ERR_UNSUPPORTED (D not 64 / 128, page_size, n_pages * Hkv * page_size or
 * B * T * Hkv at least 2^31, Hkv > 65535), SWA_ERR_MISALIGNED, SWA_ERR_CUDA.
 */
SWA_API int swa_attn_kv8_write(const void* kh, const void* vp, const int* slots, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, int B, int T, int Hkv, int D, int n_pages,
                               int page_size, swa_stream_t stream);

/*
 * swa_attn_kv8_read: the reverse, kh, vp bf16 (B, T, Hkv, D) = code * scale of the given slots, exact (for
 * a request that is moved: what is read here and written to other pages keeps its values).  Slots may
 * repeat.  Rows with a negative slot, or one past the cache (recorded), are zeros.  Errors as
 * swa_attn_kv8_write.
 */
SWA_API int swa_attn_kv8_read(const int* slots, const void* k_cache, const void* v_cache, const float* k_scale,
                              const float* v_scale, void* kh, void* vp, int B, int T, int Hkv, int D,
                              int n_pages, int page_size, swa_stream_t stream);

/*
 * swa_attn_kv8_decode: one generation step over the paged cache, as swa_attn_decode_doc with a length for
 * each request.  Request b has n_b = seq_len[b] tokens, its new one at position n_b - 1:
 *   1. the prologue of swa_attn_decode at that position; khat and v' go into its slot (as
 *      swa_attn_kv8_write).  k = v = NULL: the token is in the cache already, only q is used (then
 *      ve, gate_x, Wg are NULL too).
 *   2. out[b,h,:] = sum_j softmax_j(qhat . k_j / sqrt(D)) v_j over the cached keys j in
 *      [max(0, n_b - window, min(doc_start[b], n_b - 1)), n_b) (window <= 0: no window; doc_start int32 (B) or
 *      NULL), lse[b,h] = ln sum_j exp(qhat . k_j / sqrt(D)); query head h reads key/value head
 *      h / (H / Hkv).  Entries of the block table before the first of these keys are not read.
 *   Requests with seq_len <= 0 are empty rows: out = 0, lse = -inf, the cache is left alone.
 *   q, out bf16 (B, H, D); k, v, ve bf16 (B, Hkv, D); gate_x bf16 (B, 32); Wg bf16 [32, Hkv]; lse fp32 (B, H) or NULL;
 *   block_table int32 (B, max_pages); seq_len int32 (B).  Two requests may share pages, but not the page
 *   that takes a new token.  workspace: swa_attn_kv8_decode_workspace_bytes() bytes, 16-byte aligned,
 *   nothing kept between calls; calls that may overlap need one each.
 * A seq_len beyond max_pages * page_size (an empty row) and pages outside the cache (their keys are not
 * visible, a token that belongs there is not stored) are recorded: swa_attn_last_device_status.
 * Scores, exponentials p_j and sums are fp32.  The products with v_j take p_j * (value scale) in 11 bits (off by at
 * most 2^-11 of it); below 2^-34 of the largest of these of a request and head, off by at most 2^-45 of that one.  p_j
 * below 2^(e - 126) of the largest are lost where the largest visible value scale is 2^e: 2^-66 of it at e = 60.
 * Errors: SWA_ERR_INVALID_ARG, SWA_ERR_UNSUPPORTED (D not 64 / 128, page_size, H / Hkv > 64, sizes beyond int32),
 * SWA_ERR_MISALIGNED, SWA_ERR_NO_MEMORY (workspace too small), SWA_ERR_CUDA.
 */
SWA_API size_t swa_attn_kv8_decode_workspace_bytes(int B, int H, int Hkv, int D);
SWA_API int swa_attn_kv8_decode(const void* q, const void* k, const void* v, const void* ve, const void* gate_x,
                                const void* Wg, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                const int* block_table, const int* seq_len, const int* doc_start, void* out,
                                float* lse, int B, int H, int Hkv, int D, int n_pages, int page_size,
                                int max_pages, int window, float rope_base, float eps, void* workspace,
                                size_t ws_bytes, swa_stream_t stream);

/*
 * Failure-detection self-test (no counterpart in the pages).  Enqueues on `stream` one block of
 * 32 threads that waits, through the bounded wait every kernel here uses, on an mbarrier that
 * nothing ever completes.  After `limit_ms` (1..10000) the wait gives up, records SWA_ERR_TIMEOUT
 * at wait site 30 in the device status word and the kernel returns normally: the device context
 * stays usable.  Read the result with swa_attn_last_device_status().  Returns SWA_OK once the
 * kernel is enqueued, SWA_ERR_INVALID_ARG for a limit out of range, else as the other calls.
 */
SWA_API int swa_attn_selftest_wait(int limit_ms, swa_stream_t stream);

/* Upper bound, in milliseconds, on any single wait inside the kernels (default 2000).
 * Returns the previous value.  Values < 1 are ignored. */
SWA_API int swa_attn_set_wait_limit_ms(int ms);

/* ABI version: major * 10000 + minor * 100 + patch. */
SWA_API int swa_attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SWA_ATTN_H_ */
