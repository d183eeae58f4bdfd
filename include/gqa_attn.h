/*
 * gqa_attn.h -- C ABI of the GB300 (sm_103a) causal grouped-query attention library.
 *
 * The library computes the attention of a hybrid local/global decoder layer:
 *
 *     O[b,h,t,:] = sum_s softmax_s( scale * <Q'[b,h,t,:], K'[b,g(h),s,:]> + M[t,s] ) V[b,g(h),s,:]
 *
 * with g(h) = floor(h / (Hq/Hkv)) (consecutive query heads share one KV head), Q' and K'
 * the split-half RoPE rotations of Q and K, and M the causal or sliding-window mask.
 * Definitions, by page and section:
 *   "PLaMo 3アーキテクチャ徹底解析" (imoz.jp):
 *     §4.2 grouped-query attention;  §4.4 the cache stores K before RoPE, positions are
 *     generated inside attention (keys 0..S-1, queries S-T..S-1), the local cache keeps
 *     the last W-1 tokens and re-numbers them;  §4.5 the attention equation, scale
 *     1/sqrt(d), no softcap;  §5.1 the masks (causal j <= i; window also i - j < W,
 *     self included);  §6.1 split-half RoPE, omega_j = theta^(-2j/d);  §6.3 YaRN
 *     frequencies and the amplitude factor on cos and sin;  §6.4 partial (p-)RoPE.
 *
 * Conventions (all entry points):
 *   - Tensors are bfloat16, dense, row-major in the layouts stated per call, in device
 *     memory, 16-byte aligned.  The caller owns every buffer, descriptor array, workspace
 *     and stream; the library allocates nothing.  Its only device state is a status word
 *     per GPU and the fixed 16 MiB scratch array of gqa_attn_decode_static, both
 *     compiled into the library; on the host it remembers, per device, which kernels
 *     have had their shared-memory limit raised (a mutex guards that record, so calls
 *     may come from several host threads and may drive several GPUs in turn).
 *   - Every call validates its arguments on the host and returns a negative gqa_status
 *     without launching anything if they are wrong.  Otherwise it enqueues its kernels on
 *     `stream` (NULL = the legacy default stream) and returns GQA_OK without waiting.
 *   - Errors found on the device (a bounded wait that expired, a full cache, an index
 *     out of range) are recorded in the device status word and returned by the next
 *     gqa_get_device_status().  Device code never traps.
 *   - Stream order holds as for any kernel.  On a stream that is not being captured,
 *     gqa_kv_append, the decode calls and the packed and paged calls launch with programmatic
 *     stream serialization
 *     and let the next kernel begin launching early.  Each of their kernels waits for its
 *     predecessor before reading.  A caller's own kernel launched after them with that
 *     attribute must likewise execute griddepcontrol.wait (cudaGridDependencySynchronize)
 *     before it reads their outputs.
 *   - Head dims: prefill and decode d in {128, 256, 512}, their packed and paged forms
 *     d = 128; kv_append, rope_apply, the packed append and the Q/K normalisation d in
 *     {64, 128, 256, 512}.  Query group G = Hq/Hkv must be an
 *     integer; decode needs G <= 8.  Other values return GQA_ERR_UNSUPPORTED.
 */
#ifndef GQA_ATTN_H
#define GQA_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *gqa_stream_t;

typedef enum gqa_status {
    GQA_OK = 0,
    GQA_ERR_INVALID_ARG = -1,     /* null pointer, non-positive size, inconsistent shape */
    GQA_ERR_UNSUPPORTED = -2,     /* head dim / group size / device not supported */
    GQA_ERR_ALIGNMENT = -3,       /* a pointer is not 16-byte aligned */
    GQA_ERR_CAPACITY = -4,        /* a linear cache is full, or a length exceeds a bound */
    GQA_ERR_CUDA = -5,            /* a CUDA runtime call failed */
    GQA_ERR_DEVICE_TIMEOUT = -6,  /* a device-side bounded wait expired */
    GQA_ERR_WORKSPACE = -7,       /* workspace missing or too small */
    GQA_ERR_RANGE = -8,           /* a position lies beyond the RoPE table */
    GQA_ERR_DEVICE_BOUNDS = -9    /* debug build only: a device-side index check failed */
} gqa_status;

/* ---- RoPE frequencies and table ---------------------------------------------------
 * gqa_rope_inv_freq (host only, no GPU needed): writes omega_j, j = 0..d/2-1, to out:
 *   omega_j = base^(-2j/d)                                        ("PLaMo 3..." §6.1)
 *   if yarn_factor != 1 (YaRN, §6.3):
 *     j_low  = (d/2) ln(yarn_L0 / (2 pi beta_fast)) / ln(base)   (not rounded)
 *     j_high = (d/2) ln(yarn_L0 / (2 pi beta_slow)) / ln(base)
 *     alpha_j = clip((j - j_low) / (j_high - j_low), 0, 1)
 *     omega_j *= (1 - alpha_j) + alpha_j / yarn_factor
 *   if rotate_fraction < 1 (p-RoPE, §6.4): omega_j = 0 for j >= round(rotate_fraction d/2);
 *     the exponent keeps the full d.
 * Returns GQA_ERR_INVALID_ARG for d odd/<= 0, base <= 1, yarn_factor < 1, or a fraction
 * outside (0, 1]. */
gqa_status gqa_rope_inv_freq(double *out, int d, double base, double yarn_factor,
                             double yarn_L0, double beta_fast, double beta_slow,
                             double rotate_fraction);

/* YaRN amplitude 1 + 0.1 ln(s) applied to both cos and sin (§6.3); host only. */
double gqa_yarn_amplitude(double s);

/* Bytes of a RoPE table for head dim d and positions 0..max_pos-1:
 * max_pos * (d/2) * 2 floats. */
size_t gqa_rope_table_bytes(int d, int max_pos);

/* Fills `table` (device, caller-owned, gqa_rope_table_bytes(d, max_pos) bytes) with
 * float pairs table[p*(d/2) + j] = (amp cos(p omega_j), amp sin(p omega_j)) for
 * p < max_pos: the angle and both functions are evaluated in double precision on the
 * device and rounded once to float.  inv_freq: host array of d/2 doubles (see above),
 * copied into the launch, so it may be freed on return.  d <= 512, amp > 0. */
gqa_status gqa_rope_table_build(float *table, const double *inv_freq, int d, double amp,
                                int max_pos, gqa_stream_t stream);

/* ---- RoPE application (§6.1) --------------------------------------------------------
 * y[b,h,t,:] = rotation of x[b,h,t,:] at position pos0 + t, pairs (j, j+d/2), using the
 * table (table_len positions).  x, y: [B, H, T, d] bf16; y may equal x (in place).
 * Each output is rounded once to bf16 from the float rotation. */
gqa_status gqa_rope_apply(const void *x, void *y, int B, int H, int T, int d, int pos0,
                          const float *table, int table_len, gqa_stream_t stream);

/* ---- Prefill (§4.4, §4.5, §5.1) ------------------------------------------------------
 * q: [B, Hq, T, d], k, v: [B, Hkv, S, d] (k before RoPE, as a cache holds it),
 * o: [B, Hq, T, d] bf16.  lse: [B, Hq, T] float32 natural-log sum of exp of the scaled
 * scores, or NULL.  T <= S; query t sits at position S - T + t, key s at position s.
 * window <= 0: full causal; window > 0: keys with q_pos - k_pos < window (self included).
 * scale multiplies the dot products (e.g. 1/sqrt(d)); the table's amplitude multiplies
 * them by amp^2 on top.  scale must be finite and > 0 (the softmax takes each row's
 * maximum before scaling), else GQA_ERR_INVALID_ARG.  table_len >= S.
 * Key tiles wholly outside [q_pos - window + 1, q_pos] are never loaded or multiplied.
 * k_is_rotated = 0: k holds keys before RoPE (as the PLaMo cache stores them, §4.4); they
 *   are rotated once at positions 0..S-1 into `workspace`, which must hold at least
 *   gqa_prefill_workspace_bytes(B, Hkv, S, d) bytes; its contents are undefined afterwards.
 * k_is_rotated = 1: k already carries RoPE (a cache that stores rotated keys, as Gemma's
 *   does, §4.4); workspace may be NULL.
 * k_is_rotated = 2 (d = 128 only, else GQA_ERR_UNSUPPORTED): k holds keys before RoPE and
 *   each K tile is rotated in shared memory as it lands, inside the attention kernel (RoPE
 *   fused into the tile load); workspace may be NULL.  Same results as 0, bit for bit.
 *   Slower than 0 on long inputs: a K tile is rotated again every time a query block
 *   reloads it, while 0 rotates each key once.  Any other value: GQA_ERR_INVALID_ARG.
 * Supports d = 128, 256, 512.  Hq % Hkv == 0. */
size_t gqa_prefill_workspace_bytes(int B, int Hkv, int S, int d);
gqa_status gqa_attn_prefill(const void *q, const void *k, const void *v, void *o,
                            float *lse, int B, int T, int S, int Hq, int Hkv, int d,
                            int window, float scale, const float *table, int table_len,
                            int k_is_rotated, void *workspace, size_t workspace_bytes,
                            gqa_stream_t stream);

/* ---- KV cache (§4.4) -----------------------------------------------------------------
 * One descriptor per sequence, in device memory, owned by the caller.
 *   k, v   : device [Hkv, cap, d] bf16, K stored before RoPE.
 *   rope   : device RoPE table for this sequence's layer type; rope_len positions.
 *            Decode at d = 512 treats a group of 32 pairs whose rows 0 and 1 are all
 *            exactly (1, 0) as never rotating (omega = 0 at amplitude 1, as
 *            gqa_rope_table_build writes p-RoPE's unrotated pairs) and reads no further
 *            rows of it.
 *   cap    : slots per KV head.
 *   count  : linear cache (is_ring = 0): tokens held; they occupy slots 0..count-1 and
 *            sit at positions equal to their slots.
 *            ring cache (is_ring = 1, cap = window W): tokens appended so far; token i
 *            lives in slot i mod cap.  Attention sees the newest min(count, cap) tokens,
 *            re-numbered 0..R-1 from oldest to newest (the last W-1 kept plus the new one).
 */
typedef struct gqa_kv_desc {
    void *k;
    void *v;
    const float *rope;
    int32_t cap;
    int32_t count;
    int32_t is_ring;
    int32_t rope_len;
} gqa_kv_desc;

/* Appends one token per sequence: k_new, v_new [nseq, Hkv, d] bf16 are written to slot
 * count (linear) or count mod cap (ring) of every KV head, then count += 1.  slots_out
 * (device int32[nseq], nullable) receives the slot written.  A full linear cache is not
 * written; its slot_out is -1 and the status word records GQA_ERR_CAPACITY. */
gqa_status gqa_kv_append(gqa_kv_desc *descs, int nseq, const void *k_new,
                         const void *v_new, int Hkv, int d, int32_t *slots_out,
                         gqa_stream_t stream);

/* ---- Chunked prefill over a cache (§4.4) ----------------------------------------------
 * A chunk of T new tokens of one sequence attends to the R tokens its cache holds
 * (linear: R = count; ring: R = min(count, cap), the newest ones, oldest first) followed
 * by itself: S = R + T keys at positions 0..S-1 and queries at R..S-1 (a local layer's
 * ring is re-numbered from 0, §4.4; its window W = cap covers every key a chunk query can
 * see).  Per chunk: gqa_prefill_gather, then gqa_attn_prefill(q [1, Hq, T, d], k_out,
 * v_out, B = 1, T, S, ..., k_is_rotated = 1), then gqa_kv_append_chunk.
 *
 * gqa_prefill_gather: desc is one device descriptor; k_new, v_new [Hkv, T, d] are the
 * chunk's keys (before RoPE) and values; k_out, v_out [Hkv, S, d] (caller-owned) receive
 * the S keys rotated at positions 0..S-1 and the S values.  S is the caller's count of
 * R + T; if the descriptor disagrees, or S > table_len, nothing is written and the status
 * word records GQA_ERR_CAPACITY (resp. GQA_ERR_RANGE).
 *
 * gqa_kv_append_chunk: k_new, v_new [nseq, Hkv, T, d]; each sequence's T tokens go to slots
 * count .. count + T - 1 (linear; if they do not fit, nothing is written and the status
 * word records GQA_ERR_CAPACITY) or (count + t) mod cap (ring; when T > cap only the last
 * cap tokens are stored), then count += T.  d in {64, 128, 256, 512}. */
gqa_status gqa_prefill_gather(const gqa_kv_desc *desc, const void *k_new, const void *v_new,
                              int T, int Hkv, int d, void *k_out, void *v_out, int S,
                              const float *table, int table_len, gqa_stream_t stream);
gqa_status gqa_kv_append_chunk(gqa_kv_desc *descs, int nseq, const void *k_new,
                               const void *v_new, int T, int Hkv, int d, gqa_stream_t stream);

/* ---- Q/K normalisation in front of attention (§3.2, §4.3, §4.4) ----------------------
 * RMSNorm with an effective gain (§3.2): N(x) = gamma * x / sqrt(mean(x^2) + eps) over
 * each (token, head) vector of d values; PLaMo's q_norm / k_norm use offset 1, so the
 * caller passes gamma = 1 + w (the stored weight w plus the offset), eps = 1e-6, and one
 * gain of d floats shared by every head (§4.3).  The order is fixed by §4.4: normalise,
 * store K in the cache (normalised, not rotated), then rotate.  Sums of squares and the
 * scaling run in fp32; each output is rounded once to bf16 (the public implementation's
 * intermediate bf16 rounding is not reproduced).  d in {64, 128, 256, 512}; gains are
 * device fp32 [d], 16-byte aligned; outputs may alias their inputs (q_out == q, k_out == k).
 *
 * Prefill form: q [B, Hq, T, d] -> q_out = N_q(q) (rotated later, inside
 * gqa_attn_prefill); k [B, Hkv, T, d] -> k_out = N_k(k) (what the cache stores, nullable)
 * and k_rot = RoPE(N_k(k)) at positions pos0 + t (nullable; pass it to gqa_attn_prefill
 * with k_is_rotated = 1).  V is not touched.  table as for gqa_rope_apply; positions
 * past table_len return GQA_ERR_RANGE. */
gqa_status gqa_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, void *k_rot,
                            int B, int Hq, int Hkv, int T, int d, int pos0,
                            const float *q_gamma, const float *k_gamma, float eps,
                            const float *table, int table_len, gqa_stream_t stream);

/* Decode form: for each sequence one new token.  q [nseq, Hq, d] -> q_out = N_q(q) (the
 * decode kernel rotates it); k_new [nseq, Hkv, d] -> N_k(k_new) and v_new [nseq, Hkv, d]
 * (unchanged, or with v_norm = 1 normalised without a gain, as Gemma 4 does) are appended
 * to each sequence's cache exactly as gqa_kv_append appends them (slot, count update,
 * slots_out, GQA_ERR_CAPACITY on a full linear cache). */
gqa_status gqa_qk_norm_append(gqa_kv_desc *descs, int nseq, const void *q, const void *k_new,
                              const void *v_new, int Hq, int Hkv, int d, const float *q_gamma,
                              const float *k_gamma, float eps, int v_norm, void *q_out,
                              int32_t *slots_out, gqa_stream_t stream);

/* ---- Shared K/V projection (Gemma 4 global layers) ---------------------------------------
 * attention_k_eq_v ("PLaMo 3..." §5.2 and the Gemma 4 comparison of §8): one projection
 * output Z [.., Hkv, .., d] per token gives both K = RoPE(N_{gamma_k}(Z)) and V = N_1(Z),
 * N_1 being RMSNorm without a gain (eps as above).  Such a layer needs to cache only
 * Zn = N_1(Z): since N_gamma(Z) = gamma * N_1(Z), the keys are recomputed from it.  The
 * library does exactly that: the stored row is Zn rounded once to bf16, and the key is
 * RoPE(gamma_k * Zn) -- the fp32 gain times the stored row, rotated in fp32 and rounded
 * once to bf16 -- in prefill and decode alike (the two may round the rotation's products
 * in a different order, at most one bf16 step apart).  Gains are device fp32
 * [d], 16-byte aligned, one per layer, shared by every head; d in {64, 128, 256, 512}
 * (decode: {128, 256, 512}).
 *
 * gqa_qk_norm_rope_kv_shared (prefill form): q [B, Hq, T, d] -> q_out = N_{q_gamma}(q)
 * (rotated later, inside gqa_attn_prefill); z [B, Hkv, T, d] -> v_out = Zn (the values,
 * and what the cache stores; nullable) and k_rot = RoPE(gamma_k * Zn) at positions
 * pos0 + t (nullable; pass it to gqa_attn_prefill with k_is_rotated = 1 and v_out as v).
 * q, q_out and q_gamma may all be NULL (then Hq is ignored) to process Z alone; at least
 * one of v_out, k_rot must be given; k_gamma and the table are needed only for k_rot.
 * Each output may alias its own input (q_out == q; v_out or k_rot == z), not another output.
 *
 * gqa_kv_shared_append (decode form): q [nseq, Hq, d] -> q_out = N_{q_gamma}(q);
 * z_new [nseq, Hkv, d] -> Zn appended to each sequence's cache at desc.k, with the slot,
 * count update, slots_out and GQA_ERR_CAPACITY of gqa_kv_append; desc.v is not written.
 *
 * gqa_attn_decode_kv_shared: as gqa_attn_decode (same arguments, workspace and results),
 * over caches of Zn at desc.k: keys RoPE(k_gamma * Zn) at positions 0..R-1, values
 * Zn; desc.v is not read.  The cache rows are read once from memory for both roles, half
 * the bytes of separate K and V caches. */
gqa_status gqa_qk_norm_rope_kv_shared(const void *q, const void *z, void *q_out, void *v_out,
                                      void *k_rot, int B, int Hq, int Hkv, int T, int d,
                                      int pos0, const float *q_gamma, const float *k_gamma,
                                      float eps, const float *table, int table_len,
                                      gqa_stream_t stream);
gqa_status gqa_kv_shared_append(gqa_kv_desc *descs, int nseq, const void *q, const void *z_new,
                                int Hq, int Hkv, int d, const float *q_gamma, float eps,
                                void *q_out, int32_t *slots_out, gqa_stream_t stream);

/* ---- Decode (§4.4, §4.5) ---------------------------------------------------------------
 * One query token per sequence: q [nseq, Hq, d] bf16 at position R-1, where R = count
 * (linear) or min(count, cap) (ring) read from the descriptors (so call after
 * gqa_kv_append).  Keys are the R logical tokens at positions 0..R-1, rotated on the fly
 * with the sequence's table.  o: [nseq, Hq, d] bf16; lse: [nseq, Hq] float or NULL.
 * max_len: an upper bound on R over the batch (sizes the split-KV grid); a sequence with
 * R > max_len or rope_len < R is skipped and flagged in the status word.
 * workspace: device scratch of gqa_decode_workspace_bytes(nseq, Hq, Hkv, d, max_len) bytes:
 * the split partials, nseq Hq nsplit (m, l) float pairs padded to a multiple of 4 floats,
 * then nseq Hq nsplit rows of d floats.  The number of splits per sequence, nsplit, and
 * the keys per split are chosen from (nseq, Hkv, d, max_len) so that the grid fills the
 * GPU; the workspace size follows the same rule, so it must be queried with the shape of
 * the call.  scale: finite and > 0.
 * d in {128, 256, 512} (Gemma-4 local / global heads), Hq/Hkv <= 8. */
size_t gqa_decode_workspace_bytes(int nseq, int Hq, int Hkv, int d, int max_len);
gqa_status gqa_attn_decode(const void *q, const gqa_kv_desc *descs, int nseq, int Hq,
                           int Hkv, int d, float scale, int max_len, void *o, float *lse,
                           void *workspace, size_t workspace_bytes, gqa_stream_t stream);

gqa_status gqa_attn_decode_kv_shared(const void *q, const gqa_kv_desc *descs, int nseq, int Hq,
                                     int Hkv, int d, float scale, const float *k_gamma,
                                     int max_len, void *o, float *lse, void *workspace,
                                     size_t workspace_bytes, gqa_stream_t stream);

/* Decode without a caller-supplied workspace; allocates nothing.  The pages have no
 * counterpart to this entry point: it is the same computation as gqa_attn_decode (same
 * kernels, same arguments and results), for callers that cannot provide scratch memory --
 * for instance because their device memory is owned by another component (a framework
 * allocator that reserved the GPU up front, a serving loop that forbids allocation), or
 * because the device synchronisation of cudaMalloc/cudaFree is unacceptable per step.
 * The split-KV partials go to a fixed 16 MiB device array inside the library, which every
 * GPU that loads the library holds until the process exits.  A call whose partials need
 * more than that, i.e. gqa_decode_workspace_bytes(nseq, Hq, Hkv, d, max_len) > 16 MiB, returns
 * GQA_ERR_WORKSPACE without launching.
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 * with that device current; make that first call before any stream capture.
 * All calls share the one array and it keeps the last call's contents (each call writes
 * every record it reads, so no clearing is needed): calls that may overlap on the GPU --
 * on different streams, or from different host threads -- race on it and must be
 * serialised by the caller. */
gqa_status gqa_attn_decode_static(const void *q, const gqa_kv_desc *descs, int nseq, int Hq,
                                  int Hkv, int d, float scale, int max_len, void *o,
                                  float *lse, gqa_stream_t stream);

/* ---- Packed sequences and the paged cache ------------------------------------------------
 * A packed batch holds the tokens of nseq sequences of different lengths behind one another:
 * sequence i owns rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 of token-major tensors
 * [total, heads, d] (cu_seqlens: device int32[nseq + 1], non-decreasing, cu_seqlens[0] >= 0).
 * `total` is the number of rows of the tensors, cu_seqlens[nseq] <= total; rows that belong to
 * no sequence are neither read nor written.  A sequence may be empty.  Each tensor has a token
 * stride in elements, a multiple of 8 and at least heads * d (heads are d apart), so that q, k
 * and v may be column slices of the rows of one fused QKV projection (§4.1: 8192 q, 1024 k,
 * 1024 v columns in PLaMo 3 31B).
 *
 * A paged cache keeps each sequence's keys and values in pages of page_size tokens of one
 * pool: token j of sequence i lies in row j mod page_size of page page_table[i][j / page_size],
 * for every KV head.  Unlike the caches of gqa_kv_desc it holds keys AFTER RoPE (a cache that
 * stores rotated keys, as Gemma's does, §4.4): each key is rotated once, when it is written,
 * and a page can be shared by sequences with a common prefix.  kv_lens[i] counts the tokens
 * of sequence i with the new ones of this step: S = kv_lens[i], T = cu_seqlens[i+1] -
 * cu_seqlens[i] new tokens at positions S - T .. S - 1, T <= S.  The struct lives in host
 * memory and is read during the call; page_table and kv_lens are device memory and are read
 * when the kernels run, so a captured call follows their later contents.
 *
 * A sequence whose numbers are inconsistent (offsets that decrease or pass `total`, T > S)
 * is skipped, its outputs left as they were, and the status word records
 * GQA_ERR_INVALID_ARG; one that exceeds a bound given by the host (max_q, max_kv, the pages
 * of its table row) is skipped and records GQA_ERR_CAPACITY.  Rows over which offsets decrease
 * (from cu_seqlens[i+1] to cu_seqlens[i]) may be written for any sequence that claims them, or
 * for none; the other sequences' rows are computed.  A page-table entry outside the
 * pool records GQA_ERR_INVALID_ARG: nothing is written there, and zeros are read instead. */
typedef struct gqa_paged_kv {
    void *k;                    /* device [num_pages, Hkv, page_size, d] bf16, after RoPE */
    void *v;                    /* device, the same shape */
    const int32_t *page_table;  /* device [nseq, max_pages] */
    const int32_t *kv_lens;     /* device [nseq] */
    int32_t num_pages;
    int32_t Hkv;
    int32_t page_size;          /* 16, 32, 64 or 128 */
    int32_t d;
    int32_t max_pages;          /* entries of a page_table row */
    int32_t reserved;           /* 0 */
} gqa_paged_kv;

/* What a step does to the new tokens between the QKV projection and attention (§4.3, §4.4):
 * for each token at position p = S - T + t of its sequence
 *   q_out = RoPE_p(N_{q_gamma}(q)),   key = RoPE_p(N_{k_gamma}(k)),   value = v,
 * the key and the value written to the sequence's page, the key also to k_out.  N is the
 * RMSNorm of the section above (fp32, gain device fp32 [d]); q_gamma NULL: q is not
 * normalised, k_gamma likewise.  Everything between the load and the one rounding to bf16 is
 * fp32.  q_out [total, Hq, d] and k_out [total, Hkv, d] are dense, either may be NULL; q_out
 * may be q (k_out may be k) if that tensor's stride is dense.  q and q_out are NULL together
 * (Hq ignored).  cache NULL: no cache is written, v is not read and may be NULL, and every
 * sequence starts at position 0 (the prompts of gqa_attn_packed).  With a cache, Hkv and d
 * must be the cache's.  (The library's own attention over such a cache takes d = 128.)  A
 * position at or past table_len records GQA_ERR_RANGE and its token is skipped.  d in {64, 128,
 * 256, 512}; total <= 2^31 - 513.  One kernel.  Two sequences of one call must not append to the
 * same page. */
gqa_status gqa_packed_rope_append(const void *q, int64_t q_stride, const void *k,
                                  int64_t k_stride, const void *v, int64_t v_stride,
                                  const int32_t *cu_seqlens, int nseq, int total, int Hq,
                                  int Hkv, int d, const float *q_gamma, const float *k_gamma,
                                  float eps, const float *table, int table_len, void *q_out,
                                  void *k_out, const gqa_paged_kv *cache,
                                  gqa_stream_t stream);

/* Attention over whole prompts of different lengths: within each sequence query t attends to
 * keys j <= t (window > 0: also t - j < window).  q, k after RoPE, q [total, Hq, d], k, v
 * [total, Hkv, d], o [total, Hq, d] with token strides; o may not alias an input.  lse
 * [Hq, total] float32 natural-log sum of exp of the scaled scores, or NULL.  scale finite and
 * > 0.  A row never depends on keys or values that its mask hides, not even through NaN or
 * infinities in them.  A row whose visible scores are all -inf is NaN, its lse -inf.  d = 128;
 * Hq / Hkv an integer of at most 64; total <= 2^30 (and see the limit on counts below). */
gqa_status gqa_attn_packed(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, void *o, int64_t o_stride,
                           float *lse, const int32_t *cu_seqlens, int nseq, int total, int Hq,
                           int Hkv, int d, int window, float scale, gqa_stream_t stream);

/* Attention of each sequence's new tokens over its paged cache (which holds them already: call
 * after gqa_packed_rope_append): T = 1 is a decode step, a few are a draft being checked, many
 * a chunk of a prompt; a batch may mix them.  Query t sits at position S - T + t and attends
 * to keys j <= S - T + t (window > 0: also with S - T + t - j < window; pages that lie wholly
 * below every window are not read and their table entries may be stale).  q [total, Hq, d]
 * after RoPE, o [total, Hq, d], lse as for gqa_attn_packed.  max_q and max_kv: upper bounds on
 * T and S over the batch (bounds far above them split the keys of chunks more coarsely, which
 * costs time; a decode step is one kernel up to max_kv = 512, two beyond, and depends little on
 * it otherwise); they and the shape choose the kernel and its split of the keys, and size the
 * workspace (gqa_attn_paged_workspace_bytes with the same arguments; 0 = none needed, or a shape
 * that the call refuses).  Its contents need no initialisation; calls that may overlap need one
 * each.  Every result is the same on every run of the same call.  d = 128; G = Hq / Hkv an
 * integer of at most 64; max_q <= max_kv <= 2^30, total <= 2^30.  The work of a call is counted
 * in 32 bits: with max_q * G <= 16, nseq * Hkv * ceil(max_kv / 64) is at most 2^31 - 153; with
 * more rows, (floor(total / (2 floor(128 / G))) + min(nseq, total)) * Hkv times the spans of the
 * keys (up to 64; 1 for gqa_attn_packed) at most 2^31 - 2.  Bounds beyond these return
 * GQA_ERR_UNSUPPORTED. */
size_t gqa_attn_paged_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq,
                                      int Hkv, int d);
gqa_status gqa_attn_paged(const void *q, int64_t q_stride, const gqa_paged_kv *cache,
                          const int32_t *cu_seqlens, int nseq, int total, int max_q, int max_kv,
                          int Hq, int window, float scale, void *o, int64_t o_stride,
                          float *lse, void *workspace, size_t workspace_bytes,
                          gqa_stream_t stream);

/* ---- The 8-bit paged cache -----------------------------------------------------------------
 * The paged cache of the section above with keys and values in 8 bits, half the bytes of a decode
 * step and of the memory.  A key or value vector x (one token, one KV head) is kept as d e4m3
 * numbers y and one power of two:
 *   e = the smallest integer in [-126, 119] with max |x| <= 448 * 2^e  (-126 for a zero vector),
 *   y_i = x_i / 2^e rounded to the nearest e4m3 number, ties to even, at most 448 in magnitude,
 * and the byte e + 127 (E8M0) in `scales`.  It reads back as y_i * 2^(byte - 127), off by at most
 * 2^-4 of |x_i| and 2^(e-10) for elements below 2^(e-6).  A vector that holds an infinity or a NaN
 * gets the byte 255 and reads back as NaN; its numbers are zeros.  Rows, pages, lengths, flagged
 * contents and the meaning of a page-table entry are those of gqa_paged_kv. */
typedef struct gqa_paged_kv_q8 {
    void *k;                    /* device [num_pages, Hkv, page_size, d] e4m3, after RoPE */
    void *v;                    /* device, the same shape */
    void *scales;               /* device [num_pages, Hkv, page_size, 2]: the key's byte, then the
                                   value's */
    const int32_t *page_table;  /* device [nseq, max_pages] */
    const int32_t *kv_lens;     /* device [nseq] */
    int32_t num_pages;
    int32_t Hkv;
    int32_t page_size;          /* 16, 32, 64 or 128 */
    int32_t d;
    int32_t max_pages;          /* entries of a page_table row */
    int32_t reserved;           /* 0 */
} gqa_paged_kv_q8;

/* As gqa_packed_rope_append (same arguments, checks and flags) into an 8-bit cache, which may not
 * be NULL.  The rotated key and the value are rounded once, from fp32, to the cache's numbers;
 * k_out, if given, receives the rotated key in bf16 (for gqa_attn_packed over the same prompts).
 * One kernel. */
gqa_status gqa_packed_rope_append_q8(const void *q, int64_t q_stride, const void *k,
                                     int64_t k_stride, const void *v, int64_t v_stride,
                                     const int32_t *cu_seqlens, int nseq, int total, int Hq,
                                     int Hkv, int d, const float *q_gamma, const float *k_gamma,
                                     float eps, const float *table, int table_len, void *q_out,
                                     void *k_out, const gqa_paged_kv_q8 *cache,
                                     gqa_stream_t stream);

/* As gqa_attn_paged over an 8-bit cache: the same arguments, masks, limits and flags, applied to the
 * numbers that the cache stands for.  A key that reads back as NaN makes every row that sees it NaN,
 * a NaN value those rows' elements; a query row with an infinity or a NaN is NaN.
 * gqa_attn_paged_q8_workspace_bytes sizes its own workspace (with the arguments of the call).  With
 * more than 96 rows (max_q * Hq / Hkv) it has room for every key that nseq and max_kv allow in bf16:
 * pass a max_kv near the longest sequence, and decode steps over long caches in a call of their own,
 * not next to a chunk that brings the whole batch over 96 rows. */
size_t gqa_attn_paged_q8_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq,
                                         int Hkv, int d);
gqa_status gqa_attn_paged_q8(const void *q, int64_t q_stride, const gqa_paged_kv_q8 *cache,
                             const int32_t *cu_seqlens, int nseq, int total, int max_q, int max_kv,
                             int Hq, int window, float scale, void *o, int64_t o_stride,
                             float *lse, void *workspace, size_t workspace_bytes,
                             gqa_stream_t stream);

/* Reads an 8-bit cache back: sequence i owns rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 of k_out
 * and v_out [total, Hkv, d] bf16 (token strides as above; either may be NULL), which receive its
 * tokens S - T .. S - 1, S = kv_lens[i], T its number of rows: all of them, or the newest; another
 * kv_lens in the struct reads another range.  Each value is rounded once to bf16, exact unless it
 * leaves bf16's range.  Rows of no sequence are not written; a page outside the pool is flagged and
 * reads as zeros.  d in {64, 128, 256, 512}; total <= 2^30.  k_out and v_out may not overlap each
 * other, or the pools. */
gqa_status gqa_paged_read_q8(const gqa_paged_kv_q8 *cache, const int32_t *cu_seqlens, int nseq,
                             int total, void *k_out, int64_t k_stride, void *v_out,
                             int64_t v_stride, gqa_stream_t stream);

/* ---- Status ----------------------------------------------------------------------------
 * Waits for `stream`, then returns and clears the current device's status word
 * (GQA_OK if no device-side error was recorded since the last call). */
gqa_status gqa_get_device_status(gqa_stream_t stream);

/* Waits for `stream`, then stores in diag[0..n) and clears the diagnostic codes of the
 * device-side bounded waits that expired since the last call (0 where none): diag[0] the
 * first overall, diag[1..4] the first of each kernel role 0..3.  A code is
 * (kernel << 24) | (role << 20) | (barrier << 16) | (tile index & 0xffff), kernel 1 =
 * prefill d=128, 2 = prefill d=256, 3 = decode, 4 = gqa_watchdog_selftest,
 * 5 = prefill d=512 (a pair of CTAs), 6 = cache append, chunk gather, RoPE pass, Q/K
 * normalisation, packed append, 7 = packed / paged prefill, 8 = paged decode.  A library
 * compiled with -DGQA_DEBUG_BOUNDS checks the indices of the
 * global accesses it derives from device-side data; the first failed check records
 * GQA_ERR_DEVICE_BOUNDS and, in diag[0], (kernel << 24) | (1 << 23) | site, and the access
 * is skipped.  For diagnosing device-side errors; gqa_get_device_status leaves the codes
 * in place. */
gqa_status gqa_get_device_diag(gqa_stream_t stream, int32_t *diag, int n);

/* Self-test of the device-side watchdog (the pages have no counterpart: this checks the
 * library's own failure detection).  Enqueues on `stream` one warp that waits on an
 * mbarrier nothing ever arrives on, bounded by limit_ns nanoseconds, with the same wait
 * and reporting code as the attention kernels.  The wait expires, the kernel records
 * GQA_ERR_DEVICE_TIMEOUT and diagnostic code 4 << 24 and returns normally: the next
 * gqa_get_device_status returns GQA_ERR_DEVICE_TIMEOUT and the context stays usable.
 * limit_ns in [1000, 2000000000] (1 us .. 2 s, the kernels' own limit), else
 * GQA_ERR_INVALID_ARG without launching. */
gqa_status gqa_watchdog_selftest(int64_t limit_ns, gqa_stream_t stream);

/* Static, human-readable text for a status code. */
const char *gqa_status_string(int status);

/* Text of the CUDA runtime error behind the most recent GQA_ERR_CUDA returned to the
 * calling host thread (static storage; "no CUDA error recorded" if there was none). */
const char *gqa_last_error_string(void);

/* GQA_OK if the current CUDA device is an sm_103 part this build can run on. */
gqa_status gqa_device_check(void);

#ifdef __cplusplus
}
#endif
#endif /* GQA_ATTN_H */
