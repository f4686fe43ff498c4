/*
 * dsa.h -- C ABI of libdsa: the DeepSeek sparse-attention (DSA) hot path on
 * one GB300 (sm_103a).
 *
 * The path has three stages, as the DeepSeek-V3.2-Exp atlas page states them
 * (MoE transformer block, "All 43 steps"):
 *
 *   1. the lightning indexer
 *        S^I_{t,s} = 1/(sqrt(H_I) sqrt(D_I)) sum_h w_{t,h} ReLU(q^I_{h,t} . k^I_s)
 *      plus the causal mask M (S~^I = S^I + M),
 *   2. the top-k selection M^sel (top_2048 of S~^I_t per query), and
 *   3. multi-head latent attention over the selected keys, computed in the
 *      absorbed form: q~_h = q^C_h W_UK,h scores against the shared latent
 *      row [c^KV | k^R] (d_c + d_r values per key), an online softmax runs
 *      over the selected keys, and W_UV maps the latent context back to the
 *      per-head values (the output before the output projection wo).
 *
 * Conventions shared by every entry point
 *   - Pointers are DEVICE pointers unless the comment says "host".  The
 *     caller owns every buffer.  The library never allocates device or host
 *     memory and never synchronises the stream; scratch memory comes from a
 *     caller buffer whose size the matching *_workspace_size call returns.
 *   - Every launch goes on `stream` (a cudaStream_t; NULL = legacy default).
 *   - Every call returns a dsa_status.  Arguments are validated on the host
 *     before anything is launched; an invalid call launches nothing.
 *     Nothing aborts the process.
 *   - A batch is a set of sequences (dsa_seqs).  Query rows of all sequences
 *     are stacked: rows cu_q[b] .. cu_q[b+1]-1 belong to sequence b, and
 *     query t of sequence b sits at absolute position p = start_pos[b] + t.
 *     Keys of sequence b are rows cu_k[b] .. cu_k[b+1]-1 of the key caches
 *     and are numbered 0 .. S_b-1 within the sequence (S_b = cu_k[b+1]-cu_k[b]).
 *     Causality: key s is visible to the query at position p iff s <= p.
 *     Every sequence must satisfy start_pos[b] + T_b <= S_b.
 *   - Element types: DSA_F32 (fp32), DSA_BF16 (bf16), DSA_E4M3 (FP8 e4m3 codes,
 *     one byte each, with fp32 power-of-two block scales).
 */
#ifndef DSA_H
#define DSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dsa_status {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARG = 1,  /* null pointer, bad size / stride / alignment, inconsistent sequences */
    DSA_ERR_UNSUPPORTED = 2,  /* a dtype / shape combination no kernel handles */
    DSA_ERR_CUDA = 3,         /* a CUDA call or launch failed: dsa_last_cuda_error() gives the code */
    DSA_ERR_TIMEOUT = 4,      /* a device-side wait gave up (reported by dsa_check_device_error) */
    DSA_ERR_WORKSPACE = 5     /* workspace pointer NULL, misaligned (256 B) or smaller than required */
} dsa_status;

typedef enum dsa_dtype {
    DSA_F32 = 0,
    DSA_BF16 = 1,
    DSA_E4M3 = 2
} dsa_dtype;

/* Largest number of sequences in one call. */
#define DSA_MAX_SEQS 1024

/* A batch of sequences.  All three arrays are HOST memory, read during the
 * call only (the library copies what the kernels need into their launch
 * parameters, so the arrays may be freed when the call returns). */
typedef struct dsa_seqs {
    int32_t B;                 /* number of sequences, 1 .. DSA_MAX_SEQS */
    const int32_t *cu_q;       /* host [B+1]: cumulative query rows, cu_q[0] = 0 */
    const int32_t *cu_k;       /* host [B+1]: cumulative keys in the caches, cu_k[0] = 0 */
    const int32_t *start_pos;  /* host [B]: absolute position of each sequence's first query */
} dsa_seqs;

/* ------------------------------------------------------------------------
 * FP8 quantisation of indexer inputs.
 * Source: config_671B_v3.2.json excerpt on the "DeepSeek-V3.2-Exp - Block
 * input" atlas page (dtype fp8, scale_fmt ue8m0).  The block recipe is a
 * reading of that: a block is 128 consecutive values; its scale is 2^e with
 * e the smallest integer such that amax <= 448 * 2^e, clamped to [-127, 127]
 * (amax = 0 gives e = 0); codes are x / 2^e rounded to nearest-even e4m3,
 * saturating at +-448.
 *
 *   x        [n_blocks * 128] values of x_dtype (DSA_F32 or DSA_BF16)
 *   codes    out [n_blocks * 128] e4m3 codes (4-byte aligned)
 *   scales   out [n_blocks] fp32 scales 2^e
 * Inf and NaN inputs are not supported.
 * Errors: DSA_ERR_INVALID_ARG (null pointer, n_blocks < 0, misaligned codes),
 * DSA_ERR_UNSUPPORTED (x_dtype not F32/BF16), DSA_ERR_CUDA.  n_blocks = 0
 * launches nothing.
 * ---------------------------------------------------------------------- */
int dsa_quant_e4m3_ue8m0(const void *x, int x_dtype, int64_t n_blocks, uint8_t *codes, float *scales,
                         void *stream);

/* ------------------------------------------------------------------------
 * Lightning-indexer scores with the causal mask.
 * Source: DeepSeek-V3.2-Exp atlas page, MoE transformer block, equations
 * S^I_{t,s} and S~^I = S^I + M; the indexer's 64 heads x 128 (nnterp
 * deepseek_v32 page, "Up to 2048 tokens ..." note and printout).
 *
 *   q_idx    [sum T, H_I, D_I] of idx_dtype (F32, BF16, or E4M3 codes)
 *   q_scale  [sum T, H_I] fp32 block scales of q_idx (E4M3 only, else NULL)
 *   k_idx    [sum S, D_I] of idx_dtype
 *   k_scale  [sum S] fp32 block scales of k_idx (E4M3 only, else NULL)
 *   w        [sum T, H_I] fp32 per-head weights
 *   scores   out [sum T, ld_scores] fp32.  Row r (query t of sequence b at
 *            position p) receives columns 0 .. S_b-1: the score for s <= p
 *            and -inf for p < s < S_b.  Columns >= S_b are not written.
 *   ld_scores >= max_b S_b, a multiple of 4 (16-byte rows); scores 16-byte aligned.
 * With E4M3 the factorisation sum_h w s_q ReLU(s_k cq.ck) = s_k sum_h (w s_q)
 * ReLU(cq.ck) holds exactly for positive power-of-two scales, so D_I must be
 * 128 (one block per head row).
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED (H_I > 128 or D_I > 256,
 * E4M3 with D_I != 128), DSA_ERR_CUDA.
 * ---------------------------------------------------------------------- */
int dsa_indexer_scores(const void *q_idx, const float *q_scale, const void *k_idx, const float *k_scale,
                       int idx_dtype, const float *w, int H_I, int D_I, const dsa_seqs *seqs,
                       float *scores, int64_t ld_scores, void *stream);

/* ------------------------------------------------------------------------
 * Top-k selection per query row.
 * Source: DeepSeek-V3.2-Exp atlas page, M^sel_{t,s} = M_{t,s} if
 * s in top_k(S~^I_t); the selection tensor is int32 key indices
 * [batch, query, min(index_topk, seq)] (nnterp deepseek_v32 page).
 *
 *   scores   [sum T, ld_scores] fp32 as written by dsa_indexer_scores; only
 *            columns 0 .. p of row r are read (the causal keys).
 *   k        1 .. 16384
 *   idx      out [sum T, k] int32: the n = min(k, p + 1) causal keys with the
 *            largest scores, then -1 padding.  The exact top-n set is returned;
 *            among keys whose score equals the n-th largest the lower key
 *            indices win.  Order within the row: keys above the threshold
 *            in increasing key order, then the tied keys in increasing order.
 *            NaN scores are not supported.
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_CUDA.
 * ---------------------------------------------------------------------- */
int dsa_topk_select(const float *scores, int64_t ld_scores, const dsa_seqs *seqs, int k, int32_t *idx,
                    void *stream);

/* ------------------------------------------------------------------------
 * Sparse multi-head latent attention over selected keys (absorbed form).
 * Source: DeepSeek-V3.2-Exp atlas page (q^C, k^C = c^KV W_UK, K_i =
 * [K^C_i; k^R], v = c^KV W_UV, M^sel); nnterp deepseek_v32 page (unselected
 * keys masked before the softmax; one rotary key shared by all heads);
 * "DeepSeek-V3.2-Exp - Attention input" page (softmax scale).
 *
 *   q_nope   [sum T, H, d_n]  (dtype)
 *   q_pe     [sum T, H, d_r]  (dtype)
 *   kv_cache latent rows c^KV: row j at kv_cache + j * ld_kv, d_c values (dtype)
 *   k_pe     rotary keys: row j at k_pe + j * ld_pe, d_r values (dtype).  A packed
 *            [sum S, d_c + d_r] cache is k_pe = kv_cache + d_c, ld_pe = ld_kv.
 *   W_UK     [H, d_n, d_c] (dtype): K^C[s,h,d] = sum_c W_UK[h,d,c] c[s,c]
 *   W_UV     [H, d_c, d_v] (dtype): V[s,h,e] = sum_c c[s,c] W_UV[h,c,e]
 *   idx      [sum T, k] int32 key indices local to the row's sequence.  Entries
 *            outside 0 .. min(p, S_b-1) (e.g. the -1 padding) are masked.
 *            Each listed index counts once per occurrence.  NULL selects the
 *            dense causal pattern: entry e of every row is key e (so a row
 *            attends to keys 0 .. min(k, p + 1, S_b) - 1).
 *   softmax_scale  multiplies q.k before the softmax (1/sqrt(d_n + d_r), or the
 *            YaRN-scaled 0.1352 of the released model)
 *   out      out [sum T, H, d_v] (dtype)
 *   lse      out [sum T, H] fp32 natural-log log-sum-exp of the scaled logits,
 *            may be NULL; a row with no live key gets out = 0, lse = -inf.
 *   workspace / ws_bytes  caller scratch, >= dsa_sparse_mla_workspace_size(),
 *            256-byte aligned.
 * Strides are in elements and must keep rows 16-byte aligned.
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_WORKSPACE, DSA_ERR_UNSUPPORTED
 * (dtype E4M3, or dims beyond H <= 256, d_n <= 256, d_r <= 128, d_c <= 1024,
 * d_v <= 256), DSA_ERR_CUDA.
 * ---------------------------------------------------------------------- */
size_t dsa_sparse_mla_workspace_size(int dtype, int H, int d_n, int d_r, int d_c, int d_v, int k,
                                     const dsa_seqs *seqs);
int dsa_sparse_mla_fwd(const void *q_nope, const void *q_pe, int dtype, const void *kv_cache, int64_t ld_kv,
                       const void *k_pe, int64_t ld_pe, const void *W_UK, const void *W_UV, int H, int d_n,
                       int d_r, int d_c, int d_v, const int32_t *idx, int k, const dsa_seqs *seqs,
                       float softmax_scale, void *out, float *lse, void *workspace, size_t ws_bytes,
                       void *stream);

/* ------------------------------------------------------------------------
 * Sparse latent attention over an FP8 latent cache.
 * Source: the "DeepSeek-V3.2-Exp - Block input" page, config_671B_v3.2.json
 * excerpt (dtype fp8, scale_fmt ue8m0), read as the storage format of the
 * latent rows c^KV: e4m3 codes with one power-of-two scale per 128 values,
 * the same block recipe as dsa_quant_e4m3_ue8m0 (which produces them).  The
 * rotary keys k_pe stay bf16.
 *
 * Computes what dsa_sparse_mla_fwd computes on the dequantised latent rows
 * c[s, j] = code[s, j] * kv_scale[s, j / 128] (exact in bf16), with the same
 * arguments except:
 *   kv_codes  [sum S, ld_kv] uint8 e4m3 codes (d_c per row; ld_kv in bytes, a
 *             multiple of 16; 16-byte aligned)
 *   kv_scale  [sum S, d_c / 128] fp32 power-of-two scales
 *   k_pe      [sum S, ld_pe] bf16
 * Only the tensor-core kernel's shapes (H = 128, d_n = 128, d_r = 64,
 * d_c = 512, d_v = 128, bf16 queries and weights) are supported.
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_WORKSPACE, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA.
 * ---------------------------------------------------------------------- */
int dsa_sparse_mla_fwd_fp8kv(const void *q_nope, const void *q_pe, const uint8_t *kv_codes, int64_t ld_kv,
                             const float *kv_scale, const void *k_pe, int64_t ld_pe, const void *W_UK, const void *W_UV,
                             int H, int d_n, int d_r, int d_c, int d_v, const int32_t *idx, int k,
                             const dsa_seqs *seqs, float softmax_scale, void *out, float *lse, void *workspace,
                             size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Sparse latent attention without a caller workspace.
 * The pages have no counterpart to this entry point: it exists for callers
 * that cannot obtain device memory when they run the attention, e.g. a
 * serving runtime that has already handed all of HBM to its own KV-cache
 * pool (a late cudaMalloc would fail or stall every stream), or a plugin
 * called from such a runtime that receives only its input and output
 * tensors.  It computes exactly what dsa_sparse_mla_fwd computes, with the
 * same arguments minus the workspace, using scratch memory that is part of
 * the library's device code (DSA_NOALLOC_SCRATCH_BYTES per device, held until
 * the process exits) instead of a caller buffer.  It allocates nothing.
 *
 *   - Limit: the call needs the same scratch as dsa_sparse_mla_workspace_size()
 *     reports; a call needing more than DSA_NOALLOC_SCRATCH_BYTES returns
 *     DSA_ERR_WORKSPACE and launches nothing.  With the 671B head shapes and
 *     this version's scratch layout that is up to 128 query rows per call,
 *     e.g. one decode step of up to 128 sequences.
 *   - When the scratch is reserved: CUDA loads the library's device code on a
 *     device lazily by default, at the first call of this entry point on that
 *     device, and the scratch is reserved then.  A call with zero query rows
 *     (cu_q[B] = 0) does this set-up and launches nothing.  A caller that
 *     hands the rest of HBM to its own pool makes that first call before
 *     carving the pool (or runs with CUDA_MODULE_LOADING=EAGER, which loads
 *     it with the context); make it before any stream capture as well.
 *   - Every call looks up the scratch's device address for the current
 *     device (a host-side lookup once loaded), so it stays right across a
 *     device reset.
 *   - Every call on a device shares the one scratch array, which keeps the
 *     previous call's contents (the attention writes every scratch byte it
 *     reads, so nothing needs clearing).  Calls that overlap on the GPU --
 *     on different streams, or from several host threads without ordering --
 *     race on it and give wrong results.
 * Errors: as dsa_sparse_mla_fwd, plus DSA_ERR_WORKSPACE beyond the limit.
 * ---------------------------------------------------------------------- */
#define DSA_NOALLOC_SCRATCH_BYTES (64u << 20)
int dsa_sparse_mla_fwd_noalloc(const void *q_nope, const void *q_pe, int dtype, const void *kv_cache,
                               int64_t ld_kv, const void *k_pe, int64_t ld_pe, const void *W_UK, const void *W_UV,
                               int H, int d_n, int d_r, int d_c, int d_v, const int32_t *idx, int k,
                               const dsa_seqs *seqs, float softmax_scale, void *out, float *lse, void *stream);

/* ------------------------------------------------------------------------
 * The step before the path: the key side of the new tokens, appended to the
 * caches.
 * Sources: "DeepSeek-V3.2-Exp - Attention input" page, mla-init and mla-kv
 * excerpts (kv = wkv_a(x); split into kv_lora_rank + qk_rope_head_dim;
 * kv_norm; apply_rotary_emb on k_pe with freqs_cis); "DeepSeek-V3.2-Exp -
 * Block input" page, RMSNorm excerpt (float32 compute, one gain per feature,
 * eps 1e-6); nnterp deepseek_v32 printout (indexer wk 7168 -> 128, k_norm
 * LayerNorm(128, eps 1e-6, gain and bias), weights_proj 7168 -> 64) and its
 * note that the rotary part is served de-interleaved.
 *
 * For token t of sequence b (position p = start_pos[b] + t, cache row
 * j = cu_k[b] + p), with Y = x . W_proj^T kept in fp32:
 *   kv_cache[j, 0 .. d_c-1]       = bf16(kv_gain * Y[0:d_c] / sqrt(mean(Y[0:d_c]^2) + 1e-6))
 *   kv_cache[j, d_c + i]          = bf16(a cos_i - b sin_i)   with (a, b) = Y[d_c + 2i], Y[d_c + 2i + 1]
 *   kv_cache[j, d_c + d_r/2 + i]  = bf16(a sin_i + b cos_i)   (cos_i, sin_i of position p)
 *   k^I = bf16(LayerNorm(Y[d_c+d_r : +D_I]) * k_gain + k_bias)  (mean, biased variance, eps 1e-6)
 *   k_cache[j] = k^I (bf16), or its e4m3 codes with k_scale[j] as
 *                dsa_quant_e4m3_ue8m0 computes them from the bf16 k^I
 *   w[r, :]    = Y[d_c+d_r+D_I : +H_I]   (r = cu_q[b] + t, the indexer's weights)
 *
 *   x          [sum T, dim] bf16: the new tokens as the attention receives them
 *   W_proj     [d_c + d_r + D_I + H_I, dim] bf16: the rows of wkv_a, then of
 *              wk, then of weights_proj (nn.Linear layout, stacked)
 *   kv_gain    [d_c] fp32; k_gain, k_bias [D_I] fp32
 *   rope_cos, rope_sin  [n_pos, d_r/2] fp32: cos and sin of the angle of
 *              frequency i at position p (row p); every appended position
 *              must be < n_pos
 *   kv_cache   [sum S, ld_kv] bf16, ld_kv >= d_c + d_r (rows written: the
 *              appended ones only)
 *   k_cache    [sum S, D_I] of k_dtype (DSA_BF16, or DSA_E4M3 with D_I = 128
 *              and k_scale [sum S] fp32)
 *   w          out [sum T, H_I] fp32
 *   workspace  >= dsa_kv_prologue_workspace_size(), 256-byte aligned (the fp32 Y)
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED (dim or the stacked width
 * not a multiple of 64, odd d_r, D_I > 256), DSA_ERR_WORKSPACE, DSA_ERR_CUDA.
 * ---------------------------------------------------------------------- */
size_t dsa_kv_prologue_workspace_size(int dim, int d_c, int d_r, int D_I, int H_I, const dsa_seqs *seqs);
int dsa_kv_prologue(const void *x, int dim, const void *W_proj, const float *kv_gain, const float *k_gain,
                    const float *k_bias, const float *rope_cos, const float *rope_sin, int n_pos, int d_c, int d_r,
                    int D_I, int H_I, const dsa_seqs *seqs, void *kv_cache, int64_t ld_kv, void *k_cache, int k_dtype,
                    float *k_scale, float *w, void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The step after the path: the output projection y = out . wo^T.
 * Source: "DeepSeek-V3.2-Exp - Attention input" page, mla-init excerpt (wo maps
 * n_heads * v_head_dim to dim); nnterp deepseek_v32 printout (o_proj,
 * 16384 -> 7168, reading every head's output side by side).
 *
 *   out   [M, in_features] bf16: the attention output [M, H, d_v] viewed as
 *         [M, H * d_v]
 *   wo    [d_model, in_features] bf16 (nn.Linear layout)
 *   y     out [M, d_model] bf16
 * in_features and d_model multiples of 64; pointers 16-byte aligned.  fp32
 * accumulation on the tensor cores.
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA.
 * ---------------------------------------------------------------------- */
int dsa_output_proj(const void *out, const void *wo, int M, int in_features, int d_model, void *y, void *stream);

/* ------------------------------------------------------------------------
 * The whole path: [quantise] -> indexer -> top-k -> sparse latent attention.
 * Sources: as for the three stages above.  Rows are processed in chunks so
 * that the fp32 score buffer stays bounded; the workspace size covers one
 * chunk of scores, the selection (unless idx_out is given), the FP8 copies
 * of q^I / k^I (idx_fp8) and the attention scratch.
 * When every row's causal prefix holds at most top_k keys (k >= S, the case
 * the deepseek_v32 note on the nnterp page calls plain causal attention), the
 * selection is every causal key and is known without scores: the quantiser,
 * indexer and top-k are not launched, the attention reads the dense causal
 * pattern, and idx_out (when given) is filled with 0 .. n-1 and -1 padding,
 * exactly what the top-k writes for such rows.
 * ---------------------------------------------------------------------- */
typedef struct dsa_problem {
    /* shapes */
    int32_t H_I, D_I, top_k;          /* indexer heads, head dim, k */
    int32_t H, d_n, d_r, d_c, d_v;    /* MLA heads and widths */
    int32_t dtype;                    /* DSA_F32 or DSA_BF16: storage type of every tensor below but w */
    int32_t idx_fp8;                  /* 1: quantise q^I, k^I to e4m3 + ue8m0 before the indexer */
    float softmax_scale;
    /* indexer inputs */
    const void *q_idx;                /* [sum T, H_I, D_I] */
    const void *k_idx;                /* [sum S, D_I] */
    const float *w;                   /* [sum T, H_I] fp32 */
    /* attention inputs (layouts as in dsa_sparse_mla_fwd) */
    const void *q_nope, *q_pe;
    const void *kv_cache;
    int64_t ld_kv;
    const void *k_pe;
    int64_t ld_pe;
    const void *W_UK, *W_UV;
    /* outputs */
    void *out;                        /* [sum T, H, d_v] (dtype) */
    float *lse;                       /* [sum T, H] or NULL */
    int32_t *idx_out;                 /* [sum T, top_k] or NULL (then kept in the workspace) */
    /* The step after the path, optional (NULL wo: not applied): the output
     * projection y = out wo^T ("DeepSeek-V3.2-Exp - Attention input" page,
     * mla-init excerpt, wo: n_heads * v_head_dim -> dim).  W_UV and wo run
     * chunk by chunk (2048 rows), so each chunk of the attention output is read
     * back from L2 right after it is written.  `out` may then be NULL (the
     * chunks live in the workspace).  bf16 only; d_model and H * d_v multiples
     * of 64. */
    const void *wo;                   /* [d_model, H * d_v] */
    int32_t d_model;
    void *y;                          /* out [sum T, d_model] */
    /* FP8 latent cache (as dsa_sparse_mla_fwd_fp8kv): kv_fp8 = 1 makes kv_cache
     * e4m3 codes with ld_kv in bytes (a multiple of 16) and kv_scale their
     * [sum S, d_c / 128] fp32 block scales; k_pe stays bf16.  bf16 only, at
     * the tensor-core kernel's head shapes. */
    int32_t kv_fp8;
    const float *kv_scale;
} dsa_problem;

size_t dsa_forward_workspace_size(const dsa_problem *p, const dsa_seqs *seqs);
int dsa_forward(const dsa_problem *p, const dsa_seqs *seqs, void *workspace, size_t ws_bytes, void *stream);

/* The forward from HOST buffers: the end-to-end call of one step.  On `stream`
 * it copies the step's inputs from host memory into the device buffers that
 * `p` names, runs dsa_forward, and copies the results back: one
 * cudaMemcpyAsync per input and output; the appended cache rows of each array
 * go in one copy to the start of `workspace` and a small kernel puts them in
 * their rows (the workspace is free until the forward starts) -- or, when that
 * staging does not fit the workspace or a row is not a multiple of 16 bytes,
 * one copy per sequence and array.  q_nope and q_pe, which only the attention
 * stage reads, are copied last and on a side stream of the library's (one per
 * host thread and device, created on first use and kept): their transfer
 * overlaps the quantiser, indexer and top-k, and the attention stage waits for
 * it on `stream`.  Everything else is enqueued on `stream`.  With
 * page-locked (pinned) host buffers every copy is asynchronous and the call
 * returns once all the work is enqueued; the caller synchronises `stream`
 * before reading the host outputs.  Pageable host memory also works, but then
 * the copies block the calling thread.
 *
 * Host inputs (NULL: the device buffer already holds that data):
 *   q_idx, w, q_nope, q_pe   the step's queries, laid out as the device tensors
 *                            of `p` ([sum T, ...] rows, dense);
 *   kv_new                   the cache rows the step appends: for every
 *                            sequence b in order, its rows start_pos[b] ..
 *                            S_b - 1 (S_b = cu_k[b+1] - cu_k[b]), each a full
 *                            row of ld_kv elements (bytes for an e4m3 cache),
 *                            written to cache rows cu_k[b] + start_pos[b] ..;
 *   k_pe_new                 the same rows of k_pe (ld_pe elements each); NULL
 *                            when k_pe lies inside the kv_cache rows that
 *                            kv_new already carries;
 *   k_idx_new                the same rows of the indexer key cache (D_I each);
 *   kv_scale_new             e4m3 cache: the same rows' d_c / 128 scales.
 * Host outputs (NULL: not copied back): out (y when p->wo is set: the
 * projected output), lse, idx (requires p->idx_out).
 * Pipelining (all NULL: none), four cudaEvent_t handles: copy_after, which
 * the input copies wait for (cudaStreamWaitEvent before the first of them);
 * copy_done, recorded once the input copies (on both streams) and the append
 * kernel are enqueued; compute_after, which the forward waits for after that;
 * and compute_done, recorded once the forward's kernels are enqueued, before
 * the output copies.  Calls on two streams with their own device buffers can
 * so chain their forwards (each waits for the previous call's compute_done)
 * while one call's copies overlap the other's kernels, and chain their input
 * copies (each waits for the previous call's copy_done) so that two calls'
 * inputs do not share the host-to-device bandwidth: the first forward then
 * waits for one call's inputs instead of two calls'.
 * Every check dsa_forward makes runs before the first copy is enqueued, so a
 * refused call changes no device buffer.
 * Returns what dsa_forward returns, DSA_ERR_INVALID_ARG when a sequence has
 * start_pos[b] > S_b with kv_new, k_pe_new, k_idx_new or kv_scale_new given, or
 * when a requested output has no device buffer in `p`, and DSA_ERR_CUDA when
 * a copy cannot be enqueued. */
typedef struct dsa_host_io {
    const void *q_idx, *w, *q_nope, *q_pe;
    const void *kv_new, *k_pe_new, *k_idx_new;
    const float *kv_scale_new;
    void *out;
    float *lse;
    int32_t *idx;
    void *compute_after, *compute_done;
    void *copy_after, *copy_done;
} dsa_host_io;
int dsa_forward_host(const dsa_problem *p, const dsa_seqs *seqs, const dsa_host_io *io, void *workspace,
                     size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Speculative decoding over a served latent cache (the pages have no
 * counterpart to these four entry points): the heads' norm and rotation at a
 * draft tree's positions, the cache written (and quantised) and read back by
 * token position, and the attention of the tree's nodes over it.
 * A call captured in a graph replays the lengths (cu_q, cu_k, start_pos) that it
 * was captured with; everything in device memory (values, positions given as
 * `pos`, masks, block tables, caches) is read at each replay.
 * ---------------------------------------------------------------------- */

/* Where a sequence's tokens sit in a cache cut into pages of page_size rows:
 * token s of sequence b is row block_table[b * ld_table + s / page_size] *
 * page_size + s % page_size.  Wherever an entry point takes a `pages` pointer,
 * NULL means a contiguous cache: token s of sequence b is row cu_k[b] + s.
 * With pages, cu_k gives only the sequences' lengths.  Entries of tokens that
 * a call does not touch are not read.  An entry outside 0 .. n_pages - 1 (e.g.
 * -1) names no page: nothing is written there, it reads as zeros, and the
 * attention masks its tokens. */
typedef struct dsa_pages {
    const int32_t *block_table;   /* device [B, ld_table] */
    int64_t ld_table;             /* row stride in entries, >= width */
    int64_t width;                /* entries of a sequence */
    int32_t page_size;            /* rows of a page: a multiple of 16 */
    int32_t n_pages;              /* pages of the cache: n_pages * page_size <= rows */
} dsa_pages;

/* A latent cache.  The storage type is DSA_F32 or DSA_BF16 values, or DSA_E4M3:
 * codes with one power-of-two scale per 128 values (the block recipe of
 * dsa_quant_e4m3_ue8m0) and bf16 rotary keys.  Rows start 16-byte aligned
 * (base and stride). */
typedef struct dsa_latent_cache {
    void *kv;                     /* [rows, ld_kv]: d_c values or codes per row */
    int64_t ld_kv;                /* elements (bytes for E4M3) */
    float *kv_scale;              /* E4M3: [rows, d_c / 128] powers of two; else NULL */
    void *k_pe;                   /* [rows, ld_pe]: d_r rotary key values per row (may lie inside kv's rows) */
    int64_t ld_pe;                /* elements */
    int32_t dtype;                /* DSA_F32, DSA_BF16 or DSA_E4M3 */
    int64_t rows;                 /* rows of every array, < 2^31 - 64 */
} dsa_latent_cache;

/* Writes the new tokens' latent rows and rotary keys into the cache, quantising
 * them on the way when it holds E4M3.  Row r = cu_q[b] + t of c_kv and k_pe
 * becomes token start_pos[b] + t of sequence b; every other row of the cache
 * stays as it was.
 *   c_kv   [sum T, ld_c] of x_dtype (DSA_F32 or DSA_BF16), d_c values per row
 *   k_pe   [sum T, ld_x] of x_dtype, d_r values per row (NULL when d_r = 0)
 * Values are rounded once, to nearest even; a DSA_F32 cache holds bf16 inputs
 * exactly.  E4M3 codes and scales are those that dsa_quant_e4m3_ue8m0 gives for
 * the same values; Inf and NaN are not supported there.  Inputs must not
 * overlap the cache.  Tokens that share a row (two sequences with one page)
 * leave that row unspecified.
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED (d_c > 1024, d_r > 128, E4M3
 * with d_c not a multiple of 128, sum T not below 2^31 - 1024), DSA_ERR_CUDA. */
int dsa_latent_cache_write(const void *c_kv, int64_t ld_c, const void *k_pe, int64_t ld_x, int x_dtype, int d_c, int d_r,
                           const dsa_latent_cache *cache, const dsa_seqs *seqs, const dsa_pages *pages, void *stream);

/* Reads tokens of the cache back as dense rows, dequantised.  Row r = cu_q[b] + t
 * is token pos[r] of sequence b, or start_pos[b] + t when pos is NULL; a pos
 * outside 0 .. S_b - 1 gives a row of zeros.  The same token may be read more
 * than once.
 *   pos    device [sum T] int32, or NULL
 *   c_kv   out [sum T, ld_c] of out_dtype (DSA_F32 or DSA_BF16), d_c values per row
 *   k_pe   out [sum T, ld_x] of out_dtype, d_r values per row (NULL when d_r = 0)
 * code * scale is exact in both types unless it leaves the type's normal range.
 * Outputs must not overlap the cache.
 * Errors: as dsa_latent_cache_write. */
int dsa_latent_cache_read(const dsa_latent_cache *cache, int d_c, int d_r, const dsa_seqs *seqs, const dsa_pages *pages,
                          const int32_t *pos, void *c_kv, int64_t ld_c, void *k_pe, int64_t ld_x, int out_dtype,
                          void *stream);

/* Attention of drafted tokens over the cache, in absorbed form.  The T_b query
 * rows of sequence b are the nodes of a tree whose root is token start_pos[b] - 1;
 * node j's key is token start_pos[b] + j of the cache (written there
 * beforehand).  A node sees every token before start_pos[b] and the nodes whose
 * bit its mask sets (its ancestors and itself):
 *   z[r,h,s] = softmax_scale (q~[r,h] . c[s] + q_pe[r,h] . k_pe[s]),  q~ = q_nope W_UK
 *   out[r,h] = (sum_s softmax_s(z) c[s]) W_UV,  lse = log sum_s exp(z)
 *   q_nope, q_pe, W_UK, W_UV, out, lse   as in dsa_sparse_mla_fwd (dense, dtype)
 *   tree_mask   device [sum T, mask_words] 64-bit words: bit j % 64 of word j / 64
 *               of a row is node j of the row's own sequence (bits of nodes >= T_b
 *               are ignored; T_b <= 64 mask_words); NULL: node t sees nodes 0 .. t
 *               (a chain: one token, or a prompt chunk)
 * A row that sees nothing gets out = 0, lse = -inf.  What a row does not see never
 * reaches it, whatever its bits (stale rows, Inf, NaN).  A row that sees a NaN is
 * NaN; visible Inf (a code times its scale too), E4M3 NaN codes and E4M3 scales that
 * are no finite power of two are not supported.  Scores and sums are fp32, the sums
 * with weights of up to 2^8 before they are divided by the row sum: visible latents
 * count in full at any finite size, but may overflow in the sum where their size times
 * the number of tokens passes 2^119.  softmax_scale is finite, also times log2(e); 0
 * and negative values are allowed.  Contiguous or paged cache (`pages`), of dtype's
 * own type, or E4M3 with dtype DSA_BF16.
 * Two kernels: tensor cores for bf16 at d_n = 128, d_r = 64, d_c = 512, d_v = 128
 * and H up to 256; a generic one for everything else within the limits of
 * dsa_sparse_mla_fwd (E4M3: d_c a multiple of 128).  start_pos[b] + T_b < 2^31 - 256,
 * sum T * H < 2^31 - 256.
 * All pointers 16-byte aligned (kv_scale too); workspace as in dsa_sparse_mla_fwd, its size
 * depends on the sequences and the current device (calls captured in graphs that may run at the same
 * time need workspaces of their own).
 * Errors: DSA_ERR_INVALID_ARG, DSA_ERR_WORKSPACE, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA. */
size_t dsa_tree_mla_workspace_size(int dtype, int H, int d_n, int d_r, int d_c, int d_v, const dsa_seqs *seqs);
int dsa_tree_mla_fwd(const void *q_nope, const void *q_pe, int dtype, const dsa_latent_cache *cache, const void *W_UK,
                     const void *W_UV, int H, int d_n, int d_r, int d_c, int d_v, const uint64_t *tree_mask,
                     int mask_words, const dsa_seqs *seqs, const dsa_pages *pages, float softmax_scale, void *out,
                     float *lse, void *workspace, size_t ws_bytes, void *stream);

/* The heads of one tensor for dsa_head_norm_rope: head h of row r starts at
 * x + r * ld_x + h * hd_x (elements), and likewise for y and y_pe. */
typedef struct dsa_heads {
    const void *x;
    int64_t ld_x, hd_x;
    int32_t n_heads;              /* 0: none (everything else is then ignored) */
    int32_t norm;                 /* DSA_NORM_* */
    const float *gain, *bias;     /* [D] fp32, NULL: 1 and 0 */
    void *y;                      /* all D dims, or with y_pe the D - d_r unrotated ones */
    int64_t ld_y, hd_y;
    void *y_pe;                   /* the d_r rotated dims, or NULL: they stay in their place in y */
    int64_t ld_pe, hd_pe;
} dsa_heads;
#define DSA_NORM_NONE  0
#define DSA_NORM_RMS   1          /* x / sqrt(mean x^2 + eps) * gain */
#define DSA_NORM_LAYER 2          /* (x - mean) / sqrt(var + eps) * gain + bias (biased variance) */
#define DSA_ROPE_PAIRS  0         /* pair (2i, 2i+1) -> dims i and d_r/2 + i (the order the caches hold) */
#define DSA_ROPE_HALVES 1         /* pair (i, d_r/2 + i) stays in place */

/* Norms every head of the queries q and keys k and rotates its d_r rotary dims to
 * the row's position, in one pass: (a, b) -> (a cos_i - b sin_i, a sin_i + b cos_i)
 * for pair i.  The rotary dims are the last d_r of the D, or the first with
 * rope_first.  Norm and rotation in fp32, rounded once to y_dtype.
 *   q, k        either may be NULL (or have n_heads 0)
 *   x_dtype, y_dtype   DSA_F32 or DSA_BF16
 *   rope_cos, rope_sin [n_pos, d_r / 2] fp32
 *   pos         device [sum T] int32 positions (a draft node's start + depth), or
 *               NULL: start_pos[b] + t.  An entry outside 0 .. n_pos - 1 leaves
 *               its row unrotated (padding)
 * y may be x itself (same address, strides and type, y_pe NULL); otherwise
 * outputs overlap neither inputs nor each other.
 * Errors: DSA_ERR_INVALID_ARG (odd d_r, d_r > D, a position that start_pos gives
 * outside the tables, y_pe with d_r = 0), DSA_ERR_UNSUPPORTED (D > 512, dtype,
 * norm or rope of another kind, sum T or the heads of q and k together not below 2^31 - 1024), DSA_ERR_CUDA. */
int dsa_head_norm_rope(const dsa_heads *q, const dsa_heads *k, int x_dtype, int y_dtype, int D, int d_r, int rope_first,
                       int rope, float eps, const float *rope_cos, const float *rope_sin, int n_pos,
                       const int32_t *pos, const dsa_seqs *seqs, void *stream);

/* ------------------------------------------------------------------------
 * From the attention's output to the next token.
 * No reference code: the pages name the layers (nnterp deepseek_v32 printout: the
 * Linear modules of the attention and the two norms of a block), the operators
 * are those that every server needs between two attentions and after the last.
 * ---------------------------------------------------------------------- */
#define DSA_ACT_NONE      0
#define DSA_ACT_RELU      1       /* max(v, 0) */
#define DSA_ACT_SILU      2       /* v / (1 + exp(-v)) */
#define DSA_ACT_GELU      3       /* v / 2 (1 + erf(v / sqrt 2)) */
#define DSA_ACT_GELU_TANH 4       /* v / 2 (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) */
#define DSA_ACT_SIGMOID   5       /* 1 / (1 + exp(-v)): gates only */

/* A linear layer, y = act(x W^T + bias) + residual, in fp32 up to one rounding to
 * y's type.
 *   x         [M, K] of dtype (DSA_BF16 or DSA_F32), row stride ld_x elements
 *   W         [N, K] of dtype (nn.Linear layout), row stride ld_w
 *   bias      [N] fp32 or NULL
 *   residual  [M, N] of y's type, row stride ld_r, or NULL
 *   y         out [M, N] of y_dtype (DSA_BF16 or DSA_F32), row stride ld_y; may be
 *             residual itself (same address and stride), otherwise overlaps no input
 * Any sizes and strides of whole elements.  bf16 rows that start on 16 bytes go to
 * the tensor cores as they are; others, and fp32 values (as three bf16 terms each,
 * six products of them), are laid out in the workspace first, but for few tokens or
 * little work.  The tensor cores cut off, step by step of 16 products, what a sum of
 * 24 bits does not hold; an fp32 y is added up from parts of at most 32 such steps,
 * a bf16 y is one sum over K (1.9e-5 of the whole at K = 16384, before it is rounded
 * to 2^-8).  Measured over K of 64 to 16384 on values of a normal distribution, an
 * fp32 y is off by at most 4.8e-7 of the whole from bf16 and 2.5e-7 from fp32 (fp32
 * arithmetic: 0.5e-7 to 15e-7 and 1.4e-7 to 23e-7, growing with K).  In fp32 a product
 * with an infinity may be NaN where a call has more tokens than the CUDA cores take
 * (4, or up to 64 with little work; these give the infinity), so it may differ with
 * the size of the batch, and terms of values below 2^-100 may be lost.
 * The workspace size depends on all that it is given here (0 where none is needed);
 * calls that overlap need a workspace each.
 * Errors: DSA_ERR_INVALID_ARG (null pointer, sizes below M >= 0, N, K >= 1, an
 * address off its element, rows of an output that overlap), DSA_ERR_UNSUPPORTED
 * (dtype, act, M, N or K not below 2^31 - 1024), DSA_ERR_WORKSPACE, DSA_ERR_CUDA. */
size_t dsa_linear_workspace_size(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N, int K);
int dsa_linear(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N, int K,
               const float *bias, int act, const void *residual, int64_t ld_r, void *y, int64_t ld_y, int y_dtype,
               void *workspace, size_t ws_bytes, void *stream);

/* One norm of dsa_block_norm: DSA_NORM_*, gain and bias [D] fp32 (NULL: 1 and 0;
 * the bias goes with DSA_NORM_LAYER only). */
typedef struct dsa_norm {
    int32_t kind;
    const float *gain, *bias;
} dsa_norm;

/* The norms on both sides of a block with its gate and its residual, row by row:
 *   h' = skip h + scale act(gate) norm_post(u),   y = norm_pre(h')
 * in fp32 (sigmoid and SiLU by a quotient good to 2 units in the last place; where
 * h' and y are both bf16 also by an exponential good to 2^-16); h' and y are each
 * rounded once, y comes from the unrounded h'. */
typedef struct dsa_block_norm_args {
    int64_t rows;                 /* >= 0 */
    int32_t D;                    /* values a row, 1 .. 16384 */
    int32_t h_dtype, x_dtype;     /* DSA_F32 or DSA_BF16: of h and h_out; of u, gate and y */
    const void *h;                /* [rows, D], row stride ld_h: the residual stream */
    int64_t ld_h;
    const void *u;                /* [rows, D], row stride ld_u: what the block gave; NULL: h' = skip h */
    int64_t ld_u;
    const void *gate;             /* [rows, D], row stride ld_gate (0: one row for all); NULL: 1 */
    int64_t ld_gate;
    int32_t gate_act;             /* DSA_ACT_NONE, DSA_ACT_SIGMOID or DSA_ACT_SILU */
    dsa_norm post, pre;           /* of u; of h' */
    float skip, scale, eps;       /* eps of both norms, >= 0 */
    void *h_out;                  /* out [rows, D], row stride ld_ho, or NULL; may be h (same stride) */
    int64_t ld_ho;
    void *y;                      /* out [rows, D], row stride ld_y, or NULL; may be u (same stride) */
    int64_t ld_y;
} dsa_block_norm_args;
/* Errors: DSA_ERR_INVALID_ARG (neither h_out nor y, gate or post norm without u, an
 * address off its element, rows of an output that overlap, other overlaps that the
 * addresses show), DSA_ERR_UNSUPPORTED (D > 16384, dtype, norm or gate_act of another
 * kind), DSA_ERR_CUDA. */
int dsa_block_norm(const dsa_block_norm_args *args, void *stream);

/* The next token of every row of logits, from given random numbers.  With z_i =
 * l_i / temperature and w_i = exp(z_i - max z), tokens in the order of falling l (equal
 * ones by rising index):
 *   1. the first top_k tokens are kept,
 *   2. of these the shortest run from the start whose sum reaches top_p times theirs,
 *   3. of these the ones with w_i >= min_p; the first one always is,
 * and token = the lowest kept index whose running sum of kept weights (in the order of
 * the indices) exceeds u times their whole sum.
 *   logits       [R, V] of dtype (DSA_F32 or DSA_BF16), row stride ld; V 1 .. 262144
 *   u            [R] fp32 in [0, 1); a value outside (or NaN) counts as the nearest inside (0)
 *   temperature  [R] fp32; below 1e-5 (or NaN): top_k is 1.  NULL: 1
 *   top_k        [R] int32; <= 0: no such limit.  NULL: none
 *   top_p        [R] fp32; >= 1 or NaN: no such limit, <= 0: the first token.  NULL: none
 *   min_p        [R] fp32; <= 0 or NaN: no such limit.  NULL: none
 *   token        out [R] int32
 *   logprob      out [R] fp32: ln of the token's share of the kept sum; NULL: not wanted
 *   kept         out [R] int32: how many tokens were kept; NULL: not wanted
 * -inf and NaN are never taken (a mask): a row of nothing else gives token -1, logprob
 * -inf and kept 0.  Where a logit is +inf, those are the only ones, with equal weights.
 * Sums are of whole numbers: weights in steps of 2^-45, each off by less than 2^-40 of
 * itself and half a step, so that the order of summation is nothing and the same inputs
 * give the same token.  The logits' differences count as far as fp32 holds them.
 * A row whose logits have not arrived within the wait limit (dsa_check_device_error tells)
 * gives what a row without a token gives.
 * Errors: DSA_ERR_INVALID_ARG (null pointer, R < 0, V < 1, an address off its element),
 * DSA_ERR_UNSUPPORTED (dtype, V > 262144), DSA_ERR_CUDA. */
int dsa_sample(const void *logits, int64_t ld, int dtype, int R, int V, const float *u, const float *temperature,
               const int32_t *top_k, const float *top_p, const float *min_p, int32_t *token, float *logprob,
               int32_t *kept, void *stream);

/* ------------------------------------------------------------------------
 * Status and diagnostics.
 * ---------------------------------------------------------------------- */
/* Human-readable name of a dsa_status. */
const char *dsa_status_string(int status);
/* The cudaError_t behind the most recent DSA_ERR_CUDA on this host thread. */
int dsa_last_cuda_error(void);
/* Waits for `stream`, then reads and clears the device error word that the
 * kernels' bounded waits set.  Returns DSA_OK, DSA_ERR_TIMEOUT (and stores
 * the recorded site in *site when non-NULL), or DSA_ERR_CUDA.  This is the
 * only entry point that synchronises. */
int dsa_check_device_error(void *stream, int *site);
/* Self-test of the failure-detection path (no counterpart on the pages: a
 * diagnostic of this library).  Launches, on `stream`, one CTA that waits on an
 * mbarrier phase that nothing completes, through the same bounded wait every
 * tensor-core kernel here uses, with a limit of `limit_cycles` SM clock cycles
 * (1 .. 2^32) instead of the kernels' ~2 s.  The wait gives up, records site 90
 * in the device error word and returns; the CTA then completes the phase and
 * checks that a second wait on it succeeds, writing 1 to *completed_ok (a device
 * int, may be NULL) when both behaved.  The GPU does not fault or hang: the
 * caller reads the outcome with dsa_check_device_error (DSA_ERR_TIMEOUT, site
 * 90), after which the context is usable as before.  Returns DSA_ERR_INVALID_ARG
 * for a limit out of range. */
int dsa_selftest_bounded_wait(int64_t limit_cycles, int *completed_ok, void *stream);
/* Wait limit of the tensor-core kernels (no counterpart on the pages: a
 * diagnostic of this library).  Every wait of the indexer, absorption,
 * attention, product and sampling kernels on a barrier phase gives up after this
 * many SM clock cycles (default, and `cycles` = 0: 2^32, about two seconds),
 * records its site in the device error word, and the CTA drains its copies and
 * MMAs already in flight
 * (those drain waits keep the default limit), frees its tensor memory and exits.
 * A short limit makes the failure path of the production kernels run without a
 * fault: the next dsa_check_device_error returns DSA_ERR_TIMEOUT with the site,
 * the outputs of the calls made meanwhile are undefined, and calls made after
 * the limit is restored behave normally.  The setting is process-wide and read
 * when a kernel is launched.  Returns DSA_ERR_INVALID_ARG for cycles < 0 or
 * above the default. */
int dsa_set_wait_limit(int64_t cycles);
/* Selects, for dsa_forward calls that follow, between the two implementations
 * of the indexer + top-k on batches of at least 304 groups of 4 query rows
 * (no counterpart on the pages: a choice of this library).  Fused: one
 * persistent kernel scores a group into a per-SM slot and selects its rows'
 * top-k from it while the next group is scored, with no [rows, S] score
 * buffer; two kernels: the indexer writes chunks of fp32 score rows and a
 * separate top-k kernel selects from them.  Both give identical selections.
 * mode 1: fused wherever it applies; 0: never; -1 (default): where it measured
 * faster, the FP8 indexer over rows that see on average >= 16384 keys.
 * Process-wide.  Returns DSA_ERR_INVALID_ARG for another mode. */
int dsa_set_fused_topk(int mode);
/* Bit mask of the kernels the last entry point launched on this host thread
 * (DSA_KERNEL_* bits), and how many kernel launches it made. */
uint32_t dsa_last_kernels(void);
int dsa_last_launch_count(void);

/* Optional timing hook.  When `events` is non-NULL, dsa_forward records
 * events[i] (cudaEvent_t handles created by the caller) on its stream at
 * these stage boundaries:
 *   0 start, 1 after FP8 quantisation, 2 after the indexer + top-k loop,
 *   3 after q~ = q_nope W_UK, 4 after the sparse attention (and its
 *   split-key combine), 5 after o_lat W_UV (the end).
 * n_events must be DSA_STAGE_EVENTS.  Pass NULL to switch it off.  The setting
 * is per host thread.  Returns DSA_ERR_INVALID_ARG for a wrong count. */
#define DSA_STAGE_EVENTS 6
int dsa_set_stage_events(void *const *events, int n_events);

#define DSA_KERNEL_QUANT        (1u << 0)
#define DSA_KERNEL_INDEXER_SIMT (1u << 1)
#define DSA_KERNEL_INDEXER_TC   (1u << 2)
#define DSA_KERNEL_INDEXER_FP8  (1u << 3)
#define DSA_KERNEL_TOPK         (1u << 4)
#define DSA_KERNEL_ABSORB_SIMT  (1u << 5)
#define DSA_KERNEL_ABSORB_TC    (1u << 6)
#define DSA_KERNEL_MLA_SIMT     (1u << 7)
#define DSA_KERNEL_MLA_TC       (1u << 8)
#define DSA_KERNEL_COMBINE      (1u << 9)
#define DSA_KERNEL_SELFTEST     (1u << 10)
#define DSA_KERNEL_DENSE_IDX    (1u << 11)
#define DSA_KERNEL_GEMM_TC      (1u << 12)
#define DSA_KERNEL_PROLOGUE     (1u << 13)
#define DSA_KERNEL_INDEXER_TOPK (1u << 14)  /* the indexer launch also selected the top-k (fused) */
#define DSA_KERNEL_APPEND       (1u << 15)  /* dsa_forward_host put staged cache rows in place */
#define DSA_KERNEL_CACHE_WRITE  (1u << 16)
#define DSA_KERNEL_CACHE_READ   (1u << 17)
#define DSA_KERNEL_TREE_SIMT    (1u << 18)
#define DSA_KERNEL_TREE_TC      (1u << 19)
#define DSA_KERNEL_TREE_COMBINE (1u << 20)
#define DSA_KERNEL_HEAD_NORM    (1u << 21)
#define DSA_KERNEL_LINEAR       (1u << 22)
#define DSA_KERNEL_LINEAR_LAYOUT (1u << 23)  /* x or W laid out in the workspace first */
#define DSA_KERNEL_LINEAR_SIMT  (1u << 24)
#define DSA_KERNEL_BLOCK_NORM   (1u << 25)
#define DSA_KERNEL_SAMPLE       (1u << 26)

#ifdef __cplusplus
}
#endif

#endif /* DSA_H */
