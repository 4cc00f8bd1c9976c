/*
 * h3enc op-level entry points: each step of the encode as its own call, for
 * parity tests and kernel benchmarks.  The encode (h3enc.h) launches exactly
 * these kernels.  All pointers are device pointers unless marked HOST; all
 * matrices are row-major bf16 with the stated leading dimension; `stream` is
 * a cudaStream_t (NULL = legacy default).  `status` is an optional device
 * int32 that kernels OR error bits into (1 = bounded wait ran out, 2 = index
 * out of bounds, 4 = visual count mismatch); NULL disables recording.
 * Return: H3ENC_OK, H3ENC_ERR_INVALID_ARG (checked before launch) or
 * H3ENC_ERR_CUDA (launch failed).
 */
#ifndef H3ENC_OPS_H
#define H3ENC_OPS_H

#include <stdint.h>
#include "h3enc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* GEMM epilogues of the projection kernel C = A * W^T (fp32 accumulation). */
enum {
    H3ENC_EPI_STORE = 0,       /* C = bf16(acc)                                   (QKV projection) */
    H3ENC_EPI_RESIDUAL = 1,    /* C = bf16(R + acc); R may equal C                (o_proj + residual) */
    H3ENC_EPI_SWIGLU = 2,      /* W packed by h3enc_op_pack_gate_up (N = 2*I rows):
                                  C[:, i] = bf16(silu(gate_i) * up_i), C has I columns (gate/up + SwiGLU) */
    H3ENC_EPI_RESIDUAL_DS = 3, /* C = bf16(R + acc), then at rows with vis_rank[r] = j in [0, n_vis):
                                  C = bf16(C + DS[j])                             (down_proj + residual + DeepStack) */
    H3ENC_EPI_GELU_TANH = 5,   /* C = bf16(gelu_tanh(acc + bias))                 (vision MLP fc1) */
    H3ENC_EPI_GELU_ERF = 6     /* C = bf16(gelu(acc + bias)), exact erf form      (vision merger fc1) */
};

/* Projection GEMM on the tcgen05 tensor cores (page "vllm-omni ... encoder.py":
 * F.linear of the QKV, o, gate/up and down projections, plus the residual adds
 * of MiniMaxH3Qwen3VLTextDecoderLayer.forward and _deepstack_process).
 *   A [M, K] (lda = K), W [N, K] (ldw = K), C [M, ldc]: ldc = N, or N/2 for SWIGLU.
 *   R [M, ldc] residual (RESIDUAL*), DS [n_vis, ldc] and vis_rank [M] (RESIDUAL_DS).
 *   workspace: NULL, or device memory of at least h3enc_op_gemm_workspace_bytes()
 *   bytes, 256-byte aligned, zero-filled once before its first use and then
 *   reused; with it the k-blocks of the tiles of a partial last wave are spread
 *   evenly over all SMs (stream-K; the result is deterministic for given M, N,
 *   K and SM count).  Calls sharing a workspace must not overlap on the GPU.
 * Requires K % 8 == 0, N % 256 == 0 (of the packed weight for SWIGLU), A and W
 * 16-byte aligned.  M may be any size >= 0. */
H3ENC_API h3enc_status h3enc_op_gemm(const void *A, const void *W, void *C, int32_t M, int32_t N, int32_t K,
                           int32_t epilogue, const void *R, const void *DS, const int32_t *vis_rank,
                           int32_t n_vis, void *workspace, int64_t workspace_bytes, int32_t *status,
                           void *stream);

/* Profiling aid: the next projection GEMM this host thread launches (through
 * h3enc_op_gemm, h3enc_op_gemm_qkv_rope, h3enc_op_gemm_noalloc or inside an
 * encode) records a timeline: CTA c writes 11 %globaltimer stamps (ns) to
 * trace[c * 11 + k]: k = 0 start, 1 prologue done, 2 last data-parallel accumulator
 * ready (epilogue start of the last tile), 3 first
 * MMA, 4 last data-parallel MMA issued, 5 data-parallel epilogues done, 6 first
 * stream-K accumulator ready, 7 stream-K partials written, 8 first tile's
 * contributor flags seen, 9 stream-K reduction done, 10 end.  The stream-K phase
 * runs before the data-parallel tiles; stamps of phases a CTA does not run, and
 * rows of CTAs beyond the grid, keep their contents.  trace: device uint64 of at
 * least 11 * SM-count entries, alive until that GEMM has run. */
H3ENC_API h3enc_status h3enc_op_gemm_trace_next(void *trace, int64_t trace_entries);

/* Profiling aid: the next attention launch on this host thread (through
 * h3enc_op_attention or inside an encode) records a timeline per persistent CTA
 * (one per SM, at most one per work item; work items = heads * sum over
 * sequences of ceil(len / 256)).  CTA c writes 9 entries at trace[c * 9]:
 * 0 start and 6 end as %globaltimer ns; 1 set-up done, 2 first Q tiles landed,
 * 3 first score tile ready, 4 last P written, 5 last P V product done as SM
 * clock64 cycles; then 7 the SM id and 8 the number of key tiles processed.
 * trace: device uint64 of at least 9 * ctas entries (ctas >= the SM count
 * covers every launch), alive until that launch has run. */
H3ENC_API h3enc_status h3enc_op_attention_trace_next(void *trace, int64_t trace_entries, int32_t ctas);

/* Failure-detection self-test (no counterpart on the pages).  Launches one
 * thread on `stream` that waits, through the library's bounded-wait helpers,
 * either until the device word *flag equals `expect` (use_mbarrier = 0) or on a
 * shared-memory mbarrier that nothing arrives on (use_mbarrier = 1).  A wait that
 * is not satisfied within the wait limit (about 2 s of SM clock) ORs ST_TIMEOUT
 * (1) into the device int32 *status and returns; the context stays usable.
 * flag: device memory (ignored when use_mbarrier = 1). */
H3ENC_API h3enc_status h3enc_op_wait_probe(const uint32_t *flag, uint32_t expect, int32_t use_mbarrier,
                                 int32_t *status, void *stream);

/* Workspace bytes h3enc_op_gemm needs on the current device (-1 without a device). */
H3ENC_API int64_t h3enc_op_gemm_workspace_bytes(void);

/* h3enc_op_gemm for callers that cannot allocate device memory (the pages have
 * no counterpart: this is a library convenience).  Some callers have no way to
 * hand over a workspace: code running inside another framework's allocator
 * callback or after a memory pool has reserved the whole device, plugins that
 * receive only their input and output buffers, hosts that forbid cudaMalloc
 * after start-up.  This entry point computes exactly what h3enc_op_gemm
 * computes with a workspace (same kernel, same split of the last wave), but its
 * scratch is a fixed array inside the library's device image:
 * h3enc_op_gemm_noalloc_scratch_bytes() bytes (40 MiB + 904 B, two 128 KiB
 * fp32 slots and one flag per SM for up to 160 SMs), held by every GPU that
 * loads the library until the process exits.  The caller passes inputs and
 * outputs only; nothing is allocated or freed.
 *   - The first call on a device looks up the array's device address and clears
 *     its flags with a memset queued on `stream` ahead of the kernel (no host or
 *     device synchronisation).  While `stream` is being captured that first call
 *     is refused (H3ENC_ERR_UNSUPPORTED): make it outside any capture.  Later
 *     calls only launch the kernel.
 *   - All calls on a device share the array and it keeps the last call's
 *     contents: calls that overlap on the GPU (other streams, other threads)
 *     race and corrupt each other's results; serialise them.
 *   - A device with more than 160 SMs would need more scratch than the array
 *     holds: the call returns H3ENC_ERR_UNSUPPORTED (message from
 *     h3enc_op_gemm_noalloc_last_error()).
 * Arguments, requirements and other errors are those of h3enc_op_gemm. */
H3ENC_API h3enc_status h3enc_op_gemm_noalloc(const void *A, const void *W, void *C, int32_t M, int32_t N, int32_t K,
                                   int32_t epilogue, const void *R, const void *DS, const int32_t *vis_rank,
                                   int32_t n_vis, int32_t *status, void *stream);

/* Bytes of the fixed scratch array h3enc_op_gemm_noalloc uses. */
H3ENC_API int64_t h3enc_op_gemm_noalloc_scratch_bytes(void);

/* Message of the last h3enc_op_gemm_noalloc error on this thread ("" if none). */
H3ENC_API const char *h3enc_op_gemm_noalloc_last_error(void);

/* Pack gate [I, K] and up [I, K] into W [2I, K] for H3ENC_EPI_SWIGLU: rows
 * [256b, 256b+128) = gate rows [128b, 128b+128), rows [256b+128, 256b+256) =
 * up rows [128b, 128b+128).  Requires I % 128 == 0. */
H3ENC_API h3enc_status h3enc_op_pack_gate_up(const void *gate, const void *up, void *W, int32_t I, int32_t K,
                                   void *stream);

/* Online-FP8 projection (page "vllm-omni ... encoder.py",
 * _validate_encoder_quant_config and the _is_quantized_linear branches): as
 * h3enc_op_gemm with e4m3 operands A [M, K] and W [N, K] (one byte per element,
 * row-major, 16-byte aligned, K % 16 == 0), their fp32 scales sa [M] (per row of
 * A) and sw [N] (per row of W, 16-byte aligned): the product is
 * (A * sa) (W * sw)^T accumulated in fp32 on the tensor cores, then the same
 * epilogues (STORE, RESIDUAL, SWIGLU, RESIDUAL_DS) and the same workspace rules. */
H3ENC_API h3enc_status h3enc_op_gemm_fp8(const void *A, const void *W, const float *sa, const float *sw, void *C,
                               int32_t M, int32_t N, int32_t K, int32_t epilogue, const void *R, const void *DS,
                               const int32_t *vis_rank, int32_t n_vis, void *workspace, int64_t workspace_bytes,
                               int32_t *status, void *stream);

/* Per-row e4m3 quantisation of a bf16 matrix x [rows, cols] (cols % 8 == 0):
 * scale[r] = amax(row r) / 448 in fp32 (1 for an all-zero row), q = e4m3(x * inv)
 * with inv = 448 / amax and the product each rounded once in fp32, then rounded
 * to nearest even, saturating at +-448 (the "fn" variant).  q [rows, cols]
 * bytes; x 16-byte aligned. */
H3ENC_API h3enc_status h3enc_op_quant_rows(const void *x, int32_t rows, int32_t cols, void *q, float *scale,
                                 void *stream);

/* RMSNorm of x [rows, cols] (as h3enc_op_rmsnorm, output rounded to bf16) followed
 * by h3enc_op_quant_rows of that bf16 output: q [rows, cols] e4m3, scale [rows]. */
H3ENC_API h3enc_status h3enc_op_rmsnorm_q8(const void *x, const void *w, void *q, float *scale, int32_t rows,
                                 int32_t cols, float eps, void *stream);

/* y = bf16(w * x / sqrt(mean(x^2) + eps)) per row, fp32 math (page "...
 * encoder.py", MiniMaxH3Qwen3VLRMSNorm).  x, y [rows, cols]; cols % 8 == 0,
 * cols <= 8192; y may equal x. */
H3ENC_API h3enc_status h3enc_op_rmsnorm(const void *x, const void *w, void *y, int32_t rows, int32_t cols,
                              float eps, void *stream);

/* M-RoPE tables (page "... encoder.py", MiniMaxH3Qwen3VLTextRotaryEmbedding and
 * _apply_interleaved_mrope): for j < head_dim/2,
 *   ang = float(positions[axis(j)][s]) * inv_freq[j],  inv_freq[j] = theta^(-2j/head_dim) (fp32),
 *   axis(j) = 1 if j%3==1 and j < 3*section[1]; 2 if j%3==2 and j < 3*section[2]; else 0,
 *   cos_tab[s][j] = cos(ang), sin_tab[s][j] = sin(ang)   (fp32, [S, head_dim/2]). */
H3ENC_API h3enc_status h3enc_op_rope_table(const int32_t *positions, int32_t S, int32_t head_dim, float theta,
                                 const int32_t *section_host, float *cos_tab, float *sin_tab,
                                 void *stream);

/* h3enc_op_rope_table with a choice of layout.  stride == 0: [S, head_dim/2] as above.
 * stride >= S (head_dim % 8 == 0): row-interleaved, the layout the encoder uses,
 *   cos_tab[((j/4) * stride + s) * 4 + j%4] = cos(ang(s, j))   (same for sin_tab),
 * i.e. [head_dim/8][stride][4]: for each group of four frequencies the rows follow one
 * another, so 32 consecutive rows read one group as 512 contiguous bytes.  Rows s >= S of
 * the padding are not written.  Each table holds stride * head_dim/2 floats (16-byte
 * aligned); a stride that is a multiple of 32 keeps every 32-row run on whole lines.
 * INVALID_ARG for 0 < stride < S or head_dim % 8 with stride > 0. */
H3ENC_API h3enc_status h3enc_op_rope_table_ex(const int32_t *positions, int32_t S, int32_t head_dim, float theta,
                                    const int32_t *section_host, int32_t stride, float *cos_tab,
                                    float *sin_tab, void *stream);

/* QKV projection with the per-head q/k RMSNorm and M-RoPE fused into the GEMM
 * epilogue (page "... encoder.py", MiniMaxH3Qwen3VLTextAttention.forward: the
 * q/k/v projections, q_norm/k_norm over head_dim, then _apply_rotary_pos_emb):
 *   qkv = A * W^T with W [(nq + 2*nkv)*d, K] (q rows, then k, then v);
 *   every q head (columns h*d) and k head (columns (nq + g)*d) of qkv becomes
 *   rope(rmsnorm(x, w_q or w_k, eps)) with, for j < d/2,
 *     rope(x)[j] = x[j]*cos[j] - x[j+d/2]*sin[j],  rope(x)[j+d/2] = x[j+d/2]*cos[j] + x[j]*sin[j]
 *   (cos/sin = the fp32 tables of h3enc_op_rope_table, [M, d/2]); v heads are the plain
 *   projection.  C [M, (nq + 2*nkv)*d].  workspace as for h3enc_op_gemm.
 * Requires head_dim in {64, 128} and (nq + 2*nkv)*d % 256 == 0. */
H3ENC_API h3enc_status h3enc_op_gemm_qkv_rope(const void *A, const void *W, void *C, int32_t M, int32_t K,
                                    int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, const void *w_q,
                                    const void *w_k, float eps, const float *cos_tab, const float *sin_tab,
                                    void *workspace, int64_t workspace_bytes, int32_t *status, void *stream);

/* RMSNorm folded into a projection (page "... encoder.py", MiniMaxH3Qwen3VLRMSNorm
 * followed by the projection that reads its output; an algebraic rearrangement the
 * encoder uses when h3enc_config.separate_norm == 0):
 *   rmsnorm(x, g) W^T = diag(1 / sqrt(mean(x^2) + eps)) x (W diag(g))^T.
 * Row statistics are sums of squares over slots of 128 columns, accumulated in fp32 in
 * column order, stored slot-major: ss[s * rows + r] = sum_{c in [128 s, 128 s + 128)} x[r][c]^2.
 *
 * h3enc_op_row_sumsq: ss [cols/128, rows] fp32 of the bf16 matrix x [rows, cols];
 * cols % 128 == 0, x 16-byte aligned. */
H3ENC_API h3enc_status h3enc_op_row_sumsq(const void *x, int32_t rows, int32_t cols, float *ss, void *stream);

/* h3enc_op_fold_cols: W[r][k] = bf16(W[r][k] * gamma[k]) in place (fp32 product rounded
 * to nearest even), W bf16 [rows, cols], gamma bf16 [cols]; cols % 8 == 0, both
 * 16-byte aligned. */
H3ENC_API h3enc_status h3enc_op_fold_cols(void *W, int32_t rows, int32_t cols, const void *gamma, void *stream);

/* h3enc_op_gemm with the folded norm: ss_in [K/128, M] (or NULL): the accumulator of row
 * r is multiplied by 1/sqrt(sum_s ss_in[s][r] / K + eps) (slots added in order) before the
 * epilogue; ss_out [N/128, M] (or NULL; STORE and RESIDUAL only): the row statistics of
 * the bf16 output C, as h3enc_op_row_sumsq would give them.  epilogue: STORE,
 * RESIDUAL or SWIGLU; other arguments as h3enc_op_gemm. */
H3ENC_API h3enc_status h3enc_op_gemm_rms(const void *A, const void *W, void *C, int32_t M, int32_t N, int32_t K,
                                         int32_t epilogue, const void *R, const float *ss_in, float *ss_out,
                                         float eps, void *workspace, int64_t workspace_bytes, int32_t *status,
                                         void *stream);

/* h3enc_op_gemm_qkv_rope reading tables of either layout of h3enc_op_rope_table_ex:
 * cs_stride == 0 for [M, d/2], else the row-interleaved tables of that stride (>= M).
 * ss_in (optional, NULL: none) and in_eps as for h3enc_op_gemm_qkv_rope_rms.  The output is
 * the same, bit for bit, in both layouts; the row-interleaved one is faster (the epilogue's
 * table loads are whole lines). */
H3ENC_API h3enc_status h3enc_op_gemm_qkv_rope_ex(const void *A, const void *W, void *C, int32_t M, int32_t K,
                                       int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, const void *w_q,
                                       const void *w_k, float eps, const float *cos_tab, const float *sin_tab,
                                       int32_t cs_stride, const float *ss_in, float in_eps, void *workspace,
                                       int64_t workspace_bytes, int32_t *status, void *stream);

/* h3enc_op_gemm_qkv_rope with the folded input norm: each row of A * W^T is first
 * multiplied by 1/sqrt(sum_s ss_in[s][r] / K + in_eps) (ss_in [K/128, M], required), then
 * the q/k RMSNorm (eps) and M-RoPE of h3enc_op_gemm_qkv_rope apply. */
H3ENC_API h3enc_status h3enc_op_gemm_qkv_rope_rms(const void *A, const void *W, void *C, int32_t M, int32_t K,
                                                  int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                  const void *w_q, const void *w_k, float eps,
                                                  const float *cos_tab, const float *sin_tab, const float *ss_in,
                                                  float in_eps, void *workspace, int64_t workspace_bytes,
                                                  int32_t *status, void *stream);

/* ---- vision tower kernels (page "... encoder.py", section "Qwen3-VL vision tower") ----
 * The tower's patch order: per grid, frames, then the m x m blocks row-major, then the
 * patches of a block row-major.  grid_thw: HOST int32 [n_grids, 3] (n_grids <= 64; rows and
 * columns multiples of merge).
 *
 * h3enc_op_layernorm: y = bf16((x - mean) / sqrt(var + eps) * w + b) per row (nn.LayerNorm,
 * biased variance, fp32); x, y [rows, cols] bf16, cols % 8 == 0, cols <= 8192. */
H3ENC_API h3enc_status h3enc_op_layernorm(const void *x, const void *w, const void *b, void *y, int32_t rows,
                                          int32_t cols, float eps, void *stream);

/* h3enc_op_vision_pos_embed (fast_pos_embed_interpolate): out[k] = bf16 of the bilinear
 * sample of the grid_side x grid_side table [grid_side^2, hidden] at patch k: the grid's
 * h x w points evenly spaced from corner to corner (i * (G-1)/(h-1) in double, rounded
 * to fp32), lower corner by truncation, upper clipped to G-1, fp32 weights and
 * products summed corner by corner.  out [n_patches, hidden] bf16. */
H3ENC_API h3enc_status h3enc_op_vision_pos_embed(const void *table, int32_t grid_side, int32_t hidden,
                                                 const int32_t *grid_thw, int32_t n_grids, int32_t merge, void *out,
                                                 void *stream);

/* h3enc_op_vision_rope_table (rot_pos_emb): cos/sin [n_patches, head_dim/2] fp32 of the
 * angles row * inv_freq[j] (j < head_dim/4) and column * inv_freq[j - head_dim/4] (the
 * rest), inv_freq[j] = theta^(-2j/(head_dim/2)) rounded once to fp32; the pairs
 * (j, j + head_dim/2) of q and k rotate by angle j as in h3enc_op_gemm_qkv_rope. */
H3ENC_API h3enc_status h3enc_op_vision_rope_table(const int32_t *grid_thw, int32_t n_grids, int32_t merge,
                                                  int32_t head_dim, float theta, float *cos_tab, float *sin_tab,
                                                  void *stream);

/* h3enc_op_gemm_bias: h3enc_op_gemm with bias [N] (bf16, 16-byte aligned) added to the
 * accumulator; epilogue H3ENC_EPI_STORE (C = bf16(acc + bias)), H3ENC_EPI_RESIDUAL
 * (C = bf16(R + acc + bias)), H3ENC_EPI_GELU_TANH or H3ENC_EPI_GELU_ERF.  Other arguments
 * and requirements as h3enc_op_gemm. */
H3ENC_API h3enc_status h3enc_op_gemm_bias(const void *A, const void *W, void *C, int32_t M, int32_t N, int32_t K,
                                          int32_t epilogue, const void *R, const void *bias, void *workspace,
                                          int64_t workspace_bytes, int32_t *status, void *stream);

/* h3enc_op_gemm_qkv_rope_bias (the vision tower's attention input): qkv = A W^T + bias with
 * W [3 * heads * head_dim, K] (q rows, k rows, v rows), then every q and k head rotated
 * with the fp32 tables cos/sin [M, head_dim/2] (no per-head norm); v heads as they are. */
H3ENC_API h3enc_status h3enc_op_gemm_qkv_rope_bias(const void *A, const void *W, void *C, int32_t M, int32_t K,
                                                   int32_t heads, int32_t head_dim, const void *bias,
                                                   const float *cos_tab, const float *sin_tab, void *workspace,
                                                   int64_t workspace_bytes, int32_t *status, void *stream);

/* h3enc_op_attention_bidir: as h3enc_op_attention with one kv head per q head and no
 * causal mask: every query attends to every key of its segment (the tower's attention
 * inside each frame, scaled_dot_product_attention with is_causal=False). */
H3ENC_API h3enc_status h3enc_op_attention_bidir(const void *qkv, void *o, int32_t S, int32_t heads,
                                                int32_t head_dim, const int32_t *cu_seqlens, int32_t n_seqs,
                                                void *stream);

/* h3enc_op_attention_bidir with a workspace (h3enc_op_attention_workspace_bytes(head_dim)
 * bytes, 16-byte aligned, zero-filled once before its first use and again after a call whose
 * device status reported a timeout; calls sharing it must not overlap on the GPU).  When the persistent kernel's last round of work items would leave
 * most SMs idle, those items are cut into up to 8 ranges of their keys; each range writes
 * its unnormalised output, running maximum and sum to the workspace and the range that
 * finishes last merges them in range order (the same result on every run).  The output
 * equals the plain call's up to fp32 rounding.  0 from the size query: head_dim not 64/128. */
H3ENC_API int64_t h3enc_op_attention_workspace_bytes(int32_t head_dim);
H3ENC_API h3enc_status h3enc_op_attention_bidir_ws(const void *qkv, void *o, int32_t S, int32_t heads,
                                                   int32_t head_dim, const int32_t *cu_seqlens, int32_t n_seqs,
                                                   void *workspace, int64_t workspace_bytes, void *stream);

/* Causal GQA attention over packed sequences (page "... encoder.py",
 * MiniMaxH3Qwen3VLTextAttention.forward: repeat_interleave of K/V, SDPA with
 * is_causal=True, scale 1/sqrt(d)).  Reads q/k/v from qkv [S, (nq+2nkv)*d]
 * (q head h at column h*d, k head g at (nq+g)*d, v head g at (nq+nkv+g)*d),
 * writes o [S, nq*d] (head h at column h*d).  cu_seqlens HOST int32 [n_seqs+1]
 * or NULL (one sequence); n_seqs <= 1024. */
H3ENC_API h3enc_status h3enc_op_attention(const void *qkv, void *o, int32_t S, int32_t n_heads,
                                int32_t n_kv_heads, int32_t head_dim, const int32_t *cu_seqlens,
                                int32_t n_seqs, void *stream);

/* out[s] = table[ids[s]] (bit-exact row copy; page "... encoder.py",
 * embed_tokens / F.embedding).  Ids outside [0, vocab) give a zero row and
 * set status bit 2.  hidden % 8 == 0. */
H3ENC_API h3enc_status h3enc_op_embed(const int32_t *ids, const void *table, int32_t vocab, int32_t hidden,
                            void *out, int32_t S, int32_t *status, void *stream);

/* vis_rank[s] = number of visual rows before s if mask[s] != 0, else -1 (the
 * row of the DeepStack features that boolean-mask assignment gives row s).
 * Sets status bit 4 if the mask holds a count other than n_vis. */
H3ENC_API h3enc_status h3enc_op_vis_rank(const uint8_t *mask, int32_t S, int32_t n_vis, int32_t *vis_rank,
                               int32_t *status, void *stream);

/* ---- decoding from a paged key/value cache ----
 * The steps that extend an encoded prompt token by token (no counterpart on the pages,
 * which stop at the prefill): a projection's q/k heads normed, rotated and stored in a
 * cache, the attention of one new token of every sequence over it, and the eviction of
 * the tokens that drew the least attention.  All three run without host synchronisation,
 * read lengths and page numbers on the device, and can be captured in a CUDA graph.
 *
 * A cache holds the keys and values of one decoder layer in pages of page_size tokens;
 * element e of kv head g of the token in place s of page p is
 *   k[p * page_stride + (g * page_size + s) * head_dim + e]   (elements; v the same).
 * A sequence's token i is in place i % page_size of page page_table[b * ld_table +
 * i / page_size].  The pages of one layer may lie apart (page_stride), so that one
 * allocation can hold K and V, or all layers, side by side.  E4M3 caches store
 * e4m3(x / scale[g]) (fp32 division, rounded to nearest even, saturating at +-448) and
 * stand for that value times scale[g].
 * Requires page_size in {16, 32, 64, 128, 256}, head_dim in {64, 128}, k and v 16-byte
 * aligned, n_kv_heads <= 65536, page_stride >= n_kv_heads * page_size * head_dim, its bytes a multiple of 16
 * and below 2^40, num_pages * page_size < 2^31.  Another dtype, head_dim or page_size is
 * H3ENC_ERR_UNSUPPORTED, the rest H3ENC_ERR_INVALID_ARG. */
typedef struct {
    void *k, *v;
    const float *k_scale, *v_scale;   /* [n_kv_heads], FP8_E4M3 only; NULL for BF16 */
    int64_t page_stride;              /* elements from one page to the next */
    int32_t num_pages, page_size, n_kv_heads, head_dim;
    int32_t dtype;                    /* H3ENC_DTYPE_BF16 or H3ENC_DTYPE_FP8_E4M3 */
} h3enc_kv_cache;

/* Per-head q/k RMSNorm and rotation of a packed projection, and the K and V heads stored
 * in a cache, in one pass (what h3enc_op_gemm_qkv_rope does in its epilogue, for a
 * projection that comes from elsewhere: h3enc_op_gemm_fp8, h3enc_op_gemm_bias, few rows).
 *   qkv [T, ld_qkv]: q head h at column h*d, k head g at (n_heads+g)*d, v head g at
 *   (n_heads+n_kv_heads+g)*d.  Each q and k head becomes rope(rmsnorm(x, w_q or w_k, eps))
 *   in fp32, rounded once: w_q / w_k NULL skips that norm, cos_tab = sin_tab = NULL the
 *   rotation; tables of either layout of h3enc_op_rope_table_ex (cs_stride as there).
 *   q_out [T, ld_q] and k_out [T, ld_k] (n_heads*d and n_kv_heads*d columns; NULL: not
 *   written) may be qkv's own q and k columns (same leading dimension), and must not
 *   overlap qkv or each other otherwise.
 *   cache (or NULL) with slots [T]: k and v of row t go to place slots[t] % page_size of page
 *   slots[t] / page_size.  A negative slot stores nothing (a padding row); one past the last
 *   page stores nothing and sets status bit 2.  Rows that share a slot overwrite each
 *   other in no stated order.
 * Requires head_dim in {64, 128}, leading dimensions that are multiples of 8, operands
 * 16-byte aligned, at least one of q_out, k_out and cache. */
H3ENC_API h3enc_status h3enc_op_qk_norm_rope(const void *qkv, int64_t ld_qkv, int32_t T, int32_t n_heads,
                                             int32_t n_kv_heads, int32_t head_dim, const void *w_q,
                                             const void *w_k, float eps, const float *cos_tab,
                                             const float *sin_tab, int32_t cs_stride, void *q_out, int64_t ld_q,
                                             void *k_out, int64_t ld_k, const h3enc_kv_cache *cache,
                                             const int32_t *slots, int32_t *status, void *stream);

/* Attention of one new token of each of n_seqs sequences over the cache (the new token's
 * own key and value already in it): for q head h, reading kv head h / (n_heads / n_kv_heads),
 *   p_i = softmax_i(q . k_i / sqrt(d)) over i < seq_lens[b],   o = sum_i p_i v_i
 * (fp32, but p enters the second sum with 16 bits, 22 for E4M3; o rounded to bf16 once; a
 * sequence of length 0 gives a zero row; weights below 2^-126 of the largest count as 0,
 * also times an infinite value, which is NaN).
 *   q [n_seqs, ld_q], o [n_seqs, ld_o]: head h at column h*d; o must not overlap q.
 *   page_table DEVICE int32 [n_seqs, ld_table], seq_lens DEVICE int32 [n_seqs]; max_len: a
 *   bound on the lengths known to the host (ld_table * page_size >= max_len).  A length
 *   outside [0, max_len] is clamped into it and a page number outside the cache reads as
 *   zero keys and values; both set status bit 2.
 *   weight_out (or NULL) [n_seqs, ld_weight], ld_weight >= max_len: for i < seq_lens[b],
 *   weight_out[b][i] = weight_in[b][i] + sum over all q heads of p_i (weight_in NULL:
 *   from 0; it may equal weight_out, and must not overlap it otherwise).  Entries
 *   from the length on are left as they were.
 *   workspace: h3enc_op_attention_decode_workspace_bytes() bytes, 256-byte aligned,
 *   zero-filled once before its first use and then reused by calls of any sizes that fit.
 *   Calls (and graphs that hold them) sharing it must not overlap on the GPU.
 * The result does not depend on timing: the same inputs give the same bits on every run.  A
 * bounded wait that runs out sets status bit 1; the outputs are then undefined.
 * Requires n_seqs <= 1024, max_len <= 2^30, n_heads % n_kv_heads == 0, leading dimensions of
 * q and o that are multiples of 8, q and o 16-byte aligned; n_seqs * n_heads * ceil(max_len / 64)
 * above 2^31 - 65 is H3ENC_ERR_UNSUPPORTED. */
H3ENC_API h3enc_status h3enc_op_attention_decode(const void *q, int64_t ld_q, void *o, int64_t ld_o,
                                                 const h3enc_kv_cache *cache, const int32_t *page_table,
                                                 int32_t ld_table, const int32_t *seq_lens, int32_t n_seqs,
                                                 int32_t n_heads, int32_t max_len, const float *weight_in,
                                                 float *weight_out, int64_t ld_weight, void *workspace,
                                                 int64_t workspace_bytes, int32_t *status, void *stream);

/* Workspace bytes of h3enc_op_attention_decode on the current device; with_weights: the
 * call passes weight_out.  -1 without a device or for sizes the call refuses. */
H3ENC_API int64_t h3enc_op_attention_decode_workspace_bytes(int32_t n_seqs, int32_t n_heads, int32_t max_len,
                                                            int32_t with_weights);

/* Eviction from the cache by accumulated attention weight.  A sequence longer than `budget`
 * keeps budget tokens: its first `sink`, its last `recent` and, of the others, those of the
 * largest weight (of equal ones the earlier; NaN counts as the smallest).  The kept tokens
 * keep their order and move, K, V and weight, to the front.  Shorter sequences keep all.
 *   page_table, seq_lens, max_len as for h3enc_op_attention_decode (lengths clamped the same way).
 *   page_table_out NULL: in place, within the pages of page_table (which must not be shared
 *   between sequences, nor appear twice in one).  Otherwise DEVICE int32 [n_seqs, ld_table_out], ld_table_out *
 *   page_size >= min(budget, max_len): token i of the result goes to page
 *   page_table_out[b][i / page_size], pages that this call does not read; the source
 *   pages stay as they were.  Tokens whose page number, on either side, lies
 *   outside the cache are not moved and set status bit 2.
 *   weight [n_seqs, ld_weight] in, weight_out [n_seqs, ld_weight_out] out (leading dimensions
 *   >= max_len, no overlap): weight_out[b][i] = weight[b][kept[b][i]] for i < new_lens[b],
 *   0 from there to max_len (tokens appended later start at 0).
 *   kept int32 [n_seqs, ld_kept], ld_kept >= budget: the places the kept tokens had,
 *   ascending, then -1 up to budget.  new_lens int32 [n_seqs] (may be seq_lens itself).
 * Requires budget >= 1, sink + recent <= budget, n_seqs <= 1024, max_len <= 2^30. */
H3ENC_API h3enc_status h3enc_op_cache_evict(const h3enc_kv_cache *cache, const int32_t *page_table, int32_t ld_table,
                                            const int32_t *page_table_out, int32_t ld_table_out,
                                            const int32_t *seq_lens, int32_t n_seqs, int32_t max_len, int32_t budget,
                                            int32_t sink, int32_t recent, const float *weight, int64_t ld_weight,
                                            float *weight_out, int64_t ld_weight_out, int32_t *kept, int64_t ld_kept,
                                            int32_t *new_lens, int32_t *status, void *stream);

/* Rotary positions, for h3enc_rope_make: the first rotary_dim elements of a head rotate in pairs, pair j by the angle
 * position * w_j with w_j = theta^(-2j / rotary_dim), scaled for contexts longer than original_len tokens:
 *   ROPE_LINEAR      w_j / factor
 *   ROPE_WAVELENGTH  with n_j = original_len w_j / 2 pi, the turns of pair j over the original context, and
 *                    s = clamp((n_j - low_turns) / (high_turns - low_turns), 0, 1):  w_j (s + (1 - s) / factor)
 *   ROPE_YARN        with dim(n) = rotary_dim ln(original_len / (2 pi n)) / (2 ln theta), a = max(floor(dim(high_turns)), 0),
 *                    e = min(ceil(dim(low_turns)), rotary_dim - 1) and s = clamp((j - a) / max(e - a, 0.001), 0, 1):
 *                    w_j (1 - s) + (w_j / factor) s
 * cos and sin are multiplied by magnitude.  Angles are exact to the last bits of fp32 at every position (they are reduced
 * as 64-bit fractions of a turn), but for w_j's own rounding to 53 bits. */
enum { H3ENC_ROPE_PLAIN = 0, H3ENC_ROPE_LINEAR = 1, H3ENC_ROPE_WAVELENGTH = 2, H3ENC_ROPE_YARN = 3 };
typedef struct {
    int32_t rotary_dim;    /* a multiple of 16, 16 to 128; at most the head_dim that it is used with */
    int32_t interleaved;   /* 0: pairs (j, j + rotary_dim/2); 1: pairs (2j, 2j + 1) */
    int32_t scaling;       /* H3ENC_ROPE_* */
    int32_t original_len;  /* WAVELENGTH and YARN: >= 1 */
    double theta;          /* > 0; YARN: > 1 */
    double factor;         /* > 0; PLAIN ignores it */
    double low_turns, high_turns;   /* WAVELENGTH, YARN: 0 < low < high; both 0: 1 and 4, YARN 1 and 32 */
    double magnitude;      /* > 0; 0: 1, YARN with a factor above 1: 0.1 ln(factor) + 1 */
    int32_t section[3];    /* {0, 0, 0}: one position per row; else three-axis positions, pair j by axis(j) of
                              h3enc_op_rope_table, and the sections sum to rotary_dim/2 */
} h3enc_rope;

/* The frequencies of an h3enc_rope as the kernel takes them: made once by h3enc_rope_make, for any number of calls. */
typedef struct {
    uint64_t turns[64];     /* 2^64 times the turns of pair j per position, modulo 2^64 */
    uint64_t axis1, axis2;  /* bit j: pair j goes by the second / third axis */
    float magnitude;
    int32_t rotary_dim, interleaved, axes;
} h3enc_rope_plan;

/* HOST only (no device, no stream).  H3ENC_ERR_INVALID_ARG for parameters outside the ranges above. */
H3ENC_API h3enc_status h3enc_rope_make(const h3enc_rope *rope, h3enc_rope_plan *plan);

/* New rows of a packed projection normed, rotated and appended to their sequences in a cache, in one pass: what
 * h3enc_op_qk_norm_rope does with slots and tables that the caller makes, by page table, lengths and positions alone.
 *   qkv [T, ld_qkv], w_q, w_k, eps, q_out, k_out and their in-place rules as for h3enc_op_qk_norm_rope.  Each q and k
 *   head becomes rotate(rmsnorm(x)) in fp32, rounded once (w_q / w_k NULL: no norm; rope NULL: no rotation).
 *   seq_lens DEVICE int32 [n_seqs]: each sequence's tokens, the new ones counted in.  cu_rows DEVICE int32 [n_seqs + 1]:
 *   rows [cu_rows[b], cu_rows[b + 1]) are the last tokens of sequence b, in order; NULL: row b is the last token
 *   of sequence b.  Rows of no sequence are left as they were in every output.
 *   positions DEVICE int32 [1 or 3 axes, ld_positions] (of any sign); NULL: a row's position is its token's index in
 *   its sequence.
 *   cache (or NULL) with page_table DEVICE int32 [n_seqs, ld_table], ld_table * page_size >= max_len: k and v of token i
 *   of sequence b go to place i % page_size of page page_table[b][i / page_size].  A token outside [0, max_len)
 *   or on a page outside the cache is not stored and sets status bit 2 (its q_out and k_out are written).
 *   Without a cache, seq_lens may be NULL too (n_seqs 0, cu_rows NULL): all T rows are rotated by `positions`, which must
 *   then be given if rope is.
 * Requires head_dim in {64, 128}, n_seqs <= 1024, max_len <= 2^30, leading dimensions that are multiples of 8, operands
 * 16-byte aligned, at least one of q_out, k_out and cache. */
H3ENC_API h3enc_status h3enc_op_rope_append(const void *qkv, int64_t ld_qkv, int32_t T, int32_t n_heads,
                                            int32_t n_kv_heads, int32_t head_dim, const void *w_q, const void *w_k,
                                            float eps, const h3enc_rope_plan *rope, const int32_t *positions,
                                            int64_t ld_positions, void *q_out, int64_t ld_q, void *k_out, int64_t ld_k,
                                            const h3enc_kv_cache *cache, const int32_t *page_table, int32_t ld_table,
                                            const int32_t *seq_lens, const int32_t *cu_rows, int32_t n_seqs,
                                            int32_t max_len, int32_t *status, void *stream);

/* Attention of one new token of each sequence behind prefixes that sequences share (an instruction, a document): as
 * h3enc_op_attention_decode, with the keys of a sequence's prefix in front of its own, read once for all sequences of the group:
 *   p_i = softmax_i(q . k_i / sqrt(d)) over the prefix_lens[s] tokens of prefix s and the seq_lens[b] own tokens of b.
 *   prefix_rows DEVICE int32 [n_prefixes + 1]: sequences [prefix_rows[s], prefix_rows[s + 1]) stand behind prefix s; those of no
 *   group have no prefix.  NULL (n_prefixes <= 1): all stand behind the one.  The offsets must not run back (they are
 *   clamped into [0, n_seqs], which sets status bit 2, and rows of two groups are undefined).
 *   prefix_table DEVICE int32 [n_prefixes, ld_prefix], prefix_lens DEVICE int32 [n_prefixes], max_prefix: pages and lengths
 *   of the prefixes, in the same cache, as page_table, seq_lens and max_len are the sequences' own (token 0 of a
 *   sequence's own tokens in place 0 of its first page), clamped and reported alike.
 *   weight_in, weight_out: of the own tokens; the prefixes' weights are not accumulated.
 *   workspace: h3enc_op_attention_decode_shared_workspace_bytes() bytes, with the rules of h3enc_op_attention_decode's
 *   (zero-filled again after a call whose status reported a timeout).
 * The weights of a prefix's tokens enter the second sum with 16 bits, as the own tokens' do (e4m3: in f16, off by up to 2^-11
 * of each, where the own tokens' have 22), and those below 2^-126 (e4m3: 2^-38) of the largest count as 0, also times an infinite
 * value (as all below 2^-108 may there), which is NaN; where all sequences together would read at most 200 MB of prefixes (by
 * max_prefix), each reads its own again in one launch, with the rounding of h3enc_op_attention_decode.
 * Requires n_prefixes <= 1024, max_prefix <= 2^30;
 * n_kv_heads * ceil(heads per kv head / 128) * (n_seqs / (2 max(128 / heads per kv head, 1)) + min(n_prefixes, n_seqs)) *
 * (max_prefix / 64 + 4) above 2e9 is H3ENC_ERR_UNSUPPORTED; the rest as for h3enc_op_attention_decode. */
H3ENC_API h3enc_status h3enc_op_attention_decode_shared(
    const void *q, int64_t ld_q, void *o, int64_t ld_o, const h3enc_kv_cache *cache, const int32_t *prefix_table,
    int32_t ld_prefix, const int32_t *prefix_lens, const int32_t *prefix_rows, int32_t n_prefixes, int32_t max_prefix,
    const int32_t *page_table, int32_t ld_table, const int32_t *seq_lens, int32_t n_seqs, int32_t n_heads, int32_t max_len,
    const float *weight_in, float *weight_out, int64_t ld_weight, void *workspace, int64_t workspace_bytes, int32_t *status,
    void *stream);

/* Workspace bytes of h3enc_op_attention_decode_shared on the current device (enough for h3enc_op_attention_decode of
 * the same sizes too).  -1 without a device or for sizes the call refuses. */
H3ENC_API int64_t h3enc_op_attention_decode_shared_workspace_bytes(int32_t n_seqs, int32_t n_heads, int32_t max_len,
                                                                   int32_t with_weights);

/* Cross attention: packed queries over packed keys and values of another length (an encoder's states through a
 * projection), without a mask; one query per sequence is a decode step.
 *   o[t] = sum_i p_i v_i, p = softmax_i(q[t] . k_i / sqrt(d)), for rows t of [cu_q[b], cu_q[b + 1]) over rows i of
 *   [cu_k[b], cu_k[b + 1]); q head h reads kv head h / (n_heads / n_kv_heads).  fp32, but p enters the second sum in bf16
 *   (up to 32 rows of queries x heads per kv head and sequence on the average: with 16 bits); o rounded to bf16 once.  Weights
 *   below 2^-126 of the largest count as 0, also times an infinite value, which is NaN.  No keys: zero rows.  Rows of no
 *   sequence are left as they were.
 *   q [Tq, ld_q], o [Tq, ld_o]: head h at column h*d; k [Tk, ld_k], v [Tk, ld_v]: kv head g at column g*d (k and v may be
 *   columns of one projection).  o must not overlap q, k or v.
 *   cu_q, cu_k DEVICE int32 [n_seqs + 1], not running back; each may be NULL with n_seqs 1 (all rows).  Offsets outside
 *   [0, Tq] or [0, Tk] are clamped; that, or one that runs back, sets status bit 2 (rows of two sequences are undefined,
 *   nothing outside o's Tq rows is written).
 *   workspace: h3enc_op_attention_cross_workspace_bytes() bytes, 256-byte aligned, zero-filled once before its first use (and
 *   again after a call whose status reported a timeout) and then reused by calls of any sizes.  Calls (and graphs that hold them) sharing it must not overlap on the GPU.
 * The result does not depend on timing: the same inputs give the same bits on every run.  A bounded wait that runs out sets
 * status bit 1; the outputs are then undefined.
 * Requires head_dim in {64, 128}, n_seqs <= 1024, Tq and Tk <= 2^30, n_heads <= 65536, n_heads % n_kv_heads == 0, leading
 * dimensions that are multiples of 8 and below 2^39, operands 16-byte aligned; n_kv_heads * ceil(heads per kv head / 128) *
 * (Tq / (2 max(128 / heads per kv head, 1)) + min(n_seqs, Tq)) * (Tk / 64 + 4) above 2e9 is H3ENC_ERR_UNSUPPORTED. */
H3ENC_API h3enc_status h3enc_op_attention_cross(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v,
                                                int64_t ld_v, void *o, int64_t ld_o, int32_t Tq, int32_t Tk,
                                                int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, const int32_t *cu_q,
                                                const int32_t *cu_k, int32_t n_seqs, void *workspace,
                                                int64_t workspace_bytes, int32_t *status, void *stream);

/* Workspace bytes of h3enc_op_attention_cross on the current device.  -1 without a device or for another head_dim. */
H3ENC_API int64_t h3enc_op_attention_cross_workspace_bytes(int32_t head_dim);

#ifdef __cplusplus
}
#endif
#endif /* H3ENC_OPS_H */
