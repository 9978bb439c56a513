/*
 * qmm.h -- C ABI of libqmm: the small-M affine-quantized matrix multiply
 *
 *     Y[M,N] = X[M,K] . dequant(Wq, scales, biases)[N,K]^T,   1 <= M <= 16
 *
 * that a speculative-decoding verify step issues with a handful of draft rows.
 * The library streams the packed weights from HBM once per call whatever M is,
 * dequantizes each weight group once and reuses it for all M rows.
 *
 * and the operators around that product in a batched verify step: quantisation
 * into the microscaled formats (qmm_quantize_mx), their product for any number of
 * rows (qmm_matmul_mx), a paged key-value cache (qmm_kv_append) with attention of
 * 1..16 new rows a sequence over it (qmm_paged_attention), and the verification
 * of drafted tokens (qmm_verify_draft); and those of a served layer beside it: the
 * experts of every token (qmm_route_experts), rotary positions on the way into the
 * cache (qmm_rope_append), attention of sequences that share a long prefix
 * (qmm_shared_prefix_attention) and the requests' own low-rank adapters
 * (qmm_lora_add).  Each is defined at its declaration.
 *
 * Sources of the product's definition (page title, section):
 *   - "MLX quantized_matmul small-M verify kernels", fact "Stock qmv streams
 *     the weight matrix once per input row": the problem (cost linear in M).
 *   - same page, fact "Fix family 1": dequantize each group once into
 *     registers and reuse it across the M rows; affine mode.
 *   - same page, fact "Fix family 2": weights as the matrix operand, split K
 *     across the warps of a block, read the bf16 activations directly.
 *   - same page, fact "Group-size mechanism": fp16 scale + fp16 bias per group
 *     (4 bytes per group).
 *   - same page, fact "Microbench": W is stored [N,K] and Y = X . W^T.
 *
 * Data formats (all row-major, all buffers owned by the caller):
 *   X       bf16 [M, K]                         device
 *   Wq      uint32 [N, K*bits/32]               device
 *           code k of row n sits in word k/(32/bits) of that row at bit
 *           offset bits*(k mod (32/bits)); codes are unsigned 0..2^bits-1,
 *           bits = 2, 4 or 8.  (The pages print no bit layout; this is the
 *           layout qmm_pack writes.  8-bit affine: same page, facts
 *           "qmv_wide speedup" (int8 at M=8) and "mlx-dspark skinny_qmm".)
 *   scales  fp16 [N, K/group_size]              device
 *   biases  fp16 [N, K/group_size]              device
 *           w[n,k] = scales[n, k/g] * q[n,k] + biases[n, k/g]
 *   Y       bf16 (round to nearest even) or fp32 [M, N]    device
 *
 * Arithmetic: codes are exact in bf16 and their products with bf16 X are
 * exact in fp32; sums are fp32; each group's scale and bias are applied once
 * to the group's fp32 partial sums.  Results are deterministic for a given
 * (variant, splits, shape): no atomics, fixed reduction order.
 *
 * Execution: every compute call is asynchronous on `stream` (a cudaStream_t
 * passed as void*, 0 = legacy default stream).  Arguments are validated on the
 * host before anything is launched; a validation failure returns an error and
 * launches nothing.  There is no CPU fallback.  The library allocates no device
 * memory and keeps no per-call state.  X, Wq, scales, biases must not overlap Y.
 * The small-M calls copy Wq, scales and biases before the stream's preceding
 * kernels have been waited for, as far as these let their dependents start early
 * (programmatic dependent launch).  So a kernel that writes weights must not
 * release its dependents early.  None of this library's does: what
 * qmm_quantize_mx, qmm_from_ggml and qmm_repack write may be the weights of the
 * next call on the stream, with nothing in between.
 */
#ifndef QMM_H_
#define QMM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QMM_OK = 0,
  QMM_ERR_NULL = 1,        /* a required pointer is null                          */
  QMM_ERR_SHAPE = 2,       /* M outside 0..16, N or K negative, K not a multiple   */
                           /* of group_size, a size that overflows, or a residual  */
                           /* that partly overlaps Y                               */
  QMM_ERR_UNSUPPORTED = 3, /* bits not in {2,4,8}, group_size not in {32,64,128},  */
                           /* unknown variant, bad split count or output dtype     */
  QMM_ERR_ALIGN = 4,       /* X or Wq not 16-byte aligned, scales/biases/Y not     */
                           /* aligned to their element size                        */
  QMM_ERR_CUDA = 5,        /* the CUDA runtime reported an error; see               */
                           /* qmm_last_cuda_error()                                 */
  QMM_ERR_TABLE = 6        /* the dispatch table is unusable: the QMM_TABLE file    */
                           /* cannot be read or holds no entry, or the shape's     */
                           /* entry names an unknown variant or split count        */
} qmm_status;

typedef enum { QMM_OUT_BF16 = 0, QMM_OUT_F32 = 1 } qmm_out_dtype;

/* Y = X . dequant(W)^T with the variant the dispatch table picks for
 * (M, N, K, bits, group_size); bf16 output.
 * M == 0 or N == 0: nothing to compute, returns QMM_OK without launching.
 * K == 0: Y is the empty sum, filled with zeros on `stream`.                    */
qmm_status qmm_small_m(const void* X, const uint32_t* Wq, const void* scales, const void* biases,
                       int M, int N, int K, int bits, int group_size, void* Y, void* stream);

/* Same, with the output dtype and an optional forced kernel variant
 * (variant = -1: dispatch table; 0 .. qmm_num_variants()-1: that variant) and
 * the number of CTAs that split K inside one thread-block cluster (splits = -1:
 * the table's or the variant's default; 1..16 otherwise).  A (variant, splits)
 * pair the shape cannot use returns QMM_ERR_UNSUPPORTED and launches nothing:
 * the "tma" variants need K/group_size (G) to be a multiple of splits and
 * 16-byte aligned scales and biases; the row-stacking "tma_w*" ones also need
 * G to be a multiple of 8, the warp-owned "tma_own_*" ones take other G when
 * N*G is a multiple of 8 and G <= 128 (each stage then holds its tile's scales
 * and biases for all G groups), shared memory permitting.                     */
qmm_status qmm_small_m_ex(const void* X, const uint32_t* Wq, const void* scales, const void* biases,
                          int M, int N, int K, int bits, int group_size, void* Y,
                          int out_dtype, int variant, int splits, void* stream);

/* Fused residual add: Y = R + X . dequant(W)^T.  R has Y's dtype and layout
 * ([M, N], bf16 or fp32 per out_dtype) and is added to the fp32 result in the
 * kernel's store, before the single rounding to Y's dtype; R may be Y itself
 * (an in-place update of a residual stream) but must not otherwise overlap it.
 * Other arguments, errors and dispatch as qmm_small_m_ex; R == NULL with a
 * non-empty output returns QMM_ERR_NULL.  K == 0 gives Y = R.
 * Source: "metal : few-row MMA mat-mul and batched copies for speculative
 * decoding" (llama.cpp PR #29869), Overview: a fusion-table entry for
 * MUL_MAT + ADD writes the residual sum from the MMA store.                    */
qmm_status qmm_small_m_residual(const void* X, const uint32_t* Wq, const void* scales, const void* biases,
                                const void* R, int M, int N, int K, int bits, int group_size, void* Y,
                                int out_dtype, int variant, int splits, void* stream);

/* Gathered form for mixture-of-experts layers at verify widths:
 *     Y[i, :] = X[lhs[i], :] . dequant(W[rhs[i]])^T,   i = 0 .. P-1
 * X bf16 [T, K]; Wq [E][N][K*bits/32], scales and biases fp16 [E][N][K/g]: a
 * stack of E matrices back to back, each in the layout above; lhs, rhs int32
 * [P] device arrays, 0 <= lhs[i] < T, 0 <= rhs[i] < E; Y [P, N].  Each expert
 * in the union of rhs is streamed once per call for all the entries that name
 * it.  P <= 256.  On the mma variants, entries per expert: at most 8 if
 * T <= 8 or P <= 8, else at most 16 (true when the k experts of each token
 * are distinct and T <= 16).
 * Source: "MLX quantized_matmul small-M verify kernels", the open question on
 * "dense and MoE (gather_qmm) verify" and the "expert-union cost per verify
 * row".
 * variant = -1: with T <= 16 and a shape the "tma_own" variants take (see
 * qmm_small_m_ex), the warp-owned kernel (the first cluster size of 1, 2, 4, 8
 * that plans) computes all T rows against each expert of the union and writes
 * the rows the entries name (then any number of entries per expert is fine);
 * otherwise the "mma" variants take each
 * expert's own entries.  A forced "tma" or "tma_own" variant takes the first
 * way (QMM_ERR_UNSUPPORTED if it cannot), a forced "mma" variant the second.
 * splits as in qmm_small_m_ex.  The index
 * lists are read on the device, after the wait for the preceding kernel: an
 * index out of range, or (mma variants) too many entries for one expert,
 * leaves the affected rows of Y unwritten and sets bit 3 of
 * qmm_device_status().  K == 0 fills Y with zeros; P == 0 or N == 0 launches
 * nothing.                                                                     */
qmm_status qmm_gather_small_m(const void* X, const uint32_t* Wq, const void* scales, const void* biases,
                              const int32_t* lhs, const int32_t* rhs, int P, int T, int E, int N, int K, int bits,
                              int group_size, void* Y, int out_dtype, int variant, int splits, void* stream);

/* ggml block formats, converted on the device to the layout above.  A row of
 * W is K/32 consecutive blocks of 32 weights; blocks of all rows are
 * contiguous, row after row.  Byte layouts (the public ggml format; the pages
 * name the formats, "metal : few-row MMA mat-mul and batched copies for
 * speculative decoding", Overview):
 *   QMM_GGML_Q4_0, 18 bytes: fp16 d; 16 bytes of 4-bit codes c, byte j holding
 *                  weight j in its low nibble and weight j + 16 in its high
 *                  nibble; w = d (c - 8).
 *   QMM_GGML_Q4_1, 20 bytes: fp16 d, fp16 m, the 16 code bytes; w = d c + m.
 *   QMM_GGML_Q8_0, 34 bytes: fp16 d, 32 signed bytes q; w = d q.                */
typedef enum { QMM_GGML_Q4_0 = 0, QMM_GGML_Q4_1 = 1, QMM_GGML_Q8_0 = 2 } qmm_ggml_type;

/* Exact conversion of a ggml matrix [N, K] (device `blocks`) into Wq
 * [N, K*bits/32], scales and biases fp16 [N, K/32] (device, caller-owned) for
 * qmm_small_m* with group_size 32 and bits = 4 (Q4_0, Q4_1) or 8 (Q8_0):
 * codes unchanged (Q4) or q + 128 (Q8_0), scale d, bias -8 d (Q4_0), m (Q4_1)
 * or -128 d (Q8_0).  Exact for every Q4_1 block, and for Q4_0 / Q8_0 blocks
 * with |d| <= 8188 / 511.75: beyond that (or for a d that is inf or NaN) the
 * bias has no finite fp16 value, the converted group is not the block, and
 * bit 4 of qmm_device_status() is set.  Asynchronous on `stream`.
 * QMM_ERR_UNSUPPORTED for an
 * unknown type, QMM_ERR_SHAPE for K not a multiple of 32, QMM_ERR_NULL /
 * QMM_ERR_ALIGN for the outputs (Wq 4-byte, scales/biases 2-byte aligned).   */
qmm_status qmm_from_ggml(int type, const void* blocks, int64_t N, int64_t K, uint32_t* Wq, void* scales,
                         void* biases, void* stream);

/* Microscaling fp modes: Y = X . W^T with w = 2^(E - 127) * value(code), one
 * E8M0 scale byte E per (row, group of 32 along K), scales uint8 [N, K/32];
 * no bias.  Codes are packed as above: QMM_MXFP4 = FP4 E2M1 (4 bits: sign, 2
 * exponent bits with bias 1, 1 mantissa bit; values 0, 0.5, 1, 1.5, 2, 3, 4,
 * 6 and negatives), QMM_MXFP8 = FP8 E4M3 (8 bits: sign, 4 exponent bits with
 * bias 7, 3 mantissa bits, exponent 0 subnormal).  Encodings: the OCP
 * microscaling format; source of the modes: "MLX quantized_matmul small-M
 * verify kernels", facts "Fix family 1" / "qmv_wide covers affine, nvfp4,
 * mxfp4, mxfp8".  variant -1 (with splits -1): the compiled-in
 * microscaling table's choice for a swept (format, N, K), at the nearest
 * measured M with as many 8-row activation tiles; else the warp-owned family
 * when it can plan the shape (K/g a multiple of the cluster size, scales
 * 16-byte aligned, and K/g a multiple of 16 or else N*K/g a multiple of 16
 * with K/g <= 256), else the first "mma" variant; a forced "mma" or
 * "tma_own" variant is used as given, a "tma" variant returns
 * QMM_ERR_UNSUPPORTED.
 * QMM_NVFP4: FP4 E2M1 codes with one FP8 E4M3 scale byte per group of 16,
 * scales uint8 [N, K/16] (a per-tensor scale, where a model has one, is left
 * to the caller).
 * K must be a multiple of 32.  NaN encodings are NaN, as the OCP format
 * defines them: an E4M3 code or nvfp4 scale byte 0x7F / 0xFF, an E8M0 scale
 * 255; every output whose sum meets one is NaN.  Errors as qmm_small_m_ex.    */
typedef enum { QMM_MXFP4 = 0, QMM_MXFP8 = 1, QMM_NVFP4 = 2 } qmm_mx_format;
qmm_status qmm_small_m_mx(const void* X, const uint32_t* Wq, const uint8_t* scales, int M, int N, int K, int format,
                          void* Y, int out_dtype, int variant, int splits, void* stream);

/* Quantisation into the microscaling formats: row r of X [R, K] (bf16 or fp32
 * by x_dtype, rows ldx >= K elements apart) is cut into groups of g = 32
 * (QMM_NVFP4: 16) along K; with a the largest |x| of a group
 *   QMM_MXFP4, QMM_MXFP8: scale byte E = clamp(floor(log2 a) - e + 127, 0, 254),
 *              e = 2 (E2M1) or 8 (E4M3), E = 0 for a = 0; s = 2^(E - 127);
 *   QMM_NVFP4: s = a / 6 (one fp32 division) rounded to E4M3, at most 448;
 * and every code is x / s rounded to the nearest value of the format, ties to
 * the even code, beyond the largest value to the largest; the sign of x stays.
 * s = 0 gives codes 0 (with x's signs).  A group that holds a NaN or an
 * infinity gets a NaN scale (255; nvfp4 0x7F) and codes +0.
 * Wq [R, K*bits/32] and scales [R, K/g] have the layout qmm_small_m_mx reads, and
 * may be the weights of the next call on the stream (see Execution).
 * values: null, or bf16 [R, K]: what the codes stand for, s * value(code) (to
 * nearest even where bf16 cannot hold it: mxfp8 below 2^-130 only).
 * K must be a multiple of 32 (QMM_ERR_SHAPE); X and values are aligned to
 * their element, Wq to 4 bytes.  R == 0 or K == 0 launches nothing.  X must
 * not overlap the outputs.                                                    */
qmm_status qmm_quantize_mx(const void* X, int x_dtype, int64_t R, int64_t K, int64_t ldx, int format, uint32_t* Wq,
                           uint8_t* scales, void* values, void* stream);

/* Product of two microscaled 4-bit matrices, any number of rows:
 *     Y[M,N] = Xv[M,K] . Wv[N,K]^T
 * Xq, Wq: E2M1 codes [M, K/8] and [N, K/8] words; x_scales, w_scales
 * [M, K/g] and [N, K/g]; format QMM_MXFP4 or QMM_NVFP4 (QMM_MXFP8:
 * QMM_ERR_UNSUPPORTED); as qmm_quantize_mx writes them.  Products of codes and
 * scales are exact, sums fp32; Y is bf16 (round to nearest even) or fp32.  NaN
 * scales give NaN outputs.  K must be a multiple of 32, M and N at most 2^30;
 * Xq and Wq are 16-byte aligned.  M == 0 or N == 0 launches nothing, K == 0
 * fills Y with zeros.                                                         */
qmm_status qmm_matmul_mx(const uint32_t* Xq, const uint8_t* x_scales, const uint32_t* Wq, const uint8_t* w_scales,
                         int M, int N, int K, int format, void* Y, int out_dtype, void* stream);

/* Experts of every token from a router's logits [T, E] (bf16 or fp32, rows ld
 * elements apart).  With the scores s = softmax(x) or sigmoid(x) and the keys
 * c = s + bias[e] (bias fp32 [E], null: none; compared in 64 bits)
 *   the E experts form `groups` groups of neighbours; a group is worth the sum of its
 *   group_best (1 or 2) best keys, and the top_groups groups worth most are open
 *   (top_groups == groups: all);
 *   the k best keys of the open groups are chosen, best first (without a bias the best
 *   logits), of equals the lowest number;
 *   weights[t, j] = scale * s, or, with renormalize, scale * s / (sum of the k scores).
 * The bias chooses; it is not part of the weights.  A NaN logit counts as -inf; an
 * expert of -inf is chosen last, has weight 0 and adds nothing to its group; +inf
 * counts as the largest finite number; a NaN key counts as -inf.  Renormalised weights
 * are ratios of scores however small; where all chosen logits are -inf they are 0.
 * experts int32 [T, k]: flattened, the list rhs of qmm_gather_small_m for T k <= 256
 * entries; weights fp32 [T, k].  E <= 512 a multiple of groups <= 32; k <= 32, at most
 * the experts of top_groups groups.  T == 0 launches nothing.                      */
typedef enum { QMM_SOFTMAX = 0, QMM_SIGMOID = 1 } qmm_scoring;
qmm_status qmm_route_experts(const void* logits, int logits_dtype, int64_t ld, const float* bias, int T, int E, int k,
                             int scoring, int groups, int top_groups, int group_best, int renormalize, float scale,
                             int32_t* experts, float* weights, void* stream);

/* Low-rank adapters of many requests beside a shared projection:
 *     Y[t] = base[t] + scales[a] * Bm[a] (A[a] X[t]),  a = adapters[t]
 * X bf16 [T, K] (rows x_ld apart), A bf16 [L, R, K] and Bm bf16 [L, N, R] contiguous,
 * adapters int32 [T], scales fp32 [L] (null: 1); base and Y bf16 or fp32 by out_dtype,
 * rows base_ld and y_ld elements apart; Y may be base (with y_ld == base_ld), and
 * nothing else may overlap Y.  Sums are fp32, and one rounding to Y's type; the
 * products with Bm keep 24 bits of A X (16 where Y is bf16).  A row with a negative
 * number has no adapter: Y[t] = base[t], and X[t] is not read.  A number >= L sets bit 3
 * of qmm_device_status() and counts as none.  R is a multiple of 8 up to 128 (an adapter
 * of a smaller rank is padded with zeros), K a multiple of 8, N any; X, A, Bm 16-byte
 * aligned, x_ld a multiple of 8.  At most some 65000 tiles of rows: T / 16 plus the
 * smaller of T and L + 1, or T / 64 where that is 32 rows an adapter (QMM_ERR_SHAPE).
 * workspace: qmm_lora_workspace(T, L, R) bytes, 16-byte aligned, not shared by calls that
 * may run at the same time.  T == 0 or N == 0 launches nothing.                      */
qmm_status qmm_lora_add(const void* base, int64_t base_ld, const void* X, int64_t x_ld, const void* A, const void* Bm,
                        const int32_t* adapters, const float* scales, int T, int N, int K, int R, int L, void* Y,
                        int64_t y_ld, int out_dtype, void* workspace, size_t workspace_bytes, void* stream);
size_t qmm_lora_workspace(int T, int L, int R);

/* A paged key-value cache.  Token j of sequence b lives in page
 * block_table[b][j / page_size] at slot j mod page_size; its key for head h
 * starts at k + page * k_page + slot * k_token + h * k_head (strides in
 * elements; the D elements of a head are contiguous), its value likewise.
 * QMM_KV_E4M3 elements stand for k_scale (v_scale) times their E4M3 value;
 * QMM_KV_BF16 ignores the scales.
 * lengths[b] counts the tokens of sequence b including its new rows.
 * A page number outside 0..num_pages-1 or a length outside
 * 0..max_pages*page_size sets bit 5 of qmm_device_status(): tokens of such a
 * page are not written and read as zeros, and the length is clamped.
 * All device arrays; page_size >= 1.                                          */
typedef enum { QMM_KV_BF16 = 0, QMM_KV_E4M3 = 1 } qmm_kv_dtype;
typedef struct {
  void* k;
  void* v;
  int64_t k_page, k_token, k_head;
  int64_t v_page, v_token, v_head;
  const int32_t* block_table; /* [B][table_stride], the first max_pages of each row are read */
  const int32_t* lengths;     /* [B] */
  int64_t table_stride;
  int64_t num_pages;
  int32_t max_pages;
  int32_t page_size;
  int32_t heads;              /* key-value heads */
  int32_t head_dim;           /* D: 64, 128 or 256 */
  int32_t dtype;              /* qmm_kv_dtype */
  float k_scale, v_scale;
} qmm_paged_cache;

/* Writes the new rows' keys and values into the cache: row i < m_b of
 * sequence b goes to position lengths[b] - m_b + i (rows whose position is
 * negative are dropped).  k_new, v_new: bf16, row b*M + i starts k_ld (v_ld)
 * elements after row 0 times that index, its heads * D elements contiguous (so
 * both may be slices of one projection's output).  m_b = q_lens[b] clamped to
 * 0..M, or M if q_lens is null.  E4M3 elements are x / scale (one fp32
 * division), nearest even, at most 448 in magnitude; NaN stays NaN.
 * k, v, k_new, v_new 16-byte aligned, strides multiples of 16 bytes (else
 * QMM_ERR_ALIGN).  Two rows of one call must not name the same slot.          */
qmm_status qmm_kv_append(const qmm_paged_cache* cache, const void* k_new, int64_t k_ld, const void* v_new, int64_t v_ld,
                         int B, int M, const int32_t* q_lens, void* stream);

/* qmm_kv_append with rotary positions on the way.  A head's elements x[0 .. rot - 1] form
 * pairs: (x[j], x[j + rot/2]), or with interleaved (x[2j], x[2j + 1]); pair j of a row at
 * position p turns by t = p * inv_freq[j]:
 *     (x1, x2) -> factor * (x1 cos t - x2 sin t, x2 cos t + x1 sin t);
 * elements from rot on stay.  Angles hold at any 32-bit position (inv_freq finite, its
 * product with p is not rounded); sums are fp32, with one rounding to the output's type.
 * q (bf16, row b*M + i q_ld elements apart, q_heads * D contiguous) goes to q_out (bf16,
 * rows q_out_ld apart; it may be q, with q_out_ld == q_ld, and nothing else may overlap
 * it), the keys to the cache; the values are not turned.  Rows i >= m_b of q_out are 0.
 * Positions: null, lengths[b] - m_b + i; or int32 [axes][B][M], pair j going by axis 0
 * for j < sections[0], by axis 1 for the next sections[1], and so on (sections add up
 * to rot/2; axes <= 4).  They turn only: a key's place in the cache is always that of
 * its row, as in qmm_kv_append, whose other rules hold too, for any M.  rot is a
 * multiple of 16 up to D.                                                          */
typedef struct {
  const float* inv_freq;    /* device, [rot / 2] */
  const int32_t* positions; /* device or null */
  int32_t rot;
  int32_t axes;
  int32_t sections[4];
  int32_t interleaved;
  float factor;
} qmm_rope;
qmm_status qmm_rope_append(const qmm_paged_cache* cache, const qmm_rope* rope, const void* q, int64_t q_ld, int q_heads,
                           void* q_out, int64_t q_out_ld, const void* k_new, int64_t k_ld, const void* v_new,
                           int64_t v_ld, int B, int M, const int32_t* q_lens, void* stream);

/* Attention of M = 1..16 new rows of each of B sequences over the cache.  Row
 * i < m_b of sequence b stands at position p = lengths[b] - m_b + i and sees
 * the tokens j <= p with window == 0, or j > p - window, or j < sinks:
 *     out[b,i,h] = sum_j softmax_j(scale * q[b,i,h] . k[j,h / G]) v[j,h / G],
 * G = q_heads / cache heads (a whole number up to 1024).  q: bf16, row b*M + i q_ld
 * elements apart, q_heads * D contiguous; out: bf16 [B, M, q_heads, D]; lse:
 * null or fp32 [B, M, q_heads], log sum_j exp(scale * q . k_j).  scale is finite,
 * and an E4M3 cache's k_scale times it too (else QMM_ERR_UNSUPPORTED).  A row that
 * sees no token, and rows i >= m_b: out 0, lse -inf.  What a row does not see
 * never reaches it, whatever is stored there.  Scores, softmax statistics and
 * sums are fp32; probabilities enter the second product as two bf16 operands
 * that hold 16 of their bits (for an E4M3 cache as one in fp16: 11 bits, fewer
 * below 2^-29 of the row's largest, none below 2^-40).
 * workspace: qmm_paged_attention_workspace() bytes, 16-byte aligned, not shared
 * by calls that may run at the same time; contents need no initialisation.
 * Alignment as qmm_kv_append (q and out too).                                 */
qmm_status qmm_paged_attention(const qmm_paged_cache* cache, const void* q, int64_t q_ld, int B, int M, int q_heads,
                               const int32_t* q_lens, float scale, int window, int sinks, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream);
size_t qmm_paged_attention_workspace(int B, int M, int q_heads, int heads, int head_dim);

/* qmm_paged_attention of sequences that share their first tokens: tokens
 * 0 .. P - 1 of every sequence, P = num_prefix_pages * page_size, lie in prefix_pages
 * (device int32), token P + j of sequence b in page block_table[b][j / page_size]
 * (max_pages counts the pages of own tokens).  lengths[b] counts all tokens, the prefix
 * and the new rows among them, and the new rows come after the prefix:
 * lengths[b] - m_b >= P.  A sequence of length 0, and one with m_b == 0, has no rows; any
 * other length below P + m_b, or beyond the table, sets bit 5 of qmm_device_status(),
 * and that sequence's rows see nothing.  Without window and sinks; otherwise arguments,
 * results and errors are qmm_paged_attention's.  The prefix is read once for all rows.
 * Probabilities enter the second product with 16 bits (for an E4M3 cache as one fp16
 * operand: 11 bits, fewer below 2^-25 of the row's largest, none below 2^-36).       */
qmm_status qmm_shared_prefix_attention(const qmm_paged_cache* cache, const int32_t* prefix_pages, int num_prefix_pages,
                                       const void* q, int64_t q_ld, int B, int M, int q_heads, const int32_t* q_lens,
                                       float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                       void* stream);
size_t qmm_shared_prefix_attention_workspace(int B, int M, int q_heads, int heads, int head_dim);

/* Verification of drafted tokens against the target's logits [B, k+1, V] (bf16
 * or fp32; row i is the target's distribution after i accepted drafts, rows
 * row_stride, sequences batch_stride elements apart), from given random
 * numbers.  With p_i = softmax(logits_i / temperature[b]) and q_i =
 * draft_probs[b, i] (fp32 [B, k, V], what the draft drew token d_i from; null:
 * the drafts were certain, q_i(d_i) = 1), draft i is accepted while
 *     uniform[b, i] * q_i(d_i) < p_i(d_i).
 * After n accepted drafts the next token is the v with the largest
 * w(v) / noise[b, v] (noise fp32 [B, V], exponentially distributed, > 0; one
 * that is NaN or negative counts as +inf; the lowest v of equals): w = max(p_n - q_n, 0) where draft n was refused
 * (w = p_n if that is 0 everywhere), w = p_n where all were accepted.
 * temperature[b] <= 0 or NaN is greedy: a draft is accepted if it is the lowest
 * argmax of its row, and the next token is the argmax of row n.
 * draft_lens (null: k everywhere): sequence b has draft_lens[b] drafts, clamped
 * to 0..k.  A draft outside 0..V-1 is refused (with draft_probs null, q_n is
 * then 0 everywhere).  A NaN logit counts as -inf, which has probability 0.  A
 * row whose largest logit is not finite (-inf everywhere, or a +inf) has no
 * softmax: no draft is accepted on it and its token is its lowest argmax.
 * tokens int32 [B, k+1]: the accepted drafts, the next token, then -1;
 * accepted int32 [B]: n.  0 <= k <= 31, 1 <= V <= 2^30.                        */
qmm_status qmm_verify_draft(const void* logits, int logits_dtype, int64_t batch_stride, int64_t row_stride,
                            const int32_t* draft_tokens, const float* draft_probs, const float* uniform,
                            const float* noise, const float* temperature, const int32_t* draft_lens, int B, int k,
                            int V, int32_t* tokens, int32_t* accepted, void* stream);

/* Number of uint32 words of a packed [N, K] matrix: N * K * bits / 32
 * (0 if bits is unsupported or K*bits is not a multiple of 32).                 */
size_t qmm_packed_words(int64_t N, int64_t K, int bits);

/* Host-side packing of codes q[N,K] (one code per byte, each < 2^bits) into the
 * word layout above.  Host pointers.  Returns QMM_ERR_SHAPE for a code out of
 * range or a K that does not fill whole words.                                 */
qmm_status qmm_pack(const uint8_t* q, int64_t N, int64_t K, int bits, uint32_t* Wq);

/* Inverse of qmm_pack (host pointers).                                          */
qmm_status qmm_unpack(const uint32_t* Wq, int64_t N, int64_t K, int bits, uint8_t* q);

/* Conversion between the canonical layout above and the layout the kernels
 * read ("native").  The kernels read the canonical layout directly (the
 * k-permutation their tensor-core fragments need is applied to the
 * activations while they are staged), so the native layout IS the canonical
 * one: both calls are a stream-ordered device-to-device copy of
 * N*K*bits/8 bytes on `stream`, and nothing when the two pointers are equal.
 * Device pointers, caller-owned; the buffers must not partly overlap.
 * QMM_ERR_UNSUPPORTED for bits not in {2,4,8}, QMM_ERR_SHAPE for a K that
 * does not fill whole words, QMM_ERR_NULL for a null pointer with a non-empty
 * matrix, QMM_ERR_CUDA if the copy cannot be queued.                            */
qmm_status qmm_repack(const uint32_t* Wq, int64_t N, int64_t K, int bits, uint32_t* Wq_native, void* stream);
qmm_status qmm_unrepack(const uint32_t* Wq_native, int64_t N, int64_t K, int bits, uint32_t* Wq, void* stream);

/* Introspection of the dispatcher: the variant and split count qmm_small_m
 * would use, or -1 (and *splits untouched) if the shape is unsupported or the
 * table is unusable.  The table is compiled in; the environment variable
 * QMM_TABLE=<path> replaces it, for the whole process, by a file in the
 * format of the compiled one (lines "{M, N, K, bits, group, variant, splits},",
 * text after "//" ignored).  QMM_FORCE_VARIANT=<name or id> and
 * QMM_FORCE_SPLITS=<n> override the choice; QMM_LOG=1 prints it to stderr.      */
int qmm_select_variant(int M, int N, int K, int bits, int group_size, int* splits);

int qmm_num_variants(void);
const char* qmm_variant_name(int variant);     /* NULL for an unknown id          */
const char* qmm_status_string(int status);
int qmm_last_cuda_error(void);                 /* cudaError_t of the last failure */

/* Device status word of the kernels, OR-ed over all kernel units: bit 0 = a
 * consumer gave up waiting for a weight tile, bit 1 = the producer gave up
 * waiting for a free stage, bit 2 = copies still in flight at exit gave up,
 * bit 3 = a gathered call had an invalid index list (see qmm_gather_small_m), or
 * qmm_lora_add an adapter's number out of range,
 * bit 4 = qmm_from_ggml met a block outside its exact range, bit 5 = a paged
 * cache call met an invalid page number or length (see qmm_paged_cache).
 * Every wait is bounded (about 2 s), so a fault shows up here instead of as a
 * hang.  Synchronizes with the device; clears the word when `clear` != 0.
 * 0xFFFFFFFF if the word could not be read.                                    */
unsigned int qmm_device_status(int clear);
const char* qmm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H_ */
