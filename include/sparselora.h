/* sparselora.h — C ABI of the contextual-sparsity LoRA hot path on gfx950.
 *
 * What the library computes (sources are the pages the method is described on):
 *   - "SparseLoRA article": the lsdiaocha.cn write-up of SparseLoRA (ICML 2025),
 *     sections 一 (dynamic contextual sparsity; L2-norm criterion for the FFN,
 *     QK-norm criterion for q/k), 二 (training-free SVD sparsity estimator,
 *     computed once offline, low-rank approximation of the activations),
 *     三 (non-uniform per-layer sparsity; context tokens sparse, output tokens
 *     dense), 六 (structured sparsity for real GPU speedups) and 七 (rank-8
 *     estimator; careful slicing of sparse weights and compute order).
 *   - "SparseLoRA abstract": the xinfinite.net page "SparseLoRA：利用上下文稀疏性
 *     高效微调大语言模型" — loss and gradients are computed on a dynamically
 *     selected sparse subset of the weights.
 *   - "SALR page": the lshu.cn article, §2.1 — LoRA notation: frozen W plus a
 *     trained product of two low-rank factors.
 *
 * Conventions shared by every entry point
 *   - Tensor arguments are DEVICE pointers to row-major, contiguous arrays,
 *     16-byte aligned, unless a comment says [host].  Element type is given by
 *     the call's sl_dtype (fp32 or bf16) unless the comment says fp32/int32.
 *   - Tokens are packed as T = batch * seq_len rows; sequence b owns rows
 *     [b*seq_len, (b+1)*seq_len).  Its first ctx_len[b] rows are context tokens
 *     (computed on the selected channels only); the remaining seq_len-ctx_len[b]
 *     rows are output (loss) tokens and are computed dense.
 *   - LoRA: y = x W^T + s (x A^T) B^T with A [r, in], B [out, r] and s = lora_scale.
 *     A dropped channel drops its LoRA part too.
 *   - Channel index sets idx [batch, k] hold, per sequence, k distinct channel
 *     numbers in ascending order (what sl_estimate_select writes).  Callers may
 *     pass their own; they are not re-validated on the device.
 *   - The library never allocates device memory.  Scratch space is the caller's
 *     `ws` buffer (query its size with the *_workspace_bytes function); state the
 *     backward needs is written by the forward into the caller's `saved` buffer.
 *     No pointer is kept after a call returns.
 *   - All work is enqueued on `stream` (a hipStream_t, NULL = default stream).
 *     Calls never synchronise, except sl_build_estimator (documented there).
 *     Calls overlap independent parts of their work on a side stream (default
 *     priority, non-blocking), forked from and joined back to `stream` with
 *     events: the call's work completes in order on `stream` as if it had all
 *     been enqueued there.  Each (device, `stream`) pair gets a side stream of
 *     its own at its first call, kept until the process ends, so calls on
 *     independent streams never wait for each other; past 256 such pairs a
 *     call keeps all of its work on `stream`.  While `stream` is being
 *     captured into a graph, all of the call's work stays on it (the graph
 *     holds no cross-stream events).
 *   - Every argument is validated on the host before anything is launched.  On
 *     error nothing is launched, the status says which class of error, and
 *     sl_last_error() (thread-local) holds a message.  Launch failures map to
 *     SL_ERR_HIP; device faults surface at the caller's next synchronisation.
 *   - Calls that share a `ws` or `saved` buffer must be stream-ordered.
 */
#ifndef SPARSELORA_H
#define SPARSELORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SL_ABI_VERSION 3
#define SL_MAX_SEQS 64  /* sequences per call (batch) */

typedef enum sl_status {
  SL_OK = 0,
  SL_ERR_NULL = 1,              /* a required pointer is NULL */
  SL_ERR_ALIGN = 2,             /* a pointer is not 16-byte aligned */
  SL_ERR_SHAPE = 3,             /* inconsistent or unsupported sizes */
  SL_ERR_DTYPE = 4,             /* unknown sl_dtype / sl_criterion */
  SL_ERR_RANGE = 5,             /* k, rank, ctx_len or batch out of range */
  SL_ERR_WORKSPACE = 6,         /* ws or saved buffer too small */
  SL_ERR_UNSUPPORTED_ARCH = 7,  /* current device is not gfx950 */
  SL_ERR_HIP = 8                /* a HIP runtime call or launch failed */
} sl_status;

typedef enum sl_dtype { SL_F32 = 0, SL_BF16 = 1 } sl_dtype;

/* Channel criteria (SparseLoRA article §一):
 *   SWIGLU_L2 — FFN: sum over context tokens of h^2, h = SiLU(g) * u with g, u
 *               the low-rank estimates of the gate and up projections.
 *   L2        — a plain projection (v; o reuses v's set): sum of v^2.
 *   QK_NORM   — q/k, in kv-channel space: ||k_c||^2 * sum over the query heads
 *               sharing kv head of c of ||q_(h,d)||^2 ((||q_c|| ||k_c||)^2 when
 *               every query head has its own kv head). */
typedef enum sl_criterion { SL_CRIT_SWIGLU_L2 = 0, SL_CRIT_L2 = 1, SL_CRIT_QK_NORM = 2 } sl_criterion;

typedef struct sl_layout {
  int32_t batch;            /* 1..SL_MAX_SEQS sequences */
  int32_t seq_len;          /* rows per sequence */
  const int32_t* ctx_len;   /* [host] batch entries, 0 <= ctx_len[b] <= seq_len */
} sl_layout;

typedef struct sl_heads {
  int32_t n_q_heads, n_kv_heads, head_dim;   /* n_q_heads % n_kv_heads == 0 */
} sl_heads;

/* Frozen weights and LoRA factors of one SwiGLU FFN layer (call dtype).
 *   Wg, Wu  [d_ff, d_model]   gate / up projection weights
 *   WdT     [d_ff, d_model]   TRANSPOSE of the down projection weight [d_model, d_ff]
 *                             (a one-time copy; the weight is frozen)
 *   Ag, Au  [r, d_model]      Bg, Bu [d_ff, r]
 *   Ad      [r, d_ff]         Bd     [d_model, r]                               */
typedef struct sl_ffn_weights {
  int64_t d_model, d_ff;
  int32_t lora_rank;
  float lora_scale;
  const void *Wg, *Wu, *WdT;
  const void *Ag, *Bg, *Au, *Bu, *Ad, *Bd;
  /* Optional 4-bit frozen base (SparseLoRA article §六: SparseLoRA over a
   * QLoRA-style quantized base).  When Wg_q is not NULL the frozen weights are
   * these, and Wg, Wu, WdT are ignored (may be NULL):
   *   Wg_q, Wu_q, WdT_q  uint8 [d_ff, d_model / 2]: element 2j of a row in the
   *                      low nibble of byte j, element 2j+1 in the high nibble,
   *                      signed two's-complement codes
   *   Wg_s, Wu_s, WdT_s  fp32 [d_ff, d_model / 64]: the scale of each block of
   *                      64 consecutive elements of a row
   * The weight element is code * scale.  bf16 calls only; d_model a multiple of
   * 64; all six 16-byte aligned.  Zero-initialised (C) or NULL: plain weights. */
  const void *Wg_q, *Wu_q, *WdT_q;
  const float *Wg_s, *Wu_s, *WdT_s;
} sl_ffn_weights;

/* LoRA gradients of one FFN layer, fp32, shapes of the factors; OVERWRITTEN. */
typedef struct sl_ffn_grads {
  float *dAg, *dBg, *dAu, *dBu, *dAd, *dBd;
} sl_ffn_grads;

/* Frozen weights and LoRA factors of one attention block's projections.
 *   Wq  [Hq*hd, d_model]   Wk, Wv [Hkv*hd, d_model]
 *   WoT [Hq*hd, d_model]   TRANSPOSE of the o projection weight [d_model, Hq*hd]
 *   Aq, Ak, Av [r, d_model]; Bq [Hq*hd, r]; Bk, Bv [Hkv*hd, r]
 *   Ao [r, Hq*hd]; Bo [d_model, r]                                             */
typedef struct sl_qkvo_weights {
  int64_t d_model;
  sl_heads heads;
  int32_t lora_rank;
  float lora_scale;
  const void *Wq, *Wk, *Wv, *WoT;
  const void *Aq, *Bq, *Ak, *Bk, *Av, *Bv, *Ao, *Bo;
  /* Optional 4-bit frozen bases, in the format of sl_ffn_weights (uint8 codes
   * [rows, d_model / 2], fp32 scales [rows, d_model / 64]).  Wq_q set: q, k and
   * v read Wq_q/Wk_q/Wv_q with Wq_s/Wk_s/Wv_s, and Wq, Wk, Wv are ignored.
   * WoT_q set: o reads WoT_q with WoT_s, and WoT is ignored.  bf16 calls
   * only; d_model a multiple of 64; 16-byte aligned.  NULL: plain weights. */
  const void *Wq_q, *Wk_q, *Wv_q, *WoT_q;
  const float *Wq_s, *Wk_s, *Wv_s, *WoT_s;
} sl_qkvo_weights;

typedef struct sl_qkvo_grads {   /* fp32, shapes of the factors; OVERWRITTEN */
  float *dAq, *dBq, *dAk, *dBk, *dAv, *dBv, *dAo, *dBo;
} sl_qkvo_grads;

int sl_abi_version(void);
const char* sl_status_string(sl_status s);
const char* sl_last_error(void);          /* thread-local message of the last error */

/* ---------------------------------------------------------------------------
 * a0 — offline estimator build (SparseLoRA article §二 and §七: truncated SVD of
 * each frozen projection weight, done once before training).
 *   W     [out_f, in_f]  frozen weight (call dtype)
 *   Pt    [rank, in_f]   (V_r diag(sigma_r))^T, call dtype      (output)
 *   Q     [rank, out_f]  U_r^T, call dtype                       (output)
 *   sigma [rank] fp32, optional (NULL = not written)            (output)
 * so that x Pt^T Q approximates x W^T.  Computed by block subspace iteration
 * on the GPU in fp32 with a host fp64 Rayleigh-Ritz step; 1 <= rank <= 64 and
 * rank <= min(out_f, in_f).  SYNCHRONISES `stream` (offline, untimed).
 * ------------------------------------------------------------------------- */
size_t sl_estimator_workspace_bytes(int64_t out_f, int64_t in_f, int32_t rank);
sl_status sl_build_estimator(sl_dtype dt, const void* W, int64_t out_f, int64_t in_f,
                             int32_t rank, int32_t iters, void* Pt, void* Q, float* sigma,
                             void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * a1-a3 — estimate, score, select (SparseLoRA article §一, §二, §三).
 *   X   [T, d_in]  layer input (call dtype); only context rows are read.
 *   SWIGLU_L2: (Pt0,Q0) = gate factors, (Pt1,Q1) = up factors, N = d_ff.
 *   L2:        (Pt0,Q0) = the projection's factors, N = its out features.
 *   QK_NORM:   (Pt0,Q0) = q factors (Q0 [rank, Hq*hd]), (Pt1,Q1) = k factors
 *              (Q1 [rank, Hkv*hd]); N = Hkv*hd (selection in kv-channel space).
 *   Pt* [rank, d_in], Q* [rank, N_proj] (call dtype), 1 <= rank <= 32.
 *   idx    [batch, k] int32 out: per sequence the k best channels, ascending;
 *          ties in score go to the lower channel index.
 *   scores [batch, N] fp32 out, optional (NULL = not written): the criterion
 *          (a sum of squares over the sequence's context tokens).
 * 1 <= k <= N <= 65536.  The workspace holds the context tokens' projections,
 * the criterion's partial sums and every sequence's N selection keys.  heads
 * is read for QK_NORM only.  The workspace size query takes the same
 * criterion, layout, heads, d_in, rank and N as the call.
 * ------------------------------------------------------------------------- */
size_t sl_estimate_select_workspace_bytes(sl_criterion crit, const sl_layout* lay,
                                          const sl_heads* heads, int64_t d_in, int32_t rank,
                                          int64_t N);
sl_status sl_estimate_select(sl_criterion crit, sl_dtype dt, const sl_layout* lay,
                             const sl_heads* heads, const void* X, int64_t d_in, int32_t rank,
                             const void* Pt0, const void* Q0, const void* Pt1, const void* Q1,
                             int64_t N, int32_t k, int32_t* idx, float* scores,
                             void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * sl_estimate_select without a workspace, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Same arguments and results as sl_estimate_select,
 * minus ws / ws_bytes: the scratch is a fixed array of SL_NOALLOC_SCRATCH_BYTES
 * in the library's device memory, one per device, held from the library's
 * load until the process ends.  A call whose sl_estimate_select_workspace_bytes
 * exceeds that size returns SL_ERR_WORKSPACE (nothing launched).  The call
 * allocates nothing.  Every call on one device shares that device's array, so
 * calls that overlap on one device (different streams, or different threads
 * without stream order) race; calls in one stream's order do not.  Nothing in
 * the array needs to start at zero: every call writes what it reads.
 * ------------------------------------------------------------------------- */
#define SL_NOALLOC_SCRATCH_BYTES (32u << 20)
sl_status sl_estimate_select_noalloc(sl_criterion crit, sl_dtype dt, const sl_layout* lay,
                                     const sl_heads* heads, const void* X, int64_t d_in, int32_t rank,
                                     const void* Pt0, const void* Q0, const void* Pt1, const void* Q1,
                                     int64_t N, int32_t k, int32_t* idx, float* scores, void* stream);

/* ---------------------------------------------------------------------------
 * a1-a3 for several criteria over one input (SparseLoRA article §一, §二, §三:
 * an attention layer scores q/k by the QK-norm and v/o by the L2 norm of the
 * same layer input).  Same results as one sl_estimate_select call per job, but
 * X is projected once onto every job's leading directions, all L2-type
 * criteria share one launch and all selections share one launch.
 *   jobs[j]: crit, heads (QK_NORM only), Pt0/Q0/Pt1/Q1, N, k, idx, scores as in
 *            sl_estimate_select; every job shares X, the layout, d_in and rank.
 * 1 <= njobs <= SL_EST_MAXJOBS, and the jobs' projections (2 for SWIGLU_L2 and
 * QK_NORM, 1 for L2) number at most 4.  Jobs must write distinct idx / scores
 * buffers.  The workspace query takes the same layout, d_in, rank and jobs
 * (only crit, heads and N are read).
 * ------------------------------------------------------------------------- */
#define SL_EST_MAXJOBS 3
typedef struct sl_est_job {
  sl_criterion crit;
  sl_heads heads;                  /* QK_NORM only */
  const void *Pt0, *Q0, *Pt1, *Q1;  /* Pt1 / Q1 unused for L2 */
  int64_t N;
  int32_t k;
  int32_t* idx;                    /* [batch, k] out */
  float* scores;                   /* [batch, N] out, optional */
} sl_est_job;
size_t sl_estimate_select_multi_workspace_bytes(const sl_layout* lay, int64_t d_in, int32_t rank,
                                                int32_t njobs, const sl_est_job* jobs);
sl_status sl_estimate_select_multi(sl_dtype dt, const sl_layout* lay, const void* X, int64_t d_in,
                                   int32_t rank, int32_t njobs, const sl_est_job* jobs, void* ws,
                                   size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * a4/a5 — sparse SwiGLU FFN forward and backward (SparseLoRA article §一, §三,
 * §六, §七; SparseLoRA abstract).  Context rows of sequence b use channels
 * idx[b, :k]; output rows use all d_ff channels.
 *   fwd:  X [T, d_model] -> Y [T, d_model]; writes `saved` for the backward.
 *   bwd:  dY [T, d_model] + saved -> dX [T, d_model] and the six LoRA gradients.
 *         X, w, k, idx and the layout must be those of the forward call.
 * d_model % 8 == 0, d_ff % 8 == 0, 1 <= lora_rank <= 32, 1 <= k <= d_ff.
 * Every matrix a call reads or writes holds fewer than 2^31 elements:
 * batch*seq_len*d_model, d_ff*d_model and the compact activation buffers
 * (sum of ctx_len * round_up(k, 8) + output rows * d_ff); SL_ERR_RANGE
 * otherwise, before anything is launched.
 * ------------------------------------------------------------------------- */
size_t sl_ffn_saved_bytes(sl_dtype dt, const sl_layout* lay, int64_t d_model, int64_t d_ff,
                          int32_t lora_rank, int32_t k);
size_t sl_ffn_workspace_bytes(sl_dtype dt, const sl_layout* lay, int64_t d_model, int64_t d_ff,
                              int32_t lora_rank, int32_t k);
sl_status sl_ffn_fwd(sl_dtype dt, const sl_layout* lay, const sl_ffn_weights* w, const void* X,
                     int32_t k, const int32_t* idx, void* Y, void* saved, size_t saved_bytes,
                     void* ws, size_t ws_bytes, void* stream);
sl_status sl_ffn_bwd(sl_dtype dt, const sl_layout* lay, const sl_ffn_weights* w, const void* X,
                     int32_t k, const int32_t* idx, const void* saved, size_t saved_bytes,
                     const void* dY, void* dX, const sl_ffn_grads* g,
                     void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * a6/a7 — sparse q/k/v/o projections (SparseLoRA article §一, §三, §六).
 * idx_qk [batch, k_qk] and idx_vo [batch, k_vo] are kv-channel sets (as written
 * by sl_estimate_select with QK_NORM and L2); q and o use them expanded to every
 * query head of the group (query head j is of the group of kv head j / (Hq / Hkv)).  At context rows, unselected channels of q, k, v are
 * written as 0 and unselected columns of the attention output a are ignored.
 *   fwd:  X [T, d_model] -> q [T, Hq*hd], k, v [T, Hkv*hd]   (if X != NULL)
 *         a [T, Hq*hd]   -> o [T, d_model]                  (if a != NULL)
 *         so a caller may run q/k/v, its attention, then o, as two calls
 *         sharing one `saved` buffer.
 *   bwd:  d_out -> da [T, Hq*hd] and dAo, dBo                (if d_out != NULL)
 *         dq, dk, dv -> dX and dAq..dBv                      (if dq != NULL)
 *         X and a (the forward's inputs) are read for the factor gradients.
 *         The d_out part reads what the forward's a part left in `saved`
 *         (z_o and the packed Bo^T, Ao^T); the dq part what its X part left
 *         (z_q, z_k, z_v).
 * d_model, Hq*hd and Hkv*hd multiples of 8; 1 <= lora_rank <= 32;
 * 1 <= k_qk, k_vo <= Hkv*hd.  Every matrix a call reads or writes holds
 * fewer than 2^31 elements (T*d_model, T*Hq*hd, Hq*hd*d_model and the compact
 * projection buffers); SL_ERR_RANGE otherwise, before anything is launched.
 * ------------------------------------------------------------------------- */
size_t sl_qkvo_saved_bytes(sl_dtype dt, const sl_layout* lay, const sl_qkvo_weights* w);
size_t sl_qkvo_workspace_bytes(sl_dtype dt, const sl_layout* lay, const sl_qkvo_weights* w,
                               int32_t k_qk, int32_t k_vo);
sl_status sl_qkvo_fwd(sl_dtype dt, const sl_layout* lay, const sl_qkvo_weights* w,
                      const void* X, const void* a,
                      int32_t k_qk, const int32_t* idx_qk, int32_t k_vo, const int32_t* idx_vo,
                      void* q, void* k, void* v, void* o, void* saved, size_t saved_bytes,
                      void* ws, size_t ws_bytes, void* stream);
sl_status sl_qkvo_bwd(sl_dtype dt, const sl_layout* lay, const sl_qkvo_weights* w,
                      const void* X, const void* a,
                      int32_t k_qk, const int32_t* idx_qk, int32_t k_vo, const int32_t* idx_vo,
                      const void* saved, size_t saved_bytes,
                      const void* dq, const void* dk, const void* dv, const void* d_out,
                      void* dX, void* da, const sl_qkvo_grads* g,
                      void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Between the q/k/v and the o projection: rotary positions, norms of the q and
 * k heads, differential attention.  q is [T, Hq*hd] and k, v [T, Hkv*hd], as
 * sl_qkvo_fwd writes them (call dtype); of the layout, batch and seq_len are
 * read (ctx_len is not).  Every call is stream-ordered on `stream` alone, never
 * synchronises, launches nothing on error, and may be captured into a graph.
 *
 * Rotary positions.  The first rot_dim values of every head are pairs: value i
 * with value i + rot_dim/2 (half layout) or 2i with 2i+1 (interleaved); pair i
 * of the row at position p turns by p * f_i and is multiplied by amplitude.
 * The rest of the head is copied.
 *   turns [rot_dim/2] uint64: f_i / (2 pi) in units of 2^-64 turns (device),
 *         as sl_rotary_table writes it on the host
 *   pos   [T] int32 positions (any sign), or NULL: row % seq_len
 * sl_rotary_table(spec): f_i = base^(-2i/rot_dim), stretched for long contexts:
 *   LINEAR      f / factor
 *   BASE        base * factor^(rot_dim/(rot_dim-2)) in place of base
 *   WAVELENGTH  pairs that turn more than high_turns times within original_len
 *               keep f, fewer than low_turns get f / factor, linear between
 *   YARN        the same ends, the ramp linear in the pair index between the
 *               indices (rounded outwards) that reach high_turns and low_turns;
 *               amplitude 0.1 ln(factor) + 1
 * base > 1, factor >= 1, 0 < low_turns < high_turns; rot_dim even, 2..256.
 * turns and amplitude are host memory; the table is made once per model.
 *
 * sl_rotary_apply: q_out / k_out = the rotated rows; inverse != 0 turns the
 * other way, which is the gradient.  q_out may be q, and k_out k; otherwise no
 * output may overlap an input or the other.  k and k_out may both be NULL.
 * head_dim even, at most 256; rot_dim even, 0..head_dim.
 * ------------------------------------------------------------------------- */
typedef enum sl_rope_scaling {
  SL_ROPE_NONE = 0, SL_ROPE_LINEAR = 1, SL_ROPE_BASE = 2, SL_ROPE_WAVELENGTH = 3, SL_ROPE_YARN = 4
} sl_rope_scaling;
typedef struct sl_rotary_spec {
  int32_t rot_dim;
  sl_rope_scaling scaling;
  double base, factor;
  int64_t original_len;             /* WAVELENGTH, YARN */
  double low_turns, high_turns;     /* WAVELENGTH, YARN */
} sl_rotary_spec;
typedef struct sl_rotary {
  int32_t rot_dim, interleaved;
  float amplitude;
  const uint64_t* turns;
  const int32_t* pos;
} sl_rotary;
sl_status sl_rotary_table(const sl_rotary_spec* spec, uint64_t* turns, float* amplitude);
sl_status sl_rotary_apply(sl_dtype dt, const sl_layout* lay, const sl_heads* heads, const sl_rotary* rot,
                          const void* q, const void* k, void* q_out, void* k_out, int32_t inverse,
                          void* stream);

/* ---------------------------------------------------------------------------
 * Norms of the q and k heads, with the rotation in the same pass:
 *   y = R(x r w),  r = (mean over the head of x^2 + eps)^(-1/2)
 * wq, wk [hd] fp32 weights shared by the heads; rot NULL (or rot_dim 0): no
 * rotation.  k, wk, k_out (and their gradients) may all be NULL, and n_kv_heads
 * is then 0 or any count.
 *   fwd: q, k -> q_out, k_out (q_out may be q, k_out k; keep x for the backward)
 *   bwd: x = q, k (the forward's inputs) and dq_out, dk_out -> dq, dk and the
 *        fp32 weight gradients dwq, dwk [hd], overwritten, summed over rows and
 *        heads in a fixed order.  dq may be dq_out or q, and dk dk_out or k.
 * Otherwise no output may overlap an input, the workspace or another output.
 * A row whose mean square and eps are both 0 has no norm: its outputs are NaN.
 * ------------------------------------------------------------------------- */
sl_status sl_head_norm_fwd(sl_dtype dt, const sl_layout* lay, const sl_heads* heads, const sl_rotary* rot,
                           float eps, const void* q, const void* k, const float* wq, const float* wk,
                           void* q_out, void* k_out, void* stream);
size_t sl_head_norm_workspace_bytes(const sl_layout* lay, const sl_heads* heads);
sl_status sl_head_norm_bwd(sl_dtype dt, const sl_layout* lay, const sl_heads* heads, const sl_rotary* rot,
                           float eps, const void* q, const void* k, const float* wq, const float* wk,
                           const void* dq_out, const void* dk_out, void* dq, void* dk,
                           float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Differential attention: query heads 2h, 2h+1 are a pair that reads the kv
 * heads 2g, 2g+1 of its group, g = h / (Hq / Hkv), and one value of 2 hd, v's
 * columns [2g*hd, 2(g+1)*hd):
 *   a[:, 2h*hd : 2(h+1)*hd] = softmax(s q_2h k_2g^T) V - lambda softmax(s q_2h+1 k_2g+1^T) V
 *   lambda = exp(lq1 . lk1) - exp(lq2 . lk2) + lambda_init
 *   lq1, lk1, lq2, lk2 [hd] fp32, 16-byte aligned: shared by the heads
 *   Query head 2h+m so meets kv head 2g+m, not (2h+m) / (Hq / Hkv).  Sparse
 *   projections around it (sl_qkvo_*, and QK_NORM, which choose and expand kv
 *   channels by their heads) take the pairs as heads, {Hq/2, Hkv/2, 2 hd}: the
 *   kept channels of q, k, v and a are then those that meet.
 *   scale   s (a positive number)
 *   causal  != 0: row i of a sequence reads keys 0..i
 *   lens    [host] batch valid lengths 0..seq_len, or NULL: every row.  Rows at
 *           or past a sequence's length are padding: they are never read, and
 *           their outputs and gradients are written as 0.
 *   fwd: q, k, v -> a [T, Hq*hd]; writes `saved` for the backward.  It uses no
 *        scratch: ws may be NULL with ws_bytes 0 (one that is given is checked
 *        for size as the backward's and left as it is).
 *   bwd: q, k, v, a (the forward's) and da -> dq, dk, dv and the fp32 gradients
 *        of the four vectors, overwritten.  Sums run in a fixed order.
 * No output may overlap an input, the buffers or another output.  The backward
 * takes the forward's inputs, p and `saved` as they were.  Every value of a valid
 * row is read: a non-finite one in row j of q, k, v, a or da, a key that the causal
 * mask hides among them, may reach any row of its sequence.  A row that reads one key has
 * no gradient to its scores.
 * bf16: sums, softmax statistics and the vectors' gradients are fp32 or fp64.
 * Operands of the matrix cores are bf16: in sequences (seq_len) of more than 256 rows
 * the weights and the score gradients of dk are rounded to it once (2^-8; a, dk and
 * dv are then off by 1.3 to 1.5 times their own rounding to bf16), in shorter ones, and for dq
 * always the score gradients, to the sum of two (2^-16).  `saved` keeps the second
 * map's output in 16 bits and a's rounding in 8.  fp32 calls round nothing.
 * |v| below 2^63 (the weights are kept relative to 2^64 of a row's first maximum).
 * Hq and Hkv even, Hq a multiple of Hkv; hd a multiple of 8, at most 128; every
 * tensor fewer than 2^31 elements.
 * ------------------------------------------------------------------------- */
typedef struct sl_diff_attn {
  sl_heads heads;
  float lambda_init, scale;
  int32_t causal;
  const int32_t* lens;
  const float *lq1, *lk1, *lq2, *lk2;
} sl_diff_attn;
typedef struct sl_diff_attn_grads { float *dlq1, *dlk1, *dlq2, *dlk2; } sl_diff_attn_grads;
size_t sl_diff_attn_saved_bytes(sl_dtype dt, const sl_layout* lay, const sl_heads* heads);
size_t sl_diff_attn_workspace_bytes(sl_dtype dt, const sl_layout* lay, const sl_heads* heads);
sl_status sl_diff_attn_fwd(sl_dtype dt, const sl_layout* lay, const sl_diff_attn* p, const void* q, const void* k,
                           const void* v, void* a, void* saved, size_t saved_bytes, void* ws, size_t ws_bytes,
                           void* stream);
sl_status sl_diff_attn_bwd(sl_dtype dt, const sl_layout* lay, const sl_diff_attn* p, const void* q, const void* k,
                           const void* v, const void* a, const void* saved, size_t saved_bytes, const void* da,
                           void* dq, void* dk, void* dv, const sl_diff_attn_grads* g, void* ws, size_t ws_bytes,
                           void* stream);

/* ---------------------------------------------------------------------------
 * Around the layers: from tokens to rows, between two layers, from logits to a
 * loss.  Of the layout batch and seq_len are read, and ctx_len by the loss alone.
 * Every call is stream-ordered on `stream` alone, never synchronises, launches
 * nothing on error, and may be captured into a graph.  Sums are fp32 and run in a
 * fixed order.  Offsets are 64-bit.
 *
 * Token embedding.
 *   E    [vocab, d_model]   ids [T] int32   Y, dY [T, d_model]
 *   fwd: Y[t] = scale * E[ids[t]]; an id outside 0..vocab-1 is no token: its row
 *        is 0 and it has no gradient (its row of dY is not read).
 *   bwd: dE [vocab, d_model] in grad_dt (fp32, or bf16: the fp32 sum rounded
 *        once), overwritten: scale * the sum of the token's rows of dY, 0 for
 *        an id without one.
 * d_model a multiple of 8, at most 65536; vocab at most 2^30, T at most 2^26.
 * No output may overlap an input or the workspace.
 * ------------------------------------------------------------------------- */
sl_status sl_embed_fwd(sl_dtype dt, const sl_layout* lay, int64_t vocab, int64_t d_model, float scale, const void* E,
                       const int32_t* ids, void* Y, void* stream);
size_t sl_embed_workspace_bytes(const sl_layout* lay, int64_t d_model);
sl_status sl_embed_bwd(sl_dtype dt, const sl_layout* lay, int64_t vocab, int64_t d_model, float scale,
                       const int32_t* ids, const void* dY, sl_dtype grad_dt, void* dE, void* ws, size_t ws_bytes,
                       void* stream);

/* ---------------------------------------------------------------------------
 * Norm of whole rows with the residual sum in the same pass.
 *   h = x + r (rounded to the call's type; without r, h is x and not written)
 *   y = (h - m) s w + b,  m = mean h,  s = (mean (h - m)^2 + eps)^(-1/2)
 *   not centered: m = 0 and b = 0
 *   w, b [d_model] fp32; b may be NULL (0)
 *   fwd: x, r -> h, y [T, d_model] and stats [T, 3] fp32 (m, what m rounded away,
 *        s; NULL: not written).  r and h both or neither.  h or y may be x, or r
 *        (without r, y in x's place leaves no h for the backward).
 *   bwd: h, stats (the forward's), dy and optionally dh, the gradient that reaches
 *        h by its other way -> dx, the gradient of x and of r alike, and the fp32
 *        gradients dw and db [d_model], overwritten (db NULL: not written).  dx
 *        may be dy, dh or h.
 * Otherwise no output may overlap an input, the workspace or another output.
 * d_model a multiple of 8, at most 16384; eps >= 0.  A row whose variance (mean
 * square) and eps are both 0 has no norm: its outputs are NaN.  Squares are fp32:
 * of rows whose values pass 10^17, s may be 0.
 * ------------------------------------------------------------------------- */
typedef struct sl_layer_norm {
  int64_t d_model;
  int32_t centered;
  float eps;
  const float *w, *b;
} sl_layer_norm;
sl_status sl_layer_norm_fwd(sl_dtype dt, const sl_layout* lay, const sl_layer_norm* p, const void* x, const void* r,
                            void* h, void* y, float* stats, void* stream);
size_t sl_layer_norm_workspace_bytes(const sl_layout* lay, int64_t d_model);
sl_status sl_layer_norm_bwd(sl_dtype dt, const sl_layout* lay, const sl_layer_norm* p, const void* h,
                            const float* stats, const void* dy, const void* dh, void* dx, float* dw, float* db,
                            void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Distillation from a teacher's top logits, mixed with hard labels.  Row t of the
 * logits [T, ld] holds z over the vocabulary, in its first `vocab` elements:
 *   p = softmax(top_logits[t] / temperature) over its `top` entries; an id
 *       outside 0..vocab-1 is no entry, the same id twice counts twice
 *   q = softmax(z / temperature),  o = softmax(z)
 *   loss = (1 - hard) temperature^2 sum_k p_k (log p_k - log q_{i_k}) - hard log o_label
 *   dlogits = dloss * the loss's gradient
 * A row without entries has no first term, one whose label is outside 0..vocab-1
 * no second.  Context rows (the first ctx_len[b] of each sequence) have neither:
 * loss 0, dlogits 0, whatever they hold; so has every row without a term.
 *   top_ids [T, top] int32, top_logits [T, top] fp32   (hard = 1: may be NULL)
 *   labels  [T] int32                                  (hard = 0: may be NULL)
 *   fwd:  logits -> loss [T] fp32 and stats [T, 4] fp32 for the backward
 *   bwd:  logits, stats, dloss [T] fp32 (NULL: ones) -> dlogits [T, ld_out]
 *   step: logits, dloss -> loss and dlogits in one call, for a loss whose weights
 *         are known beforehand: one launch, and most of logits read from memory once
 *   A row whose dloss is 0 gets zeros.
 * dlogits may be logits (with ld_out = ld); otherwise no output may overlap an
 * input or another output.  Elements of a row behind the vocabulary are neither
 * read nor written.  ld, ld_out >= vocab, any number; logits and dlogits need no
 * more than the alignment of their elements (by which, row by row, the order of the
 * sums goes).
 * Logits of -inf have probability 0.  A row of -inf alone, or with +inf or NaN,
 * has no distribution: its loss and its gradient are NaN; so is the loss of a
 * teacher's entry of +inf or NaN, and the gradient there.  The first term is
 * temperature^2 times a difference of fp32 logarithms and has their rounding that
 * many times.
 * 0 <= hard <= 1, temperature in [1e-6, 1e6], 1 <= top <= SL_DISTILL_MAX_TOP, vocab <= 2^30.
 * ------------------------------------------------------------------------- */
#define SL_DISTILL_MAX_TOP 256
typedef struct sl_distill {
  int64_t vocab;
  int32_t top;
  float temperature, hard;
  const int32_t* top_ids;
  const float* top_logits;
  const int32_t* labels;
} sl_distill;
sl_status sl_distill_fwd(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits, int64_t ld,
                         float* loss, float* stats, void* stream);
sl_status sl_distill_bwd(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits, int64_t ld,
                         const float* stats, const float* dloss, void* dlogits, int64_t ld_out, void* stream);
sl_status sl_distill_step(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits, int64_t ld,
                          const float* dloss, float* loss, void* dlogits, int64_t ld_out, void* stream);

/* ---------------------------------------------------------------------------
 * Offline quantization of a frozen weight to the 4-bit base of sl_ffn_weights
 * (SparseLoRA article §六: SparseLoRA over a QLoRA-style quantized base; the
 * pages name no format, this is the plainest 4-bit one).  W [rows, cols] in dt
 * -> codes uint8 [rows, cols/2] and scales fp32 [rows, cols/64]: each block of
 * 64 consecutive row elements gets s = max|w| / 7 (0 for an all-zero block)
 * and codes q = rint(w / s) in [-7, 7] (IEEE fp32 division, ties to even);
 * element 2j of a row sits in the low nibble of byte j, element 2j+1 in the
 * high nibble (two's complement).  cols a positive multiple of 64; all
 * pointers device, 16-byte aligned; the caller owns every buffer.  Stream-
 * ordered, never synchronises.  Errors: SL_ERR_NULL, SL_ERR_DTYPE,
 * SL_ERR_SHAPE, SL_ERR_RANGE, SL_ERR_ALIGN, SL_ERR_UNSUPPORTED_ARCH,
 * SL_ERR_HIP; nothing is launched on error.
 * ------------------------------------------------------------------------- */
sl_status sl_quantize_q4(sl_dtype dt, const void* W, int64_t rows, int64_t cols, void* codes, float* scales,
                         void* stream);

/* ---------------------------------------------------------------------------
 * Diagnostics (not part of the computation).  When enabled, the library's main
 * launches are bracketed by HIP events on the caller's stream and attributed
 * to the slots below, so a caller can time individual kernels inside a timed
 * region.  The timer state is per calling thread: it covers the calls that
 * thread makes.  sl_timer_enable(n) keeps room for n
 * launches (0 disables and frees the events); sl_timer_read waits for the
 * recorded events and returns the slot's total milliseconds and launch count
 * since the last sl_timer_reset.  sl_timer_select(mask) records only the slots
 * whose bit (1 << slot) is set (all after sl_timer_enable), so that a timed
 * region carries events around the kernels of interest only.
 * ------------------------------------------------------------------------- */
typedef enum sl_timer_slot {
  SL_TS_ESTIMATE = 0,   /* estimator stage 1 + criterion (a1, a2) */
  SL_TS_SELECT = 1,     /* top-k (a3) */
  SL_TS_GU_FWD = 2,     /* gate/up gather-GEMM + SwiGLU (a4) */
  SL_TS_DOWN_FWD = 3,   /* down K-gather GEMM (a4) */
  SL_TS_DH_BWD = 4,     /* dH gather-GEMM + SwiGLU backward (a5) */
  SL_TS_DX_BWD = 5,     /* dX K-gather GEMM (a5) */
  SL_TS_QKV_FWD = 6, SL_TS_O_FWD = 7, SL_TS_DA_BWD = 8, SL_TS_DXQKV_BWD = 9
} sl_timer_slot;
int sl_timer_enable(int max_launches);
void sl_timer_select(uint32_t slot_mask);
void sl_timer_reset(void);
int sl_timer_read(int slot, double* total_ms, int* count);

/* ---------------------------------------------------------------------------
 * GEMM variants (tuning and testing; results agree to the same tolerance).
 * The gather-GEMMs run as 128 x 256 tiles staged through registers, as wide
 * 128 x 512 N-gather tiles fed by LDS-DMA, or as tall 256 x 256 tiles (N- or
 * K-gather) fed by LDS-DMA.  The LDS-DMA tiles need bf16 calls with every
 * operand 16-byte aligned (N-gather: K a multiple of 8); the tall tiles are
 * taken when their grid moves fewer operand bytes per CU than the other
 * variant's.  `variants` is a bit mask of what the calling thread allows: 1 =
 * wide tiles, 2 = tall tiles, 4 = tall tiles whatever their grid (with 2); 0 =
 * 128 x 256 tiles only; a negative value leaves the setting.  Default 3.
 * Returns the previous setting.  The setting is per calling thread and
 * applies to the calls that thread makes.
 * ------------------------------------------------------------------------- */
int sl_gemm_config(int variants);

#ifdef __cplusplus
}
#endif
#endif /* SPARSELORA_H */
