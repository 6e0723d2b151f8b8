// Distillation from a teacher's top logits, mixed with hard labels.  A row t
// with loss has logits z over the vocabulary, the teacher's K entries (i_k, t_k) and
// a label:
//   p = softmax(t / tau) over the entries (an id outside the vocabulary is no entry),
//   q = softmax(z / tau),  o = softmax(z),
//   loss = (1 - hard) tau^2 sum_k p_k (log p_k - log q_{i_k}) - hard log o_label,
//   dz_v = dloss [(1 - hard) tau (q_v - sum_{k: i_k = v} p_k) + hard (o_v - [v = label])].
// Rows of context have neither loss nor gradient and are not read.
//
// One block a row.  The first walk over the row keeps, per thread, the running
// maximum and the running sums of exp((z - max) / tau) and exp(z - max), rescaled
// where the maximum moves, and joins them over the block.  The second walk forms
// the gradient; behind it the few ids of the teacher's entries and the label are
// written again with their subtrahends.  A step (loss and gradient in one call)
// does both walks in one launch, the second from the caches.  Rows need not be
// aligned (an odd vocabulary): a vector is 16 bytes at any element.
#include <cmath>

#include "sl_rows.hpp"

namespace sl {

constexpr int kTop = SL_DISTILL_MAX_TOP;   // most entries of the teacher
constexpr int kRowThreads = 512;

enum DistillMode { DM_FWD, DM_BWD, DM_STEP };

struct DistillArgs {
  const void* z;
  void* dz;
  const int* top_ids;
  const float* top_logits;
  const int* labels;
  const float* dloss;       // NULL: 1
  float* loss;
  float* stats;             // [T][4]: the maximum, the sums of exp((z - max) / tau) and of exp(z - max), 0
  long long ld, ld_out;     // elements from row to row
  int V, top, L, rows;
  float tau, inv_tau, hard;
  int ctx[SL_MAX_SEQS];
};

constexpr float kLog2e = 1.44269504088896341f;

// 16 bytes of row elements, at any element's address
template <typename T> struct RowVec;
template <> struct RowVec<bf16> {
  typedef uint16_t Raw __attribute__((ext_vector_type(8), aligned(2)));
  static constexpr int W = 8;
  __device__ static inline float get(uint16_t x) { return bf2f(x); }
  __device__ static inline uint16_t put(float x) { return f2el<bf16>(x).v; }
};
template <> struct RowVec<float> {
  typedef float Raw __attribute__((ext_vector_type(4), aligned(4)));
  static constexpr int W = 4;
  __device__ static inline float get(float x) { return x; }
  __device__ static inline float put(float x) { return x; }
};

// e^((z - m) scale), z <= m; scale includes log2 e.  z - m first: lowest values and
// infinities of a mask then behave (equal ones count 1, -inf below a finite maximum 0).
__device__ inline float exp_below(float z, float m, float scale) { return __builtin_amdgcn_exp2f((z - m) * scale); }

// Running maximum and the two sums relative to it; an empty one has m = -inf.
struct Sums {
  float m, s[2];
};
template <bool TWO> __device__ inline void rebase(Sums& a, float m, const float* scale) {
  // (a row of -inf alone, or of NaN, keeps m = -inf: relative to 0 its sums stay what they are)
  const float from = a.m == -INFINITY ? m : a.m;
  a.s[0] *= m == -INFINITY ? 1.f : exp_below(from, m, scale[0]);
  if (TWO) a.s[1] *= m == -INFINITY ? 1.f : exp_below(from, m, scale[1]);
  a.m = m;
}

// The values of one vector into the running sums.
template <bool TWO, int N> __device__ inline void absorb(Sums& a, const float (&x)[N], const float* scale) {
  float m = a.m;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, x[j]);
  if (m > a.m) rebase<TWO>(a, m, scale);
  const float at = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    a.s[0] += exp_below(x[j], at, scale[0]);
    if (TWO) a.s[1] += exp_below(x[j], at, scale[1]);
  }
}

// TWO: the teacher's term at tau and the label's at 1 need an exponential each.
// With one of the terms alone, or with tau = 1, one serves.
template <typename T, int MODE, bool TWO>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(const DistillArgs a) {
  using RV = RowVec<T>;
  using Raw = typename RV::Raw;
  constexpr int W = RV::W, U = 4, kWaves = kRowThreads / 64;
  __shared__ float red[3][kWaves];
  __shared__ int ids[kTop + 1];                 // the teacher's entries and, behind them, the label; -1: none
  __shared__ float ptop[kTop], ztop[kTop + 1];  // the entries' logits, the student's at these ids
  __shared__ float teacher[2];                  // maximum and sum of the entries; sum 0: none
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool soft = a.hard < 1.f, hard = a.hard > 0.f;
  const int K = soft ? a.top : 0;
  const float scale[2] = {(soft ? a.inv_tau : 1.f) * kLog2e, kLog2e};
  const int nvec = a.V / W;

  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* const z = reinterpret_cast<const T*>(a.z) + row * a.ld;
    T* const dz = reinterpret_cast<T*>(a.dz) + row * a.ld_out;
    const int seq = (int)(row / a.L);
    const float g = MODE == DM_FWD ? 0.f : a.dloss ? a.dloss[row] : 1.f;
    bool read = (int)(row - (long long)seq * a.L) >= a.ctx[seq] && (MODE != DM_BWD || g != 0.f);
    __syncthreads();                            // the last row's shared values have been read
    if (read && tid <= K) {
      int id = tid < K ? a.top_ids[row * a.top + tid] : hard ? a.labels[row] : -1;
      if ((unsigned)id >= (unsigned)a.V) id = -1;
      ids[tid] = id;
      ztop[tid] = id >= 0 ? ldv<T>(z, id) : 0.f;
      if (tid < K) ptop[tid] = id >= 0 ? a.top_logits[row * a.top + tid] : -INFINITY;
    }
    __syncthreads();
    if (read && wave == 0) {
      float m = -INFINITY, bad = 0.f, s = 0.f;
      for (int k = lane; k < K; k += 64) {
        m = fmaxf(m, ptop[k]);
        if (!(ptop[k] < INFINITY)) bad = 1.f;   // infinite or NaN: no distribution
      }
      m = wave_max(m);
      bad = wave_add(bad);
      if (m > -INFINITY)
        for (int k = lane; k < K; k += 64) s += exp_below(ptop[k], m, scale[0]);
      s = wave_add(s);
      if (lane == 0) {
        teacher[0] = m;
        teacher[1] = bad > 0.f ? NAN : s;
      }
    }
    __syncthreads();
    const float tmax = teacher[0], tsum = teacher[1];
    const bool taught = read && !(tsum == 0.f), labelled = read && ids[K] >= 0;
    read = taught || labelled;                  // with neither the row has no loss
    if (!read) {
      if (MODE != DM_BWD && tid == 0) a.loss[row] = 0.f;
      if (MODE == DM_FWD && tid < 4) a.stats[row * 4 + tid] = 0.f;
      if (MODE != DM_FWD) {
        const Raw zero = {};
        for (int c = tid; c < nvec; c += kRowThreads) *reinterpret_cast<Raw*>(dz + (long long)c * W) = zero;
        if (tid < a.V - nvec * W) stv<T>(dz, nvec * W + tid, 0.f);
      }
      continue;
    }

    Sums run = {-INFINITY, {0.f, 0.f}};
    if constexpr (MODE == DM_BWD) {
      run = {a.stats[row * 4], {a.stats[row * 4 + 1], a.stats[row * 4 + 2]}};
    } else {
      int c = tid;
      for (; c + (U - 1) * kRowThreads < nvec; c += kRowThreads * U) {
        Raw v[U];
        float x[U * W];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const Raw*>(z + (long long)(c + u * kRowThreads) * W);
#pragma unroll
        for (int j = 0; j < U * W; ++j) x[j] = RV::get(v[j / W][j % W]);
        absorb<TWO>(run, x, scale);
      }
      for (; c < nvec; c += kRowThreads) {
        const Raw v = *reinterpret_cast<const Raw*>(z + (long long)c * W);
        float x[W];
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = RV::get(v[j]);
        absorb<TWO>(run, x, scale);
      }
      if (tid < a.V - nvec * W) {
        const float x[1] = {ldv<T>(z, nvec * W + tid)};
        absorb<TWO>(run, x, scale);
      }
      rebase<TWO>(run, wave_max(run.m), scale);
#pragma unroll
      for (int i = 0; i < 1 + TWO; ++i) run.s[i] = wave_add(run.s[i]);
      if (lane == 0) {
        red[0][wave] = run.m;
        red[1][wave] = run.s[0];
        red[2][wave] = run.s[1];
      }
      __syncthreads();
      float m = red[0][0];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) m = fmaxf(m, red[0][i]);
      run = {m, {0.f, 0.f}};
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        Sums p = {red[0][i], {red[1][i], red[2][i]}};
        rebase<TWO>(p, m, scale);
        run.s[0] += p.s[0];
        run.s[1] += p.s[1];
      }
      if (m == -INFINITY) run.s[0] = run.s[1] = NAN;   // nothing to choose from: no distribution
      if (MODE == DM_FWD && tid < 4) a.stats[row * 4 + tid] = tid == 0 ? run.m : tid == 1 ? run.s[0] : tid == 2 ? run.s[1] : 0.f;
    }
    const float s_soft = run.s[0], s_hard = run.s[TWO];

    if (MODE != DM_BWD && wave == 0) {
      float kl = 0.f;
      const float lp = logf(tsum), lq = logf(s_soft);
      if (taught)
        for (int k = lane; k < K; k += 64) {
          const float p = exp_below(ptop[k], tmax, scale[0]) / tsum;
          if (!(p == 0.f)) kl += p * (((ptop[k] - tmax) * a.inv_tau - lp) - ((ztop[k] - run.m) * a.inv_tau - lq));
        }
      kl = wave_add(kl);
      if (lane == 0) {
        float l = taught ? (1.f - a.hard) * a.tau * a.tau * kl : 0.f;
        if (labelled) l += a.hard * (logf(s_hard) - (ztop[K] - run.m));
        a.loss[row] = l;
      }
    }
    if constexpr (MODE != DM_FWD) {
      const float cs = taught ? g * (1.f - a.hard) * a.tau : 0.f, ch = labelled ? g * a.hard : 0.f;
      const float as = (TWO ? cs : cs + ch) / s_soft, ah = ch / s_hard, at = run.m == -INFINITY ? 0.f : run.m;
      auto grad = [&](float x) __attribute__((always_inline)) {
        const float d = exp_below(x, at, scale[0]) * as;
        return TWO ? fmaf(exp_below(x, at, scale[1]), ah, d) : d;
      };
      auto vec = [&](const Raw& v) __attribute__((always_inline)) {
        Raw o;
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = RV::put(grad(RV::get(v[j])));
        return o;
      };
      int c = tid;
      for (; c + (U - 1) * kRowThreads < nvec; c += kRowThreads * U) {
        Raw v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const Raw*>(z + (long long)(c + u * kRowThreads) * W);
#pragma unroll
        for (int u = 0; u < U; ++u) *reinterpret_cast<Raw*>(dz + (long long)(c + u * kRowThreads) * W) = vec(v[u]);
      }
      for (; c < nvec; c += kRowThreads)
        *reinterpret_cast<Raw*>(dz + (long long)c * W) = vec(*reinterpret_cast<const Raw*>(z + (long long)c * W));
      if (tid < a.V - nvec * W) stv<T>(dz, nvec * W + tid, grad(ldv<T>(z, nvec * W + tid)));
      __syncthreads();
      // the entries and the label, their q and o from before dz may have been written
      // over z; an id that comes twice gets the same value from each of its entries
      if (tid <= K && ids[tid] >= 0) {
        const int id = ids[tid];
        float d = grad(ztop[tid]);
        if (taught)
          for (int k = 0; k < K; ++k)
            if (ids[k] == id) d -= cs * (exp_below(ptop[k], tmax, scale[0]) / tsum);
        if (labelled && ids[K] == id) d -= ch;
        stv<T>(dz, id, d);
      }
    }
  }
}

static sl_status distill_args(DistillArgs& a, sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* z,
                              int64_t ld, const void* dz, int64_t ld_out) {
  sl_status st = check_dtype(dt);
  if (st == SL_OK) st = check_tokens(lay);
  if (st != SL_OK) return st;
  if (!lay->ctx_len) SL_FAIL(SL_ERR_NULL, "layout.ctx_len is NULL");
  if (!p || !z) SL_FAIL(SL_ERR_NULL, "the targets and logits required");
  if (p->vocab < 1 || p->vocab > (1LL << 30)) SL_FAIL(SL_ERR_RANGE, "vocabulary of %lld outside [1, 2^30]", (long long)p->vocab);
  if (!(p->hard >= 0.f && p->hard <= 1.f)) SL_FAIL(SL_ERR_RANGE, "hard must be in [0, 1]");
  if (!(p->temperature > 0.f) || !std::isfinite(p->temperature) || !std::isfinite(1.f / p->temperature))
    SL_FAIL(SL_ERR_RANGE, "temperature must be positive and finite");
  if (p->hard < 1.f) {
    if (p->top < 1 || p->top > kTop) SL_FAIL(SL_ERR_RANGE, "top = %d outside [1, %d]", p->top, kTop);
    if (!p->top_ids || !p->top_logits) SL_FAIL(SL_ERR_NULL, "top_ids and top_logits required");
  }
  if (p->hard > 0.f && !p->labels) SL_FAIL(SL_ERR_NULL, "labels required");
  if (ld < p->vocab || (dz && ld_out < p->vocab))
    SL_FAIL(SL_ERR_SHAPE, "rows of %lld and %lld elements hold no %lld logits", (long long)ld, (long long)ld_out, (long long)p->vocab);
  if (!aligned16(z) || !aligned16(dz) || !aligned16(p->top_ids) || !aligned16(p->top_logits) || !aligned16(p->labels))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  a = DistillArgs{};
  a.z = z; a.ld = ld; a.ld_out = ld_out;
  a.top_ids = p->top_ids; a.top_logits = p->top_logits; a.labels = p->labels;
  a.V = (int)p->vocab; a.top = p->top;
  a.L = lay->seq_len; a.rows = lay->batch * lay->seq_len;
  a.tau = p->temperature; a.inv_tau = 1.f / p->temperature; a.hard = p->hard;
  for (int b = 0; b < lay->batch; ++b) {
    a.ctx[b] = lay->ctx_len[b];
    if (a.ctx[b] < 0 || a.ctx[b] > lay->seq_len)
      SL_FAIL(SL_ERR_RANGE, "ctx_len[%d] = %d outside [0, %d]", b, a.ctx[b], lay->seq_len);
  }
  return SL_OK;
}

template <int MODE> static sl_status run_distill(sl_dtype dt, const DistillArgs& a, void* stream) {
  sl_status st = check_arch();
  if (st != SL_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid = walk_grid(a.rows), block(kRowThreads);
  const bool two = a.hard > 0.f && a.hard < 1.f && a.tau != 1.f;
  if (dt == SL_BF16) {
    if (two) hipLaunchKernelGGL((distill_kernel<bf16, MODE, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((distill_kernel<bf16, MODE, false>), grid, block, 0, s, a);
  } else {
    if (two) hipLaunchKernelGGL((distill_kernel<float, MODE, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((distill_kernel<float, MODE, false>), grid, block, 0, s, a);
  }
  SL_HIP(hipGetLastError());
  return SL_OK;
}

}  // namespace sl

using namespace sl;

extern "C" sl_status sl_distill_fwd(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits,
                                    int64_t ld, float* loss, float* stats, void* stream) {
  if (!loss || !stats) SL_FAIL(SL_ERR_NULL, "loss and stats required");
  DistillArgs a;
  sl_status st = distill_args(a, dt, lay, p, logits, ld, nullptr, 0);
  if (st != SL_OK) return st;
  if (!aligned16(loss) || !aligned16(stats)) SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  a.loss = loss; a.stats = stats;
  return run_distill<DM_FWD>(dt, a, stream);
}

extern "C" sl_status sl_distill_bwd(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits,
                                    int64_t ld, const float* stats, const float* dloss, void* dlogits, int64_t ld_out,
                                    void* stream) {
  if (!stats || !dlogits) SL_FAIL(SL_ERR_NULL, "stats and dlogits required");
  DistillArgs a;
  sl_status st = distill_args(a, dt, lay, p, logits, ld, dlogits, ld_out);
  if (st != SL_OK) return st;
  if (!aligned16(stats) || !aligned16(dloss)) SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  a.stats = const_cast<float*>(stats); a.dloss = dloss; a.dz = dlogits;
  return run_distill<DM_BWD>(dt, a, stream);
}

extern "C" sl_status sl_distill_step(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits,
                                     int64_t ld, const float* dloss, float* loss, void* dlogits, int64_t ld_out,
                                     void* stream) {
  if (!loss || !dlogits) SL_FAIL(SL_ERR_NULL, "loss and dlogits required");
  DistillArgs a;
  sl_status st = distill_args(a, dt, lay, p, logits, ld, dlogits, ld_out);
  if (st != SL_OK) return st;
  if (!aligned16(loss) || !aligned16(dloss)) SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  a.loss = loss; a.dloss = dloss; a.dz = dlogits;
  return run_distill<DM_STEP>(dt, a, stream);
}
