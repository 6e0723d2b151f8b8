// Distillation from a teacher's top logits, mixed with hard labels.  A row t
// with loss has logits z over the vocabulary, the teacher's K entries (i_k, t_k) and
// a label:
//   p = softmax(t / tau) over the entries (an id outside the vocabulary is no entry),
//   q = softmax(z / tau),  o = softmax(z),
//   loss = (1 - hard) tau^2 sum_k p_k (log p_k - log q_{i_k}) - hard log o_label,
//   dz_v = dloss [(1 - hard) tau (q_v - sum_{k: i_k = v} p_k) + hard (o_v - [v = label])].
// Rows of context have neither loss nor gradient and are not read.
//
// One block a row, the rows with a loss first, so that the context rows' zeros fill the
// time in which the last of them end.  The first walk over a row keeps, per thread, the
// running maximum and the running sums of exp((z - max) / tau) and exp(z - max),
// rescaled where the maximum moves, and joins them over the block.  The second walk
// forms the gradient; behind it the few ids of the teacher's entries and the label are
// written again with their subtrahends.  A step (loss and gradient in one call) does
// both walks in one launch, the second from the caches.  Both load the next four
// vectors of a thread before they work on these.  A row's vectors start at
// its first 16-byte border (an odd vocabulary has it elsewhere in every row); in a
// gradient whose rows stand otherwise they are stored where they fall.
//
// Measured (bf16): step of 4096 rows of 128256 logits 457 us: 1.05 GB read and as much written,
// and 0.8 GB read again (what LDS does not keep of a 256 KB row), 6.3 TB/s together, where an
// elementwise copy runs at 6.2; of 2048 rows of 32000 (whole rows kept) 72 us; of 4 x 512 with 384
// context rows each 36 us, 131 MB of it written.  What bounds it: memory, and in short launches a row's own length, about 10 us of loads, an
// exchange between the waves, and stores, two rows to a CU at a time.
#include <cmath>
#include <type_traits>

#include "sl_rows.hpp"

namespace sl {

constexpr int kTop = SL_DISTILL_MAX_TOP;   // most entries of the teacher
constexpr int kRowThreads = 512;           // most threads of a row
constexpr int kVecs = 4;                   // vectors that a thread loads at a time
constexpr int kKept = 2;                   // such loads of a step that stay in LDS between the walks

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
  int V, top, rows;
  float tau, inv_tau, hard;
  float scale;              // log2(e) / tau rounded once (log2(e) where the label's term stands alone)
  SeqTab st;
};

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// 16 bytes of row elements, at any element's address
template <typename T> struct RowVec;
template <> struct RowVec<bf16> {
  typedef uint16_t Raw __attribute__((ext_vector_type(8), aligned(2)));
  static constexpr int W = 8;
  __device__ static inline float get(uint16_t x) { return bf2f(x); }
  __device__ static inline uint16_t put(float x) { return f2el<bf16>(x).v; }
  __device__ static inline Raw none() { return (Raw)(uint16_t)0xFF80; }   // -inf
};
template <> struct RowVec<float> {
  typedef float Raw __attribute__((ext_vector_type(4), aligned(4)));
  static constexpr int W = 4;
  __device__ static inline float get(float x) { return x; }
  __device__ static inline float put(float x) { return x; }
  __device__ static inline Raw none() { return (Raw)(-INFINITY); }
};

template <typename R, typename T> __device__ inline R* vec_at(T* row, int c) {
  return reinterpret_cast<R*>(row) + c;
}

// Running maximum m and the two sums of 2^(z scale - top), top = m scale rounded once
// (then a number like any other: one rounding of the small difference is all an
// exponent gets).  Past 2^20 that one rounding would reach the exponents' range: there,
// and where m is infinite, the sums are of 2^((z - m) scale), so that equal lowest values
// of a mask count 1 each.  An empty one has m = -inf.
struct Sums {
  float m, s[2], top[2];
  bool near;                                    // |top| below 2^20
};
template <bool TWO> __device__ inline void set_top(Sums& a, float m, const float* scale) {
  a.m = m;
  a.top[0] = rounded(m * scale[0]);
  a.near = fabsf(a.top[0]) < 0x1p20f;
  if (TWO) {
    a.top[1] = rounded(m * scale[1]);
    a.near = a.near && fabsf(a.top[1]) < 0x1p20f;
  }
}
// 2^(z scale - top) of a value z <= m; m = -inf (nothing but -inf or NaN so far) counts as 0
template <bool NEAR> __device__ inline float term(const Sums& a, float z, float scale, int i) {
  const float y = NEAR ? fmaf(z, scale, -a.top[i]) : (z - (a.m == -INFINITY ? 0.f : a.m)) * scale;
  return __builtin_amdgcn_exp2f(y);
}
// The sums relative to another maximum, at least the old one.  Where one of the two is
// within 2^20 and the other past it, the step is between a rounded product and one that is
// not: the rounding, up to 2^-5 there, is part of it.
template <bool TWO> __device__ inline void rebase(Sums& a, float m, const float* scale) {
  const Sums old = a;
  set_top<TWO>(a, m, scale);
  if (old.m == -INFINITY) return;               // (the sums are 0, or NaN)
  float by[1 + TWO];
#pragma unroll
  for (int i = 0; i < 1 + TWO; ++i) by[i] = old.near ? old.top[i] - a.top[i] : (old.m - m) * scale[i];
  if (__builtin_expect(__ballot(old.near != a.near) != 0, 0)) {   // a branch, not two more operations in every step
#pragma unroll
    for (int i = 0; i < 1 + TWO; ++i)
      if (old.near != a.near) by[i] = old.near ? -fmaf(m, scale[i], -old.top[i]) : fmaf(old.m, scale[i], -a.top[i]);
  }
#pragma unroll
  for (int i = 0; i < 1 + TWO; ++i) a.s[i] *= __builtin_amdgcn_exp2f(by[i]);
}

// The values of some vectors into the running sums.
template <bool TWO, int N> __device__ inline void absorb(Sums& a, const float (&x)[N], const float* scale) {
  float m = a.m;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, x[j]);
  if (m > a.m) rebase<TWO>(a, m, scale);
  if (a.near) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 1 + TWO; ++i) a.s[i] += __builtin_amdgcn_exp2f(fmaf(x[j], scale[i], -a.top[i]));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 1 + TWO; ++i) a.s[i] += term<false>(a, x[j], scale[i], i);
  }
}

__device__ inline float top_term(float t, float m, float scale) { return __builtin_amdgcn_exp2f((t - m) * scale); }

// Token row of row i of the context rows.
__device__ inline int context_token(const SeqTab& st, int i) {
  int lo = 0, hi = st.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (st.ctx_pre[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo * st.L + (i - st.ctx_pre[lo]);
}

// TWO: the teacher's term at tau and the label's at 1 need an exponential each.
// With one of the terms alone, or with tau = 1, one serves.
// NT: past the caches, 1 the gradient's stores, 2 the logits' loads too.
// Loss or gradient alone: at most 80 registers, with which a CU takes three blocks (loss of 2048
// rows of 32000 bf16: 32 us, with 83 registers 37); the loss with two exponentials needs 87.  The
// gradient's kernel spills up to 20 bytes a thread for it: with 90 registers and none, 2048 rows of
// 32000 take 57.3 us in place of 55.3, 748 of 50021 41.5 for 40.1, 4096 of 128256 400 for 403.
template <typename T, int MODE, bool TWO, int NT>
__global__ void __launch_bounds__(kRowThreads, MODE == DM_BWD || (MODE == DM_FWD && !TWO) ? 6 : 4) distill_kernel(const DistillArgs a) {
  using RV = RowVec<T>;
  using Raw = typename RV::Raw;
  constexpr int W = RV::W, U = kVecs;
  __shared__ float red[3][kRowThreads / 64];
  __shared__ int ids[kTop + 1];                 // the teacher's entries and, behind them, the label; -1: none
  __shared__ float ptop[kTop], ztop[kTop + 1];  // the entries' logits, the student's at these ids
  __shared__ float dtop[MODE == DM_FWD ? 1 : kTop + 1];   // the gradient there
  typedef uint32_t Line __attribute__((ext_vector_type(4)));
  extern __shared__ Line kept[];                // step: the first loads of the row, a thread's where it left them
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
  const bool soft = a.hard < 1.f, hard = a.hard > 0.f;
  const int K = soft ? a.top : 0;
  const float scale[2] = {a.scale, kLog2e};
  const int batch = threads * U;

  for (long long it = blockIdx.x; it < a.rows; it += gridDim.x) {
    const bool out = it < a.st.T_out;
    const long long row = out ? out_token(a.st, (int)it) : context_token(a.st, (int)it - a.st.T_out);
    const T* const z = reinterpret_cast<const T*>(a.z) + row * a.ld;
    T* const dz = reinterpret_cast<T*>(a.dz) + row * a.ld_out;
    const float g = MODE == DM_FWD || !out ? 0.f : a.dloss ? a.dloss[row] : 1.f;
    // the row: the elements up to a vector's border, the vectors, the elements behind
    const int to_border = (int)(-reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T));
    const int nhead = to_border < a.V ? to_border : a.V, nvec = (a.V - nhead) / W, ntail = a.V - nhead - nvec * W;
    const T* const zv = z + nhead;
    T* const dv = dz + nhead;
    const int kept_end = MODE == DM_STEP ? kKept * batch < nvec ? kKept * batch : nvec : 0;   // vectors kept
    auto odd_ones = [&](auto f) __attribute__((always_inline)) {
      if (tid < nhead) f(tid);
      if (tid < ntail) f(nhead + nvec * W + tid);
    };
    auto fetch = [&](int c, Raw (&v)[U]) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u * threads >= nvec) v[u] = RV::none();
        else if (NT == 2) v[u] = __builtin_nontemporal_load(vec_at<const Raw>(zv, c + u * threads));
        else v[u] = *vec_at<const Raw>(zv, c + u * threads);
    };
    auto store = [&](int c, Raw o) __attribute__((always_inline)) {
      if (NT) __builtin_nontemporal_store(o, vec_at<Raw>(dv, c));
      else *vec_at<Raw>(dv, c) = o;
    };
    Raw v[U], next[U];
    Sums run = {-INFINITY, {0.f, 0.f}, {0.f, 0.f}, false};
    bool taught = false, labelled = false;
    float tmax = -INFINITY, tsum = 0.f, e[kTop / 64];
    int eid[kTop / 64];
    if (out) {
      __syncthreads();                          // the last row's shared values have been read
      if constexpr (MODE == DM_BWD) {
        set_top<TWO>(run, a.stats[row * 4], scale);
        run.s[0] = a.stats[row * 4 + 1];
        run.s[1] = a.stats[row * 4 + 2];
      }
      // an entry a thread (more where the block is small): its id at once, the logit there
      // behind the first vectors, both in LDS when the first walk is over
      auto entry = [&](int k, int& id, float& t) __attribute__((always_inline)) {
        id = k < K ? a.top_ids[row * a.top + k] : hard ? a.labels[row] : -1;
        t = k < K ? a.top_logits[row * a.top + k] : 0.f;
      };
      auto share = [&](int k, int id, float t) __attribute__((always_inline)) {
        if ((unsigned)id >= (unsigned)a.V) id = -1;
        ids[k] = id;
        if (k < K) ptop[k] = id >= 0 ? t : -INFINITY;
      };
      int id0 = -1;
      float t0 = 0.f, z0 = 0.f;
      if (tid <= K) entry(tid, id0, t0);
      fetch(tid, v);
      if ((unsigned)id0 < (unsigned)a.V) z0 = ldv<T>(z, id0);
      for (int k = tid + threads; k <= K; k += threads) {
        int id;
        float t;
        entry(k, id, t);
        share(k, id, t);
        ztop[k] = ids[k] >= 0 ? ldv<T>(z, ids[k]) : 0.f;
      }
      if constexpr (MODE != DM_BWD) {
        for (int c = tid; c - tid < nvec; c += batch) {
          fetch(c + batch, next);
          if (c < kept_end)
#pragma unroll
            for (int u = 0; u < U; ++u) kept[c + u * threads] = __builtin_bit_cast(Line, v[u]);
          // half a batch at a time: a whole one unpacked took the loss's kernel from 79 registers to 90, three
          // blocks a CU to two (2048 rows of 32000 bf16, one temperature: 30 us to 36; 4096 of 50021: 84 to 93)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[U * W / 2];
#pragma unroll
            for (int j = 0; j < U * W / 2; ++j) x[j] = RV::get(v[h * U / 2 + j / W][j % W]);
            absorb<TWO>(run, x, scale);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) v[u] = next[u];
        }
        odd_ones([&](int i) __attribute__((always_inline)) {
          const float x[1] = {ldv<T>(z, i)};
          absorb<TWO>(run, x, scale);
        });
        if (MODE == DM_STEP) fetch(kKept * batch + tid, v);   // the second walk's first, behind what is kept
        rebase<TWO>(run, wave_max(run.m), scale);
#pragma unroll
        for (int i = 0; i < 1 + TWO; ++i) run.s[i] = wave_add(run.s[i]);
        if (lane == 0) {
          red[0][wave] = run.m;
          red[1][wave] = run.s[0];
          red[2][wave] = run.s[1];
        }
      }
      if (tid <= K) {
        share(tid, id0, t0);
        ztop[tid] = z0;
      }
      __syncthreads();
      // every wave for itself: lane l holds entries l, l + 64, ...
      float bad = 0.f;
#pragma unroll
      for (int j = 0; j < kTop / 64; ++j) {
        const int k = lane + 64 * j;
        eid[j] = k < K ? ids[k] : -1;
        e[j] = k < K ? ptop[k] : -INFINITY;
        tmax = fmaxf(tmax, e[j]);
        if (!(e[j] < INFINITY)) bad = 1.f;      // infinite or NaN: no distribution
      }
      tmax = wave_max(tmax);
#pragma unroll
      for (int j = 0; j < kTop / 64; ++j) {
        e[j] = tmax > -INFINITY ? top_term(e[j], tmax, scale[0]) : 0.f;
        tsum += e[j];
      }
      tsum = wave_add(tsum);
      if (wave_add(bad) > 0.f) tsum = NAN;
      taught = !(tsum == 0.f);
      labelled = ids[K] >= 0;
    }
    auto no_gradient = [&]() __attribute__((always_inline)) {
      for (int c = tid; c < nvec; c += threads) store(c, Raw{});
      odd_ones([&](int i) { stv<T>(dz, i, 0.f); });
    };
    if ((!taught && !labelled) || (MODE == DM_BWD && g == 0.f)) {   // no loss, or none that counts
      if (MODE != DM_BWD && tid == 0) a.loss[row] = 0.f;
      if (MODE == DM_FWD && tid < 4) a.stats[row * 4 + tid] = 0.f;
      if (MODE != DM_FWD) no_gradient();
      continue;
    }
    if constexpr (MODE != DM_BWD) {
      const int waves = threads >> 6;
      float m = red[0][0];
      for (int i = 1; i < waves; ++i) m = fmaxf(m, red[0][i]);
      set_top<TWO>(run, m, scale);
      run.s[0] = run.s[1] = 0.f;
      for (int i = 0; i < waves; ++i) {
        Sums p;
        set_top<TWO>(p, red[0][i], scale);
        p.s[0] = red[1][i];
        p.s[1] = red[2][i];
        rebase<TWO>(p, m, scale);
        run.s[0] += p.s[0];
        run.s[1] += p.s[1];
      }
      if (m == -INFINITY) run.s[0] = run.s[1] = NAN;   // nothing to choose from: no distribution
      if (MODE == DM_FWD && tid < 4) a.stats[row * 4 + tid] = tid == 0 ? run.m : tid == 1 ? run.s[0] : tid == 2 ? run.s[1] : 0.f;
    }
    const float s_soft = run.s[0], s_hard = run.s[TWO];

    if (MODE != DM_BWD && wave == 0) {
      // the natural logarithm of a term
      auto below = [&](float x, int i) __attribute__((always_inline)) {
        return kLn2 * (run.near ? fmaf(x, scale[i], -run.top[i]) : (x - run.m) * scale[i]);
      };
      float kl = 0.f;
      const float lp = logf(tsum), lq = logf(s_soft);
      if (taught)
#pragma unroll
        for (int j = 0; j < kTop / 64; ++j) {
          const int k = lane + 64 * j;
          const float p = e[j] / tsum;
          if (k < K && !(p == 0.f)) kl += p * (((ptop[k] - tmax) * a.inv_tau - lp) - (below(ztop[k], 0) - lq));
        }
      kl = wave_add(kl);
      if (lane == 0) {
        float l = taught ? (1.f - a.hard) * a.tau * a.tau * kl : 0.f;
        if (labelled) l += a.hard * (logf(s_hard) - below(ztop[K], TWO));
        a.loss[row] = l;
      }
    }
    if (MODE == DM_STEP && g == 0.f) {
      no_gradient();
      continue;
    }
    if constexpr (MODE != DM_FWD) {
      const float cs = taught ? g * (1.f - a.hard) * a.tau : 0.f, ch = labelled ? g * a.hard : 0.f;
      const float as = (TWO ? cs : cs + ch) / s_soft, ah = ch / s_hard;
      auto walk = [&](auto near) __attribute__((always_inline)) {
        auto grad = [&](float x) __attribute__((always_inline)) {
          const float d = term<decltype(near)::value>(run, x, scale[0], 0) * as;
          return TWO ? fmaf(term<decltype(near)::value>(run, x, scale[1], 1), ah, d) : d;
        };
        // at the entries' ids and the label; an id that comes twice gets the same value
        // from each of its entries
        for (int k0 = wave * 64; k0 <= K; k0 += threads) {      // whole waves: lanes read each other's entries
          const int k = k0 + lane, id = k <= K ? ids[k] : -1;
          float p = 0.f;
#pragma unroll
          for (int j = 0; j < kTop / 64; ++j)
            for (int i = 0; i < 64 && i + 64 * j < K; ++i)
              p += __builtin_amdgcn_readlane(eid[j], i) == id ? lane_value(e[j], i) : 0.f;
          if (k <= K) {
            float d = grad(ztop[k]);
            if (taught) d -= cs * (p / tsum);
            if (labelled && ids[K] == id) d -= ch;
            dtop[k] = d;
          }
        }
        auto put = [&](int c, Raw x) __attribute__((always_inline)) {
          Raw o;
#pragma unroll
          for (int j = 0; j < W; ++j) o[j] = RV::put(grad(RV::get(x[j])));
          if (c < nvec) store(c, o);
        };
        for (int c = (MODE == DM_STEP ? kKept * batch : 0) + tid; c - tid < nvec; c += batch) {
          fetch(c + batch, next);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            put(c + u * threads, v[u]);
            v[u] = next[u];
          }
        }
        for (int c = tid; c < kept_end; c += threads) put(c, __builtin_bit_cast(Raw, kept[c]));
        odd_ones([&](int i) __attribute__((always_inline)) { stv<T>(dz, i, grad(ldv<T>(z, i))); });
      };
      if (run.near) walk(std::true_type());
      else walk(std::false_type());
      __syncthreads();                          // the row is written, and dtop
      for (int k = tid; k <= K; k += threads)
        if (ids[k] >= 0) stv<T>(dz, ids[k], dtop[k]);
    }
  }
}

static sl_status distill_args(DistillArgs& a, sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* z,
                              int64_t ld, const void* dz, int64_t ld_out) {
  sl_status st = check_dtype(dt);
  if (st == SL_OK) st = build_seqtab(lay, a.st);
  if (st != SL_OK) return st;
  if (!p || !z) SL_FAIL(SL_ERR_NULL, "the targets and logits required");
  if (p->vocab < 1 || p->vocab > (1LL << 30)) SL_FAIL(SL_ERR_RANGE, "vocabulary of %lld outside [1, 2^30]", (long long)p->vocab);
  if (!(p->hard >= 0.f && p->hard <= 1.f)) SL_FAIL(SL_ERR_RANGE, "hard must be in [0, 1]");
  if (!(p->temperature >= 1e-6f && p->temperature <= 1e6f)) SL_FAIL(SL_ERR_RANGE, "temperature must be in [1e-6, 1e6]");
  if (p->hard < 1.f) {
    if (p->top < 1 || p->top > kTop) SL_FAIL(SL_ERR_RANGE, "top = %d outside [1, %d]", p->top, kTop);
    if (!p->top_ids || !p->top_logits) SL_FAIL(SL_ERR_NULL, "top_ids and top_logits required");
  }
  if (p->hard > 0.f && !p->labels) SL_FAIL(SL_ERR_NULL, "labels required");
  if (ld < p->vocab || (dz && ld_out < p->vocab))
    SL_FAIL(SL_ERR_SHAPE, "rows of %lld and %lld elements hold no %lld logits", (long long)ld, (long long)ld_out, (long long)p->vocab);
  const uintptr_t es = dt == SL_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(dz)) % es)
    SL_FAIL(SL_ERR_ALIGN, "logits and dlogits must be aligned to their elements");
  if (!aligned16(p->top_ids) || !aligned16(p->top_logits) || !aligned16(p->labels))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  a.z = z; a.ld = ld; a.ld_out = ld_out;
  a.top_ids = p->top_ids; a.top_logits = p->top_logits; a.labels = p->labels;
  a.V = (int)p->vocab; a.top = p->top;
  a.rows = lay->batch * lay->seq_len;
  a.tau = p->temperature; a.inv_tau = 1.f / p->temperature; a.hard = p->hard;
  a.scale = p->hard < 1.f ? (float)(1.4426950408889634 / (double)p->temperature) : kLog2e;
  return SL_OK;
}

template <typename T, int MODE, bool TWO> static void launch_distill(const DistillArgs& a, hipStream_t s) {
  // as few threads as load a row at once (8192 rows of 2000 bf16, loss: 64 threads 12 us, 512 72)
  int threads = 64;
  while (threads < kRowThreads && threads * kVecs < a.V / RowVec<T>::W) threads *= 2;
  const dim3 grid = walk_grid(a.rows), block(threads);
  const size_t lds = MODE == DM_STEP ? (size_t)kKept * threads * kVecs * 16 : 0;
  // What is used once goes past the caches, in rows of whole vectors, from 112 MiB (117 MB, of the last
  // cache's 256 MiB) on: the gradient's stores by all rows, context rows' zeros among them, and in calls
  // of loss or gradient alone the loads by the rows with a loss, which alone are read.  Measured in us,
  // bf16, through the caches and past them.  Stores: step of 4096 rows of 128256 481, 438; with the products
  // that make the logits and read the gradient, 1750 rows of 32000 (112 MB) 287, 296, 2000 (128 MB) 302, 302,
  // 2500 364, 358, 4 x 1024 of 768 context rows each 398, 390; 4 x 512 of 384 (131 MB, 98 of them
  // zeros) 240, 260, the step alone 41.5, 37.7.  Loads: loss and gradient with those products, 1750 rows
  // 300, 313, 2000 311, 312, 2500 367, 372, 4096 490, 484, without them 2048 rows 88, 85; 4 x 512 of 384
  // context rows (33 MB read) 45, 49.
  const bool whole = (a.ld | a.ld_out) * (long long)sizeof(T) % 16 == 0 && aligned16(a.z) && aligned16(a.dz);
  const long long row = a.V * (long long)sizeof(T);
  const bool stores = whole && a.rows * row >= 112LL << 20, loads = whole && a.st.T_out * row >= 112LL << 20;
  auto go = [&](auto nt) { hipLaunchKernelGGL((distill_kernel<T, MODE, TWO, decltype(nt)::value>), grid, block, lds, s, a); };
  using None = std::integral_constant<int, 0>;
  using Stores = std::integral_constant<int, 1>;
  using Both = std::integral_constant<int, 2>;
  if constexpr (MODE == DM_STEP) stores ? go(Stores()) : go(None());
  else if constexpr (MODE == DM_BWD) loads ? go(Both()) : stores ? go(Stores()) : go(None());
  else loads ? go(Both()) : go(None());
}

template <int MODE> static sl_status run_distill(sl_dtype dt, const DistillArgs& a, void* stream) {
  sl_status st = check_arch();
  if (st != SL_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool two = a.hard > 0.f && a.hard < 1.f && a.tau != 1.f;
  if (dt == SL_BF16) two ? launch_distill<bf16, MODE, true>(a, s) : launch_distill<bf16, MODE, false>(a, s);
  else two ? launch_distill<float, MODE, true>(a, s) : launch_distill<float, MODE, false>(a, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}

}  // namespace sl

using namespace sl;

extern "C" sl_status sl_distill_fwd(sl_dtype dt, const sl_layout* lay, const sl_distill* p, const void* logits,
                                    int64_t ld, float* loss, float* stats, void* stream) {
  if (!loss || !stats) SL_FAIL(SL_ERR_NULL, "loss and stats required");
  DistillArgs a{};
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
  DistillArgs a{};
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
  DistillArgs a{};
  sl_status st = distill_args(a, dt, lay, p, logits, ld, dlogits, ld_out);
  if (st != SL_OK) return st;
  if (!aligned16(loss) || !aligned16(dloss)) SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  a.loss = loss; a.dloss = dloss; a.dz = dlogits;
  return run_distill<DM_STEP>(dt, a, stream);
}
