// Rotary positions and per-head norms of the q and k rows that the q/k/v
// projections write, forward and backward, in one pass over the data.
//
// Rotation: the first rot_dim values of a head are pairs (a, b); with the
// angle phi = position * frequency of its pair,
//   a' = c a - s b,  b' = c b + s a,   c = amplitude cos phi, s = amplitude sin phi.
// The rest of the head is copied.  The gradient is the same with -phi.
// Head norm: u = x r w with r = (mean x^2 + eps)^-1/2, then the rotation.  With
// g the gradient turned back and h = g w:
//   dx = r (h - x r^2 mean(h x)),  dw = sum over rows of g x r.
//
// Angles: a table holds each pair's frequency as a whole number of 2^-64 turns,
// so position * frequency is an integer product that drops whole turns exactly,
// at any position; its upper 32 bits are the angle to 1.5e-9 rad.  Sine and
// cosine are their Taylor polynomials on [-pi/4, pi/4] (the first dropped terms
// are below 2e-9, under half a step of fp32) and a quarter-turn swap.
//
// What bounds it: HBM (each row read once and written once), as long as the
// vector work stays below it.  A block forms the sines and cosines of its tokens
// once, in LDS, and walks its rows (the tokens' heads, one behind the other).  A
// thread owns one "unit" of a head, two vectors of V values: V pairs, or 2 V
// values behind the rotated part; the lanes of one head stand next to each
// other, so a norm's sums are shuffles.  The next row is loaded before this one
// is worked on.  Measured (bf16, heads of 128): rotation of 2 x 1024 tokens of 64
// heads 13 us, 5.2 TB/s; norms of 2 x 8192 tokens of 40 heads 67 us forward, 5.0
// TB/s, and 111 us backward, 4.5 TB/s, where a copy of 2 GiB runs at 4.9 and one of
// 64 MiB at 6.8.
#include <cmath>

#include "sl_common.hpp"
#include "sl_host.hpp"

namespace sl {

enum RotMode { RM_ROTATE, RM_NORM_FWD, RM_NORM_BWD };

struct RotArgs {
  const void* x[2];     // q, k: rotate / norm input
  const void* dy[2];    // norm backward: gradients of the rotated rows
  void* y[2];           // out: rotated rows, or dx
  const float* w[2];    // norm weights [hd]
  float* part;          // norm backward: [grid][2][hd] sums of g x r
  const unsigned long long* turns;
  const int* pos;
  int nh[2];            // heads of q and of k
  int hd, rot, L, T;
  int tokens;           // tokens a block takes at a time
  int lph_log2;         // lanes per head, log2
  float amp, sign, eps, inv_hd;
};

constexpr int kTokens = 4;   // most tokens a block takes at a time

// V values, moved as one
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };

template <typename T> __device__ inline float el2f(T x);
template <> __device__ inline float el2f<float>(float x) { return x; }
template <> __device__ inline float el2f<bf16>(bf16 x) { return bf2f(x.v); }
template <typename T> __device__ inline T f2el(float x);
template <> __device__ inline float f2el<float>(float x) { return x; }
template <> __device__ inline bf16 f2el<bf16>(float x) { return __builtin_bit_cast(bf16, (__bf16)x); }   // to nearest even

// cos and sin of 2 pi * phase / 2^32
__device__ inline void cos_sin_turn(uint32_t phase, float& c, float& s) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(phase - (quarter << 30)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
  const float x2 = x * x;
  float sn = fmaf(x2, 2.7557319223985893e-6f, -1.9841269841269841e-4f);
  sn = fmaf(x2, sn, 8.3333333333333333e-3f);
  sn = fmaf(x2, sn, -1.6666666666666666e-1f);
  sn = fmaf(x2 * sn, x, x);
  float cs = fmaf(x2, -2.7557319223985888e-7f, 2.4801587301587302e-5f);
  cs = fmaf(x2, cs, -1.3888888888888889e-3f);
  cs = fmaf(x2, cs, 4.1666666666666666e-2f);
  cs = fmaf(x2, cs, -0.5f);
  cs = fmaf(x2, cs, 1.0f);
  const bool swap = quarter & 1u;
  const float a = swap ? sn : cs, b = swap ? cs : sn;
  c = (quarter + 1u) & 2u ? -a : a;
  s = quarter & 2u ? -b : b;
}

template <typename T, int V, bool INTER, int MODE>
__global__ void __launch_bounds__(256) rotary_kernel(const RotArgs a) {
  constexpr int NU = V == 1 ? 2 : 1;   // units per lane (256-wide heads of single pairs need two)
  constexpr int W = 2 * V;             // values of a unit
  constexpr bool NORM = MODE != RM_ROTATE, BWD = MODE == RM_NORM_BWD;
  using VT = Vec<T, V>;
  __shared__ __attribute__((aligned(32))) float trig[2][kTokens * 128];   // cosines, sines of the block's tokens
  __shared__ __attribute__((aligned(16))) float red[BWD ? 256 * NU * W : 4];
  const int lph = 1 << a.lph_log2;
  const int ul = threadIdx.x & (lph - 1);          // unit (and ul + lph)
  const int slot = threadIdx.x >> a.lph_log2, nslot = 256 >> a.lph_log2;
  const int nunit = a.hd / W, npair = a.rot / W, np2 = a.rot / 2;

  int off[NU][2];
  bool live[NU], pair[NU];
  float acc[2][NU][W];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = ul + n * lph;
    live[n] = u < nunit;
    pair[n] = u < npair;
    if (pair[n]) {
      off[n][0] = INTER ? W * u : V * u;
      off[n][1] = INTER ? W * u + V : a.rot / 2 + V * u;
    } else {
      off[n][0] = live[n] ? W * u : 0;             // behind the pairs: units tile the head in order
      off[n][1] = live[n] ? W * u + V : 0;
    }
    if constexpr (BWD) {
#pragma unroll
      for (int j = 0; j < W; ++j) acc[0][n][j] = acc[1][n][j] = 0.f;
    }
  }

  for (int tok0 = blockIdx.x * a.tokens; tok0 < a.T; tok0 += gridDim.x * a.tokens) {
    const int ntok = a.T - tok0 < a.tokens ? a.T - tok0 : a.tokens;
    if (tok0 != (int)blockIdx.x * a.tokens) __syncthreads();   // the last tokens' angles are still read
    for (int i = threadIdx.x; i < ntok * np2; i += 256) {
      const int t = i / np2, j = i - t * np2;
      const int pos = a.pos ? a.pos[tok0 + t] : (tok0 + t) % a.L;
      const unsigned long long f = a.turns[j];
      const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32), ps = (uint32_t)pos;
      float c, sn;
      // upper word of f * pos (pos signed)
      cos_sin_turn(__umulhi(lo, ps) + hi * ps - (pos < 0 ? lo : 0u), c, sn);
      trig[0][t * np2 + j] = c * a.amp;
      trig[1][t * np2 + j] = sn * a.amp * a.sign;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int nh = a.nh[p], items = ntok * nh;   // rows of hd values, one behind the other
      if (slot - (slot & (64 / lph - 1)) >= items) continue;   // none for this wave
      float w[NU][W];
      if constexpr (NORM) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int j = 0; j < W; ++j) w[n][j] = live[n] ? a.w[p][off[n][j / V] + j % V] : 0.f;
      }
      const long long base = (long long)tok0 * nh * a.hd;
      const T* src = reinterpret_cast<const T*>(BWD ? a.dy[p] : a.x[p]) + base;
      const T* xin = reinterpret_cast<const T*>(a.x[p]) + base;
      T* dst = reinterpret_cast<T*>(a.y[p]) + base;
      VT rv[NU][2], rx[NU][2];
      auto load = [&](int it) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NU; ++n)
          if (it < items && live[n]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              rv[n][e] = *reinterpret_cast<const VT*>(src + (long long)it * a.hd + off[n][e]);
              if constexpr (BWD) rx[n][e] = *reinterpret_cast<const VT*>(xin + (long long)it * a.hd + off[n][e]);
            }
          }
      };
      int t = slot / nh, h = slot - t * nh;
      const int dt = nslot / nh, dh = nslot - dt * nh;
      load(slot);
      // (the lanes of a wave leave together, so that the shuffles are whole)
      for (int it = slot; it - (slot & (64 / lph - 1)) < items; it += nslot) {
        const bool on = it < items;
        float v[NU][W], x[NU][W];
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int j = 0; j < W; ++j) {
            v[n][j] = on && live[n] ? el2f<T>(rv[n][j / V].v[j % V]) : 0.f;
            if constexpr (BWD) x[n][j] = on && live[n] ? el2f<T>(rx[n][j / V].v[j % V]) : 0.f;
          }
        load(it + nslot);
        if constexpr (MODE == RM_NORM_FWD) {
          float ss = 0.f;
#pragma unroll
          for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int j = 0; j < W; ++j) ss = fmaf(v[n][j], v[n][j], ss);
          for (int o = lph >> 1; o; o >>= 1) ss += __shfl_xor(ss, o);
          const float r = rsqrtf(fmaf(ss, a.inv_hd, a.eps));
#pragma unroll
          for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int j = 0; j < W; ++j) v[n][j] = v[n][j] * r * w[n][j];
        }
        // the pairs of a unit: value j of both vectors, or neighbours across them
#pragma unroll
        for (int n = 0; n < NU; ++n)
          if (pair[n]) {
            const float* const tc = &trig[0][(on ? t : 0) * np2 + (ul + n * lph) * V];
            const float* const ts = &trig[1][(on ? t : 0) * np2 + (ul + n * lph) * V];
            const Vec<float, V> cs = *reinterpret_cast<const Vec<float, V>*>(tc);
            const Vec<float, V> sn = *reinterpret_cast<const Vec<float, V>*>(ts);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : V + j;
              const float va = v[n][ia], vb = v[n][ib];
              v[n][ia] = va * cs.v[j] - vb * sn.v[j];
              v[n][ib] = vb * cs.v[j] + va * sn.v[j];
            }
          }
        if constexpr (BWD) {
          float ss = 0.f, hx = 0.f;
#pragma unroll
          for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int j = 0; j < W; ++j) {
              ss = fmaf(x[n][j], x[n][j], ss);
              hx = fmaf(v[n][j] * w[n][j], x[n][j], hx);
            }
          for (int o = lph >> 1; o; o >>= 1) {
            ss += __shfl_xor(ss, o);
            hx += __shfl_xor(hx, o);
          }
          const float r = rsqrtf(fmaf(ss, a.inv_hd, a.eps));
          const float m = hx * a.inv_hd * r * r;
#pragma unroll
          for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const float g = v[n][j];
              // a lane without a row holds zeros, and r may be infinite
              if (on) acc[p][n][j] = fmaf(g, x[n][j] * r, acc[p][n][j]);
              v[n][j] = r * (g * w[n][j] - x[n][j] * m);
            }
        }
#pragma unroll
        for (int n = 0; n < NU; ++n)
          if (on && live[n]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              VT r;
#pragma unroll
              for (int j = 0; j < V; ++j) r.v[j] = f2el<T>(v[n][e * V + j]);
              *reinterpret_cast<VT*>(dst + (long long)it * a.hd + off[n][e]) = r;
            }
          }
        t += dt;
        h += dh;
        if (h >= nh) {
          h -= nh;
          ++t;
        }
      }
    }
  }
  if constexpr (BWD) {
    // sum the head slots in order; unit u's values of slot s at [s][u][j]
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int j = 0; j < W; ++j) red[(slot * (NU * lph) + ul + n * lph) * W + j] = acc[p][n][j];
      __syncthreads();
      for (int c = threadIdx.x; c < a.hd; c += 256) {   // c counts in unit order
        const int u = c / W, j = c % W;
        float s = 0.f;
        for (int k = 0; k < nslot; ++k) s += red[(k * (NU * lph) + u) * W + j];
        // the head position of value j of unit u
        int at = c;
        if (!INTER && u < npair) at = (j / V) * (a.rot / 2) + V * u + j % V;
        a.part[((long long)blockIdx.x * 2 + p) * a.hd + at] = s;
      }
    }
  }
}

// dw = the blocks' sums, added in a fixed order: 128 row groups of 8 columns,
// then the groups in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int nblk, int hd,
                                                       float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sm[128][9];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int col = blockIdx.x * 8 + c;
  float s = 0.f;
  if (col < 2 * hd) {
#pragma unroll 8
    for (int i = g; i < nblk; i += 128) s += part[(long long)i * 2 * hd + col];
  }
  sm[g][c] = s;
  __syncthreads();
  if (threadIdx.x < 64) {   // 8 sums of 16 groups for each column, then those 8
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sm[(threadIdx.x >> 3) * 16 + i][c];
    for (int o = 8; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if (threadIdx.x < 8 && col < 2 * hd) {
      if (col < hd) dwq[col] = s;
      else if (dwk) dwk[col - hd] = s;
    }
  }
}

// Tokens per block and blocks.  Up to four tokens share a block's set-up where
// that leaves 512 blocks, two to a CU (norms of 2048 tokens of 64 heads of 128 in
// bf16, forward and backward: 53-57 us with four, 64 us with one); a launch holds
// fewer than 2^32 threads, so past 2^20 blocks they walk on.  The norm's backward walks from 1024 blocks,
// whose weight-gradient sums one more launch adds.
constexpr int kNormBwdBlocks = 1024;
inline int rot_tokens(long long T) { return T >= 512 * kTokens ? kTokens : T >= 1024 ? 2 : 1; }
inline int rot_blocks(long long T, int most) {
  const long long n = (T + rot_tokens(T) - 1) / rot_tokens(T);
  return (int)(n < most ? n : most);
}

template <typename T, int V, bool INTER>
static void launch_mode(int mode, const RotArgs& a, dim3 grid, hipStream_t s) {
  if (mode == RM_ROTATE) hipLaunchKernelGGL((rotary_kernel<T, V, INTER, RM_ROTATE>), grid, dim3(256), 0, s, a);
  else if (mode == RM_NORM_FWD) hipLaunchKernelGGL((rotary_kernel<T, V, INTER, RM_NORM_FWD>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((rotary_kernel<T, V, INTER, RM_NORM_BWD>), grid, dim3(256), 0, s, a);
}

template <typename T>
static void launch_vec(int V, bool inter, int mode, const RotArgs& a, dim3 grid, hipStream_t s) {
#define SL_ROT_V(N)                                          \
  case N:                                                    \
    if (inter) launch_mode<T, N, true>(mode, a, grid, s);    \
    else launch_mode<T, N, false>(mode, a, grid, s);         \
    break;
  switch (V) {
    case 8:
      if constexpr (sizeof(T) == 2) {
        if (inter) launch_mode<T, 8, true>(mode, a, grid, s);
        else launch_mode<T, 8, false>(mode, a, grid, s);
      }
      break;
    SL_ROT_V(4)
    SL_ROT_V(2)
    SL_ROT_V(1)
  }
#undef SL_ROT_V
}

static sl_status run_rotary(int mode, sl_dtype dt, RotArgs& a, int inter, hipStream_t s) {
  const int es = dt == SL_BF16 ? 2 : 4;
  // the widest vector (up to 16 bytes) that tiles the rotated part and the head
  int V = 16 / es;
  while (V > 1 && (a.rot % (2 * V) || a.hd % (2 * V))) V >>= 1;
  const int nunit = a.hd / (2 * V), per_lane = V == 1 ? 2 : 1;
  int lg = 0;
  while ((per_lane << lg) < nunit) ++lg;
  a.lph_log2 = lg;
  a.tokens = rot_tokens(a.T);
  a.inv_hd = 1.0f / a.hd;
  const int blocks = rot_blocks(a.T, mode == RM_NORM_BWD ? kNormBwdBlocks : 1 << 20);
  if (dt == SL_BF16) launch_vec<bf16>(V, inter != 0, mode, a, dim3((unsigned)blocks), s);
  else launch_vec<float>(V, inter != 0, mode, a, dim3((unsigned)blocks), s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}

static sl_status check_heads(const sl_heads* h, bool has_k) {
  if (!h) SL_FAIL(SL_ERR_NULL, "heads is NULL");
  if (h->n_q_heads < 1 || (has_k && h->n_kv_heads < 1) || h->n_q_heads > 65536 || h->n_kv_heads > 65536)
    SL_FAIL(SL_ERR_SHAPE, "head counts %d, %d must be in [1, 65536]", h->n_q_heads, h->n_kv_heads);
  if (h->head_dim < 2 || h->head_dim > 256 || h->head_dim % 2)
    SL_FAIL(SL_ERR_SHAPE, "head_dim %d must be even and at most 256", h->head_dim);
  return SL_OK;
}

// Fill the arguments shared by every mode; rot may be NULL for the norms.
static sl_status rot_args(RotArgs& a, sl_dtype dt, const sl_layout* lay, const sl_heads* heads,
                          const sl_rotary* rot, bool has_k, float sign, int* inter) {
  if (dt != SL_BF16 && dt != SL_F32) SL_FAIL(SL_ERR_DTYPE, "dtype must be SL_F32 or SL_BF16");
  if (!lay) SL_FAIL(SL_ERR_NULL, "layout is NULL");
  if (lay->batch < 1 || lay->batch > SL_MAX_SEQS)
    SL_FAIL(SL_ERR_RANGE, "batch %d outside [1, %d]", lay->batch, SL_MAX_SEQS);
  if (lay->seq_len < 1) SL_FAIL(SL_ERR_RANGE, "seq_len %d < 1", lay->seq_len);
  if ((long long)lay->batch * lay->seq_len > (1LL << 30)) SL_FAIL(SL_ERR_RANGE, "too many tokens");
  sl_status st = check_heads(heads, has_k);
  if (st != SL_OK) return st;
  a = RotArgs{};
  a.T = lay->batch * lay->seq_len;
  a.L = lay->seq_len;
  a.hd = heads->head_dim;
  a.nh[0] = heads->n_q_heads;
  a.nh[1] = has_k ? heads->n_kv_heads : 0;
  a.amp = 1.f;
  a.sign = sign;
  *inter = 0;
  if (rot) {
    if (rot->rot_dim < 0 || rot->rot_dim % 2 || rot->rot_dim > a.hd)
      SL_FAIL(SL_ERR_SHAPE, "rot_dim %d must be even and at most head_dim %d", rot->rot_dim, a.hd);
    if (rot->rot_dim > 0 && !rot->turns) SL_FAIL(SL_ERR_NULL, "rotary turns is NULL");
    if (!aligned16(rot->turns) || !aligned16(rot->pos))
      SL_FAIL(SL_ERR_ALIGN, "rotary turns and pos must be 16-byte aligned");
    if (!(std::isfinite(rot->amplitude))) SL_FAIL(SL_ERR_RANGE, "rotary amplitude is not finite");
    a.rot = rot->rot_dim;
    a.turns = reinterpret_cast<const unsigned long long*>(rot->turns);
    a.pos = rot->pos;
    a.amp = rot->amplitude;
    *inter = rot->interleaved != 0;
  }
  return SL_OK;
}

}  // namespace sl

using namespace sl;

extern "C" sl_status sl_rotary_table(const sl_rotary_spec* sp, uint64_t* turns, float* amplitude) {
  if (!sp || !turns || !amplitude) SL_FAIL(SL_ERR_NULL, "spec, turns and amplitude must be non-NULL");
  if (sp->rot_dim < 2 || sp->rot_dim > 256 || sp->rot_dim % 2)
    SL_FAIL(SL_ERR_SHAPE, "rot_dim %d must be even and in [2, 256]", sp->rot_dim);
  if (!(sp->base > 1.0) || !std::isfinite(sp->base)) SL_FAIL(SL_ERR_RANGE, "base must be finite and above 1");
  if (sp->scaling < SL_ROPE_NONE || sp->scaling > SL_ROPE_YARN)
    SL_FAIL(SL_ERR_DTYPE, "unknown rotary scaling %d", (int)sp->scaling);
  if (sp->scaling != SL_ROPE_NONE && (!(sp->factor >= 1.0) || !std::isfinite(sp->factor)))
    SL_FAIL(SL_ERR_RANGE, "scaling factor must be finite and at least 1");
  if (sp->scaling >= SL_ROPE_WAVELENGTH &&
      (sp->original_len < 1 || !(sp->low_turns > 0.0) || !(sp->high_turns > sp->low_turns) ||
       !std::isfinite(sp->high_turns)))
    SL_FAIL(SL_ERR_RANGE, "original_len >= 1 and 0 < low_turns < high_turns required");
  const long double two_pi = 6.283185307179586476925286766559L;
  const int rot = sp->rot_dim, n = rot / 2;
  const long double s = sp->scaling == SL_ROPE_NONE ? 1.0L : (long double)sp->factor;
  long double base = sp->base;
  if (sp->scaling == SL_ROPE_BASE && rot > 2) base *= powl(s, (long double)rot / (rot - 2));
  // yarn: the pairs between which the stretch ramps up
  double lo = 0, span = 1;
  if (sp->scaling == SL_ROPE_YARN) {
    auto index = [&](double turns_at) {
      return rot * std::log(sp->original_len / (turns_at * (double)two_pi)) / (2 * std::log(sp->base));
    };
    lo = std::fmax(std::floor(index(sp->high_turns)), 0.0);
    const double hi = std::fmin(std::ceil(index(sp->low_turns)), rot - 1.0);
    span = std::fmax(hi - lo, 0.001);
  }
  for (int i = 0; i < n; ++i) {
    long double f = powl(base, -2.0L * i / rot);
    long double stretch = 0;   // share of the frequency divided by the factor
    if (sp->scaling == SL_ROPE_LINEAR) stretch = 1;
    if (sp->scaling == SL_ROPE_WAVELENGTH) {
      const long double t = sp->original_len * f / two_pi;   // turns within the original length
      stretch = 1.0L - fminl(fmaxl((t - sp->low_turns) / (sp->high_turns - sp->low_turns), 0.0L), 1.0L);
    }
    if (sp->scaling == SL_ROPE_YARN) stretch = std::fmin(std::fmax((i - lo) / span, 0.0), 1.0);
    f = f / s * stretch + f * (1.0L - stretch);
    turns[i] = (uint64_t)(f / two_pi * 18446744073709551616.0L + 0.5L);   // f <= 1: below a sixth of a turn
  }
  *amplitude = sp->scaling == SL_ROPE_YARN ? (float)(0.1 * std::log(sp->factor) + 1.0) : 1.0f;
  return SL_OK;
}

extern "C" sl_status sl_rotary_apply(sl_dtype dt, const sl_layout* lay, const sl_heads* heads, const sl_rotary* rot,
                                     const void* q, const void* k, void* q_out, void* k_out, int32_t inverse,
                                     void* stream) {
  if (!rot) SL_FAIL(SL_ERR_NULL, "rot is NULL");
  if (!q || !q_out || (k == nullptr) != (k_out == nullptr))
    SL_FAIL(SL_ERR_NULL, "q and q_out required; k and k_out both or neither");
  RotArgs a;
  int inter;
  sl_status st = rot_args(a, dt, lay, heads, rot, k != nullptr, inverse ? -1.f : 1.f, &inter);
  if (st != SL_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
    SL_FAIL(SL_ERR_ALIGN, "q, k, q_out and k_out must be 16-byte aligned");
  st = check_arch();
  if (st != SL_OK) return st;
  a.x[0] = q; a.x[1] = k; a.y[0] = q_out; a.y[1] = k_out;
  return run_rotary(RM_ROTATE, dt, a, inter, reinterpret_cast<hipStream_t>(stream));
}

extern "C" sl_status sl_head_norm_fwd(sl_dtype dt, const sl_layout* lay, const sl_heads* heads, const sl_rotary* rot,
                                      float eps, const void* q, const void* k, const float* wq, const float* wk,
                                      void* q_out, void* k_out, void* stream) {
  if (!q || !q_out || !wq || (k == nullptr) != (k_out == nullptr) || (k && !wk))
    SL_FAIL(SL_ERR_NULL, "q, wq and q_out required; k, wk and k_out all or none");
  RotArgs a;
  int inter;
  sl_status st = rot_args(a, dt, lay, heads, rot, k != nullptr, 1.f, &inter);
  if (st != SL_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) SL_FAIL(SL_ERR_RANGE, "eps must be finite and >= 0");
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(wq) || !aligned16(wk))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  st = check_arch();
  if (st != SL_OK) return st;
  a.x[0] = q; a.x[1] = k; a.y[0] = q_out; a.y[1] = k_out; a.w[0] = wq; a.w[1] = wk;
  a.eps = eps;
  return run_rotary(RM_NORM_FWD, dt, a, inter, reinterpret_cast<hipStream_t>(stream));
}

extern "C" size_t sl_head_norm_workspace_bytes(const sl_layout* lay, const sl_heads* heads) {
  RotArgs a;
  int inter;
  // (the size does not depend on k; without kv heads it is asked for calls without k)
  if (rot_args(a, SL_F32, lay, heads, nullptr, heads && heads->n_kv_heads != 0, 1.f, &inter) != SL_OK) return 0;
  return (size_t)rot_blocks(a.T, kNormBwdBlocks) * 2 * a.hd * sizeof(float);
}

extern "C" sl_status sl_head_norm_bwd(sl_dtype dt, const sl_layout* lay, const sl_heads* heads, const sl_rotary* rot,
                                      float eps, const void* q, const void* k, const float* wq, const float* wk,
                                      const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                                      float* dwk, void* ws, size_t ws_bytes, void* stream) {
  if (!q || !dq_out || !dq || !wq || !dwq) SL_FAIL(SL_ERR_NULL, "q, wq, dq_out, dq and dwq required");
  if (k ? (!wk || !dk_out || !dk || !dwk) : (dk_out || dk || dwk))
    SL_FAIL(SL_ERR_NULL, "k, wk, dk_out, dk and dwk all or none");
  RotArgs a;
  int inter;
  sl_status st = rot_args(a, dt, lay, heads, rot, k != nullptr, -1.f, &inter);
  if (st != SL_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) SL_FAIL(SL_ERR_RANGE, "eps must be finite and >= 0");
  if (!aligned16(q) || !aligned16(k) || !aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) ||
      !aligned16(wq) || !aligned16(wk) || !aligned16(dwq) || !aligned16(dwk) || !aligned16(ws))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  const int nblk = rot_blocks(a.T, kNormBwdBlocks);
  if (!ws || ws_bytes < (size_t)nblk * 2 * a.hd * sizeof(float))
    SL_FAIL(SL_ERR_WORKSPACE, "head norm workspace too small (%zu bytes)", ws_bytes);
  st = check_arch();
  if (st != SL_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  a.x[0] = q; a.x[1] = k; a.dy[0] = dq_out; a.dy[1] = dk_out; a.y[0] = dq; a.y[1] = dk; a.w[0] = wq; a.w[1] = wk;
  a.eps = eps;
  a.part = reinterpret_cast<float*>(ws);
  st = run_rotary(RM_NORM_BWD, dt, a, inter, s);
  if (st != SL_OK) return st;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)ceil_div(2 * a.hd, 8)), dim3(1024), 0, s, a.part, nblk, a.hd,
                     dwq, dwk);
  SL_HIP(hipGetLastError());
  return SL_OK;
}
