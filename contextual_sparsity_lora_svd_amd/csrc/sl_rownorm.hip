// Norms of whole rows with the residual sum in the same pass:
//   h = x + r,  u = (h - m) s,  y = u w + b,
//   m = mean of the row (0 where it is not centred),  s = (mean (h - m)^2 + eps)^(-1/2).
// Backward, with g = dy w and the gradient dres that reaches h by its other way:
//   dx = s (g - mean g - u mean(g u)) + dres,  dw = sum over rows of dy u,  db = sum over rows of dy.
//
// A row belongs to a group of lanes, 8 to 64 of one wave or several whole waves,
// and stays in registers from its loads to its stores.  The variance is formed from
// differences, never from mean h^2 - m^2: each wave takes the mean of its own
// values and sums the squares of their distances from it, and the waves' means and
// sums are joined (the squares about the row's mean are those about the wave's and
// n (m_wave - m)^2), with one exchange through LDS a row.  The rounding error of the
// mean comes out of the same sums and is kept beside it.  A group walks over
// rows and loads the next row before it works on this one.  The backward keeps the
// sums of dw and db of its rows in registers; a block adds its groups' sums in LDS,
// and one more launch the blocks' in a fixed order.
//
// Measured (bf16, with the residual sum and its gradient): 2 x 8192 rows of 5120, not centred:
// forward 114 us, 5.9 TB/s, backward 137 and 5 for the last launch, 4.7 TB/s, where an elementwise
// copy runs at 6.2; 2 x 1024 rows of 4096: 17, 17 and 4.  What bounds it: memory where there are rows enough
// to fill it.  Below that, forward: the first loads and the last stores of two or three rows a
// block, three blocks to a CU.  Backward: one block of 8 waves to a CU walks over eight rows with one
// loaded ahead, some 24 KB in flight; more blocks cost more in partial sums than they bring, more waves
// a block more in joining groups (figures at norm_bwd_blocks).  Narrow rows, many groups to a block:
// that join, one group behind the other.
#include <cmath>
#include <type_traits>

#include "sl_rows.hpp"

namespace sl {

struct RowNormArgs {
  const void *x, *r;         // forward: summands; backward: x is h
  const void *dy, *dres;
  void *y, *h;               // forward: outputs; backward: y is dx
  const float *w, *b;
  float* stats;              // [T][3]: m, what m rounded away, s
  float* part;               // backward: [blocks][2][D]
  int T, nvec, D;
  int group;                 // lanes of a row
  float eps, inv_d;
};

constexpr int kNormWaves = 16;   // most waves of a block

// Sum over a row's lanes where they are of one wave.
__device__ inline float group_add(float x, int group) {
  if (group == 64) return wave_add(x);
  x += dpp<kXor1>(x);
  x += dpp<kXor2>(x);
  x += dpp<kMirror8>(x);
  if (group >= 16) x += dpp<kMirror16>(x);
  if (group >= 32) x += __shfl_xor(x, 16);
  return x;
}

// Lanes of a wave that hold values in place e of their vectors.
__device__ inline int live_lanes(const RowNormArgs& a, int wave, int e) {
  const int n = a.nvec - e * a.group - wave * 64;
  return n < 0 ? 0 : n < 64 ? n : 64;
}

template <typename T, int N> __device__ inline void load_floats(const float* p, float (&v)[N], int at) {
#pragma unroll
  for (int j = 0; j < 16 / (int)sizeof(T); j += 4) {
    const Vec<float, 4> x = *reinterpret_cast<const Vec<float, 4>*>(p + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[at + j + i] = x.v[i];
  }
}

// A row's exchange between waves takes the two halves of an LDS array in turn, so
// one barrier a row is enough: a half is written again only behind the next row's.
template <typename T, int NV, bool CENTERED>
__global__ void __launch_bounds__(64 * kNormWaves, NV == 1 ? 8 : 4) row_norm_fwd_kernel(const RowNormArgs a) {
  using VT = Pack<T>;
  constexpr int W = VT::W, N = NV * W;
  __shared__ float red[2][3][kNormWaves];
  const int groups = blockDim.x / a.group, group = threadIdx.x / a.group, lane = threadIdx.x - group * a.group;
  const int wave = threadIdx.x >> 6, per = a.group >> 6;
  const long long step = (long long)gridDim.x * groups;
  long long row = (long long)blockIdx.x * groups + group;
  int half = 0;
  bool live[NV];
  float w[N], b[N];
  VT vx[NV], vr[NV];
#pragma unroll
  for (int e = 0; e < NV; ++e) live[e] = lane + e * a.group < a.nvec;
  auto load = [&](long long t) __attribute__((always_inline)) {
    if (t >= a.T) return;
#pragma unroll
    for (int e = 0; e < NV; ++e)
      if (live[e]) {
        const long long at = t * a.nvec + lane + e * a.group;
        vx[e] = reinterpret_cast<const VT*>(a.x)[at];
        if (a.r) vr[e] = reinterpret_cast<const VT*>(a.r)[at];
      }
  };
  load(row);
#pragma unroll
  for (int e = 0; e < NV; ++e)
    if (live[e]) {
      load_floats<T>(a.w + (lane + e * a.group) * W, w, e * W);
      if (CENTERED && a.b) load_floats<T>(a.b + (lane + e * a.group) * W, b, e * W);
    }
  // the groups of a block go through the barriers together
  for (long long t0 = (long long)blockIdx.x * groups; t0 < a.T; t0 += step, row += step) {
    const bool on = row < a.T;
    float h[N];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      if (on && live[e] && a.r) {
#pragma unroll
        for (int j = 0; j < W; j += 2) vx[e].put(j, vx[e].get(j) + vr[e].get(j), vx[e].get(j + 1) + vr[e].get(j + 1));
        reinterpret_cast<VT*>(a.h)[row * a.nvec + lane + e * a.group] = vx[e];
      }
#pragma unroll
      for (int j = 0; j < W; ++j) h[e * W + j] = on && live[e] ? vx[e].get(j) : 0.f;   // the sum as it is kept
    }
    load(row + step);
    // m + off: the mean and what its rounding lost; ss: the squares about it
    float m = 0.f, off = 0.f, ss = 0.f;
    if constexpr (CENTERED) {
      int n = a.nvec * W;
      if (a.group > 64) {
        n = 0;
#pragma unroll
        for (int e = 0; e < NV; ++e) n += live_lanes(a, wave - group * per, e) * W;
      }
      const float inv = n ? 1.f / n : 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) m += h[j];
      m = rounded(group_add(m, a.group < 64 ? a.group : 64) * inv);
#pragma unroll
      for (int e = 0; e < NV; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float d = live[e] ? h[e * W + j] - m : 0.f;
          off += d;
          ss = fmaf(d, d, ss);
        }
      off = group_add(off, a.group < 64 ? a.group : 64);
      ss = group_add(ss, a.group < 64 ? a.group : 64);
      if (a.group > 64) {
        if ((threadIdx.x & 63) == 0) {
          red[half][0][wave] = m;
          red[half][1][wave] = off;
          red[half][2][wave] = ss;
        }
        __syncthreads();
        const int w0 = group * per;
        m = 0.f;
        for (int k = 0; k < per; ++k) {
          int c = 0;
#pragma unroll
          for (int e = 0; e < NV; ++e) c += live_lanes(a, k, e) * W;
          m = fmaf((float)c, red[half][0][w0 + k], m);
        }
        m = rounded(m * a.inv_d);
        off = ss = 0.f;
        for (int k = 0; k < per; ++k) {
          int c = 0;
#pragma unroll
          for (int e = 0; e < NV; ++e) c += live_lanes(a, k, e) * W;
          // about the wave's mean: off_k, ss_k; about m: those moved by the distance
          const float d = red[half][0][w0 + k] - m, o = red[half][1][w0 + k];
          off += fmaf((float)c, d, o);
          ss += fmaf(d, fmaf((float)c, d, 2.f * o), red[half][2][w0 + k]);
        }
        half ^= 1;
      }
      off *= a.inv_d;
      const float var = fmaf(-off, off, ss * a.inv_d);
      ss = var < 0.f ? 0.f : var;
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) ss = fmaf(h[j], h[j], ss);
      ss = group_add(ss, a.group < 64 ? a.group : 64);
      if (a.group > 64) {
        if ((threadIdx.x & 63) == 0) red[half][0][wave] = ss;
        __syncthreads();
        ss = 0.f;
        for (int k = 0; k < per; ++k) ss += red[half][0][group * per + k];
        half ^= 1;
      }
      ss *= a.inv_d;
    }
    const float s = 1.f / sqrtf(ss + a.eps);
    if (on) {
      if (a.stats && lane < 3) a.stats[row * 3 + lane] = lane == 0 ? m : lane == 1 ? off : s;
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (live[e]) {
          VT o;
#pragma unroll
          for (int j = 0; j < W; j += 2) {
            float y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int n = e * W + j + i;
              const float u = (CENTERED ? (h[n] - m) - off : h[n]) * s;
              y[i] = CENTERED && a.b ? fmaf(u, w[n], b[n]) : u * w[n];
            }
            o.put(j, y[0], y[1]);
          }
          reinterpret_cast<VT*>(a.y)[row * a.nvec + lane + e * a.group] = o;
        }
    }
  }
}

template <typename T, int NV, bool CENTERED>
__global__ void __launch_bounds__(64 * kNormWaves) row_norm_bwd_kernel(const RowNormArgs a) {
  using VT = Pack<T>;
  constexpr int W = VT::W, N = NV * W;
  __shared__ float red[2][2][kNormWaves];
  // Rows of over 1024 vectors fill the registers of a block of 1024 threads: the weight is
  // then kept in LDS and the next row is not loaded ahead (2048 rows of 16384 bf16: 71 us;
  // loaded ahead 77, with the weight in registers too, 104: the compiler spills, as it still
  // does with the four vectors of fp32 rows past 8192).
  constexpr bool WLDS = NV > 1;
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [2][D] where a block has several groups; the weight
  const int groups = blockDim.x / a.group, group = threadIdx.x / a.group, lane = threadIdx.x - group * a.group;
  const int wave = threadIdx.x >> 6, per = a.group >> 6;
  const long long step = (long long)gridDim.x * groups;
  long long row = (long long)blockIdx.x * groups + group;
  int half = 0;
  bool live[NV];
  float w[WLDS ? 1 : N], dw[N], db[N];
  VT vh[NV], vg[NV], vd[NV];
  float st[3] = {0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < NV; ++e) live[e] = lane + e * a.group < a.nvec;
#pragma unroll
  for (int j = 0; j < N; ++j) dw[j] = db[j] = 0.f;
  auto load = [&](long long t) __attribute__((always_inline)) {
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < 3; ++i) st[i] = a.stats[t * 3 + i];
#pragma unroll
    for (int e = 0; e < NV; ++e)
      if (live[e]) {
        const long long at = t * a.nvec + lane + e * a.group;
        vh[e] = reinterpret_cast<const VT*>(a.x)[at];
        vg[e] = reinterpret_cast<const VT*>(a.dy)[at];
        if (a.dres) vd[e] = reinterpret_cast<const VT*>(a.dres)[at];
      }
  };
  if (!WLDS) load(row);
  if constexpr (WLDS) {
    for (int i = threadIdx.x * 4; i < a.D; i += blockDim.x * 4)
      *reinterpret_cast<Vec<float, 4>*>(sums + i) = *reinterpret_cast<const Vec<float, 4>*>(a.w + i);
    __syncthreads();
  } else if (live[0]) {
    load_floats<T>(a.w + lane * W, w, 0);
  }
  for (long long t0 = (long long)blockIdx.x * groups; t0 < a.T; t0 += step, row += step) {
    const bool on = row < a.T;
    if (WLDS) load(row);
    const float m = st[0], off = st[1], s = st[2];
    float u[N], g[N];
    VT other[NV];
    float cu = 0.f, cg = 0.f;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      other[e] = vd[e];
      float we[W];
      if constexpr (WLDS) {
        if (live[e]) load_floats<T>(sums + (lane + e * a.group) * W, we, 0);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) we[j] = w[j];
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int n = e * W + j;
        u[n] = g[n] = 0.f;
        if (on && live[e]) {
          const float h = vh[e].get(j), dy = vg[e].get(j);
          u[n] = (CENTERED ? (h - m) - off : h) * s;
          dw[n] = fmaf(dy, u[n], dw[n]);
          if (CENTERED) db[n] += dy;
          g[n] = dy * we[j];
          cu = fmaf(g[n], u[n], cu);
          if (CENTERED) cg += g[n];
        }
      }
    }
    if (!WLDS) load(row + step);
    cu = group_add(cu, a.group < 64 ? a.group : 64);
    if (CENTERED) cg = group_add(cg, a.group < 64 ? a.group : 64);
    if (a.group > 64) {
      if ((threadIdx.x & 63) == 0) {
        red[half][0][wave] = cu;
        red[half][1][wave] = cg;
      }
      __syncthreads();
      cu = cg = 0.f;
      for (int k = 0; k < per; ++k) {
        cu += red[half][0][group * per + k];
        if (CENTERED) cg += red[half][1][group * per + k];
      }
      half ^= 1;
    }
    cu *= a.inv_d;
    cg *= a.inv_d;
    if (on)
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (live[e]) {
          VT o;
#pragma unroll
          for (int j = 0; j < W; j += 2) {
            float y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int n = e * W + j + i;
              const float d = (CENTERED ? g[n] - cg : g[n]) - u[n] * cu;
              y[i] = a.dres ? fmaf(s, d, other[e].get(j + i)) : s * d;
            }
            o.put(j, y[0], y[1]);
          }
          reinterpret_cast<VT*>(a.y)[row * a.nvec + lane + e * a.group] = o;
        }
  }
  float* const out = a.part + (long long)blockIdx.x * 2 * a.D;
  if (groups == 1) {
#pragma unroll
    for (int e = 0; e < NV; ++e)
      if (live[e]) {
        const int at = (lane + e * a.group) * W;
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          *reinterpret_cast<Vec<float, 4>*>(out + at + j) = {{dw[e * W + j], dw[e * W + j + 1], dw[e * W + j + 2], dw[e * W + j + 3]}};
          if (CENTERED)
            *reinterpret_cast<Vec<float, 4>*>(out + a.D + at + j) = {{db[e * W + j], db[e * W + j + 1], db[e * W + j + 2], db[e * W + j + 3]}};
        }
      }
    return;
  }
  // the block's groups, one behind the other
  for (int k = 0; k < groups; ++k) {
    __syncthreads();
    if (group == k)
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (live[e])
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const int n = e * W + j, at = (lane + e * a.group) * W + j;
            sums[at] = dw[n] + (k ? sums[at] : 0.f);
            if (CENTERED) sums[a.D + at] = db[n] + (k ? sums[a.D + at] : 0.f);
          }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (CENTERED ? 2 : 1) * a.D; i += blockDim.x) out[i] = sums[i];
}

// dw and db from the blocks' sums, in a fixed order: 64 row groups of 64 columns
// (4 a thread), then the groups.
__global__ void __launch_bounds__(1024) row_norm_sum_kernel(const float* __restrict__ part, int nblk, int D,
                                                            float* __restrict__ dw, float* __restrict__ db) {
  __shared__ Vec<float, 4> sm[64][16];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const long long col = ((long long)blockIdx.x * 16 + c) * 4;
  Vec<float, 4> s = {{0.f, 0.f, 0.f, 0.f}};
  if (col < 2 * D && (col < D || db)) {
#pragma unroll 4
    for (int i = g; i < nblk; i += 64) {
      const Vec<float, 4> v = *reinterpret_cast<const Vec<float, 4>*>(part + (long long)i * 2 * D + col);
#pragma unroll
      for (int j = 0; j < 4; ++j) s.v[j] += v.v[j];
    }
  }
  sm[g][c] = s;
  __syncthreads();
  for (int n = 32; n; n >>= 1) {
    if (g < n)
#pragma unroll
      for (int j = 0; j < 4; ++j) sm[g][c].v[j] += sm[g + n][c].v[j];
    __syncthreads();
  }
  if (g == 0 && col < 2 * D) {
    if (col < D) *reinterpret_cast<Vec<float, 4>*>(dw + col) = sm[0][c];
    else if (db) *reinterpret_cast<Vec<float, 4>*>(db + col - D) = sm[0][c];
  }
}

struct NormShape {
  int nv, group, block;   // vectors of a lane, lanes of a row, threads of a block
  NormShape(sl_dtype dt, long long D) {
    const int nvec = (int)(D * (dt == SL_BF16 ? 2 : 4) / 16);
    nv = nvec <= 1024 ? 1 : nvec <= 2048 ? 2 : 4;
    const int lanes = (nvec + nv - 1) / nv;
    if (lanes <= 64) for (group = 8; group < lanes;) group *= 2;
    else group = (lanes + 63) / 64 * 64;
    block = group >= 512 ? group : 512 / group * group;
  }
};

// Blocks of a forward launch; past that they walk on.  A whole number to each of 256
// CUs, as they all have the same work: three of up to 512 threads, two wider ones
// (2 x 8192 rows of 5120 bf16 in blocks of 640: one to a CU 116 us, two 121, three 148; 1 x 2048
// rows of 4096 in blocks of 512: one 19.3, two 15.3, three 14.0, four 14.7; 2048 of 8192: 37, 32, 33).
inline unsigned norm_fwd_blocks(int T, const NormShape& sh) {
  return walk_grid(ceil_div(T, sh.block / sh.group), 256 * (sh.block <= 512 ? 3 : 2)).x;
}

// Blocks of a backward launch, whose sums the last launch adds: one to a CU (2048 rows
// of 4096, with the last launch: 128 blocks 25.0 us, 256 19.3, 512 21.3, 1024 28.7), and
// at least two rows to each (256 rows: 128 blocks 9.4 us, 256 11.9).  Other widths, with
// 128, 256, 512 and 1024 blocks: 16384 rows of 5120 208, 133, 142, 150 us, of 1024 48, 33.5, 34.5, 40;
// 131072 of 64 54, 49.5, 48.7, 84.  Blocks of 1024 threads in place of 512 (16 waves to a CU) lose
// where groups have to join: 2048 rows of 4096 21.5 us, of 1024 12.4 to 15.2, of 64 39 to 73.
inline int norm_bwd_blocks(int T, const NormShape& sh) {
  const int n = ceil_div(T, 2 * (sh.block / sh.group));
  return n < 256 ? n : 256;
}

static sl_status check_norm(const sl_layout* lay, int64_t D) {
  sl_status st = check_tokens(lay);
  if (st != SL_OK) return st;
  if (D < 8 || D % 8 || D > 16384) SL_FAIL(SL_ERR_SHAPE, "d_model %lld must be a multiple of 8 in [8, 16384]", (long long)D);
  return SL_OK;
}

static sl_status norm_args(RowNormArgs& a, sl_dtype dt, const sl_layout* lay, const sl_layer_norm* p) {
  sl_status st = check_dtype(dt);
  if (st != SL_OK) return st;
  if (!p) SL_FAIL(SL_ERR_NULL, "the norm is NULL");
  st = check_norm(lay, p->d_model);
  if (st != SL_OK) return st;
  if (!p->w) SL_FAIL(SL_ERR_NULL, "w required");
  if (p->b && !p->centered) SL_FAIL(SL_ERR_SHAPE, "a norm that is not centred has no bias");
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) SL_FAIL(SL_ERR_RANGE, "eps must be finite and >= 0");
  if (!aligned16(p->w) || !aligned16(p->b)) SL_FAIL(SL_ERR_ALIGN, "w and b must be 16-byte aligned");
  a = RowNormArgs{};
  a.T = lay->batch * lay->seq_len;
  a.D = (int)p->d_model;
  a.nvec = a.D * (dt == SL_BF16 ? 2 : 4) / 16;
  a.w = p->w;
  a.b = p->b;
  a.eps = p->eps;
  a.inv_d = 1.0f / a.D;
  return SL_OK;
}

template <typename T, bool CENTERED, bool BWD>
static void launch_norm(const NormShape& sh, const RowNormArgs& a, unsigned blocks, hipStream_t s) {
  const dim3 grid(blocks), block(sh.block);
  // (several groups to a block: rows of at most 256 lanes)
  const size_t lds = !BWD ? 0 : sh.nv > 1 ? (size_t)a.D * sizeof(float) : sh.block == sh.group ? 0 : (size_t)2 * a.D * sizeof(float);
  auto launch = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if constexpr (BWD) hipLaunchKernelGGL((row_norm_bwd_kernel<T, NV, CENTERED>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((row_norm_fwd_kernel<T, NV, CENTERED>), grid, block, lds, s, a);
  };
  if (sh.nv == 1) launch(std::integral_constant<int, 1>());
  else if (sizeof(T) == 2 || sh.nv == 2) launch(std::integral_constant<int, 2>());
  else if constexpr (sizeof(T) == 4) launch(std::integral_constant<int, 4>());
}

template <bool BWD>
static sl_status run_norm(sl_dtype dt, bool centered, const NormShape& sh, const RowNormArgs& a, unsigned blocks, hipStream_t s) {
  if (dt == SL_BF16) centered ? launch_norm<bf16, true, BWD>(sh, a, blocks, s) : launch_norm<bf16, false, BWD>(sh, a, blocks, s);
  else centered ? launch_norm<float, true, BWD>(sh, a, blocks, s) : launch_norm<float, false, BWD>(sh, a, blocks, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}

}  // namespace sl

using namespace sl;

extern "C" sl_status sl_layer_norm_fwd(sl_dtype dt, const sl_layout* lay, const sl_layer_norm* p, const void* x,
                                       const void* r, void* h, void* y, float* stats, void* stream) {
  if (!x || !y || (r == nullptr) != (h == nullptr)) SL_FAIL(SL_ERR_NULL, "x and y required; r and h both or neither");
  RowNormArgs a;
  sl_status st = norm_args(a, dt, lay, p);
  if (st != SL_OK) return st;
  if (!aligned16(x) || !aligned16(r) || !aligned16(h) || !aligned16(y) || !aligned16(stats))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  st = check_arch();
  if (st != SL_OK) return st;
  a.x = x; a.r = r; a.h = h; a.y = y; a.stats = stats;
  const NormShape sh(dt, a.D);
  a.group = sh.group;
  return run_norm<false>(dt, p->centered != 0, sh, a, norm_fwd_blocks(a.T, sh), reinterpret_cast<hipStream_t>(stream));
}

extern "C" size_t sl_layer_norm_workspace_bytes(const sl_layout* lay, int64_t d_model) {
  if (check_norm(lay, d_model) != SL_OK) return 0;
  // the most blocks that a call of either type has
  const int T = lay->batch * lay->seq_len;
  int most = 0;
  for (sl_dtype dt : {SL_F32, SL_BF16}) {
    const NormShape sh(dt, d_model);
    const int n = norm_bwd_blocks(T, sh);
    most = n > most ? n : most;
  }
  return (size_t)most * 2 * d_model * sizeof(float);
}

extern "C" sl_status sl_layer_norm_bwd(sl_dtype dt, const sl_layout* lay, const sl_layer_norm* p, const void* h,
                                       const float* stats, const void* dy, const void* dh, void* dx, float* dw,
                                       float* db, void* ws, size_t ws_bytes, void* stream) {
  if (!h || !stats || !dy || !dx || !dw) SL_FAIL(SL_ERR_NULL, "h, stats, dy, dx and dw required");
  RowNormArgs a;
  sl_status st = norm_args(a, dt, lay, p);
  if (st != SL_OK) return st;
  if (db && !p->centered) SL_FAIL(SL_ERR_SHAPE, "a norm that is not centred has no bias gradient");
  if (!aligned16(h) || !aligned16(stats) || !aligned16(dy) || !aligned16(dh) || !aligned16(dx) || !aligned16(dw) ||
      !aligned16(db) || !aligned16(ws))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  const NormShape sh(dt, a.D);
  const int blocks = norm_bwd_blocks(a.T, sh);
  if (!ws || ws_bytes < (size_t)blocks * 2 * a.D * sizeof(float))
    SL_FAIL(SL_ERR_WORKSPACE, "layer norm workspace too small (%zu bytes)", ws_bytes);
  st = check_arch();
  if (st != SL_OK) return st;
  a.x = h; a.stats = const_cast<float*>(stats); a.dy = dy; a.dres = dh; a.y = dx;
  a.part = reinterpret_cast<float*>(ws);
  a.group = sh.group;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  st = run_norm<true>(dt, p->centered != 0, sh, a, blocks, s);
  if (st != SL_OK) return st;
  hipLaunchKernelGGL(row_norm_sum_kernel, dim3((unsigned)ceil_div(2 * a.D, 64)), dim3(1024), 0, s, a.part, blocks, a.D, dw, db);
  SL_HIP(hipGetLastError());
  return SL_OK;
}
