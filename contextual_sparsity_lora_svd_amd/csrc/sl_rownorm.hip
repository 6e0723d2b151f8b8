// Norms of whole rows with the residual sum in the same pass:
//   h = x + r,  u = (h - m) s,  y = u w + b,
//   m = mean of the row (0 where it is not centred),  s = (mean (h - m)^2 + eps)^(-1/2).
// Backward, with g = dy w and the gradient dres that reaches h by its other way:
//   dx = s (g - mean g - u mean(g u)) + dres,  dw = sum over rows of dy u,  db = sum over rows of dy.
//
// A row belongs to a group of lanes, 8 to 64 of one wave or several whole waves,
// and stays in registers from its loads to its stores; its sums are added over
// the lanes, and over the waves through LDS.  The variance is formed from
// h - m, not from mean h^2 - m^2, and the mean's own rounding error is taken out
// of both with the same sums.  A group walks over rows and loads the next row
// before it works on this one.  The backward keeps the sums of dw and db of its
// rows in registers; a block adds its groups' sums in LDS, and one more launch the
// blocks' in a fixed order.
#include <cmath>

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
  int group, group_log2;     // lanes of a row; log2 below a wave
  float eps, inv_d;
};

constexpr int kNormThreads = 1024;   // most threads of a block

// Sums over a row's lanes.  Groups of whole waves go through LDS: calls take the
// two halves of `red` in turn, so one barrier a call is enough (a half is written
// again only behind the next call's barrier).
template <int N>
__device__ inline void row_add(float (&v)[N], const RowNormArgs& a, float (*red)[2][kNormThreads / 64], int& half) {
  if (a.group < 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] += dpp<kXor1>(v[i]);
      v[i] += dpp<kXor2>(v[i]);
      v[i] += dpp<kMirror8>(v[i]);
      if (a.group >= 16) v[i] += dpp<kMirror16>(v[i]);
      if (a.group >= 32) v[i] += __shfl_xor(v[i], 16);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_add(v[i]);
  if (a.group == 64) return;
  const int wave = threadIdx.x >> 6, per = a.group >> 6, first = wave - wave % per;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[half][i][wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = red[half][i][first];
  for (int k = 1; k < per; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[half][i][first + k];
  half ^= 1;
}

template <typename T, int NV, bool CENTERED>
__global__ void __launch_bounds__(kNormThreads) row_norm_fwd_kernel(const RowNormArgs a) {
  constexpr int W = 16 / sizeof(T), N = NV * W;
  using VT = Vec<T, W>;
  __shared__ float red[2][2][kNormThreads / 64];
  const int groups = blockDim.x / a.group, group = threadIdx.x / a.group, lane = threadIdx.x % a.group;
  const long long step = (long long)gridDim.x * groups;
  long long row = (long long)blockIdx.x * groups + group;
  int half = 0;
  bool live[NV];
  float w[N], b[N];
  VT vx[NV], vr[NV];
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int c = lane + e * a.group;
    live[e] = c < a.nvec;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      w[e * W + j] = live[e] ? a.w[c * W + j] : 0.f;
      b[e * W + j] = live[e] && a.b ? a.b[c * W + j] : 0.f;
    }
  }
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
  // the groups of a block go through the barriers together
  for (long long t0 = (long long)blockIdx.x * groups; t0 < a.T; t0 += step, row += step) {
    const bool on = row < a.T;
    float h[N];
    VT vh[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float v = 0.f;
        if (on && live[e]) {
          v = el2f<T>(vx[e].v[j]);
          if (a.r) v += el2f<T>(vr[e].v[j]);
          vh[e].v[j] = f2el<T>(v);
          v = el2f<T>(vh[e].v[j]);        // the norm is of the sum as it is kept
        }
        h[e * W + j] = v;
      }
    if (on && a.h)
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (live[e]) reinterpret_cast<VT*>(a.h)[row * a.nvec + lane + e * a.group] = vh[e];
    load(row + step);
    float m = 0.f, off = 0.f, ss;
    if constexpr (CENTERED) {
      float s1[1] = {0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) s1[0] += h[j];
      row_add(s1, a, red, half);
      m = s1[0] * a.inv_d;
      float s2[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < NV; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float d = live[e] ? h[e * W + j] - m : 0.f;
          h[e * W + j] = d;
          s2[0] += d;
          s2[1] = fmaf(d, d, s2[1]);
        }
      row_add(s2, a, red, half);
      off = s2[0] * a.inv_d;
      ss = fmaxf(fmaf(-off, off, s2[1] * a.inv_d), 0.f);
      if (!(s2[1] == s2[1])) ss = s2[1];   // (a row with a NaN stays one)
    } else {
      float s2[1] = {0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) s2[0] = fmaf(h[j], h[j], s2[0]);
      row_add(s2, a, red, half);
      ss = s2[0] * a.inv_d;
    }
    const float s = 1.f / sqrtf(ss + a.eps);
    if (on) {
      if (a.stats && lane == 0) {
        a.stats[row * 3] = m;
        a.stats[row * 3 + 1] = off;
        a.stats[row * 3 + 2] = s;
      }
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (live[e]) {
          VT o;
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const float u = (CENTERED ? h[e * W + j] - off : h[e * W + j]) * s;
            o.v[j] = f2el<T>(fmaf(u, w[e * W + j], b[e * W + j]));
          }
          reinterpret_cast<VT*>(a.y)[row * a.nvec + lane + e * a.group] = o;
        }
    }
  }
}

template <typename T, int NV, bool CENTERED>
__global__ void __launch_bounds__(kNormThreads) row_norm_bwd_kernel(const RowNormArgs a) {
  constexpr int W = 16 / sizeof(T), N = NV * W;
  using VT = Vec<T, W>;
  __shared__ float red[2][2][kNormThreads / 64];
  extern __shared__ float sums[];              // [2][D]
  const int groups = blockDim.x / a.group, group = threadIdx.x / a.group, lane = threadIdx.x % a.group;
  const long long step = (long long)gridDim.x * groups;
  long long row = (long long)blockIdx.x * groups + group;
  int half = 0;
  bool live[NV];
  float w[N], dw[N], db[N];
  VT vh[NV], vg[NV], vd[NV];
  float st[3] = {0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int c = lane + e * a.group;
    live[e] = c < a.nvec;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      w[e * W + j] = live[e] ? a.w[c * W + j] : 0.f;
      dw[e * W + j] = db[e * W + j] = 0.f;
    }
  }
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
  load(row);
  for (long long t0 = (long long)blockIdx.x * groups; t0 < a.T; t0 += step, row += step) {
    const bool on = row < a.T;
    const float m = st[0], off = st[1], s = st[2];
    float u[N], g[N], other[N];
    float c[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int n = e * W + j;
        u[n] = g[n] = other[n] = 0.f;
        if (on && live[e]) {
          const float h = el2f<T>(vh[e].v[j]), dy = el2f<T>(vg[e].v[j]);
          u[n] = CENTERED ? ((h - m) - off) * s : h * s;
          if (a.dres) other[n] = el2f<T>(vd[e].v[j]);
          dw[n] = fmaf(dy, u[n], dw[n]);
          if (CENTERED) db[n] += dy;
          g[n] = dy * w[n];
          c[0] = fmaf(g[n], u[n], c[0]);
          if (CENTERED) c[1] += g[n];
        }
      }
    load(row + step);
    row_add(c, a, red, half);
    const float cu = c[0] * a.inv_d, cg = CENTERED ? c[1] * a.inv_d : 0.f;
    if (on)
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (live[e]) {
          VT o;
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const int n = e * W + j;
            o.v[j] = f2el<T>(fmaf(s, (g[n] - cg) - u[n] * cu, other[n]));
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
        *reinterpret_cast<Vec<float, W>*>(out + at) = *reinterpret_cast<const Vec<float, W>*>(dw + e * W);
        *reinterpret_cast<Vec<float, W>*>(out + a.D + at) = *reinterpret_cast<const Vec<float, W>*>(db + e * W);
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
            sums[a.D + at] = db[n] + (k ? sums[a.D + at] : 0.f);
          }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) out[i] = sums[i];
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
  NormShape(sl_dtype dt, long long D, bool bwd) {
    const int nvec = (int)(D * (dt == SL_BF16 ? 2 : 4) / 16);
    nv = nvec <= 64 ? 1 : nvec <= 2048 ? 2 : 4;
    const int lanes = (nvec + nv - 1) / nv;
    if (lanes <= 64) for (group = 8; group < lanes;) group *= 2;
    else group = (lanes + 63) / 64 * 64;
    const int want = bwd ? 512 : 256;
    block = group >= want ? group : want / group * group;
  }
};

// Blocks of a backward launch, whose sums the last launch adds.
inline int norm_bwd_blocks(int T, int rows) {
  const int n = ceil_div(T, rows);
  return n < 512 ? n : 512;
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

template <typename T, bool CENTERED>
static void launch_fwd(int nv, const RowNormArgs& a, dim3 grid, dim3 block, hipStream_t s) {
  if (nv == 1) hipLaunchKernelGGL((row_norm_fwd_kernel<T, 1, CENTERED>), grid, block, 0, s, a);
  else if (nv == 2) hipLaunchKernelGGL((row_norm_fwd_kernel<T, 2, CENTERED>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((row_norm_fwd_kernel<T, 4, CENTERED>), grid, block, 0, s, a);
}

template <typename T, bool CENTERED>
static void launch_bwd(int nv, const RowNormArgs& a, dim3 grid, dim3 block, hipStream_t s) {
  // (several groups to a block: rows of at most 256 lanes, two vectors each)
  const size_t lds = (int)block.x == a.group ? 0 : (size_t)2 * a.D * sizeof(float);
  if (nv == 1) hipLaunchKernelGGL((row_norm_bwd_kernel<T, 1, CENTERED>), grid, block, lds, s, a);
  else if (nv == 2) hipLaunchKernelGGL((row_norm_bwd_kernel<T, 2, CENTERED>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((row_norm_bwd_kernel<T, 4, CENTERED>), grid, block, lds, s, a);
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
  const NormShape sh(dt, a.D, false);
  a.group = sh.group;
  const int rows = sh.block / sh.group;
  const dim3 grid = walk_grid(ceil_div(a.T, rows), 2048 * 256 / sh.block), block(sh.block);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dt == SL_BF16) p->centered ? launch_fwd<bf16, true>(sh.nv, a, grid, block, s) : launch_fwd<bf16, false>(sh.nv, a, grid, block, s);
  else p->centered ? launch_fwd<float, true>(sh.nv, a, grid, block, s) : launch_fwd<float, false>(sh.nv, a, grid, block, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}

extern "C" size_t sl_layer_norm_workspace_bytes(const sl_layout* lay, int64_t d_model) {
  if (check_norm(lay, d_model) != SL_OK) return 0;
  // the most blocks that a call of either type has
  const int T = lay->batch * lay->seq_len;
  int most = 0;
  for (sl_dtype dt : {SL_F32, SL_BF16}) {
    const NormShape sh(dt, d_model, true);
    const int n = norm_bwd_blocks(T, sh.block / sh.group);
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
  const NormShape sh(dt, a.D, true);
  const int blocks = norm_bwd_blocks(a.T, sh.block / sh.group);
  if (!ws || ws_bytes < (size_t)blocks * 2 * a.D * sizeof(float))
    SL_FAIL(SL_ERR_WORKSPACE, "layer norm workspace too small (%zu bytes)", ws_bytes);
  st = check_arch();
  if (st != SL_OK) return st;
  a.x = h; a.stats = const_cast<float*>(stats); a.dy = dy; a.dres = dh; a.y = dx;
  a.part = reinterpret_cast<float*>(ws);
  a.group = sh.group;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid(blocks), block(sh.block);
  if (dt == SL_BF16) p->centered ? launch_bwd<bf16, true>(sh.nv, a, grid, block, s) : launch_bwd<bf16, false>(sh.nv, a, grid, block, s);
  else p->centered ? launch_bwd<float, true>(sh.nv, a, grid, block, s) : launch_bwd<float, false>(sh.nv, a, grid, block, s);
  hipLaunchKernelGGL(row_norm_sum_kernel, dim3((unsigned)ceil_div(2 * a.D, 64)), dim3(1024), 0, s, a.part, blocks, a.D, dw, db);
  SL_HIP(hipGetLastError());
  return SL_OK;
}
