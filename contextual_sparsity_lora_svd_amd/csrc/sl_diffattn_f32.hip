// Differential attention in fp32: forward and backward kernels.
#include "sl_diffattn.hpp"

namespace sl {

// Block -> (row block, head pair or part, sequence); where lengths differ each row
// block starts one further, since workgroups go round the XCDs.
__device__ inline void place(int bid, const DiffArgs& a, int units, int& blk, int& unit, int& b) {
  const int n = units * a.B;
  blk = bid / n;
  const int u = (bid % n + (a.mix ? blk : 0)) % n;
  unit = u / a.B;
  b = u % a.B;
}

// ---------------------------------------------------------------------------
// The fp32 matrix instructions run at a sixteenth of the bf16 rate, so L1 and L2
// feed the walked tiles directly, each operand read two groups of 8 instructions
// before its use and its loads between them.  Only the workgroup's own 32 rows lie
// in LDS: read by rows they would take a cache line per lane each time (1 x 2048
// causal tokens, 8 heads of 128: dQ 310 -> 238 us, dK/dV 415 -> 346).  The waves
// take every fourth tile and add their sums in order in the end, so that short
// sequences and few heads still fill the GPU.
//
// Forward: four waves per map, each with a running maximum and sum.  The transposed
// score tile (keys x queries) leaves a query in a lane pair: the softmax needs one
// exchange per tile and its weights feed the second product from registers.  A
// wave per map, not both in one, leaves registers for a second wave on the SIMD (1
// x 1024 tokens, 16 heads, 8 kv, of 128: 158 -> 142 us).
//
// Bound by the fp32 matrix instructions and, about as much, by what L1 delivers: that
// call runs at 90 (forward), 92 (dQ) and 92 TFLOP/s (dK/dV) where a large fp32
// product reaches 153.
template <int D>
__global__ void __launch_bounds__(512, 2) diff_fwd_direct(const DiffArgs a) {
  using T = float;
  constexpr int KS = D / 16, NT = D / 16;   // NT: 32-value tiles of the 2 D wide output
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ __attribute__((aligned(16))) float sm[2][NT * 1024];
  __shared__ float smx[2][4][64], ssum[2][4][64];
  __shared__ float4 own[2 * (D / 16) * 128];
  const int m = wave >> 2, kq = wave & 3;               // map, key tiles
  const int nqb = (a.L + 31) / 32;
  int blk, pair, b;
  place(blockIdx.x, a, a.hp, blk, pair, b);
  const int qb = nqb - 1 - blk;                         // the longest rows first
  const int g = pair / (a.hp / a.gp), len = a.lens[b];
  float e1, e2;
  const float lam = lambda_of(a, e1, e2);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.lam[0] = lam;
    a.lam[1] = e1;
    a.lam[2] = e2;
  }
  const int row = qb * 32 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const T* qp = reinterpret_cast<const T*>(a.q) + (tok0 + qb * 32) * ldq + pair * 2 * a.hd;
  const T* kp = reinterpret_cast<const T*>(a.k) + tok0 * ldk + g * 2 * a.hd;
  const T* vp = reinterpret_cast<const T*>(a.v) + tok0 * ldk + g * 2 * a.hd;
  const bool rok = row < len;
  f32x16 o[NT];
  // ms: the running maximum times sc as it was rounded, which the weights are relative
  // to.  Only differences of such values rescale: mx * sc formed again (and fused with a
  // subtraction) is off by its rounding, at every tile
  float mx = -INFINITY, ms = -INFINITY, sum = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) zero16(o[t]);
  const float sc = a.scale * kLog2e;
  int kend = len;
  if (a.causal && kend > qb * 32 + 32) kend = qb * 32 + 32;
  if (qb * 32 >= len) kend = 0;
  if (kend > 0) put_own(own + m * KS * 128, KS, qp + (rok ? c : 0) * ldq + m * a.hd, a.hd, kq, lane);   // (past the end: any)
  __syncthreads();
  // products over the columns, then over the keys; an operand is read AHEAD groups
  // of 8 matrix instructions before its use
  constexpr int NG = KS + 2 * NT, AHEAD = 2;
  for (int k0 = 32 * kq; k0 < kend; k0 += 128) {
    const T* const kt = kp + (long long)k0 * ldk + m * a.hd;
    const T* const vt = vp + (long long)k0 * ldk;
    Rows32 r;
    r.init(c, h, len - 1 - k0, (unsigned)ldk);
    const float4* const mine = own + m * KS * 128 + opaque(lane);
    const int cz = c + opaque(0), hz = h + opaque(0);    // offsets of columns are made where they are used
    f32x16 s;
    Frag<T> fa[AHEAD + 1], fb[AHEAD + 1];
    zero16(s);
    auto fetch = [&](auto gc, int j) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, x = g % (AHEAD + 1);
      if constexpr (g < KS) {
        read_row(fa[x], j, kt, r.row + first_if_past(g * 16 + hz * 8, a.hd));
        read_own(fb[x], j - 2, mine, g);
      } else if constexpr (g < NG) {
        read_col(fa[x], j, vt, r, (g - KS) / NT, last_if_past((g - KS) % NT * 32 + cz, 2 * a.hd));
      }
    };
    each<8 * AHEAD>([&](auto i) __attribute__((always_inline)) { fetch(std::integral_constant<int, decltype(i)::value / 8>{}, decltype(i)::value % 8); });
    each<NG>([&](auto gc) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, x = g % (AHEAD + 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fetch(std::integral_constant<int, g + AHEAD>{}, j);
        if constexpr (g < KS) mma1(s, fa[x], fb[x].v[j], j);
        else mma1(o[(g - KS) % NT], fa[x], s[8 * ((g - KS) / NT) + j], j);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (g == KS - 1) {
        float tm = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = k0 + 8 * (i >> 2) + 4 * h + (i & 3);
          if (key >= len || (a.causal && key > row)) s[i] = -INFINITY;
          tm = fmaxf(tm, s[i]);
        }
        tm = fmaxf(tm, __shfl_xor(tm, 32));
        mx = fmaxf(mx, tm);
        const float ns = mx * sc, rel = ns == -INFINITY ? 0.f : ns;   // nothing seen yet: weights 0
        const float f = ns == ms ? 1.f : fast_exp2(ms - rel);
        float ts = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = fast_exp2(fmaf(s[i], sc, -rel));
          ts += s[i];
        }
        sum = sum * f + ts;
        ms = ns;
        if (__any(f != 1.f)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] *= f;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  smx[m][kq][lane] = ms;
  ssum[m][kq][lane] = sum;
  __syncthreads();
  float top = smx[m][0][lane], l = 0.f;
#pragma unroll
  for (int w = 1; w < 4; ++w) top = fmaxf(top, smx[m][w][lane]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float x = smx[m][w][lane];
    if (x > -INFINITY) l = fmaf(fast_exp2(x - top), ssum[m][w][lane], l);   // else it saw no key
  }
  const float f = ms > -INFINITY ? fast_exp2(ms - top) : 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[t][i] *= f;
  l += __shfl_xor(l, 32);
  const float inv = rok ? 1.f / l : 0.f;
  if (kq == 0 && h == 0 && row < a.L) {
    float* const at = a.lse + ((long long)(b * a.hp + pair) * 2 + m) * a.ls + row;
    *at = rok ? top + log2f(l) : INFINITY;
    if (row == a.L - 1) at[1] = INFINITY;
  }
  add_waves(o, sm[m], kq, lane);
  // the last waves hold the maps' sums; the second map's hands over O_2
  const long long orow = (tok0 + row) * ldq + pair * 2 * a.hd;
  const bool put = kq == 3 && row < a.L;
  float4* const y4 = reinterpret_cast<float4*>(sm[1]) + lane;
  if (m == 1 && kq == 3) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int dv = 32 * t + 2 * i + 4 * h;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = rok ? o[t][i + e] * inv : 0.f;
        y4[(t * 4 + i / 4) * 64] = make_float4(y[0], y[1], y[2], y[3]);
        if (put && dv < 2 * a.hd) store4<T>(reinterpret_cast<T*>(a.o2) + orow + dv, y[0], y[1], y[2], y[3]);
      }
  }
  __syncthreads();
  if (m == 0 && put) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int dv = 32 * t + 2 * i + 4 * h;
        if (dv >= 2 * a.hd) continue;
        const float4 y = y4[(t * 4 + i / 4) * 64];
        store4<T>(reinterpret_cast<T*>(a.o) + orow + dv, rok ? o[t][i] * inv - lam * y.x : 0.f, rok ? o[t][i + 1] * inv - lam * y.y : 0.f,
                  rok ? o[t][i + 2] * inv - lam * y.z : 0.f, rok ? o[t][i + 3] * inv - lam * y.w : 0.f);
      }
  }
}

// ---------------------------------------------------------------------------
// dQ: 32 queries per workgroup, every fourth key tile per wave.  D_1 = dO . (O +
// lambda O_2) and D_2 = dO . O_2 of the rows come first (a launch of their own took
// 4 us at 2 x 64 tokens); dK and dV read them from memory.  The sum of P_2 dP
// is -dlambda.
template <int D>
__global__ void __launch_bounds__(256, 1) diff_dq_direct(const DiffArgs a) {
  using T = float;
  constexpr int DT = D / 32;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ __attribute__((aligned(16))) float sm[DT * 1024];
  __shared__ float4 own[(D / 4) * 128];
  __shared__ float sds[2][4][32];
  const int nqb = (a.L + 31) / 32;
  int blk, pair, b;
  place(blockIdx.x, a, a.hp, blk, pair, b);
  const int qb = nqb - 1 - blk;
  const int g = pair / (a.hp / a.gp), len = a.lens[b];
  const float lam = a.lam[0];
  const int row = qb * 32 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long qoff = (tok0 + row) * ldq + pair * 2 * a.hd, koff = tok0 * ldk + g * 2 * a.hd;
  const long long toff = (tok0 + qb * 32) * ldq + pair * 2 * a.hd;
  const T* qp = reinterpret_cast<const T*>(a.q) + toff;
  const T* dop = reinterpret_cast<const T*>(a.da) + toff;
  const T* kp = reinterpret_cast<const T*>(a.k) + koff;
  const T* vp = reinterpret_cast<const T*>(a.v) + koff;
  const bool rok = row < len;
  float lse[2], ds[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const long long at = ((long long)(b * a.hp + pair) * 2 + m) * a.ls + row;
    lse[m] = rok ? a.lse[at] : INFINITY;
    ds[m] = 0.f;
  }
  if (rok) {                       // every eighth chunk of 4 columns
    const T* op = reinterpret_cast<const T*>(a.a) + qoff;
    const T* o2p = reinterpret_cast<const T*>(a.o2) + qoff;
    const T* gp = reinterpret_cast<const T*>(a.da) + qoff;
    for (int i = 4 * (2 * wave + h); i < 2 * a.hd; i += 32) {
      const float4 g4 = *reinterpret_cast<const float4*>(gp + i), o4 = *reinterpret_cast<const float4*>(op + i);
      const float4 y4 = *reinterpret_cast<const float4*>(o2p + i);
      ds[0] = fmaf(g4.x, fmaf(lam, y4.x, o4.x), ds[0]);
      ds[0] = fmaf(g4.y, fmaf(lam, y4.y, o4.y), ds[0]);
      ds[0] = fmaf(g4.z, fmaf(lam, y4.z, o4.z), ds[0]);
      ds[0] = fmaf(g4.w, fmaf(lam, y4.w, o4.w), ds[0]);
      ds[1] = fmaf(g4.x, y4.x, fmaf(g4.y, y4.y, fmaf(g4.z, y4.z, fmaf(g4.w, y4.w, ds[1]))));
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    ds[m] += __shfl_xor(ds[m], 32);
    if (h == 0) sds[m][wave][c] = ds[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    ds[m] = ((sds[m][0][c] + sds[m][1][c]) + sds[m][2][c]) + sds[m][3][c];
    if (wave == 0 && h == 0 && row < a.L) {
      float* const at = a.dsum + ((long long)(b * a.hp + pair) * 2 + m) * a.ls + row;
      *at = ds[m];
      if (row == a.L - 1) at[1] = 0.f;
    }
  }
  f32x16 dq[2][DT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dq[m][t]);
  const float sc = a.scale * kLog2e;
  double dlam = 0.0;
  int kend = len;
  if (a.causal && kend > qb * 32 + 32) kend = qb * 32 + 32;
  if (qb * 32 >= len) kend = 0;
  if (kend > 0) {                                      // (a row past the end: any)
    const long long at = (rok ? c : 0) * ldq;
    put_own(own, D / 8, dop + at, 2 * a.hd, wave, lane);
    for (int m = 0; m < 2; ++m) put_own(own + (2 + m) * (D / 16) * 128, D / 16, qp + at + m * a.hd, a.hd, wave, lane);
  }
  __syncthreads();
  // products in order dP, S_1, S_2, then over the keys; operands read as in the forward
  constexpr int N0 = D / 8, KS = D / 16, N1 = 2 * KS, NG = N0 + N1 + 4 * DT, AHEAD = 2;
  for (int k0 = 32 * wave; k0 < kend; k0 += 128) {
    const T* const kt = kp + (long long)k0 * ldk;
    const T* const vt = vp + (long long)k0 * ldk;
    Rows32 r;
    r.init(c, h, len - 1 - k0, (unsigned)ldk);
    const float4* const mine = own + opaque(lane);
    const int cz = c + opaque(0), hz = h + opaque(0);
    f32x16 dp, s[2];
    float part = 0.f;
    Frag<T> fa[AHEAD + 1], fb[AHEAD + 1];
    zero16(dp);
    zero16(s[0]);
    zero16(s[1]);
    auto fetch = [&](auto gc, int j) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, x = g % (AHEAD + 1);
      if constexpr (g < N0) {
        const unsigned col = first_if_past(g * 16 + hz * 8, 2 * a.hd);
        read_row(fa[x], j, vt, r.row + col);
        read_own(fb[x], j - 2, mine, g);
      } else if constexpr (g < N0 + N1) {
        const int m = (g - N0) / KS;
        const unsigned col = first_if_past((g - N0) % KS * 16 + hz * 8, a.hd);
        read_row(fa[x], j, kt + m * a.hd, r.row + col);
        read_own(fb[x], j - 2, mine, g);
      } else if constexpr (g < NG) {
        constexpr int y = g - N0 - N1;
        read_col(fa[x], j, kt + y / (2 * DT) * a.hd, r, y / DT % 2, last_if_past(y % DT * 32 + cz, a.hd));
      }
    };
    each<8 * AHEAD>([&](auto i) __attribute__((always_inline)) { fetch(std::integral_constant<int, decltype(i)::value / 8>{}, decltype(i)::value % 8); });
    each<NG>([&](auto gc) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, x = g % (AHEAD + 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fetch(std::integral_constant<int, g + AHEAD>{}, j);
        if constexpr (g < N0) {
          mma1(dp, fa[x], fb[x].v[j], j);
        } else if constexpr (g < N0 + N1) {
          mma1(s[(g - N0) / KS], fa[x], fb[x].v[j], j);
        } else {
          constexpr int y = g - N0 - N1, m = y / (2 * DT);
          mma1(dq[m][y % DT], fa[x], s[m][8 * (y / DT % 2) + j], j);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (g >= N0 && g < N0 + N1 && (g - N0) % KS == KS - 1) {
        constexpr int m = (g - N0) / KS;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = k0 + 8 * (i >> 2) + 4 * h + (i & 3);
          const bool hidden = key >= len || (a.causal && key > row) || !rok;
          const float p = hidden ? 0.f : fast_exp2(fmaf(s[m][i], sc, -lse[m]));
          if (m == 1) part = fmaf(p, dp[i], part);
          s[m][i] = p * (dp[i] - ds[m]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    dlam += (double)part;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) dlam += __shfl_xor(dlam, o);
  if (lane == 0) a.dlam_part[blockIdx.x * 4 + wave] = dlam;
  add_waves(dq[0], sm, wave, lane);
  add_waves(dq[1], sm, wave, lane);
  if (wave != 3 || row >= a.L) return;
  T* out = reinterpret_cast<T*>(a.dq) + qoff;
  const bool some = !one_key(a, row, len);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float f = m ? -lam * a.scale : a.scale;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d >= a.hd) continue;
        store4<T>(out + m * a.hd + d, some ? dq[m][t][i] * f : 0.f, some ? dq[m][t][i + 1] * f : 0.f,
                  some ? dq[m][t][i + 2] * f : 0.f, some ? dq[m][t][i + 3] * f : 0.f);
      }
  }
}

// dK and dV: 32 keys per workgroup, every fourth of the group's query tiles per wave.
template <int D>
__global__ void __launch_bounds__(256, 1) diff_dkv_direct(const DiffArgs a) {
  using T = float;
  constexpr int DT = D / 32, NT = D / 16;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ __attribute__((aligned(16))) float sm[NT * 1024];
  __shared__ float4 own[(D / 4) * 128];
  if (blockIdx.x == gridDim.x - 1) {
    dlambda_block(a, reinterpret_cast<double*>(sm));
    return;
  }
  int kb, gs, b;
  place(blockIdx.x, a, a.gp * a.split, kb, gs, b);    // causal: the first keys have the most queries
  const int g = gs / a.split, hpart = gs % a.split;
  const int grp = a.hp / a.gp, len = a.lens[b];
  const float lam = a.lam[0];
  const int key = kb * 32 + c;
  const bool kok = key < len;                                  // else: its results are 0
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long koff = (tok0 + key) * ldk + g * 2 * a.hd;
  const long long toff = (tok0 + kb * 32) * ldk + g * 2 * a.hd;
  const T* kp = reinterpret_cast<const T*>(a.k) + toff;
  const T* vp = reinterpret_cast<const T*>(a.v) + toff;
  f32x16 dk[2][DT], dv[NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dk[m][t]);
#pragma unroll
  for (int t = 0; t < NT; ++t) zero16(dv[t]);
  const float sc = a.scale * kLog2e;
  const int t0 = a.causal ? kb : 0, ntile = kb * 32 < len ? (len + 31) / 32 - t0 : 0;
  const int nh = grp / a.split, pr0 = g * grp + hpart * nh;
  if (ntile > 0) {                                             // (a key past the end: any)
    const long long at = (kok ? c : 0) * ldk;
    put_own(own, D / 8, vp + at, 2 * a.hd, wave, lane);
    for (int m = 0; m < 2; ++m) put_own(own + (2 + m) * (D / 16) * 128, D / 16, kp + at + m * a.hd, a.hd, wave, lane);
  }
  __syncthreads();
  // products in order dP, S_1, S_2, dV, dK; operands read as in the forward
  constexpr int N0 = D / 8, KS = D / 16, N1 = 2 * KS, N2 = 2 * NT, NG = N0 + N1 + N2 + 4 * DT, AHEAD = 2;
  for (int x = wave; x < ntile * nh; x += 4) {
    const int pr = pr0 + x / ntile, q0 = (t0 + x % ntile) * 32;
    const T* const qt = reinterpret_cast<const T*>(a.q) + (tok0 + q0) * ldq + pr * 2 * a.hd;
    const T* const gt = reinterpret_cast<const T*>(a.da) + (tok0 + q0) * ldq + pr * 2 * a.hd;
    Rows32 r;
    r.init(c, h, len - 1 - q0, (unsigned)ldq);
    const float4* const mine = own + opaque(lane);
    const float* const lse = a.lse + (long long)(b * a.hp + pr) * 2 * a.ls;
    const float* const dsm = a.dsum + (long long)(b * a.hp + pr) * 2 * a.ls;
    const int cz = c + opaque(0), hz = h + opaque(0);
    f32x16 dp, s[2], w;
    float sl[16], sd[16];
    Frag<T> fa[AHEAD + 1], fb[AHEAD + 1];
    zero16(dp);
    zero16(s[0]);
    zero16(s[1]);
    auto fetch = [&](auto gc, int j) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, y = g % (AHEAD + 1);
      if constexpr (g < N0) {
        const unsigned col = first_if_past(g * 16 + hz * 8, 2 * a.hd);
        read_row(fa[y], j, gt, r.row + col);
        read_own(fb[y], j - 2, mine, g);
      } else if constexpr (g < N0 + N1) {
        const int m = (g - N0) / KS;
        const unsigned col = first_if_past((g - N0) % KS * 16 + hz * 8, a.hd);
        read_row(fa[y], j, qt + m * a.hd, r.row + col);
        read_own(fb[y], j - 2, mine, g);
      } else if constexpr (g < N0 + N1 + N2) {
        constexpr int z = g - N0 - N1;
        read_col(fa[y], j, gt, r, z / NT, last_if_past(z % NT * 32 + cz, 2 * a.hd));
      } else if constexpr (g < NG) {
        constexpr int z = g - N0 - N1 - N2;
        read_col(fa[y], j, qt + z / (2 * DT) * a.hd, r, z / DT % 2, last_if_past(z % DT * 32 + cz, a.hd));
      }
    };
    each<8 * AHEAD>([&](auto i) __attribute__((always_inline)) { fetch(std::integral_constant<int, decltype(i)::value / 8>{}, decltype(i)::value % 8); });
    each<NG>([&](auto gc) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, y = g % (AHEAD + 1);
      if constexpr (g >= N0 && g < N0 + N1 && (g - N0) % KS == 0) {
        constexpr int m = (g - N0) / KS;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int q = q0 + 8 * (i >> 2) + 4 * h + (i & 3), at = m * a.ls + (q < len ? q : len);   // past the end: weights 0
          sl[i] = lse[at];
          sd[i] = dsm[at];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        fetch(std::integral_constant<int, g + AHEAD>{}, j);
        if constexpr (g < N0) {
          mma1(dp, fa[y], fb[y].v[j], j);
        } else if constexpr (g < N0 + N1) {
          mma1(s[(g - N0) / KS], fa[y], fb[y].v[j], j);
        } else if constexpr (g < N0 + N1 + N2) {
          constexpr int z = g - N0 - N1;
          mma1(dv[z % NT], fa[y], w[8 * (z / NT) + j], j);
        } else {
          constexpr int z = g - N0 - N1 - N2, m = z / (2 * DT);
          mma1(dk[m][z % DT], fa[y], s[m][8 * (z / DT % 2) + j], j);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (g >= N0 && g < N0 + N1 && (g - N0) % KS == KS - 1) {
        constexpr int m = (g - N0) / KS;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int q = q0 + 8 * (i >> 2) + 4 * h + (i & 3);
          const float p = a.causal && key > q ? 0.f : fast_exp2(fmaf(s[m][i], sc, -sl[i]));
          w[i] = m ? w[i] - lam * p : p;
          s[m][i] = one_key(a, q, len) ? 0.f : p * (dp[i] - sd[i]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  add_waves(dv, sm, wave, lane);
  add_waves(dk[0], sm, wave, lane);
  add_waves(dk[1], sm, wave, lane);
  if (wave != 3 || key >= a.L) return;
  const long long poff = (long long)hpart * a.B * a.L * ldk + koff;
  T* dkp = (a.split > 1 ? a.dk_part + poff : reinterpret_cast<T*>(a.dk) + koff);
  T* dvp = (a.split > 1 ? a.dv_part + poff : reinterpret_cast<T*>(a.dv) + koff);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = 32 * t + 2 * i + 4 * h;
      if (d < 2 * a.hd) store4<T>(dvp + d, kok ? dv[t][i] : 0.f, kok ? dv[t][i + 1] : 0.f, kok ? dv[t][i + 2] : 0.f, kok ? dv[t][i + 3] : 0.f);
    }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float f = kok ? (m ? -lam * a.scale : a.scale) : 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d < a.hd)
          store4<T>(dkp + m * a.hd + d, dk[m][t][i] * f, dk[m][t][i + 1] * f, dk[m][t][i + 2] * f, dk[m][t][i + 3] * f);
      }
  }
}

void launch_diff_fwd_f32(const DiffArgs& a, hipStream_t s) {
  by_width(a.hd, [&](auto d) {
    hipLaunchKernelGGL(diff_fwd_direct<decltype(d)::value>, dim3((unsigned)((a.L + 31) / 32 * a.B * a.hp)), dim3(512), 0, s, a);
  });
}

void launch_diff_bwd_f32(const DiffArgs& a, hipStream_t s) {
  const int blocks = (a.L + 31) / 32 * a.B;
  by_width(a.hd, [&](auto d) {
    constexpr int D = decltype(d)::value;
    hipLaunchKernelGGL(diff_dq_direct<D>, dim3((unsigned)(blocks * a.hp)), dim3(256), 0, s, a);
    hipLaunchKernelGGL(diff_dkv_direct<D>, dim3((unsigned)(blocks * a.gp * a.split + 1)), dim3(256), 0, s, a);
  });
  if (a.split > 1) {
    const long long n = 2 * ((long long)a.B * a.L * a.gp * 2 * a.hd / 4);
    hipLaunchKernelGGL(diff_dkv_sum<float>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  }
}

}  // namespace sl
