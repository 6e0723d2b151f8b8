// Differential attention in fp32, operands straight from memory: the fp32
// matrix instructions run at a sixteenth of the bf16 rate, so L1 and L2 feed
// them (2 bytes per cycle and wave at full rate) and LDS would only add waits.
#pragma once

#include "sl_diffattn.hpp"

namespace sl {

// ---------------------------------------------------------------------------
// Operands straight from memory.  One wave per 32 rows; the transposed score
// tile (keys x queries) leaves a query in a lane pair, so the softmax needs one
// exchange per tile and its weights feed the second product from registers.
template <int D>
__global__ void __launch_bounds__(256, 1) diff_fwd_direct(const DiffArgs a) {
  using T = float;
  constexpr int NT = D / 16;   // 32-value tiles of the 2 D wide output
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int nqb = (a.L + 31) / 32;
  if (wave >= nqb * a.hp * a.B) return;
  const int qb = nqb - 1 - wave / (a.hp * a.B);       // the longest rows first
  const int pair = (wave / a.B) % a.hp, b = wave % a.B;
  const int g = pair / (a.hp / a.gp), len = a.lens[b];
  float e1, e2;
  const float lam = lambda_of(a, e1, e2);
  if (wave == 0 && lane == 0) {
    a.lam[0] = lam;
    a.lam[1] = e1;
    a.lam[2] = e2;
  }
  const int row = qb * 32 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const T* qp = reinterpret_cast<const T*>(a.q) + (tok0 + row) * ldq + pair * 2 * a.hd;
  const T* kp = reinterpret_cast<const T*>(a.k) + tok0 * ldk + g * 2 * a.hd;
  const T* vp = reinterpret_cast<const T*>(a.v) + tok0 * ldk + g * 2 * a.hd;
  const bool rok = row < len;
  f32x16 o[2][NT];
  float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) zero16(o[m][t]);
  const float sc = a.scale * kLog2e;
  int kend = len;
  if (a.causal && kend > qb * 32 + 32) kend = qb * 32 + 32;
  if (qb * 32 >= len) kend = 0;
  for (int k0 = 0; k0 < kend; k0 += 32) {
    const int kz = opaque(0);
    f32x16 s[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      zero16(s[m]);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int col = ks * 16 + h * 8;
        const bool cok = col < a.hd;
        const Frag<T> kf = load_row<T>(kp + (long long)(k0 + c) * ldk + m * a.hd + col, cok && k0 + c < len);
        const Frag<T> qf = load_row<T>(qp + m * a.hd + col + kz, cok && rok);
        mma(s[m], kf, qf);
      }
      float tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = k0 + 8 * (i >> 2) + 4 * h + (i & 3);
        if (key >= len || (a.causal && key > row)) s[m][i] = -INFINITY;
        tm = fmaxf(tm, s[m][i]);
      }
      tm = fmaxf(tm, __shfl_xor(tm, 32));
      const float nm = fmaxf(mx[m], tm);
      const float ms = nm == -INFINITY ? 0.f : nm * sc;   // nothing seen yet: weights 0
      const float f = exp2f(mx[m] * sc - ms);
      float ts = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[m][i] = exp2f(fmaf(s[m][i], sc, -ms));
        ts += s[m][i];
      }
      sum[m] = sum[m] * f + ts;
      mx[m] = nm;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[m][t][i] *= f;
    }
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      const Frag<T> p0 = acc_frag<T>(s[0], cc), p1 = acc_frag<T>(s[1], cc);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int dv = 32 * t + c;
        const Frag<T> vf = load_col(vp + dv, ldk, k0 + 16 * cc, len, h, dv < 2 * a.hd);
        mma(o[0][t], vf, p0);
        mma(o[1][t], vf, p1);
      }
    }
  }
  if (row >= a.L) return;
  float inv[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float l = sum[m] + __shfl_xor(sum[m], 32);
    inv[m] = rok ? 1.f / l : 0.f;
    if (h == 0) a.lse[((long long)(b * a.hp + pair) * 2 + m) * a.L + row] = rok ? mx[m] * sc + log2f(l) : INFINITY;
  }
  const long long orow = (tok0 + row) * ldq + pair * 2 * a.hd;
  T* op = reinterpret_cast<T*>(a.o) + orow;
  T* o2p = reinterpret_cast<T*>(a.o2) + orow;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int dv = 32 * t + 2 * i + 4 * h;
      if (dv >= 2 * a.hd) continue;
      float x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] = rok ? o[1][t][i + e] * inv[1] : 0.f;
        x[e] = rok ? o[0][t][i + e] * inv[0] - lam * y[e] : 0.f;
      }
      store4<T>(op + dv, x[0], x[1], x[2], x[3]);
      store4<T>(o2p + dv, y[0], y[1], y[2], y[3]);
    }
}

// dQ: one wave per 32 queries, keys in order.  It also sums P_2 dP, whose total
// is -dlambda, in fp32 (D_2 of the saved, rounded O_2 would not be exact enough).
template <int D>
__global__ void __launch_bounds__(256, 1) diff_dq_direct(const DiffArgs a) {
  using T = float;
  constexpr int DT = D / 32;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int nqb = (a.L + 31) / 32;
  if (wave >= nqb * a.hp * a.B) {
    if (lane == 0) a.dlam_part[wave] = 0.0;
    return;
  }
  const int qb = nqb - 1 - wave / (a.hp * a.B);
  const int pair = (wave / a.B) % a.hp, b = wave % a.B;
  const int g = pair / (a.hp / a.gp), len = a.lens[b];
  const float lam = a.lam[0];
  const int row = qb * 32 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long qoff = (tok0 + row) * ldq + pair * 2 * a.hd, koff = tok0 * ldk + g * 2 * a.hd;
  const T* qp = reinterpret_cast<const T*>(a.q) + qoff;
  const T* dop = reinterpret_cast<const T*>(a.da) + qoff;
  const T* kp = reinterpret_cast<const T*>(a.k) + koff;
  const T* vp = reinterpret_cast<const T*>(a.v) + koff;
  const bool rok = row < len;
  float lse[2], ds[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const long long at = ((long long)(b * a.hp + pair) * 2 + m) * a.L + row;
    lse[m] = rok ? a.lse[at] : INFINITY;
    ds[m] = rok ? a.dsum[at] : 0.f;
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
  for (int k0 = 0; k0 < kend; k0 += 32) {
    const int kz = opaque(0);
    f32x16 dp, s[2];
    float part = 0.f;
    zero16(dp);
#pragma unroll
    for (int ks = 0; ks < D / 8; ++ks) {
      const int col = ks * 16 + h * 8;
      const bool cok = col < 2 * a.hd;
      const Frag<T> vf = load_row<T>(vp + (long long)(k0 + c) * ldk + col, cok && k0 + c < len);
      const Frag<T> gf = load_row<T>(dop + col + kz, cok && rok);
      mma(dp, vf, gf);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      zero16(s[m]);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int col = ks * 16 + h * 8;
        const bool cok = col < a.hd;
        const Frag<T> kf = load_row<T>(kp + (long long)(k0 + c) * ldk + m * a.hd + col, cok && k0 + c < len);
        const Frag<T> qf = load_row<T>(qp + m * a.hd + col + kz, cok && rok);
        mma(s[m], kf, qf);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = k0 + 8 * (i >> 2) + 4 * h + (i & 3);
        const bool hidden = key >= len || (a.causal && key > row) || !rok;
        const float p = hidden ? 0.f : exp2f(fmaf(s[m][i], sc, -lse[m]));
        if (m == 1) part = fmaf(p, dp[i], part);
        s[m][i] = p * (dp[i] - ds[m]);
      }
    }
    dlam += (double)part;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const Frag<T> sf = acc_frag<T>(s[m], cc);
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const int d = 32 * t + c;
          const Frag<T> kf = load_col(kp + m * a.hd + d, ldk, k0 + 16 * cc, len, h, d < a.hd);
          mma(dq[m][t], kf, sf);
        }
      }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) dlam += __shfl_xor(dlam, o);
  if (lane == 0) a.dlam_part[wave] = dlam;
  if (row >= a.L) return;
  T* out = reinterpret_cast<T*>(a.dq) + qoff;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float f = m ? -lam * a.scale : a.scale;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d >= a.hd) continue;
        store4<T>(out + m * a.hd + d, dq[m][t][i] * f, dq[m][t][i + 1] * f, dq[m][t][i + 2] * f, dq[m][t][i + 3] * f);
      }
  }
}

// dK and dV: one wave per 32 keys; the query pairs of the group in order, their
// queries in order.
template <int D>
__global__ void __launch_bounds__(256, 1) diff_dkv_direct(const DiffArgs a) {
  using T = float;
  constexpr int DT = D / 32, NT = D / 16;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int nkb = (a.L + 31) / 32;
  if (wave >= nkb * a.gp * a.B) return;
  const int kb = wave / (a.gp * a.B);                 // causal: the first keys have the most queries
  const int g = (wave / a.B) % a.gp, b = wave % a.B;
  const int grp = a.hp / a.gp, len = a.lens[b];
  const float lam = a.lam[0];
  const int key = kb * 32 + c;
  const bool kok = key < len;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long koff = (tok0 + key) * ldk + g * 2 * a.hd;
  const T* kp = reinterpret_cast<const T*>(a.k) + koff;
  const T* vp = reinterpret_cast<const T*>(a.v) + koff;
  f32x16 dk[2][DT], dv[NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dk[m][t]);
#pragma unroll
  for (int t = 0; t < NT; ++t) zero16(dv[t]);
  const float sc = a.scale * kLog2e;
  const int qbeg = a.causal ? kb * 32 : 0;
  for (int pr = g * grp; pr < (g + 1) * grp; ++pr) {
    const T* qp = reinterpret_cast<const T*>(a.q) + tok0 * ldq + pr * 2 * a.hd;
    const T* dop = reinterpret_cast<const T*>(a.da) + tok0 * ldq + pr * 2 * a.hd;
    const float* lse = a.lse + (long long)(b * a.hp + pr) * 2 * a.L;
    const float* dsm = a.dsum + (long long)(b * a.hp + pr) * 2 * a.L;
    for (int q0 = kb * 32 < len ? qbeg : len; q0 < len; q0 += 32) {
      const int kz = opaque(0);
      f32x16 dp, s[2], w;
      zero16(dp);
#pragma unroll
      for (int ks = 0; ks < D / 8; ++ks) {
        const int col = ks * 16 + h * 8;
        const bool cok = col < 2 * a.hd;
        const Frag<T> gf = load_row<T>(dop + (long long)(q0 + c) * ldq + col, cok && q0 + c < len);
        const Frag<T> vf = load_row<T>(vp + col + kz, cok && kok);
        mma(dp, gf, vf);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        zero16(s[m]);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int col = ks * 16 + h * 8;
          const bool cok = col < a.hd;
          const Frag<T> qf = load_row<T>(qp + (long long)(q0 + c) * ldq + m * a.hd + col, cok && q0 + c < len);
          const Frag<T> kf = load_row<T>(kp + m * a.hd + col + kz, cok && kok);
          mma(s[m], qf, kf);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int q = q0 + 8 * (i >> 2) + 4 * h + (i & 3);
          const bool hidden = q >= len || (a.causal && key > q) || !kok;
          const int qq = q < len ? q : 0;
          const float p = hidden ? 0.f : exp2f(fmaf(s[m][i], sc, -lse[m * a.L + qq]));
          w[i] = m ? w[i] - lam * p : p;
          s[m][i] = p * (dp[i] - dsm[m * a.L + qq]);
        }
      }
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const Frag<T> wf = acc_frag<T>(w, cc);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int d = 32 * t + c;
          const Frag<T> gf = load_col(dop + d, ldq, q0 + 16 * cc, len, h, d < 2 * a.hd);
          mma(dv[t], gf, wf);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const Frag<T> sf = acc_frag<T>(s[m], cc);
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            const int d = 32 * t + c;
            const Frag<T> qf = load_col(qp + m * a.hd + d, ldq, q0 + 16 * cc, len, h, d < a.hd);
            mma(dk[m][t], qf, sf);
          }
        }
      }
    }
  }
  if (key >= a.L) return;
  T* dkp = reinterpret_cast<T*>(a.dk) + koff;
  T* dvp = reinterpret_cast<T*>(a.dv) + koff;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = 32 * t + 2 * i + 4 * h;
      if (d < 2 * a.hd) store4<T>(dvp + d, dv[t][i], dv[t][i + 1], dv[t][i + 2], dv[t][i + 3]);
    }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float f = m ? -lam * a.scale : a.scale;
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

}  // namespace sl
