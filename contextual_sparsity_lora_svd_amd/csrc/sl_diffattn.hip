// Differential attention, forward and backward.
//
// Per head pair, with S_m = s q_m k_m^T (causal or within the sequence's length):
//   P_m = softmax(S_m),  O = P_1 V - lambda P_2 V
//   dP = dO V^T,  D_m = rowsum(P_m dP) = dO . (P_m V)
//   dS_1 = P_1 (dP - D_1),  dS_2 = -lambda P_2 (dP - D_2)
//   dQ_m = s dS_m K_m,  dK_m = s dS_m^T Q_m,  dV = (P_1 - lambda P_2)^T dO
//   dlambda = -sum D_2
// The two maps share V, dP and dV's product.  The forward keeps the running
// maximum and sum of each map (one pass over the keys) and saves each row's
// log2-sum-exp and O_2 = P_2 V; the backward forms the weights again from them.
#include <cmath>

#include "sl_common.hpp"
#include "sl_host.hpp"

namespace sl {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct DiffArgs {
  const void *q, *k, *v, *a, *da;
  void *o, *o2;              // forward: output and P_2 V (also read by the backward)
  float* lse;                // [batch][pairs][2][L], log2 units
  float* dsum;               // [batch][pairs][2][L] row sums D_1, D_2
  void *dq, *dk, *dv;
  float* dlam_part;          // one partial sum of D_2 per wave of the dQ kernel
  float *dlq1, *dlk1, *dlq2, *dlk2;
  const float *lq1, *lk1, *lq2, *lk2;
  float lambda_init, scale;
  int B, L, hp, gp, hd;      // hp query pairs, gp kv pairs
  int causal, npart;
  int lens[SL_MAX_SEQS];
};

template <typename T> struct Frag;          // 8 consecutive k values of one row
template <> struct Frag<bf16> { bf16x8 v; };
template <> struct Frag<float> { float v[8]; };

template <typename T> __device__ inline Frag<T> load_row(const T* p, bool ok);
template <> __device__ inline Frag<bf16> load_row<bf16>(const bf16* p, bool ok) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  return Frag<bf16>{__builtin_bit_cast(bf16x8, ok ? *reinterpret_cast<const uint4*>(p) : z)};
}
template <> __device__ inline Frag<float> load_row<float>(const float* p, bool ok) {
  Frag<float> f;
  float4 x = make_float4(0, 0, 0, 0), y = x;
  if (ok) {
    x = *reinterpret_cast<const float4*>(p);
    y = *reinterpret_cast<const float4*>(p + 4);
  }
  f.v[0] = x.x; f.v[1] = x.y; f.v[2] = x.z; f.v[3] = x.w;
  f.v[4] = y.x; f.v[5] = y.y; f.v[6] = y.z; f.v[7] = y.w;
  return f;
}

// acc (32 x 32) += A (32 x 16) B (16 x 32).  Lane l holds row l % 32 of A and
// column l % 32 of B, 8 k values of half l / 32; any order of k serves as long
// as both operands use it.  acc[i] is row 8 (i / 4) + 4 (l / 32) + i % 4 of
// column l % 32.
__device__ inline void mma(f32x16& acc, const Frag<bf16>& a, const Frag<bf16>& b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ inline void mma(f32x16& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], acc, 0, 0, 0);
}

// Accumulator values 8 c .. 8 c + 7 as the k values of an operand: k position j
// of half h is row 16 c + 8 (j / 4) + 4 h + j % 4.
template <typename T> __device__ inline Frag<T> acc_frag(const f32x16& x, int c);
template <> __device__ inline Frag<bf16> acc_frag<bf16>(const f32x16& x, int c) {
  Frag<bf16> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = (__bf16)x[8 * c + j];
  return f;
}
template <> __device__ inline Frag<float> acc_frag<float>(const f32x16& x, int c) {
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = x[8 * c + j];
  return f;
}

// The matching operand from memory: column `col` of rows row0 + 16 c + 8 (j / 4)
// + 4 h + j % 4, rows at or past `rows` as 0.
template <typename T> __device__ inline Frag<T> load_col(const T* base, long long ld, int row0, int rows, int h, bool ok) {
  Frag<T> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = row0 + 8 * (j >> 2) + 4 * h + (j & 3);
    if constexpr (sizeof(T) == 2) {
      const uint16_t x = ok && r < rows ? base[r * ld].v : (uint16_t)0;
      f.v[j] = __builtin_bit_cast(__bf16, x);
    } else {
      f.v[j] = ok && r < rows ? base[r * ld] : 0.f;
    }
  }
  return f;
}

// four consecutive values of a row
template <typename T> __device__ inline void store4(T* p, float a, float b, float c, float d);
template <> __device__ inline void store4<bf16>(bf16* p, float a, float b, float c, float d) {
  uint2 w;
  w.x = (uint32_t)f2bf(a) | ((uint32_t)f2bf(b) << 16);
  w.y = (uint32_t)f2bf(c) | ((uint32_t)f2bf(d) << 16);
  *reinterpret_cast<uint2*>(p) = w;
}
template <> __device__ inline void store4<float>(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

__device__ inline float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// lambda, and the two exponentials it is made of; every lane gets them
__device__ inline float lambda_of(const DiffArgs& a, float& e1, float& e2) {
  const int lane = threadIdx.x & 63;
  float s1 = 0.f, s2 = 0.f;
  for (int i = lane; i < a.hd; i += 64) {
    s1 = fmaf(a.lq1[i], a.lk1[i], s1);
    s2 = fmaf(a.lq2[i], a.lk2[i], s2);
  }
  e1 = expf(wave_sum(s1));
  e2 = expf(wave_sum(s2));
  return e1 - e2 + a.lambda_init;
}

constexpr float kLog2e = 1.44269504088896341f;

__device__ inline void zero16(f32x16& x) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
}

// Keep a loop from hoisting (and then spilling) the loads behind an offset.
__device__ inline int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// ---------------------------------------------------------------------------
// Operands straight from memory.  One wave per 32 rows; the transposed score
// tile (keys x queries) leaves a query in a lane pair, so the softmax needs one
// exchange per tile and its weights feed the second product from registers.
template <typename T, int D>
__global__ void __launch_bounds__(256, 1) diff_fwd_direct(const DiffArgs a) {
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
        const Frag<T> vf = load_col<T>(vp + dv, ldk, k0 + 16 * cc, len, h, dv < 2 * a.hd);
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

// D_1 = dO . (O + lambda O_2), D_2 = dO . O_2, one wave per row and head pair.
template <typename T>
__global__ void __launch_bounds__(256) diff_dsum(const DiffArgs a) {
  const int lane = threadIdx.x & 63;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const long long rows = (long long)a.B * a.L;
  if (w >= rows * a.hp) return;
  const int pair = (int)(w % a.hp);
  const long long tok = w / a.hp;
  const int b = (int)(tok / a.L), row = (int)(tok % a.L);
  float e1, e2;
  const float lam = lambda_of(a, e1, e2);
  float d1 = 0.f, d2 = 0.f;
  if (row < a.lens[b]) {
    const long long at = (tok * a.hp + pair) * 2 * a.hd;
    const T* dop = reinterpret_cast<const T*>(a.da) + at;
    const T* op = reinterpret_cast<const T*>(a.a) + at;
    const T* o2p = reinterpret_cast<const T*>(a.o2) + at;
    for (int i = lane; i < 2 * a.hd; i += 64) {
      const float g = ldv(dop, i), y = ldv(o2p, i);
      d1 = fmaf(g, ldv(op, i) + lam * y, d1);
      d2 = fmaf(g, y, d2);
    }
  }
  d1 = wave_sum(d1);
  d2 = wave_sum(d2);
  if (lane < 2) a.dsum[((long long)(b * a.hp + pair) * 2 + lane) * a.L + row] = lane ? d2 : d1;
}

// dQ: one wave per 32 queries, keys in order.  It also sums P_2 dP, whose total
// is -dlambda, in fp32 (D_2 of the saved, rounded O_2 would not be exact enough).
template <typename T, int D>
__global__ void __launch_bounds__(256, 1) diff_dq_direct(const DiffArgs a) {
  constexpr int DT = D / 32;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int nqb = (a.L + 31) / 32;
  if (wave >= nqb * a.hp * a.B) return;
  const int qb = nqb - 1 - wave / (a.hp * a.B);
  const int pair = (wave / a.B) % a.hp, b = wave % a.B;
  const int g = pair / (a.hp / a.gp), len = a.lens[b];
  float e1, e2;
  const float lam = lambda_of(a, e1, e2);
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
  float dlam = 0.f;
  int kend = len;
  if (a.causal && kend > qb * 32 + 32) kend = qb * 32 + 32;
  if (qb * 32 >= len) kend = 0;
  for (int k0 = 0; k0 < kend; k0 += 32) {
    const int kz = opaque(0);
    f32x16 dp, s[2];
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
        if (m == 1) dlam = fmaf(p, dp[i], dlam);
        s[m][i] = p * (dp[i] - ds[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const Frag<T> sf = acc_frag<T>(s[m], cc);
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const int d = 32 * t + c;
          const Frag<T> kf = load_col<T>(kp + m * a.hd + d, ldk, k0 + 16 * cc, len, h, d < a.hd);
          mma(dq[m][t], kf, sf);
        }
      }
  }
  dlam = wave_sum(dlam);
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
template <typename T, int D>
__global__ void __launch_bounds__(256, 1) diff_dkv_direct(const DiffArgs a) {
  constexpr int DT = D / 32, NT = D / 16;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int nkb = (a.L + 31) / 32;
  if (wave >= nkb * a.gp * a.B) return;
  const int kb = wave / (a.gp * a.B);                 // causal: the first keys have the most queries
  const int g = (wave / a.B) % a.gp, b = wave % a.B;
  const int grp = a.hp / a.gp, len = a.lens[b];
  float e1, e2;
  const float lam = lambda_of(a, e1, e2);
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
          const Frag<T> gf = load_col<T>(dop + d, ldq, q0 + 16 * cc, len, h, d < 2 * a.hd);
          mma(dv[t], gf, wf);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const Frag<T> sf = acc_frag<T>(s[m], cc);
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            const int d = 32 * t + c;
            const Frag<T> qf = load_col<T>(qp + m * a.hd + d, ldq, q0 + 16 * cc, len, h, d < a.hd);
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

// dlambda = -(sum of the partial sums, in a fixed order); the four vectors' gradients.
__global__ void __launch_bounds__(1024) diff_dlambda(const DiffArgs a) {
  __shared__ float sm[16];
  float e1, e2;
  lambda_of(a, e1, e2);
  float s = 0.f;
  for (int i = threadIdx.x; i < a.npart; i += 1024) s += a.dlam_part[i];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < 16; ++i) s += sm[i];
  const int i = threadIdx.x;
  if (i < a.hd) {
    const float g1 = -s * e1, g2 = s * e2;
    const float q1 = a.lq1[i], k1 = a.lk1[i], q2 = a.lq2[i], k2 = a.lk2[i];
    a.dlq1[i] = g1 * k1;
    a.dlk1[i] = g1 * q1;
    a.dlq2[i] = g2 * k2;
    a.dlk2[i] = g2 * q2;
  }
}

// ---------------------------------------------------------------------------
// host side
struct DiffPlan {
  size_t lse, o2, saved;           // offsets and size of the saved buffer
  size_t dsum, dlam, ws;           // of the workspace
  int npart;
};

static sl_status diff_plan(sl_dtype dt, const sl_layout* lay, const sl_heads* hs, DiffPlan& pl) {
  if (dt != SL_BF16 && dt != SL_F32) SL_FAIL(SL_ERR_DTYPE, "dtype must be SL_F32 or SL_BF16");
  if (!lay || !hs) SL_FAIL(SL_ERR_NULL, "layout and heads must be non-NULL");
  if (lay->batch < 1 || lay->batch > SL_MAX_SEQS)
    SL_FAIL(SL_ERR_RANGE, "batch %d outside [1, %d]", lay->batch, SL_MAX_SEQS);
  if (lay->seq_len < 1) SL_FAIL(SL_ERR_RANGE, "seq_len %d < 1", lay->seq_len);
  const int hq = hs->n_q_heads, hkv = hs->n_kv_heads, hd = hs->head_dim;
  if (hq < 2 || hkv < 2 || hq % 2 || hkv % 2 || hq % hkv || hq > 65536)
    SL_FAIL(SL_ERR_SHAPE, "differential heads come in pairs: %d query heads must be a multiple of %d kv heads, both even",
            hq, hkv);
  if (hd < 8 || hd > 128 || hd % 8) SL_FAIL(SL_ERR_SHAPE, "head_dim %d must be a multiple of 8 and at most 128", hd);
  const long long T = (long long)lay->batch * lay->seq_len;
  sl_status st = check_extent("q", T, (long long)hq * hd);
  if (st != SL_OK) return st;
  const long long stats = T * hq;   // two rows of statistics per head pair
  Bump s, w;
  pl.lse = s.take(stats * 4);
  pl.o2 = s.take(T * hq * hd * (dt == SL_BF16 ? 2 : 4));
  pl.saved = s.off;
  const long long nqb = (lay->seq_len + 31) / 32;
  if (nqb * (hq / 2) * lay->batch > 0x7fffffffLL / 4) SL_FAIL(SL_ERR_RANGE, "too many rows");
  pl.npart = (int)(nqb * (hq / 2) * lay->batch);
  pl.dsum = w.take(stats * 4);
  pl.dlam = w.take((size_t)pl.npart * 4);
  pl.ws = w.off;
  return SL_OK;
}

static sl_status diff_args(DiffArgs& a, const sl_layout* lay, const sl_diff_attn* p) {
  a = DiffArgs{};
  a.B = lay->batch;
  a.L = lay->seq_len;
  a.hp = p->heads.n_q_heads / 2;
  a.gp = p->heads.n_kv_heads / 2;
  a.hd = p->heads.head_dim;
  a.causal = p->causal != 0;
  a.lambda_init = p->lambda_init;
  a.scale = p->scale;
  a.lq1 = p->lq1; a.lk1 = p->lk1; a.lq2 = p->lq2; a.lk2 = p->lk2;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) SL_FAIL(SL_ERR_RANGE, "scale must be positive and finite");
  if (!std::isfinite(p->lambda_init)) SL_FAIL(SL_ERR_RANGE, "lambda_init is not finite");
  if (!a.lq1 || !a.lk1 || !a.lq2 || !a.lk2) SL_FAIL(SL_ERR_NULL, "lq1, lk1, lq2 and lk2 must be non-NULL");
  if (!aligned16(a.lq1) || !aligned16(a.lk1) || !aligned16(a.lq2) || !aligned16(a.lk2))
    SL_FAIL(SL_ERR_ALIGN, "lq1, lk1, lq2 and lk2 must be 16-byte aligned");
  for (int b = 0; b < a.B; ++b) {
    a.lens[b] = p->lens ? p->lens[b] : a.L;
    if (a.lens[b] < 0 || a.lens[b] > a.L) SL_FAIL(SL_ERR_RANGE, "lens[%d] = %d outside [0, %d]", b, a.lens[b], a.L);
  }
  return SL_OK;
}

template <typename F> static void by_width(int hd, F f) {
  if (hd <= 32) f(std::integral_constant<int, 32>{});
  else if (hd <= 64) f(std::integral_constant<int, 64>{});
  else if (hd <= 96) f(std::integral_constant<int, 96>{});
  else f(std::integral_constant<int, 128>{});
}

template <typename T> static void launch_fwd(const DiffArgs& a, int waves, hipStream_t s) {
  by_width(a.hd, [&](auto d) {
    hipLaunchKernelGGL((diff_fwd_direct<T, decltype(d)::value>), dim3((waves + 3) / 4), dim3(256), 0, s, a);
  });
}

template <typename T> static void launch_bwd(const DiffArgs& a, int waves, hipStream_t s) {
  const long long rows = (long long)a.B * a.L * a.hp;
  hipLaunchKernelGGL(diff_dsum<T>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, a);
  const int kwaves = (a.L + 31) / 32 * a.gp * a.B;
  by_width(a.hd, [&](auto d) {
    hipLaunchKernelGGL((diff_dq_direct<T, decltype(d)::value>), dim3((waves + 3) / 4), dim3(256), 0, s, a);
    hipLaunchKernelGGL((diff_dkv_direct<T, decltype(d)::value>), dim3((kwaves + 3) / 4), dim3(256), 0, s, a);
  });
  hipLaunchKernelGGL(diff_dlambda, dim3(1), dim3(1024), 0, s, a);
}

}  // namespace sl

using namespace sl;

extern "C" size_t sl_diff_attn_saved_bytes(sl_dtype dt, const sl_layout* lay, const sl_heads* heads) {
  DiffPlan pl;
  return diff_plan(dt, lay, heads, pl) == SL_OK ? pl.saved : 0;
}

extern "C" size_t sl_diff_attn_workspace_bytes(sl_dtype dt, const sl_layout* lay, const sl_heads* heads) {
  DiffPlan pl;
  return diff_plan(dt, lay, heads, pl) == SL_OK ? pl.ws : 0;
}

extern "C" sl_status sl_diff_attn_fwd(sl_dtype dt, const sl_layout* lay, const sl_diff_attn* p, const void* q,
                                      const void* k, const void* v, void* o, void* saved, size_t saved_bytes, void* ws,
                                      size_t ws_bytes, void* stream) {
  if (!p || !q || !k || !v || !o) SL_FAIL(SL_ERR_NULL, "p, q, k, v and a must be non-NULL");
  DiffPlan pl;
  DiffArgs a;
  sl_status st = diff_plan(dt, lay, &p->heads, pl);
  if (st != SL_OK) return st;
  st = diff_args(a, lay, p);
  if (st != SL_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(saved) || !aligned16(ws))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  if (!saved || saved_bytes < pl.saved)
    SL_FAIL(SL_ERR_WORKSPACE, "saved buffer too small: %zu of %zu bytes", saved_bytes, pl.saved);
  if (!ws || ws_bytes < pl.ws) SL_FAIL(SL_ERR_WORKSPACE, "workspace too small: %zu of %zu bytes", ws_bytes, pl.ws);
  st = check_arch();
  if (st != SL_OK) return st;
  a.q = q; a.k = k; a.v = v; a.o = o;
  a.lse = reinterpret_cast<float*>(reinterpret_cast<char*>(saved) + pl.lse);
  a.o2 = reinterpret_cast<char*>(saved) + pl.o2;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dt == SL_BF16) launch_fwd<bf16>(a, pl.npart, s);
  else launch_fwd<float>(a, pl.npart, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}

extern "C" sl_status sl_diff_attn_bwd(sl_dtype dt, const sl_layout* lay, const sl_diff_attn* p, const void* q,
                                      const void* k, const void* v, const void* o, const void* saved,
                                      size_t saved_bytes, const void* da, void* dq, void* dk, void* dv,
                                      const sl_diff_attn_grads* g, void* ws, size_t ws_bytes, void* stream) {
  if (!p || !q || !k || !v || !o || !da || !dq || !dk || !dv || !g || !g->dlq1 || !g->dlk1 || !g->dlq2 || !g->dlk2)
    SL_FAIL(SL_ERR_NULL, "p, q, k, v, a, da and every gradient must be non-NULL");
  DiffPlan pl;
  DiffArgs a;
  sl_status st = diff_plan(dt, lay, &p->heads, pl);
  if (st != SL_OK) return st;
  st = diff_args(a, lay, p);
  if (st != SL_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(da) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned16(saved) || !aligned16(ws) || !aligned16(g->dlq1) ||
      !aligned16(g->dlk1) || !aligned16(g->dlq2) || !aligned16(g->dlk2))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  if (!saved || saved_bytes < pl.saved)
    SL_FAIL(SL_ERR_WORKSPACE, "saved buffer too small: %zu of %zu bytes", saved_bytes, pl.saved);
  if (!ws || ws_bytes < pl.ws) SL_FAIL(SL_ERR_WORKSPACE, "workspace too small: %zu of %zu bytes", ws_bytes, pl.ws);
  st = check_arch();
  if (st != SL_OK) return st;
  a.q = q; a.k = k; a.v = v; a.a = o; a.da = da; a.dq = dq; a.dk = dk; a.dv = dv;
  a.lse = reinterpret_cast<float*>(reinterpret_cast<char*>(const_cast<void*>(saved)) + pl.lse);
  a.o2 = reinterpret_cast<char*>(const_cast<void*>(saved)) + pl.o2;
  a.dsum = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + pl.dsum);
  a.dlam_part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + pl.dlam);
  a.npart = pl.npart;
  a.dlq1 = g->dlq1; a.dlk1 = g->dlk1; a.dlq2 = g->dlq2; a.dlk2 = g->dlk2;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dt == SL_BF16) launch_bwd<bf16>(a, pl.npart, s);
  else launch_bwd<float>(a, pl.npart, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}
