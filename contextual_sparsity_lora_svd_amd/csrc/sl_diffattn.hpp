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
#pragma once

#include <utility>

#include <cmath>

#include "sl_common.hpp"
#include "sl_host.hpp"

namespace sl {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct DiffArgs {
  const void *q, *k, *v, *a, *da;
  void *o, *o2;              // forward: output and O_2 = P_2 V (also read by the backward): fp32, or
                             // 16-bit integers times the row's rsc[1]
  signed char* res;          // bf16 calls: what rounding O to bf16 dropped, times the row's rsc[0]
  float* rsc;                // [batch][pairs][2][ls]
  float* lam;                // lambda and its two exponentials, written by the forward
  float* lse;                // [batch][pairs][2][ls], log2 units; +inf for rows past the length
  float* fix;                // bf16 calls: [batch][pairs][ls], the second map's weights times 1 + this are free of the lse's rounding
  float* dsum;               // [batch][pairs][2][ls] row sums D_1, D_2; 0 for rows past the length
  void *dq, *dk, *dv;
  float *dk_part, *dv_part;  // [split][tokens][kv columns] sums of the heads' parts, split > 1
  double* dlam_part;         // one partial sum of D_2 per wave of the dQ kernel
  float *dlq1, *dlk1, *dlq2, *dlk2;
  const float *lq1, *lk1, *lq2, *lk2;
  float lambda_init, scale;
  int B, L, hp, gp, hd;      // hp query pairs, gp kv pairs
  int ls;                    // L + 1: statistics of one row more than there are, past every length
  int causal, mix, npart, split;   // mix: the sequences' lengths differ
  int dq_rows, dkv_rows;     // bf16: rows, or keys, of a workgroup
  int fine;                  // bf16: weights and score gradients enter their products as two bf16 values
  int lens[SL_MAX_SEQS];
};

template <typename T> struct Frag;          // 8 consecutive k values of one row
template <> struct Frag<bf16> { bf16x8 v; };
template <> struct Frag<float> { float v[8]; };

template <typename T> __device__ inline Frag<T> load_row(const T* p, bool ok);
template <> __device__ inline Frag<bf16> load_row<bf16>(const bf16* p, bool ok) {
  uint4 x = make_uint4(0, 0, 0, 0);
  if (ok) x = *reinterpret_cast<const uint4*>(p);
  return Frag<bf16>{__builtin_bit_cast(bf16x8, x)};
}

// acc (32 x 32) += A (32 x 16) B (16 x 32).  Lane l holds row l % 32 of A and
// column l % 32 of B, 8 k values of half l / 32; any order of k serves as long
// as both operands use it.  acc[i] is row 8 (i / 4) + 4 (l / 32) + i % 4 of
// column l % 32.
__device__ inline void mma(f32x16& acc, const Frag<bf16>& a, const Frag<bf16>& b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ inline void mma1(f32x16& acc, const Frag<float>& a, float b, int j) {   // one of the 8 k values
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b, acc, 0, 0, 0);
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

// fp32 operands come straight from memory, each read some products before its
// use.  A tile is 32 rows; rows past the sequence's last read that one again
// (their weights are zero, or their results dropped), columns past the width the
// first or the last (the other operand is zero there; as columns of a result they
// are dropped).
struct Rows32 {
  unsigned row, col[16];     // bytes from the tile's first row: of row l % 32; of rows 8 (j / 4) + 4 h + j % 4
  __device__ inline void init(int c, int h, int last, unsigned ld) {
    row = (unsigned)(c < last ? c : last) * ld * 4u;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int r = 8 * (j >> 2) + 4 * h + (j & 3);
      col[j] = (unsigned)(r < last ? r : last) * ld * 4u;
    }
  }
};
// Part j of 8 of an operand: 8 values of a row from byte `at` on (parts 0 and 1) ...
__device__ inline void read_row(Frag<float>& f, int j, const float* base, unsigned at) {
  if (j != 0 && j != 1) return;
  const float4 x = reinterpret_cast<const float4*>(reinterpret_cast<const char*>(base) + at)[j];
  f.v[4 * j] = x.x; f.v[4 * j + 1] = x.y; f.v[4 * j + 2] = x.z; f.v[4 * j + 3] = x.w;
}
// ... or the column at byte `at` of row j of half cc
__device__ inline void read_col(Frag<float>& f, int j, const float* base, const Rows32& r, int cc, unsigned at) {
  f.v[j] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(base) + (r.col[8 * cc + j] + at));
}
__device__ inline unsigned first_if_past(int col, int w) { return (col < w ? col : 0) * 4u; }
__device__ inline unsigned last_if_past(int col, int w) { return (col < w ? col : w - 1) * 4u; }
// The workgroup's own 32 rows of `w` values in LDS, as operands: operand f is columns
// 16 f + 8 h on, zero past the width.  A wave writes every fourth.
__device__ inline void put_own(float4* own, int nf, const float* row, int w, int wave, int lane) {
  for (int f = wave; f < nf; f += 4) {
    const int col = f * 16 + (lane >> 5) * 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (col < w) {
      x = *reinterpret_cast<const float4*>(row + col);
      y = *reinterpret_cast<const float4*>(row + col + 4);
    }
    own[f * 128 + lane] = x;
    own[f * 128 + 64 + lane] = y;
  }
}
__device__ inline void read_own(Frag<float>& f, int j, const float4* own, int n) {   // own: + lane
  if (j != 0 && j != 1) return;
  const float4 x = own[n * 128 + j * 64];
  f.v[4 * j] = x.x; f.v[4 * j + 1] = x.y; f.v[4 * j + 2] = x.z; f.v[4 * j + 3] = x.w;
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

// Whether a row reads a single key.  Its weights are 1 whatever the scores, so its
// score gradients are 0, which D, summed from rounded values, leaves only nearly so.
__device__ inline bool one_key(const DiffArgs& a, int row, int len) { return len == 1 || (a.causal && row == 0); }

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

__device__ inline float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }   // subnormal results are 0

// The four waves' values added in order; the last wave ends with the sum.  sm holds
// N tiles of 1024 floats.
template <int N> __device__ inline void add_waves(f32x16 (&x)[N], float* sm, int wave, int lane) {
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          float4* const p = reinterpret_cast<float4*>(sm + (n * 4 + i / 4) * 256) + lane;
          if (w > 0) {
            const float4 y = *p;
            x[n][i] += y.x; x[n][i + 1] += y.y; x[n][i + 2] += y.z; x[n][i + 3] += y.w;
          }
          if (w < 3) *p = make_float4(x[n][i], x[n][i + 1], x[n][i + 2], x[n][i + 3]);
        }
    }
    __syncthreads();
  }
}

// f(0) .. f(N - 1) with compile-time indices, unrolled however long.
template <typename F, int... I>
__device__ inline __attribute__((always_inline)) void each_of(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ inline __attribute__((always_inline)) void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// Run f with the row width D that serves head_dim hd.
template <typename F> inline void by_width(int hd, F f) {
  if (hd <= 32) f(std::integral_constant<int, 32>{});
  else if (hd <= 64) f(std::integral_constant<int, 64>{});
  else if (hd <= 96) f(std::integral_constant<int, 96>{});
  else f(std::integral_constant<int, 128>{});
}

// dlambda = -(the waves' sums of D_2, added in a fixed order) and the four
// vectors' gradients: the work of one block of 256 threads.
__device__ inline void dlambda_block(const DiffArgs& a, double* sm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < a.npart; i += 256) s += a.dlam_part[i];
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = s;
  __syncthreads();
  s = ((sm[0] + sm[1]) + sm[2]) + sm[3];
  const int i = threadIdx.x;
  if (i < a.hd) {
    const float g1 = -(float)s * a.lam[1], g2 = (float)s * a.lam[2];
    const float q1 = a.lq1[i], k1 = a.lk1[i], q2 = a.lq2[i], k2 = a.lk2[i];
    a.dlq1[i] = g1 * k1;
    a.dlk1[i] = g1 * q1;
    a.dlq2[i] = g2 * k2;
    a.dlk2[i] = g2 * q2;
  }
}

// dK and dV from the parts' sums, in order; 4 values per thread.
template <typename T> __global__ void __launch_bounds__(256) diff_dkv_sum(const DiffArgs a) {
  const long long n = (long long)a.B * a.L * a.gp * 2 * a.hd / 4;
  long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool v = i >= n;
  if (v) i -= n;
  if (i >= n) return;
  const float4* src = reinterpret_cast<const float4*>(v ? a.dv_part : a.dk_part) + i;
  float4 x = src[0];
  for (int p = 1; p < a.split; ++p) {
    const float4 y = src[p * n];
    x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
  }
  store4<T>(reinterpret_cast<T*>(v ? a.dv : a.dk) + 4 * i, x.x, x.y, x.z, x.w);
}

// Blocks of `rows` rows that hold any of a sequence.
inline long long filled(const DiffArgs& a, int rows) {
  long long n = 0;
  for (int b = 0; b < a.B; ++b) n += (a.lens[b] + rows - 1) / rows;
  return n;
}

// Enqueue the forward, and the backward, of one type on s.
void launch_diff_fwd_bf16(const DiffArgs& a, hipStream_t s);
void launch_diff_bwd_bf16(const DiffArgs& a, hipStream_t s);
void launch_diff_fwd_f32(const DiffArgs& a, hipStream_t s);
void launch_diff_bwd_f32(const DiffArgs& a, hipStream_t s);

}  // namespace sl
