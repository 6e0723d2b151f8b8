// Shared by the operators that walk token rows: vectors of values, sums over
// the lanes of a wave, and the checks of their arguments.
#pragma once

#include "sl_common.hpp"
#include "sl_host.hpp"

namespace sl {

// V values, moved as one
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T v[V]; };

template <typename T> __device__ inline float el2f(T x);
template <> __device__ inline float el2f<float>(float x) { return x; }
template <> __device__ inline float el2f<bf16>(bf16 x) { return bf2f(x.v); }
template <typename T> __device__ inline T f2el(float x);
template <> __device__ inline float f2el<float>(float x) { return x; }
template <> __device__ inline bf16 f2el<bf16>(float x) { return __builtin_bit_cast(bf16, (__bf16)x); }   // to nearest even

// 16 bytes of row elements as the four registers they are loaded into; values are
// taken out where they are used.
template <typename T> struct Pack;
template <> struct Pack<bf16> {
  static constexpr int W = 8;
  typedef uint32_t Raw __attribute__((ext_vector_type(4)));
  Raw r;
  __device__ float get(int j) const { return __builtin_bit_cast(float, j & 1 ? r[j / 2] & 0xFFFF0000u : r[j / 2] << 16); }
  __device__ void put(int j, float lo, float hi) {   // values j and j + 1
    typedef __bf16 Two __attribute__((ext_vector_type(2)));
    r[j / 2] = __builtin_bit_cast(uint32_t, Two{(__bf16)lo, (__bf16)hi});
  }
};
template <> struct Pack<float> {
  static constexpr int W = 4;
  typedef float Raw __attribute__((ext_vector_type(4)));
  Raw r;
  __device__ float get(int j) const { return r[j]; }
  __device__ void put(int j, float lo, float hi) {
    r[j] = lo;
    r[j + 1] = hi;
  }
};

// The value of the lane at a fixed place in the same 16 lanes (a DPP move).
template <int CTRL> __device__ inline float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;   // lane ^ 1, ^ 2, 7 - lane, 15 - lane

// x of lane l, the same for the whole wave
__device__ inline float lane_value(float x, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}

// Sum over the wave's 64 lanes of whole numbers.
__device__ inline int wave_count(int x) {
  x += __builtin_amdgcn_mov_dpp(x, kXor1, 0xf, 0xf, true);
  x += __builtin_amdgcn_mov_dpp(x, kXor2, 0xf, 0xf, true);
  x += __builtin_amdgcn_mov_dpp(x, kMirror8, 0xf, 0xf, true);
  x += __builtin_amdgcn_mov_dpp(x, kMirror16, 0xf, 0xf, true);
  return __builtin_amdgcn_readlane(x, 0) + __builtin_amdgcn_readlane(x, 16) + __builtin_amdgcn_readlane(x, 32) +
         __builtin_amdgcn_readlane(x, 48);
}

// Sum and maximum over the wave's 64 lanes: over each 16 by DPP moves, then the
// four 16s.  Every lane adds the same pairs, so all hold the same bits.
__device__ inline float wave_add(float x) {
  x += dpp<kXor1>(x);
  x += dpp<kXor2>(x);
  x += dpp<kMirror8>(x);
  x += dpp<kMirror16>(x);
  return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}
__device__ inline float wave_max(float x) {   // NaN only where every lane holds one
  x = fmaxf(x, dpp<kXor1>(x));
  x = fmaxf(x, dpp<kXor2>(x));
  x = fmaxf(x, dpp<kMirror8>(x));
  x = fmaxf(x, dpp<kMirror16>(x));
  return fmaxf(fmaxf(lane_value(x, 0), lane_value(x, 16)), fmaxf(lane_value(x, 32), lane_value(x, 48)));
}

// A product as it is rounded: the compiler may not fuse it into the difference that
// it goes into (which would be to another number than the one kept elsewhere).
__device__ inline float rounded(float x) {
  asm("" : "+v"(x));
  return x;
}

// batch and seq_len of a layout (ctx_len is not looked at)
inline sl_status check_tokens(const sl_layout* lay) {
  if (!lay) SL_FAIL(SL_ERR_NULL, "layout is NULL");
  if (lay->batch < 1 || lay->batch > SL_MAX_SEQS)
    SL_FAIL(SL_ERR_RANGE, "batch %d outside [1, %d]", lay->batch, SL_MAX_SEQS);
  if (lay->seq_len < 1) SL_FAIL(SL_ERR_RANGE, "seq_len %d < 1", lay->seq_len);
  if ((long long)lay->batch * lay->seq_len > (1LL << 30)) SL_FAIL(SL_ERR_RANGE, "too many tokens");
  return SL_OK;
}

inline sl_status check_dtype(sl_dtype dt) {
  if (dt != SL_BF16 && dt != SL_F32) SL_FAIL(SL_ERR_DTYPE, "dtype must be SL_F32 or SL_BF16");
  return SL_OK;
}

// A grid for n pieces of work; past `most` blocks they walk on (a launch holds
// fewer than 2^32 threads).
inline dim3 walk_grid(long long n, long long most = 1 << 20) { return dim3((unsigned)(n < 1 ? 1 : n < most ? n : most)); }

}  // namespace sl
