// Differential attention in bf16: tiles of K and V (or Q and dO) rows staged in
// LDS by LDS-DMA, operands kept in registers, products on the bf16 matrix cores.
//
// Row tiles.  32 token rows of one head pair, 2 hd values each, lie in LDS as
// rows of 4 D bytes (D = hd rounded up to 32), written by global_load_lds as
// they come, 64 chunks of 16 bytes per instruction.  Two kinds of reads follow:
// a product over hd reads 16 bytes of 32 rows (ds_read_b128), a product over
// the rows reads 4 rows of 32 columns (the transposing ds_read_b64_tr_b16).  Row
// r's chunks are XORed with swz(r), so that 8 or 16 consecutive rows of the
// first kind and the 4 rows of the second fall on different banks; the XOR is
// applied to the address that a lane loads from, since the DMA writes in order.
//
// Columns past hd read the head's first chunk again (their partner in the
// other operand is zero, or their results are dropped), rows past the
// sequence's length read its last row again (their weight is zero): nothing
// outside the sequence is read.
#pragma once

#include <utility>

#include "sl_diffattn.hpp"

namespace sl {

typedef short v4i16 __attribute__((ext_vector_type(4)));

// 4-bit XOR where a row is whole 256-byte lines (D = 64, 128), 3-bit where it
// ends in half a line (D = 32, 96).
template <int D> __device__ inline unsigned swz(unsigned r) {
  const unsigned r0 = r & 1, r1 = (r >> 1) & 1, r2 = (r >> 2) & 1, r3 = (r >> 3) & 1;
  return D % 64 == 0 ? ((r1 ^ r3) << 3) | (r0 << 2) | (r1 << 1) | r2 : (r1 << 2) | ((r0 ^ r3) << 1) | r2;
}

template <int D> struct RowTile {
  static constexpr int PITCH = 4 * D;             // bytes of a row: 2 D values
  static constexpr int CH = D / 4;                // chunks of a row
  static constexpr int BYTES = 32 * PITCH;
  static constexpr int NDMA = BYTES / 1024;       // DMA instructions per tile
  static constexpr int PER_WAVE = NDMA / 4;       // of each of 4 waves
  static constexpr int LINE = D % 64 == 0 ? 16 : 8;   // chunks that the XOR permutes

  // Source of this lane's chunk of DMA instruction `instr`: row in the tile and
  // byte offset in the row.
  static __device__ inline void source(int instr, int lane, int hd, int& row, unsigned& col) {
    const unsigned p = (unsigned)(instr * 64 + lane);
    row = (int)(p / CH);
    const unsigned c = (p % CH) ^ swz<D>((unsigned)row);
    const unsigned m = c / (D / 8), d = (c % (D / 8)) * 8;
    col = (m * hd + (d < (unsigned)hd ? d : 0u)) * 2u;
  }
};

__device__ inline unsigned lds_addr(const unsigned char* p) {
  return (unsigned)(uintptr_t)(const __attribute__((address_space(3))) unsigned char*)p;
}

// 64 chunks of 16 bytes from base + off (per lane) to LDS at dst (uniform), in lane order.
// (A load to LDS may read m0 one wait state after it was written, and the compiler
// adds none inside an asm string: the s_nop.)
__device__ inline void dma16(const void* base, unsigned off, unsigned dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2"
               :: "v"(off), "s"(dst), "s"(base) : "memory", "m0");
}

__device__ inline const void* uniform(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo);
}

// At most N vector memory operations of this wave outstanding (the DMA's are
// not tracked by the compiler).
template <int N> __device__ inline void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}
// Every wave's LDS reads so far are done and every DMA it waited for is visible.
__device__ inline void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ inline Frag<bf16> lds_row(const unsigned char* p) {
  return Frag<bf16>{*reinterpret_cast<const bf16x8*>(p)};
}
__device__ inline v4i16 lds_tr(const unsigned char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4i16*)((__attribute__((address_space(3))) unsigned char*)p));
}

// Addresses of a lane in a row tile.  row(): 8 values of row l % 32 (chunk 2 s
// + l / 32 of map m) for the K-step s.  col(): column 32 t + l % 32 of the rows
// 16 c + 8 (j / 4) + 4 (l / 32) + j % 4.
template <int D> struct TileAddr {
  using R = RowTile<D>;
  static constexpr int NV = R::LINE / 2, NW = R::LINE / 4;
  unsigned r[NV], w[2][NW];
  __device__ inline void init(int lane, bool rows, bool cols) {
    const unsigned c = lane & 31, h = lane >> 5;
    if (rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) r[j] = c * R::PITCH + 16 * ((2 * j) ^ (h ^ swz<D>(c)));
    }
    if (cols) {
      const unsigned grp = lane >> 4, gi = lane & 15;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const unsigned row = 8 * jj + 4 * (grp >> 1) + (gi >> 2);
        const unsigned sub = 2 * (grp & 1) + ((gi & 3) >> 1);
#pragma unroll
        for (int v = 0; v < NW; ++v)
          w[jj][v] = row * R::PITCH + 16 * ((4 * v + sub) ^ swz<D>(row)) + 8 * (gi & 1);
      }
    }
  }
  __device__ inline Frag<bf16> row(const unsigned char* tile, int chunk0) const {   // chunk0 = chunk of half 0
    return lds_row(tile + r[(chunk0 % R::LINE) / 2] + (chunk0 / R::LINE) * (R::LINE * 16));
  }
  __device__ inline Frag<bf16> col(const unsigned char* tile, int t, int c) const {
    v4i16 x[2];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj)
      x[jj] = lds_tr(tile + w[jj][t % NW] + (t / NW) * (R::LINE * 16) + 16 * c * R::PITCH);
    return Frag<bf16>{__builtin_bit_cast(bf16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7))};
  }
};

// The larger (or the sum) of a value and its partner 32 lanes away.
__device__ inline float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float pair_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Block -> (row block, head pair, sequence): the longest causal rows first, and
// the pairs of a kv group (`grp` of `hp`) on one XCD (blocks go round the 8 XCDs),
// whose L2 then holds the group's K and V.  Where lengths differ (`mix`) each row
// block starts one XCD further, so that none has the long sequences alone (4 x 777
// tokens, lengths 777 to 0: forward 33 -> 28 us, dQ 41 -> 31).
__device__ inline void locate(int bid, int B, int hp, int grp, bool mix, int& blk, int& pair, int& b) {
  const int n = hp * B;
  blk = bid / n;
  const int u = xcd_remap((bid % n + (mix ? blk : 0)) % n, n), v = u / grp;
  b = v % B;
  pair = v / B * grp + u % grp;
}

// Two values rounded to bf16 (to nearest even), the first in the low half; and
// their place in an operand.
__device__ inline uint32_t round2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
__device__ inline void set2(Frag<bf16>& f, int i, uint32_t v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 w = __builtin_bit_cast(u32x4, f.v);
  w[i / 2] = v;
  f.v = __builtin_bit_cast(bf16x8, w);
}

// Accumulator values as operands rounded to bf16 (half a step, 2^-8) and, if FINE, what
// the rounding dropped as second operands (2^-16 left).
template <bool FINE> __device__ inline void operand(const f32x16& x, Frag<bf16> (&hi)[2], Frag<bf16> (&lo)[2]) {
  hi[0] = acc_frag<bf16>(x, 0);
  hi[1] = acc_frag<bf16>(x, 1);
  if constexpr (FINE) {
#pragma unroll
    for (int e = 0; e < 16; ++e) lo[e / 8].v[e % 8] = (__bf16)(x[e] - (float)hi[e / 8].v[e % 8]);
  }
}

// Accumulators to LDS, and added to from there; 4 KB per tile.
template <int N> __device__ inline void put_acc(const f32x16 (&x)[N], unsigned char* p, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      reinterpret_cast<float4*>(p + (n * 4 + i / 4) * 1024)[lane] = make_float4(x[n][i], x[n][i + 1], x[n][i + 2], x[n][i + 3]);
}
template <int N> __device__ inline void add_acc(f32x16 (&x)[N], const unsigned char* p, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 y = reinterpret_cast<const float4*>(p + (n * 4 + i / 4) * 1024)[lane];
      x[n][i] += y.x; x[n][i + 1] += y.y; x[n][i + 2] += y.z; x[n][i + 3] += y.w;
    }
}

// 32 rows that a wave has laid out in LDS (`pitch` bytes apart) to memory, 16
// bytes a lane and whole rows at a time: an accumulator tile's own layout would
// write 8 bytes of 32 rows per instruction.
__device__ inline void store_rows(const unsigned char* stage, int pitch, void* dst, long long ld_bytes, int row_bytes,
                                  int rows, int lane) {
  const int nch = row_bytes / 16, n = rows * nch;
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the rows are written before other lanes read them
  unsigned char* d = reinterpret_cast<unsigned char*>(dst);
  for (int i = lane; i < n; i += 64) {
    const int r = i / nch, ch = i - r * nch;
    *reinterpret_cast<uint4*>(d + r * ld_bytes + ch * 16) = *reinterpret_cast<const uint4*>(stage + r * pitch + ch * 16);
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // ... and read before they are written again
}

}  // namespace sl
