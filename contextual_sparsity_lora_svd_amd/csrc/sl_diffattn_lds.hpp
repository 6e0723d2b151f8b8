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

  // Source of this lane's chunk of the wave's DMA instruction i: row in the
  // tile and byte offset in the row.
  static __device__ inline void source(int wave, int i, int lane, int hd, int& row, unsigned& col) {
    const unsigned p = (unsigned)((wave * PER_WAVE + i) * 64 + lane);
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
__device__ inline void dma16(const void* base, unsigned off, unsigned dst) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, %2"
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

__device__ inline float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }   // subnormal results are 0

// Block -> (row block, head pair, sequence): the longest causal rows first, and
// the pairs of a kv group on one XCD (blocks go round the 8 XCDs), whose L2
// then holds the group's K and V.
__device__ inline void locate(int bid, int n, int hp, int& blk, int& pair, int& b) {
  blk = bid / n;
  const int u = xcd_remap(bid % n, n);
  b = u / hp;
  pair = u % hp;
}

// ---------------------------------------------------------------------------
// Forward.  A wave owns 32 queries and both maps: the score tiles are formed
// transposed (keys x queries), so a lane holds 16 keys of one query, the softmax
// exchanges one value per tile between the two lane halves, and the weights
// are the next product's operand as they stand; V's fragments serve both maps.
// The weights are taken relative to the maximum of the row's first tile and the
// accumulators never rescaled (fp32 and bf16 reach 2^127 alike, and a sum of at
// least 1 loses nothing to small weights).  A row whose sum passes 2^64 makes
// the workgroup go again, after a pass that finds every row's maximum.
// Rescaling as the maximum grows would put vector instructions on the
// accumulators, which then leave the matrix cores' register half every tile.
// PIPE (D > 64, one wave per SIMD): the next tile's scores are computed beside
// this tile's exponentials.  Otherwise two workgroups share a CU and their
// waves cover each other.
template <int D>
__global__ void __launch_bounds__(256, D > 64 ? 1 : 2) diff_fwd_lds(const DiffArgs a) {
  using R = RowTile<D>;
  constexpr int NT = D / 16, KS = D / 16, NST = 4, PW = R::PER_WAVE;
  constexpr bool PIPE = D > 64;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * NST * R::BYTES];
  unsigned char* const sk = smem;
  unsigned char* const sv = smem + NST * R::BYTES;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nqb = (a.L + 127) / 128;
  int blk, pair, b;
  locate(blockIdx.x, a.hp * a.B, a.hp, blk, pair, b);
  const int q0 = (nqb - 1 - blk) * 128, len = a.lens[b], g = pair / (a.hp / a.gp);
  const int row = q0 + wave * 32 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long qoff = (tok0 + row) * ldq + pair * 2 * a.hd;
  const bf16* kbase = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.k) + tok0 * ldk + g * 2 * a.hd));
  const bf16* vbase = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.v) + tok0 * ldk + g * 2 * a.hd));
  const bool rok = row < len;

  int kend = q0 < len ? len : 0, wend = q0 + wave * 32 < len ? len : 0;
  if (a.causal) {
    kend = kend < q0 + 128 ? kend : q0 + 128;
    wend = wend < q0 + wave * 32 + 32 ? wend : q0 + wave * 32 + 32;
  }
  const int nt = (kend + 31) / 32, wt = (wend + 31) / 32;      // key tiles of the workgroup, of this wave
  // tiles from here on hold keys that some query of the wave does not read
  const int wfull = a.causal ? ((q0 + wave * 32 + 1 < len ? q0 + wave * 32 + 1 : len) / 32) : len / 32;

  Frag<bf16> q[2][KS];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int col = s * 16 + h * 8;
      q[m][s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.q) + qoff + m * a.hd + col, rok && col < a.hd);
    }
  int srow[PW];
  unsigned scol[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) R::source(wave, i, lane, a.hd, srow[i], scol[i]);
  const unsigned ldb = (unsigned)ldk * 2u;
  const int last = len - 1;
  auto issue = [&](const bf16* base, unsigned char* ring, int tile) __attribute__((always_inline)) {
    const unsigned dst = __builtin_amdgcn_readfirstlane(
        lds_addr(ring) + (unsigned)((tile & (NST - 1)) * R::BYTES + wave * PW * 1024));
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      int r = tile * 32 + srow[i];
      r = r < last ? r : last;
      dma16(base, (unsigned)r * ldb + scol[i], dst + i * 1024);
    }
  };
  // group j: K of tile j + 1 (PIPE; else of tile j) and V of tile j
  auto issue_group = [&](int j) __attribute__((always_inline)) {
    issue(kbase, sk, j + (PIPE ? 1 : 0));
    issue(vbase, sv, j);
  };

  TileAddr<D> ad;
  ad.init(lane, true, true);
  f32x16 o[2][NT];
  float mx[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) zero16(o[m][t]);
  const float sc = a.scale * kLog2e;

  auto scores = [&](f32x16 (&s)[2], int tile) __attribute__((always_inline)) {
    const unsigned char* kt = sk + (tile & (NST - 1)) * R::BYTES;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      zero16(s[m]);
#pragma unroll
      for (int x = 0; x < KS; ++x) mma(s[m], ad.row(kt, m * (D / 8) + 2 * x), q[m][x]);
    }
  };
  auto mask = [&](f32x16 (&s)[2], int tile) __attribute__((always_inline)) {
    const int lim = a.causal && row + 1 < len ? row + 1 : len;   // keys this query reads
    const int k0 = tile * 32 + 4 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool hidden = k0 + 8 * (i >> 2) + (i & 3) >= lim;
      s[0][i] = hidden ? -INFINITY : s[0][i];
      s[1][i] = hidden ? -INFINITY : s[1][i];
    }
  };
  auto tile_max = [&](const f32x16& s) __attribute__((always_inline)) {
    float t = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) t = fmaxf(t, s[i]);
    return pair_max(t);
  };
  auto weights = [&](f32x16& s, int m) __attribute__((always_inline)) {
    const float ms = mx[m] * sc;
    float ts = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = fast_exp2(fmaf(s[i], sc, -ms));
      ts += s[i];
    }
    sum[m] += ts;
  };
  auto values = [&](const Frag<bf16> (&p)[2][2], int tile) __attribute__((always_inline)) {
    const unsigned char* vt = sv + (tile & (NST - 1)) * R::BYTES;
#pragma unroll
    for (int cc = 0; cc < 2; ++cc)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Frag<bf16> vf = ad.col(vt, t, cc);
        mma(o[0][t], vf, p[0][cc]);
        mma(o[1][t], vf, p[1][cc]);
      }
  };

  // one tile's step: weights of tile i, scores of tile i + 1 (PIPE) or i
  auto step = [&](f32x16 (&s)[2], int i) __attribute__((always_inline)) {
    f32x16 nx[2];
    Frag<bf16> p[2][2];
    if constexpr (PIPE) {
      scores(nx, i + 1);
    } else {
      scores(s, i);
      if (i >= wfull) mask(s, i);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      weights(s[m], m);
      p[m][0] = acc_frag<bf16>(s[m], 0);
      p[m][1] = acc_frag<bf16>(s[m], 1);
    }
    values(p, i);
    if constexpr (PIPE) {
      if (i + 1 >= wfull) mask(nx, i + 1);
      s[0] = nx[0];
      s[1] = nx[1];
    }
  };
  auto advance = [&](int i) __attribute__((always_inline)) {
    wait_vm<4 * PW>();            // group i has landed, i + 1 and i + 2 may be in flight
    lds_barrier();                // ... for every wave, and all are done with group i - 1
    issue_group(i + 3);           // past the last tile: rows of the end again, read by none
  };
  for (bool exact = false;; exact = true) {
    float big = 0.f;
    if (nt > 0) {
      f32x16 s[2];
      if (exact) {
        for (int i = 0; i < nt; ++i) {
          issue(kbase, sk, i);
          wait_vm<0>();
          lds_barrier();
          if (i < wt) {
            scores(s, i);
            if (i >= wfull) mask(s, i);
#pragma unroll
            for (int m = 0; m < 2; ++m) mx[m] = i == 0 ? tile_max(s[m]) : fmaxf(mx[m], tile_max(s[m]));
          }
        }
        lds_barrier();
      }
      if constexpr (PIPE) issue(kbase, sk, 0);
      issue_group(0);
      issue_group(1);
      issue_group(2);
      if (PIPE || !exact) {
        if constexpr (PIPE) wait_vm<6 * PW>();
        else wait_vm<4 * PW>();
        lds_barrier();
        scores(s, 0);
        if (wfull <= 0) mask(s, 0);
        if (!exact) {
          mx[0] = tile_max(s[0]);
          mx[1] = tile_max(s[1]);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        sum[m] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) zero16(o[m][t]);
      }
      for (int i = 0; i < wt; ++i) {
        advance(i);
        step(s, i);
      }
      for (int i = wt; i < nt; ++i) advance(i);
      wait_vm<0>();               // no DMA outlives the sweep
      big = fmaxf(pair_sum(sum[0]), pair_sum(sum[1]));
      if (sum[0] != sum[0] || sum[1] != sum[1]) big = INFINITY;
    }
    if (exact) break;
    if (!__any(rok && !(big < 0x1p64f))) big = 0.f;
    lds_barrier();
    if (lane == 0) reinterpret_cast<float*>(smem)[wave] = big;
    lds_barrier();
    const float4 w = *reinterpret_cast<const float4*>(smem);
    lds_barrier();
    if (w.x + w.y + w.z + w.w == 0.f) break;
  }

  float e1, e2;
  const float lam = lambda_of(a, e1, e2);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.lam[0] = lam;
    a.lam[1] = e1;
    a.lam[2] = e2;
  }
  float inv[2], st[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float l = pair_sum(sum[m]);
    inv[m] = rok ? 1.f / l : 0.f;
    st[m] = rok ? mx[m] * sc + __log2f(l) : INFINITY;
  }
  // O_2 and the part of O that its bf16 rounding drops, to 16 and 8 bits of the
  // row's largest: with them D_m = dO . (P_m V) is exact to 2^-16 in the
  // backward, where an error of D would add up over the whole row of keys
  float big2 = 0.f, bigr = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool in = (32 * t) % D + 8 * (i >> 2) + 4 * h < a.hd;   // 4 neighbours are in or out together
      const float y = rok && in ? o[1][t][i] * inv[1] : 0.f;
      const float x = rok && in ? fmaf(-lam, y, o[0][t][i] * inv[0]) : 0.f;
      o[1][t][i] = y;
      o[0][t][i] = x;
      big2 = fmaxf(big2, fabsf(y));
      bigr = fmaxf(bigr, fabsf(x - bf2f(f2bf(x))));
    }
  big2 = pair_max(big2);
  bigr = pair_max(bigr);
  if (row >= a.L) return;
  if (h == 0) {
    const long long at = (long long)(b * a.hp + pair) * 2 * a.L + row;
    a.lse[at] = st[0];
    a.lse[at + a.L] = st[1];
    a.rsc[at] = bigr / 127.f;
    a.rsc[at + a.L] = big2 / 32767.f;
  }
  const float f2 = big2 > 0.f ? 32767.f / big2 : 0.f, fr = bigr > 0.f ? 127.f / bigr : 0.f;
  bf16* op = reinterpret_cast<bf16*>(a.o) + qoff;
  short* o2p = reinterpret_cast<short*>(a.o2) + qoff;
  signed char* rp = a.res + qoff;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      // V's tile has D columns per half, hd of them in use
      const int e0 = (32 * t) % D + 2 * i + 4 * h, dv = 32 * t / D * a.hd + e0;
      if (e0 >= a.hd) continue;
      uint32_t r4 = 0;
      short y4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = o[0][t][i + e];
        y4[e] = (short)__float2int_rn(o[1][t][i + e] * f2);
        r4 |= ((uint32_t)__float2int_rn((x - bf2f(f2bf(x))) * fr) & 0xFFu) << (8 * e);
      }
      store4<bf16>(op + dv, o[0][t][i], o[0][t][i + 1], o[0][t][i + 2], o[0][t][i + 3]);
      *reinterpret_cast<uint2*>(o2p + dv) =
          make_uint2((uint16_t)y4[0] | ((uint32_t)(uint16_t)y4[1] << 16), (uint16_t)y4[2] | ((uint32_t)(uint16_t)y4[3] << 16));
      *reinterpret_cast<uint32_t*>(rp + dv) = r4;
    }
}

// ---------------------------------------------------------------------------
// dQ.  As the forward: a wave owns 32 queries (their rows of Q and dO are held
// in registers) and walks the key tiles, scores and dP = V dO^T transposed, so
// that P and dS stay where they are formed.  K's tile is read twice, by rows
// for the scores and by columns for dQ^T += K^T dS^T.
template <int D>
__global__ void __launch_bounds__(256, D > 64 ? 1 : 2) diff_dq_lds(const DiffArgs a) {
  using R = RowTile<D>;
  constexpr int DT = D / 32, KS = D / 16, NST = 4, PW = R::PER_WAVE;
  constexpr bool PIPE = D > 64;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * NST * R::BYTES];
  unsigned char* const sk = smem;
  unsigned char* const sv = smem + NST * R::BYTES;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nqb = (a.L + 127) / 128;
  int blk, pair, b;
  locate(blockIdx.x, a.hp * a.B, a.hp, blk, pair, b);
  const int q0 = (nqb - 1 - blk) * 128, len = a.lens[b], g = pair / (a.hp / a.gp);
  const int row = q0 + wave * 32 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long qoff = (tok0 + row) * ldq + pair * 2 * a.hd;
  const bf16* kbase = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.k) + tok0 * ldk + g * 2 * a.hd));
  const bf16* vbase = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.v) + tok0 * ldk + g * 2 * a.hd));
  const bool rok = row < len;
  int kend = q0 < len ? len : 0, wend = q0 + wave * 32 < len ? len : 0;
  if (a.causal) {
    kend = kend < q0 + 128 ? kend : q0 + 128;
    wend = wend < q0 + wave * 32 + 32 ? wend : q0 + wave * 32 + 32;
  }
  const int nt = (kend + 31) / 32, wt = (wend + 31) / 32;
  const int wfull = a.causal ? ((q0 + wave * 32 + 1 < len ? q0 + wave * 32 + 1 : len) / 32) : len / 32;
  const float lam = a.lam[0];

  Frag<bf16> q[2][KS], go[2 * KS];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int col = s * 16 + h * 8;
      const bool ok = rok && col < a.hd;
      q[m][s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.q) + qoff + m * a.hd + col, ok);
      // dO's columns follow the tile's: D per half, hd of them in use
      go[m * KS + s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.da) + qoff + m * a.hd + col, ok);
    }
  float lse[2], ds[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const long long at = ((long long)(b * a.hp + pair) * 2 + m) * a.L + row;
    lse[m] = rok ? a.lse[at] : INFINITY;      // weights of rows past the end: 0
    ds[m] = rok ? a.dsum[at] : 0.f;
  }
  int srow[PW];
  unsigned scol[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) R::source(wave, i, lane, a.hd, srow[i], scol[i]);
  const unsigned ldb = (unsigned)ldk * 2u;
  const int last = len - 1;
  auto issue_tile = [&](int tile) __attribute__((always_inline)) {
    const unsigned d0 = __builtin_amdgcn_readfirstlane((unsigned)((tile & (NST - 1)) * R::BYTES + wave * PW * 1024));
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      int r = tile * 32 + srow[i];
      r = r < last ? r : last;
      const unsigned off = (unsigned)r * ldb + scol[i];
      dma16(kbase, off, lds_addr(sk) + d0 + i * 1024);
      dma16(vbase, off, lds_addr(sv) + d0 + i * 1024);
    }
  };

  TileAddr<D> ad;
  ad.init(lane, true, true);
  f32x16 dq[2][DT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dq[m][t]);
  const float sc = a.scale * kLog2e;
  double dlam = 0.0;

  auto scores = [&](f32x16 (&s)[2], f32x16& dp, int tile) __attribute__((always_inline)) {
    const unsigned char* kt = sk + (tile & (NST - 1)) * R::BYTES;
    const unsigned char* vt = sv + (tile & (NST - 1)) * R::BYTES;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      zero16(s[m]);
#pragma unroll
      for (int x = 0; x < KS; ++x) mma(s[m], ad.row(kt, m * (D / 8) + 2 * x), q[m][x]);
    }
    zero16(dp);
#pragma unroll
    for (int x = 0; x < 2 * KS; ++x) mma(dp, ad.row(vt, 2 * x), go[x]);
  };
  auto mask = [&](f32x16 (&s)[2], int tile) __attribute__((always_inline)) {
    const int lim = a.causal && row + 1 < len ? row + 1 : len;
    const int k0 = tile * 32 + 4 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool hidden = k0 + 8 * (i >> 2) + (i & 3) >= lim;
      s[0][i] = hidden ? -INFINITY : s[0][i];
      s[1][i] = hidden ? -INFINITY : s[1][i];
    }
  };
  // S and dP of a tile -> dS of both maps
  auto grads = [&](f32x16 (&s)[2], const f32x16& dp) __attribute__((always_inline)) {
    float part = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = fast_exp2(fmaf(s[m][i], sc, -lse[m]));
        if (m == 1) part = fmaf(p, dp[i], part);
        s[m][i] = p * (dp[i] - ds[m]);
      }
    dlam += (double)part;
  };
  auto accumulate = [&](const f32x16 (&s)[2], int tile) __attribute__((always_inline)) {
    const unsigned char* kt = sk + (tile & (NST - 1)) * R::BYTES;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const Frag<bf16> sf = acc_frag<bf16>(s[m], cc);
#pragma unroll
        for (int t = 0; t < DT; ++t) mma(dq[m][t], ad.col(kt, m * DT + t, cc), sf);
      }
  };

  if (nt > 0) {
    // PIPE: tile i + 1's products run in iteration i, which still needs K of tile i
    constexpr int AHEAD = PIPE ? 1 : 0;
    f32x16 s[2], dp;
    if constexpr (PIPE) issue_tile(0);
    issue_tile(AHEAD);
    issue_tile(AHEAD + 1);
    if constexpr (PIPE) {
      wait_vm<4 * PW>();
      lds_barrier();
      scores(s, dp, 0);
      if (wfull <= 0) mask(s, 0);
    }
    auto advance = [&](int i) __attribute__((always_inline)) {
      wait_vm<2 * PW>();          // tile i + AHEAD has landed
      lds_barrier();
      issue_tile(i + AHEAD + 2);  // into the slot of tile i - 1 or i - 2
    };
    for (int i = 0; i < wt; ++i) {
      advance(i);
      f32x16 nx[2], ndp;
      if constexpr (PIPE) {
        scores(nx, ndp, i + 1);
      } else {
        scores(s, dp, i);
        if (i >= wfull) mask(s, i);
      }
      grads(s, dp);
      accumulate(s, i);
      if constexpr (PIPE) {
        if (i + 1 >= wfull) mask(nx, i + 1);
        s[0] = nx[0];
        s[1] = nx[1];
        dp = ndp;
      }
    }
    for (int i = wt; i < nt; ++i) advance(i);
    wait_vm<0>();
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) dlam += __shfl_xor(dlam, o);
  if (lane == 0) a.dlam_part[blockIdx.x * 4 + wave] = dlam;
  if (row >= a.L) return;
  bf16* out = reinterpret_cast<bf16*>(a.dq) + qoff;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float f = m ? -lam * a.scale : a.scale;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d >= a.hd) continue;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = rok ? dq[m][t][i + e] * f : 0.f;
        store4<bf16>(out + m * a.hd + d, x[0], x[1], x[2], x[3]);
      }
  }
}

// ---------------------------------------------------------------------------
// dK and dV.  A wave owns 32 keys (K's rows in registers; V's rows in registers
// up to D = 64, else in LDS) and walks the query tiles of its group's heads:
// scores and dP = dO V^T with a key per lane, then dV^T += dO^T (P_1 - lambda P_2)
// and dK_m^T += Q_m^T dS_m with the tile's rows read by columns.  A key's column
// never meets another's, so keys past the end need no mask: their results are
// written as 0.  The heads of a group are cut into `split` parts where one
// workgroup per key block would leave CUs idle; the parts' sums are then fp32
// and diff_dkv_sum adds them in order.
template <int D>
__global__ void __launch_bounds__(256, 1) diff_dkv_lds(const DiffArgs a) {
  using R = RowTile<D>;
  constexpr int DT = D / 32, NT = D / 16, KS = D / 16, NST = 2, PW = R::PER_WAVE;
  constexpr bool VREG = D <= 64;
  constexpr int STAT = 4 * 64 * 4;      // lse and D of both maps for 64 rows (32 in use)
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * NST * R::BYTES + (VREG ? 0 : 4 * R::BYTES) + NST * STAT];
  unsigned char* const sq = smem;
  unsigned char* const sg = smem + NST * R::BYTES;
  unsigned char* const sv = smem + 2 * NST * R::BYTES;
  unsigned char* const ss = sv + (VREG ? 0 : 4 * R::BYTES);
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int blk, gs, b;
  locate(blockIdx.x, a.gp * a.split * a.B, a.gp * a.split, blk, gs, b);
  const int g = gs / a.split, part = gs % a.split;
  const int grp = a.hp / a.gp, nh = grp / a.split, len = a.lens[b];
  const int k0 = blk * 128, key = k0 + wave * 32 + c;           // causal: the first keys have the most queries
  const bool kok = key < len;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long koff = (tok0 + key) * ldk + g * 2 * a.hd;
  const float lam = a.lam[0];
  const int pr0 = g * grp + part * nh;
  const int t0 = a.causal ? k0 / 32 : 0;                        // first query tile
  const int ntile = k0 < len ? (len + 31) / 32 - t0 : 0, total = ntile * nh;

  int srow[PW];
  unsigned scol[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) R::source(wave, i, lane, a.hd, srow[i], scol[i]);
  const int last = len - 1;
  Frag<bf16> kf[2][KS], vf[VREG ? 2 * KS : 1];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int col = s * 16 + h * 8;
      const bool ok = kok && col < a.hd;
      kf[m][s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.k) + koff + m * a.hd + col, ok);
      if constexpr (VREG) vf[m * KS + s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.v) + koff + m * a.hd + col, ok);
    }
  if constexpr (!VREG) {
    // the workgroup's 128 rows of V, zeros where dO's tile repeats columns
    for (int i = threadIdx.x; i < 128 * R::CH; i += 256) {
      const int r = i / R::CH, p = i % R::CH, cl = p ^ (int)swz<D>((unsigned)r & 31);
      const int m = cl / (D / 8), d = (cl % (D / 8)) * 8;
      const bool ok = k0 + r < len && d < a.hd;
      const Frag<bf16> x = load_row<bf16>(reinterpret_cast<const bf16*>(a.v) + (tok0 + k0 + r) * ldk + g * 2 * a.hd + m * a.hd + d, ok);
      *reinterpret_cast<bf16x8*>(sv + r * R::PITCH + p * 16) = x.v;
    }
  }
  const unsigned ldb = (unsigned)ldq * 2u;
  int it_pr = pr0, it_t = t0;                                   // the next tile to load
  // statistics: wave w loads lse (w < 2) or D of map w % 2, 64 rows
  const float* const sbase = (wave < 2 ? a.lse : a.dsum) + (long long)b * a.hp * 2 * a.L + (wave & 1) * a.L;
  auto issue_next = [&](int it) __attribute__((always_inline)) {
    const unsigned d0 = __builtin_amdgcn_readfirstlane((unsigned)((it & 1) * R::BYTES + wave * PW * 1024));
    const bf16* qb = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.q) + tok0 * ldq + it_pr * 2 * a.hd));
    const bf16* gb = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.da) + tok0 * ldq + it_pr * 2 * a.hd));
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      int r = it_t * 32 + srow[i];
      r = r < last ? r : last;
      const unsigned off = (unsigned)r * ldb + scol[i];
      dma16(qb, off, lds_addr(sq) + d0 + i * 1024);
      dma16(gb, off, lds_addr(sg) + d0 + i * 1024);
    }
    int r = it_t * 32 + lane;
    r = r < last ? r : last;
    const float* sb = reinterpret_cast<const float*>(uniform(sbase + (long long)it_pr * 2 * a.L));
    const unsigned sd = __builtin_amdgcn_readfirstlane(lds_addr(ss) + (unsigned)((it & 1) * STAT + wave * 256));
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, %2"
                 :: "v"((unsigned)r * 4u), "s"(sd), "s"(sb) : "memory", "m0");
    if (++it_t == t0 + ntile) {
      it_t = t0;
      if (it_pr + 1 < pr0 + nh) ++it_pr;                        // past the last: read again, used by none
    }
  };

  TileAddr<D> ad;
  ad.init(lane, true, true);
  f32x16 dk[2][DT], dv[NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dk[m][t]);
#pragma unroll
  for (int t = 0; t < NT; ++t) zero16(dv[t]);
  const float sc = a.scale * kLog2e;

  if (total > 0) {
    issue_next(0);
    int it = 0;
    auto advance = [&]() __attribute__((always_inline)) {
      wait_vm<0>();               // tile `it` has landed
      lds_barrier();              // ... for every wave, and the other slot is read by none
      issue_next(it + 1);
    };
    const int skip = a.causal ? (wave < ntile ? wave : ntile) : 0;   // tiles before this wave's keys
    for (int n = 0; n < nh; ++n) {
      for (int j = 0; j < skip; ++j, ++it) advance();
      for (int j = skip; j < ntile; ++j, ++it) {
        advance();
        const int q0 = (t0 + j) * 32;
        const unsigned char* qt = sq + (it & 1) * R::BYTES;
        const unsigned char* gt = sg + (it & 1) * R::BYTES;
        const float* st = reinterpret_cast<const float*>(ss + (it & 1) * STAT);
        f32x16 dp, s, w;
        zero16(dp);
#pragma unroll
        for (int x = 0; x < 2 * KS; ++x) {
          if constexpr (VREG) mma(dp, ad.row(gt, 2 * x), vf[x]);
          else mma(dp, ad.row(gt, 2 * x), ad.row(sv + wave * R::BYTES, 2 * x));
        }
        const bool masked = q0 + 32 > len || (a.causal && q0 < k0 + wave * 32 + 31);
        const int first = a.causal ? key : 0;                   // queries that read this key: first .. len - 1
        Frag<bf16> df[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          zero16(s);
#pragma unroll
          for (int x = 0; x < KS; ++x) mma(s, ad.row(qt, m * (D / 8) + 2 * x), kf[m][x]);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(st + m * 64 + 2 * i + 4 * h);
            const float4 d4 = *reinterpret_cast<const float4*>(st + (2 + m) * 64 + 2 * i + 4 * h);
            const float le[4] = {l4.x, l4.y, l4.z, l4.w}, de[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float p = fast_exp2(fmaf(s[i + e], sc, -le[e]));
              if (masked) {
                const int qr = q0 + 2 * i + 4 * h + e;
                p = qr < first || qr >= len ? 0.f : p;
              }
              w[i + e] = m ? fmaf(-lam, p, w[i + e]) : p;
              s[i + e] = p * (dp[i + e] - de[e]);
            }
          }
          df[m][0] = acc_frag<bf16>(s, 0);
          df[m][1] = acc_frag<bf16>(s, 1);
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const Frag<bf16> wf = acc_frag<bf16>(w, cc);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(dv[t], ad.col(gt, t, cc), wf);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < DT; ++t) mma(dk[m][t], ad.col(qt, m * DT + t, cc), df[m][cc]);
        }
      }
    }
    wait_vm<0>();
  }
  if (key >= a.L) return;
  const long long pofs = (long long)part * a.B * a.L * ldk + koff;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int e = (32 * t) % D + 2 * i + 4 * h, m = 32 * t / D;
      if (e >= a.hd) continue;
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = kok ? dv[t][i + j] : 0.f;
      if (a.split > 1) store4<float>(a.dv_part + pofs + m * a.hd + e, x[0], x[1], x[2], x[3]);
      else store4<bf16>(reinterpret_cast<bf16*>(a.dv) + koff + m * a.hd + e, x[0], x[1], x[2], x[3]);
    }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float f = m ? -lam * a.scale : a.scale;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d >= a.hd) continue;
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = kok ? dk[m][t][i + j] * f : 0.f;
        if (a.split > 1) store4<float>(a.dk_part + pofs + m * a.hd + d, x[0], x[1], x[2], x[3]);
        else store4<bf16>(reinterpret_cast<bf16*>(a.dk) + koff + m * a.hd + d, x[0], x[1], x[2], x[3]);
      }
  }
}

// dK and dV from the parts' sums, in order; 4 values per thread.
__global__ void __launch_bounds__(256) diff_dkv_sum(const DiffArgs a) {
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
  store4<bf16>(reinterpret_cast<bf16*>(v ? a.dv : a.dk) + 4 * i, x.x, x.y, x.z, x.w);
}

// D_1 = dO . (O + lambda O_2) and D_2 = dO . O_2 from the saved integers.  LP
// lanes (a power of two) per row and head pair, 8 values each.
__global__ void __launch_bounds__(256) diff_dsum_q(const DiffArgs a, int lp_log2) {
  const int lp = 1 << lp_log2, sub = threadIdx.x & (lp - 1);
  const long long n = (long long)a.B * a.L * a.hp;
  const float lam = a.lam[0];
  const long long w = ((long long)blockIdx.x * 256 + threadIdx.x) >> lp_log2;
  const bool on = w < n;
  const int pair = on ? (int)(w % a.hp) : 0;
  const long long tok = on ? w / a.hp : 0;
  const int b = (int)(tok / a.L), row = (int)(tok % a.L);
  const long long st = (long long)(b * a.hp + pair) * 2 * a.L + row;
  float d1 = 0.f, d2 = 0.f, r1 = 0.f;
  if (on && row < a.lens[b] && 8 * sub < 2 * a.hd) {
    const long long at = (tok * a.hp + pair) * 2 * a.hd + 8 * sub;
    const uint4 gv = *reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.da) + at);
    const uint4 ov = *reinterpret_cast<const uint4*>(reinterpret_cast<const bf16*>(a.a) + at);
    const uint4 yv = *reinterpret_cast<const uint4*>(reinterpret_cast<const short*>(a.o2) + at);
    const uint2 rv = *reinterpret_cast<const uint2*>(a.res + at);
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, ow[4] = {ov.x, ov.y, ov.z, ov.w}, yw[4] = {yv.x, yv.y, yv.z, yv.w};
    const uint32_t rw[2] = {rv.x, rv.y};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gx = bf2f((uint16_t)(gw[j >> 1] >> (16 * (j & 1)))), ox = bf2f((uint16_t)(ow[j >> 1] >> (16 * (j & 1))));
      const float y = (float)(short)(yw[j >> 1] >> (16 * (j & 1)));
      const float r = (float)(signed char)(rw[j >> 2] >> (8 * (j & 3)));
      d1 = fmaf(gx, ox, d1);
      r1 = fmaf(gx, r, r1);
      d2 = fmaf(gx, y, d2);
    }
    d2 *= a.rsc[st + a.L];
    d1 = fmaf(r1, a.rsc[st], d1);
    d1 = fmaf(lam, d2, d1);
  }
  for (int o = lp >> 1; o; o >>= 1) {
    d1 += __shfl_xor(d1, o);
    d2 += __shfl_xor(d2, o);
  }
  if (on && sub == 0) {
    a.dsum[st] = d1;
    a.dsum[st + a.L] = d2;
  }
}

}  // namespace sl
