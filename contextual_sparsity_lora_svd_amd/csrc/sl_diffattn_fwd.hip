// Differential attention: forward kernels.
#include "sl_diffattn_lds.hpp"

namespace sl {

// ---------------------------------------------------------------------------
// Forward.  A workgroup of 8 waves owns 128 queries of a head pair; a wave owns
// 32 of them and one map (both maps' accumulators of 2 D columns would leave no
// registers for a second wave on the SIMD).  The score tiles are formed
// transposed (keys x queries), so a lane holds 16 keys of one query: the weights
// are the next product's operand as they stand and nothing is exchanged
// between lanes.
//
// The weights are taken relative to the maximum of the row's first tile and the
// accumulators never rescaled (fp32 and bf16 reach 2^127 alike, and a sum of at
// least 1 loses nothing to small weights).  A row whose sum passes 2^64 makes
// the workgroup go again, after a pass that finds every row's maximum.
//
// The weights are rounded to bf16 for the matrix cores (half a step, 2^-8), in short
// sequences to the sum of two (FINE; where and why: kFineRows); their sum is not.
//
// Bound by the matrix cores and, beside them, the issue of two waves' other
// instructions: 1 x 4096 tokens, 32 heads, 8 kv, of 128, take 375 to 404
// us (1100 to 1020 TFLOP/s, where a large product reaches 1144 to 1244), causal 198, and
// 220 to 232 in the first milliseconds after the GPU was idle.
//
// RB blocks of 32 queries per workgroup.  Four, with tiles loaded two ahead, move
// the fewest bytes.  Two, loaded one ahead, leave room for a second workgroup on
// the CU: causal ones of very different lengths then share it, a long one with a
// short one (they are dispatched in that order), and the long one has the SIMDs to
// itself once the other is done; and where there is no second one, it has them
// from the start: taken while the 128-row workgroups are no more than one round of
// 256 (causal), or the 64-row ones (not causal).  Measured with four / two, heads of
// 128 (128-row workgroups in brackets), causal: 4 x 512 tokens of 32 heads (256) 52 / 49 us,
// of 48 (384) 71 / 73, 2 x 1024 of 32 (256) 67 / 62, 2 x 1280 of 32 (320) 77 / 82, 1 x 2048 of
// 8 (64) 82 / 65, of 32 (256) 97 / 89, of 48 (384) 111 / 125, 1 x 4096 of 16 (256) 160 / 144,
// of 24 (384) 181 / 200, of 32 (512) 217 / 253; not causal, 1 x 1024 of 32 (128) 62 / 57, 1 x
// 1280 of 32 (160) 70 / 81, 1 x 2048 of 32 (256) 115 / 126.
template <int D, int RB, bool FINE>
__global__ void __launch_bounds__(RB * 128, 2) diff_fwd_lds(const DiffArgs a) {
  using R = RowTile<D>;
  constexpr int NT = D / 16, KS = D / 16, WAVES = 2 * RB, ROWS = 32 * RB;
  constexpr int NST = RB == 4 ? 4 : 2, DIST = NST / 2;    // tiles in the ring, tiles loaded ahead
  constexpr int PW = (R::NDMA + WAVES - 1) / WAVES;       // DMA per wave; the last may be issued twice
  constexpr int P2 = 4 * D + 16, P1 = 2 * D + 16;         // staged result rows: 2-byte and 1-byte values
  constexpr int STAGED = WAVES * 32 * P2;
  constexpr int RING = 2 * NST * R::BYTES > STAGED ? 2 * NST * R::BYTES : STAGED;
  static_assert(RB * NT * 4096 <= RING, "four waves' P_2 V fit the ring");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[RING + 64];
  unsigned char* const sk = smem;
  unsigned char* const sv = smem + NST * R::BYTES;
  float* const slam = reinterpret_cast<float*>(smem + RING);
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = wave / RB, rb = wave % RB;                // map, block of 32 rows
  const int nqb = (a.L + ROWS - 1) / ROWS;
  int blk, pair, b;
  locate(blockIdx.x, a.B, a.hp, a.hp / a.gp, a.mix, blk, pair, b);
  // the longest rows first; with two workgroups to a CU, the second half of the
  // blocks the other way round
  if (RB == 2 && 2 * blk >= nqb) blk = nqb - 1 - (blk - (nqb + 1) / 2);
  const int q0 = (nqb - 1 - blk) * ROWS, len = a.lens[b], g = pair / (a.hp / a.gp);
  const int row0 = q0 + rb * 32, row = row0 + c;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long qoff = (tok0 + row) * ldq + pair * 2 * a.hd;
  const bf16* kbase = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.k) + tok0 * ldk + g * 2 * a.hd));
  const bf16* vbase = reinterpret_cast<const bf16*>(uniform(reinterpret_cast<const bf16*>(a.v) + tok0 * ldk + g * 2 * a.hd));
  const bool rok = row < len;

  int kend = q0 < len ? len : 0, wend = row0 < len ? len : 0;
  if (a.causal) {
    kend = kend < q0 + ROWS ? kend : q0 + ROWS;
    wend = wend < row0 + 32 ? wend : row0 + 32;
  }
  const int nt = (kend + 31) / 32, wt = (wend + 31) / 32;      // key tiles of the workgroup, of this wave
  // tiles from here on hold keys that some query of the wave does not read
  const int wfull = (a.causal && row0 + 1 < len ? row0 + 1 : len) / 32;

  Frag<bf16> q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int col = s * 16 + h * 8;
    q[s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.q) + qoff + m * a.hd + col, rok && col < a.hd);
  }
  int srow[PW], sins[PW];
  unsigned scol[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) {
    sins[i] = wave * PW + i < R::NDMA ? wave * PW + i : R::NDMA - 1;
    R::source(sins[i], lane, a.hd, srow[i], scol[i]);
  }
  const unsigned ldb = (unsigned)ldk * 2u;
  const int last = len - 1;
  auto issue_part = [&](const bf16* base, unsigned char* ring, int tile, int i) __attribute__((always_inline)) {
    int r = tile * 32 + srow[i];
    r = r < last ? r : last;
    dma16(base, (unsigned)r * ldb + scol[i],
          __builtin_amdgcn_readfirstlane(lds_addr(ring) + (unsigned)((tile & (NST - 1)) * R::BYTES + sins[i] * 1024)));
  };
  auto issue = [&](const bf16* base, unsigned char* ring, int tile) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PW; ++i) issue_part(base, ring, tile, i);
  };
  // group j: V of tile j, K of the tile after it
  auto issue_group = [&](int j) __attribute__((always_inline)) {
    issue(kbase, sk, j + 1);
    issue(vbase, sv, j);
  };

  TileAddr<D> ad;
  ad.init(lane, false, true);
  unsigned kx[KS];                // this wave's map in a row of K
#pragma unroll
  for (int x = 0; x < KS; ++x)
    kx[x] = (unsigned)c * R::PITCH + 16 * (((unsigned)(m * (D / 8) + 2 * x) + h) ^ swz<D>((unsigned)c));
  f32x16 o[NT];
  float mx = 0.f, sum = 0.f, rest = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) zero16(o[t]);
  const float sc = a.scale * kLog2e;

  auto scores = [&](f32x16& s, int tile) __attribute__((always_inline)) {
    const unsigned char* kt = sk + (tile & (NST - 1)) * R::BYTES;
    zero16(s);
#pragma unroll
    for (int x = 0; x < KS; ++x) mma(s, lds_row(kt + kx[x]), q[x]);
  };
  auto mask = [&](f32x16& s, int tile) __attribute__((always_inline)) {
    const int lim = a.causal && row + 1 < len ? row + 1 : len;   // keys this query reads
    const int k0 = tile * 32 + 4 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = k0 + 8 * (i >> 2) + (i & 3) >= lim ? -INFINITY : s[i];
  };
  auto tile_max = [&](const f32x16& s) __attribute__((always_inline)) {
    float t = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) t = fmaxf(t, s[i]);
    return pair_max(t);
  };

  if (wave == 0) {
    float e1, e2;
    const float lam = lambda_of(a, e1, e2);
    if (lane == 0) {
      slam[0] = lam;
      if (blockIdx.x == 0) {
        a.lam[0] = lam;
        a.lam[1] = e1;
        a.lam[2] = e2;
      }
    }
  }
  for (bool exact = false;; exact = true) {
    float big = 0.f;
    if (nt > 0) {
      f32x16 s;
      if (exact) {
        for (int i = 0; i < nt; ++i) {
          issue(kbase, sk, i);
          wait_vm<0>();
          lds_barrier();
          if (i < wt) {
            scores(s, i);
            if (i >= wfull) mask(s, i);
            mx = i == 0 ? tile_max(s) : fmaxf(mx, tile_max(s));
          }
        }
        lds_barrier();
      }
      issue(kbase, sk, 0);
      issue_group(0);
      if constexpr (DIST == 2) issue_group(1);
      wait_vm<2 * DIST * PW>();
      lds_barrier();
      scores(s, 0);
      if (wfull <= 0) mask(s, 0);
      if (!exact) mx = tile_max(s);
      sum = rest = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t) zero16(o[t]);
      // after it, tile n's step (or the wave's wait for the others) loads group
      // n + DIST; past the last tile that is rows of the end again, read by none
      auto arrive = [&]() __attribute__((always_inline)) {
        wait_vm<2 * (DIST - 1) * PW>();   // group n has landed, a later one may be in flight
        lds_barrier();                    // ... for every wave, and all are done with group n - 1
      };
      // A tile's step in a fixed order: the next tile's scores, then the values
      // times the first and the second half of the weights; each operand is read
      // from LDS AHEAD products before its use, and the exponentials of a half
      // stand between the products before it.
      constexpr int NG = KS + 2 * NT, AHEAD = 2;
      auto step = [&](int i, auto masked) __attribute__((always_inline)) {
        const unsigned char* vt = sv + (i & (NST - 1)) * R::BYTES;
        const unsigned char* kt = sk + ((i + 1) & (NST - 1)) * R::BYTES;
        f32x16 nx;
        Frag<bf16> p[2], lo[2], fa[AHEAD];
        const float ms = mx * sc;
        float ts = 0.f;
        zero16(nx);
        auto read = [&](auto gc) __attribute__((always_inline)) {
          constexpr int g = decltype(gc)::value, x = g % AHEAD;
          if constexpr (g < KS) fa[x] = lds_row(kt + kx[g]);
          else if constexpr (g < NG) fa[x] = ad.col(vt, (g - KS) % NT, (g - KS) / NT);
        };
        auto weigh = [&](int half, int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
          for (int e = e0; e < e1; ++e) {
            const float w = fast_exp2(fmaf(s[8 * half + e], sc, -ms));
            ts += w;
            p[half].v[e] = (__bf16)w;
            if constexpr (FINE) lo[half].v[e] = (__bf16)(w - (float)p[half].v[e]);
          }
        };
        each<AHEAD>(read);
        each<NG>([&](auto gc) __attribute__((always_inline)) {
          constexpr int g = decltype(gc)::value;
          if constexpr (g < KS) mma(nx, fa[g % AHEAD], q[g]);
          else mma(o[(g - KS) % NT], fa[g % AHEAD], p[(g - KS) / NT]);
          if constexpr (FINE && g >= KS) mma(o[(g - KS) % NT], fa[g % AHEAD], lo[(g - KS) / NT]);
          read(std::integral_constant<int, g + AHEAD>{});
          if constexpr (g % 2 == 1 && g / 2 < PW) {
            issue_part(kbase, sk, i + DIST + 1, g / 2);
            issue_part(vbase, sv, i + DIST, g / 2);
          }
          if constexpr (g < KS) weigh(0, 8 * g / KS, 8 * (g + 1) / KS);
          else if constexpr (g < KS + NT) weigh(1, 8 * (g - KS) / NT, 8 * (g - KS + 1) / NT);
          __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (decltype(masked)::value) mask(nx, i + 1);   // (past the last tile: unused)
        // the tiles' sums, with what each addition dropped
        const float both = sum + ts;
        rest += ts - (both - sum);
        sum = both;
        s = nx;
      };
      int i = 0;
      for (; i + 1 < wfull && i < wt; ++i) {
        arrive();
        step(i, std::false_type{});
      }
      for (; i < wt; ++i) {
        arrive();
        step(i, std::true_type{});
      }
      for (; i < nt; ++i) {
        arrive();
        issue_group(i + DIST);
      }
      wait_vm<0>();               // no DMA outlives the sweep
      if (rok && !(pair_sum(sum) < 0x1p64f)) big = 1.f;
    }
    lds_barrier();
    if (exact) break;
    const bool again = __any(big != 0.f);
    if (lane == 0) reinterpret_cast<int*>(smem)[wave] = again;
    lds_barrier();
    int any = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) any |= reinterpret_cast<const int*>(smem)[w];
    lds_barrier();
    if (!any) break;
  }

  // The sweep's last barrier is behind every wave: the ring is free, and lambda
  // is there.  The second map's waves hand P_2 V over in fp32.  For the backward
  // O_2 is kept as 16-bit integers of its row's largest value, and what O's
  // rounding to bf16 drops in 8 bits: D_m = dO . (P_m V) is then exact to 2^-16,
  // where an error of D would add up over the whole row of keys.
  const float lam = slam[0];
  const long long stat = (long long)(b * a.hp + pair) * 2 * a.ls + row;
  const long long goff = (tok0 + row0) * ldq + pair * 2 * a.hd;   // the wave's first row
  const int rows = a.L - row0 < 32 ? a.L - row0 : 32;
  const float l = pair_sum(sum) + pair_sum(rest), inv = rok ? 1.f / l : 0.f;
  if (h == 0 && row < a.L) {
    // log2-sum-exp, from l = f 2^e; and, for the second map, by how much its
    // rounding to fp32 makes the weights too small
    int e;
    const float lf = __log2f(frexpf(l, &e));
    const double exact = (double)(mx * sc) + ((double)e + (double)lf);   // the weights were taken relative to mx sc
    float* const at = a.lse + stat + m * a.ls;
    *at = rok ? (float)exact : INFINITY;
    if (row == a.L - 1) at[1] = INFINITY;
    if (m == 1) a.fix[((long long)b * a.hp + pair) * a.ls + row] = (float)((double)(float)exact - exact) * 0.693147181f;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[t][i] = rok ? o[t][i] * inv : 0.f;
  // column of accumulator value (t, i): V's tile has D per half, hd of them in
  // use, and 4 neighbours are in or out together
  auto column = [&](int t, int i, bool& in) __attribute__((always_inline)) {
    const int e0 = (32 * t) % D + 2 * i + 4 * h;
    in = e0 < a.hd;
    return 32 * t / D * a.hd + e0;
  };
  unsigned char* const xch = smem + rb * NT * 4096 + lane * 16;
  if (m == 1) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(xch + (t * 4 + (i >> 2)) * 1024) =
            make_float4(o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]);
  }
  lds_barrier();
  if (m == 0) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 y = *reinterpret_cast<const float4*>(xch + (t * 4 + (i >> 2)) * 1024);
        o[t][i] = fmaf(-lam, y.x, o[t][i]);
        o[t][i + 1] = fmaf(-lam, y.y, o[t][i + 1]);
        o[t][i + 2] = fmaf(-lam, y.z, o[t][i + 2]);
        o[t][i + 3] = fmaf(-lam, y.w, o[t][i + 3]);
      }
  }
  lds_barrier();
  unsigned char* const st = smem + wave * 32 * P2;
  if (m == 1) {
    float top = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((32 * t) % D + 8 * (i >> 2) + 4 * h < a.hd) top = fmaxf(top, fabsf(o[t][i]));
    top = pair_max(top);
    const float f = top > 0.f ? 32767.f / top : 0.f;
    if (h == 0 && row < a.L) a.rsc[stat + a.ls] = top / 32767.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        bool in;
        const int dv = column(t, i, in);
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (uint32_t)__float2int_rn(o[t][i + e] * f) & 0xFFFFu;
        if (in) *reinterpret_cast<uint2*>(st + c * P2 + 2 * dv) = make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
      }
    store_rows(st, P2, reinterpret_cast<short*>(a.o2) + goff, ldq * 2, 4 * a.hd, rows, lane);
  }
  if (m == 0) {
    float top = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        bool in;
        const int dv = column(t, i, in);
        if (in)
          store4<bf16>(reinterpret_cast<bf16*>(st + c * P2) + dv, o[t][i], o[t][i + 1], o[t][i + 2], o[t][i + 3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[t][i + e] -= bf2f(f2bf(o[t][i + e]));
          top = fmaxf(top, in ? fabsf(o[t][i + e]) : 0.f);
        }
      }
    top = pair_max(top);
    if (h == 0 && row < a.L) a.rsc[stat] = top / 127.f;
    const float f = top > 0.f ? 127.f / top : 0.f;
    store_rows(st, P2, reinterpret_cast<bf16*>(a.o) + goff, ldq * 2, 4 * a.hd, rows, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        bool in;
        const int dv = column(t, i, in);
        uint32_t r4 = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) r4 |= ((uint32_t)__float2int_rn(o[t][i + e] * f) & 0xFFu) << (8 * e);
        if (in) *reinterpret_cast<uint32_t*>(st + c * P1 + dv) = r4;
      }
    store_rows(st, P1, a.res + goff, ldq, 2 * a.hd, rows, lane);
  }
}

void launch_diff_fwd_bf16(const DiffArgs& a, hipStream_t s) {
  const int n = a.hp * a.B;
  auto grid = [&](int rows) { return dim3((unsigned)((a.L + rows - 1) / rows * n)); };
  by_width(a.hd, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const bool four = filled(a, a.causal ? 128 : 64) * a.hp > 256;
    if (a.fine) {
      if (four) hipLaunchKernelGGL((diff_fwd_lds<D, 4, true>), grid(128), dim3(512), 0, s, a);
      else hipLaunchKernelGGL((diff_fwd_lds<D, 2, true>), grid(64), dim3(256), 0, s, a);
    } else {
      if (four) hipLaunchKernelGGL((diff_fwd_lds<D, 4, false>), grid(128), dim3(512), 0, s, a);
      else hipLaunchKernelGGL((diff_fwd_lds<D, 2, false>), grid(64), dim3(256), 0, s, a);
    }
  });
}

}  // namespace sl
