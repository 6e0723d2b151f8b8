// Differential attention: backward kernels.
#include "sl_diffattn_lds.hpp"

namespace sl {

// ---------------------------------------------------------------------------
// dQ.  As the forward: a wave owns 32 queries (their rows of Q and dO are held
// in registers) and walks the key tiles, scores and dP = V dO^T transposed, so
// that P and dS stay where they are formed.  K's tile is read twice, by rows
// for the scores and by columns for dQ^T += K^T dS^T.
//
// dS goes to the matrix cores as the sum of two bf16 (2^-16): a row of dS sums to
// zero, so what one rounding of 2^-8 leaves behind is not small beside dQ where
// the keys have something in common.  It costs a third more products (1 x 4096,
// 8 kv heads of 128: dQ's error 1.5 to 1.1 times that of its own rounding to bf16).
// H = 1: four row blocks to a workgroup, tiles loaded two ahead.  H = 2: two row
// blocks, each with two waves that take every other tile and add their sums in the
// end (where each kind pays: bwd_rows).
// Bound by what its one wave per SIMD can issue (55 % of its cycles; 27 % wait for
// loads and barriers): 1 x 2048 tokens, 32 heads, 8 kv, of 128, 146 us, 706 TFLOP/s
// of scores, dP and dQ (dS counted once).
// The sum of P_2 dP, which is -dlambda, stays in fp32 over a tile and in fp64
// beyond, with what the log-sum-exp's rounding did to the row taken out again.
template <int D, int H>
__global__ void __launch_bounds__(256, 1) diff_dq_lds(const DiffArgs a) {
  using R = RowTile<D>;
  constexpr int DT = D / 32, KS = D / 16, PW = R::PER_WAVE, P2 = 4 * D + 16;
  constexpr int STEP = H * R::BYTES, ROWS = 128 / H;
  constexpr int DIST = H == 1 ? 2 : 1;                    // steps that tiles are loaded ahead
  constexpr int NK = H == 1 ? 4 : 3, NV = H == 1 ? 4 : 2; // ring; K is read for one step more than V
  constexpr int RING = (NK + NV) * STEP;
  static_assert(4 / H * 32 * P2 <= RING && 4 * DT * 4096 <= RING, "the halves and the staged results fit the ring");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[RING];
  unsigned char* const sk = smem;
  unsigned char* const sv = smem + NK * STEP;
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rb = wave / H, half = wave % H;               // block of 32 rows, every H-th key tile
  const int nqb = (a.L + ROWS - 1) / ROWS;
  int blk, pair, b;
  locate(blockIdx.x, a.B, a.hp, a.hp / a.gp, a.mix, blk, pair, b);
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
  // steps of H tiles: of the workgroup, of this wave, and those that need no mask
  const int nt = (kend + 32 * H - 1) / (32 * H), wt = ((wend + 31) / 32 + H - 1 - half) / H;
  const int wfull = ((a.causal && row0 + 1 < len ? row0 + 1 : len) / 32 + H - 1 - half) / H;
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
    const long long at = ((long long)(b * a.hp + pair) * 2 + m) * a.ls + row;
    lse[m] = rok ? a.lse[at] : INFINITY;      // weights of rows past the end: 0
    ds[m] = 0.f;
  }
  // D_2 = dO . O_2 and D_1 = dO . (O + lambda O_2) of the row, from the saved
  // integers; dK and dV read them from memory
  {
    const long long st = (long long)(b * a.hp + pair) * 2 * a.ls + row;
    float dres = 0.f;
#pragma unroll
    for (int x = 0; x < 2 * KS; ++x) {
      const int col = (x % KS) * 16 + h * 8;
      if (rok && col < a.hd) {
        const long long at = qoff + x / KS * a.hd + col;
        const Frag<bf16> of = load_row<bf16>(reinterpret_cast<const bf16*>(a.a) + at, true);
        const uint4 yv = *reinterpret_cast<const uint4*>(reinterpret_cast<const short*>(a.o2) + at);
        const uint2 rv = *reinterpret_cast<const uint2*>(a.res + at);
        const uint32_t yw[4] = {yv.x, yv.y, yv.z, yv.w}, rw[2] = {rv.x, rv.y};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gx = (float)go[x].v[e];
          ds[0] = fmaf(gx, (float)of.v[e], ds[0]);
          ds[1] = fmaf(gx, (float)(short)(yw[e >> 1] >> (16 * (e & 1))), ds[1]);
          dres = fmaf(gx, (float)(signed char)(rw[e >> 2] >> (8 * (e & 3))), dres);
        }
      }
    }
    if (rok) {
      ds[1] = pair_sum(ds[1]) * a.rsc[st + a.ls];
      ds[0] = fmaf(lam, ds[1], fmaf(pair_sum(dres), a.rsc[st], pair_sum(ds[0])));
    }
    if (h == 0 && half == 0 && row < a.L) {
      a.dsum[st] = ds[0];
      a.dsum[st + a.ls] = ds[1];
      if (row == a.L - 1) a.dsum[st + 1] = a.dsum[st + a.ls + 1] = 0.f;
    }
  }
  int srow[PW];
  unsigned scol[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) R::source(wave * PW + i, lane, a.hd, srow[i], scol[i]);
  const unsigned ldb = (unsigned)ldk * 2u;
  const int last = len - 1;
  auto issue_part = [&](int step, int i) __attribute__((always_inline)) {   // i < PW: the first tile
    const unsigned d0 = (unsigned)(i / PW * R::BYTES + (wave * PW + i % PW) * 1024);
    int r = step * 32 * H + i / PW * 32 + srow[i % PW];
    r = r < last ? r : last;
    const unsigned off = (unsigned)r * ldb + scol[i % PW];
    dma16(kbase, off, __builtin_amdgcn_readfirstlane(lds_addr(sk) + (unsigned)(step % NK * STEP) + d0));
    dma16(vbase, off, __builtin_amdgcn_readfirstlane(lds_addr(sv) + (unsigned)(step % NV * STEP) + d0));
  };
  auto issue_step = [&](int step) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < H * PW; ++i) issue_part(step, i);
  };

  TileAddr<D> ad;
  ad.init(lane, true, true);
  f32x16 dq[2][DT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dq[m][t]);
  const float sc = a.scale * kLog2e;
  const double fix = rok ? 1.0 + (double)a.fix[((long long)b * a.hp + pair) * a.ls + row] : 1.0;
  double dlam = 0.0;

  auto mask = [&](f32x16 (&s)[2], int step) __attribute__((always_inline)) {
    const int lim = a.causal && row + 1 < len ? row + 1 : len;
    const int k0 = (H * step + half) * 32 + 4 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool hidden = k0 + 8 * (i >> 2) + (i & 3) >= lim;
      s[0][i] = hidden ? -INFINITY : s[0][i];
      s[1][i] = hidden ? -INFINITY : s[1][i];
    }
  };
  // Step i in a fixed order: the scores of tile i, while the first map's dS of
  // tile i - 1 is formed; the first map's dQ, while the second's dS is; the second
  // map's dQ and then dP of tile i, while the weights of tile i are.  Operands are
  // read AHEAD products early.
  constexpr int N1 = 2 * KS, N2 = 2 * DT, NG = 2 * N1 + 2 * N2, AHEAD = 3;
  constexpr int GAP = H == 1 ? NG / PW : 2;               // products between loads
  f32x16 s[2], dp;
  auto step = [&](int i, auto has_prev, auto has_next, auto masked) __attribute__((always_inline)) {
    constexpr bool PREV = decltype(has_prev)::value, NEXT = decltype(has_next)::value;
    const unsigned char* kt = sk + i % NK * STEP + half * R::BYTES;
    const unsigned char* vt = sv + i % NV * STEP + half * R::BYTES;
    const unsigned char* kp = sk + (i + NK - 1) % NK * STEP + half * R::BYTES;
    f32x16 n[2], ndp;
    Frag<bf16> hi[2][2], lo[2][2], fa[AHEAD];
    float part = 0.f;
    zero16(n[0]);
    zero16(n[1]);
    zero16(ndp);
    auto read = [&](auto gc) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value, x = g % AHEAD;
      if constexpr (g < N1) {
        if constexpr (NEXT) fa[x] = ad.row(kt, (g / KS) * (D / 8) + 2 * (g % KS));
      } else if constexpr (g < N1 + 2 * N2) {
        constexpr int m = (g - N1) / N2, j = (g - N1) % N2;
        if constexpr (PREV) fa[x] = ad.col(kp, m * DT + j % DT, j / DT);
      } else if constexpr (g < NG) {
        if constexpr (NEXT) fa[x] = ad.row(vt, 2 * (g - N1 - 2 * N2));
      }
    };
    // dS of elements e0 .. e1 - 1 (pairs) of map m, as the sum of two bf16
    auto grads = [&](int m, int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
      for (int x = e0; x < e1; x += 2) {
        if (m == 1) part = fmaf(s[1][x], dp[x], fmaf(s[1][x + 1], dp[x + 1], part));
        const float g0 = s[m][x] * (dp[x] - ds[m]), g1 = s[m][x + 1] * (dp[x + 1] - ds[m]);
        const uint32_t top = round2(g0, g1);
        set2(hi[m][x / 8], x % 8, top);
        set2(lo[m][x / 8], x % 8, round2(g0 - __uint_as_float(top << 16), g1 - __uint_as_float(top & 0xFFFF0000u)));
      }
    };
    auto weigh = [&](int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
      for (int e = e0; e < e1; ++e) n[e / 16][e % 16] = fast_exp2(fmaf(n[e / 16][e % 16], sc, -lse[e / 16]));
    };
    each<AHEAD>(read);
    each<NG>([&](auto gc) __attribute__((always_inline)) {
      constexpr int g = decltype(gc)::value;
      if constexpr (g < N1) {
        if constexpr (NEXT) mma(n[g / KS], fa[g % AHEAD], q[g / KS][g % KS]);
      } else if constexpr (g < N1 + 2 * N2) {
        constexpr int m = (g - N1) / N2, j = (g - N1) % N2;
        if constexpr (PREV) {
          mma(dq[m][j % DT], fa[g % AHEAD], hi[m][j / DT]);
          mma(dq[m][j % DT], fa[g % AHEAD], lo[m][j / DT]);
        }
      } else {
        if constexpr (NEXT) mma(ndp, fa[g % AHEAD], go[g - N1 - 2 * N2]);
      }
      read(std::integral_constant<int, g + AHEAD>{});
      if constexpr (NEXT && g % GAP == 1 && g / GAP < H * PW) issue_part(i + DIST, g / GAP);
      if constexpr (g < N1 && PREV) grads(0, 2 * (8 * g / N1), 2 * (8 * (g + 1) / N1));
      if constexpr (g >= N1 && g < N1 + N2 && PREV) grads(1, 2 * (8 * (g - N1) / N2), 2 * (8 * (g - N1 + 1) / N2));
      if constexpr (g == N1 - 1 && NEXT && decltype(masked)::value) mask(n, i);
      if constexpr (g >= N1 + N2 && NEXT) weigh(32 * (g - N1 - N2) / (N1 + N2), 32 * (g - N1 - N2 + 1) / (N1 + N2));
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (PREV) dlam = fma((double)part, fix, dlam);
    if constexpr (NEXT) {
      s[0] = n[0];
      s[1] = n[1];
      dp = ndp;
    }
  };

  if (nt > 0) {
    issue_step(0);
    if (DIST == 2) issue_step(1);
    // after it, step i (or the wave's wait for the others) loads the tiles of step i + DIST
    auto arrive = [&]() __attribute__((always_inline)) {
      wait_vm<2 * PW * (DIST - 1)>();   // the tiles of step i have landed
      lds_barrier();                    // ... for every wave, and all are done with step i - 1
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    int i = 0;
    if (wt > 0) {
      arrive();
      if (wfull > 0) step(0, no, yes, no);
      else step(0, no, yes, yes);
      for (i = 1; i < wfull && i < wt; ++i) {
        arrive();
        step(i, yes, yes, no);
      }
      for (; i < wt; ++i) {
        arrive();
        step(i, yes, yes, yes);
      }
      step(i, yes, no, no);       // K of step wt - 1: refilled from step wt + 1's arrival on
    }
    for (; i < nt; ++i) {
      arrive();
      issue_step(i + DIST);
    }
    wait_vm<0>();
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) dlam += __shfl_xor(dlam, o);
  if (lane == 0) a.dlam_part[blockIdx.x * 4 + wave] = dlam;
  // the two waves of a row block: the first ends with the sum of map 1, the second of map 2
  lds_barrier();                  // the ring is free
  if constexpr (H == 2) {
    unsigned char* const mine = smem + wave * DT * 4096;
    unsigned char* const other = smem + (wave ^ 1) * DT * 4096;
    if (half) put_acc(dq[0], mine, lane);
    else put_acc(dq[1], mine, lane);
    lds_barrier();
    if (half) add_acc(dq[1], other, lane);
    else add_acc(dq[0], other, lane);
    lds_barrier();
  }
  unsigned char* const st = smem + rb * 32 * P2;
  const bool some = rok && !one_key(a, row, len);
  auto stage = [&](const f32x16 (&x)[DT], int m, float f) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d >= a.hd) continue;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = some ? x[t][i + e] * f : 0.f;
        store4<bf16>(reinterpret_cast<bf16*>(st + c * P2) + m * a.hd + d, y[0], y[1], y[2], y[3]);
      }
  };
  if (H == 1 || half == 0) stage(dq[0], 0, a.scale);
  if (H == 1 || half == 1) stage(dq[1], 1, -lam * a.scale);
  if (H == 2) lds_barrier();
  constexpr int NR = 32 / H;
  const int r0 = row0 + NR * half, rows = a.L - r0 < NR ? a.L - r0 : NR;
  store_rows(st + NR * half * P2, P2, reinterpret_cast<bf16*>(a.dq) + (tok0 + r0) * ldq + pair * 2 * a.hd, ldq * 2, 4 * a.hd,
             rows, lane);
}

// ---------------------------------------------------------------------------
// dK and dV.  A wave owns 32 keys (K's rows in registers; V's rows in registers
// up to D = 64, else in LDS) and walks the query tiles of its group's heads:
// scores and dP = dO V^T with a key per lane, then dV^T += dO^T (P_1 - lambda P_2)
// and dK_m^T += Q_m^T dS_m with the tile's rows read by columns.  A key's column
// never meets another's, so keys past the end need no mask: their results are
// written as 0.  H as in dQ, of key blocks and query tiles.  The heads of a group
// are cut into `split` parts where one workgroup per key block would leave CUs
// idle; the parts' sums are then fp32 and diff_dkv_sum adds them in order.
//
// P_1 - lambda P_2 and dS are rounded to bf16 for the matrix cores, dS once where dQ's
// is the sum of two: a key's column of dS does not sum to zero.  In short sequences
// both are the sum of two (FINE; where and why: kFineRows).
//
// Bound as dQ (62 % of the wave's cycles issue, 23 % wait; at D = 128 144 of 344
// vector instructions a tile move accumulators): the same call 157 us, 875 TFLOP/s.
template <int D, int H, bool FINE>
__global__ void __launch_bounds__(256, 1) diff_dkv_lds(const DiffArgs a) {
  using R = RowTile<D>;
  constexpr int DT = D / 32, NT = D / 16, KS = D / 16, NST = 2, PW = R::PER_WAVE, STEP = H * R::BYTES, NB = 4 / H;
  // V's operands in registers, the others in LDS as they are read; at D = 128 one
  // makes room for the statistics in 160 KB
  constexpr int VR = D <= 64 ? 2 * KS : D == 128 && H == 2 ? 1 : 0, VL = 2 * KS - VR;
  constexpr int STAT = 4 * 64 * 4;      // lse and D of both maps for 64 rows, a step's or more
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * NST * STEP + NB * VL * 1024 + NST * STAT];
  unsigned char* const sq = smem;
  unsigned char* const sg = smem + NST * STEP;
  unsigned char* const sv = smem + 2 * NST * STEP;
  unsigned char* const ss = sv + NB * VL * 1024;
  if (blockIdx.x == gridDim.x - 1) {   // the last block sums up dlambda, beside the others
    dlambda_block(a, reinterpret_cast<double*>(smem));
    return;
  }
  const int lane = threadIdx.x & 63, h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rb = wave / H, half = wave % H;                     // block of 32 keys, every H-th query tile
  int blk, gs, b;
  locate(blockIdx.x, a.B, a.gp * a.split, a.split, a.mix, blk, gs, b);
  const int g = gs / a.split, part = gs % a.split;
  const int grp = a.hp / a.gp, nh = grp / a.split, len = a.lens[b];
  const int k0 = blk * 32 * NB, key = k0 + rb * 32 + c;              // causal: the first keys have the most queries
  const bool kok = key < len;
  const long long ldq = (long long)a.hp * 2 * a.hd, ldk = (long long)a.gp * 2 * a.hd, tok0 = (long long)b * a.L;
  const long long koff = (tok0 + key) * ldk + g * 2 * a.hd;
  const float lam = a.lam[0];
  const int pr0 = g * grp + part * nh;
  const int t0 = a.causal ? k0 / 32 : 0;                        // first query tile
  const int ntile = k0 < len ? (len + 31) / 32 - t0 : 0, ns = (ntile + H - 1) / H;   // steps of H tiles

  int srow[PW];
  unsigned scol[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) R::source(wave * PW + i, lane, a.hd, srow[i], scol[i]);
  const int last = len - 1;
  unsigned char* const vt = sv + rb * VL * 1024 + lane * 16;    // this lane's operands of V
  Frag<bf16> kf[2][KS], vf[VR > 0 ? VR : 1];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int col = s * 16 + h * 8;
      const bool ok = kok && col < a.hd;
      kf[m][s] = load_row<bf16>(reinterpret_cast<const bf16*>(a.k) + koff + m * a.hd + col, ok);
      const Frag<bf16> x = load_row<bf16>(reinterpret_cast<const bf16*>(a.v) + koff + m * a.hd + col, ok);
      if (m * KS + s < VR) vf[m * KS + s] = x;
      else if (half == s % H) *reinterpret_cast<bf16x8*>(vt + (m * KS + s - VR) * 1024) = x.v;
    }
  const unsigned ldb = (unsigned)ldq * 2u;
  int it_pr = pr0, it_t = t0;                                   // the next tile to load
  // statistics: wave w loads lse (w < 2) or D of map w % 2, 64 rows
  const float* const sbase = (wave < 2 ? a.lse : a.dsum) + (long long)b * a.hp * 2 * a.ls + (wave & 1) * a.ls;
  auto issue_part = [&](int it, int i) __attribute__((always_inline)) {   // i < PW: the first tile
    const unsigned d0 = __builtin_amdgcn_readfirstlane((unsigned)((it & 1) * STEP + i / PW * R::BYTES + (wave * PW + i % PW) * 1024));
    const long long ofs = tok0 * ldq + it_pr * 2 * a.hd;
    int r = (it_t + i / PW) * 32 + srow[i % PW];
    r = r < last ? r : last;
    const unsigned off = (unsigned)r * ldb + scol[i % PW];
    dma16(uniform(reinterpret_cast<const bf16*>(a.q) + ofs), off, lds_addr(sq) + d0);
    dma16(uniform(reinterpret_cast<const bf16*>(a.da) + ofs), off, lds_addr(sg) + d0);
  };
  auto issue_stats = [&](int it) __attribute__((always_inline)) {
    int r = it_t * 32 + lane;
    r = r < len ? r : len;                                      // lse there is +inf: weights 0
    const float* sb = reinterpret_cast<const float*>(uniform(sbase + (long long)it_pr * 2 * a.ls));
    const unsigned sd = __builtin_amdgcn_readfirstlane(lds_addr(ss) + (unsigned)((it & 1) * STAT + wave * 256));
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, %2"
                 :: "v"((unsigned)r * 4u), "s"(sd), "s"(sb) : "memory", "m0");
  };
  auto issued = [&]() __attribute__((always_inline)) {
    it_t += H;
    if (it_t >= t0 + ntile) {
      it_t = t0;
      if (it_pr + 1 < pr0 + nh) ++it_pr;                        // past the last: read again, used by none
    }
  };
  auto issue_next = [&](int it) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < H * PW; ++i) issue_part(it, i);
    issue_stats(it);
    issued();
  };

  TileAddr<D> ad;
  ad.init(lane, true, true);
  f32x16 dk[2][DT], dv[2][DT];   // dV's columns as the two halves of its tile
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < DT; ++t) zero16(dk[m][t]);
#pragma unroll
  for (int t = 0; t < NT; ++t) zero16(dv[t / DT][t % DT]);
  const float sc = a.scale * kLog2e;

  if (ns > 0) {
    issue_next(0);
    int it = 0;
    // after it, step `it` (or the wave's wait for the others) loads the next one's tiles
    auto arrive = [&]() __attribute__((always_inline)) {
      wait_vm<0>();               // the tiles of step `it` have landed
      lds_barrier();              // ... for every wave, and the other slot is read by none
    };
    // One query tile: the products in order S_1, S_2, dP, dV, dK, each with its
    // operand read from LDS `AHEAD` products before, and between them the
    // vector work that is ready (the weights while dP is formed, the score
    // gradients while dV is) and the next tile's loads.  One wave has the SIMD to itself, so only this
    // order covers the LDS reads and the exponentials.
    constexpr int N1 = 2 * KS, N2 = 2 * KS, N3 = 2 * NT, N4 = 4 * DT, NOP = N1 + N2 + N3 + N4, AHEAD = 3;
    auto tile = [&](int q0, auto diag) __attribute__((always_inline)) {
      constexpr bool DIAG = decltype(diag)::value;
      const unsigned char* qt = sq + (it & 1) * STEP + half * R::BYTES;
      const unsigned char* gt = sg + (it & 1) * STEP + half * R::BYTES;
      const float* st = reinterpret_cast<const float*>(ss + (it & 1) * STAT) + 32 * half + 4 * h;
      f32x16 s[2], dp, w;
      Frag<bf16> wf[2], wl[2], df[2][2], dl[2][2], fa[AHEAD], fb[AHEAD];
      float4 l4[2], d4[2];
      zero16(s[0]);
      zero16(s[1]);
      zero16(dp);
      auto read = [&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value, x = i % AHEAD;
        if constexpr (i < N1) {
          fa[x] = ad.row(qt, (i / KS) * (D / 8) + 2 * (i % KS));
        } else if constexpr (i < N1 + N2) {
          fa[x] = ad.row(gt, 2 * (i - N1));
          if constexpr (i - N1 >= VR) fb[x] = lds_row(vt + (i - N1 - VR) * 1024);
        } else if constexpr (i < N1 + N2 + N3) {
          fa[x] = ad.col(gt, (i - N1 - N2) % NT, (i - N1 - N2) / NT);
        } else if constexpr (i < NOP) {
          fa[x] = ad.col(qt, (i - N1 - N2 - N3) % (2 * DT), (i - N1 - N2 - N3) / (2 * DT));
        }
      };
      // statistics of elements e .. e + 3 (map e / 16): lse while weights are formed, then D
      auto stats = [&](float4 (&x)[2], int e, int which) __attribute__((always_inline)) {
        if (e < 32) x[(e / 4) & 1] = *reinterpret_cast<const float4*>(st + (which + e / 16) * 64 + 2 * (e % 16));
      };
      auto part4 = [](const float4& x, int e) __attribute__((always_inline)) {
        return e % 4 == 0 ? x.x : e % 4 == 1 ? x.y : e % 4 == 2 ? x.z : x.w;
      };
      each<AHEAD>(read);
      each<NOP>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < N1) {
          mma(s[i / KS], fa[i % AHEAD], kf[i / KS][i % KS]);
        } else if constexpr (i < N1 + N2) {
          if constexpr (i - N1 < VR) mma(dp, fa[i % AHEAD], vf[i - N1]);
          else mma(dp, fa[i % AHEAD], fb[i % AHEAD]);
        } else if constexpr (i < N1 + N2 + N3) {
          mma(dv[(i - N1 - N2) % NT / DT][(i - N1 - N2) % DT], fa[i % AHEAD], wf[(i - N1 - N2) / NT]);
          if constexpr (FINE) mma(dv[(i - N1 - N2) % NT / DT][(i - N1 - N2) % DT], fa[i % AHEAD], wl[(i - N1 - N2) / NT]);
        } else {
          constexpr int j = i - N1 - N2 - N3, mt = j % (2 * DT);
          mma(dk[mt / DT][mt % DT], fa[i % AHEAD], df[mt / DT][j / (2 * DT)]);
          if constexpr (FINE) mma(dk[mt / DT][mt % DT], fa[i % AHEAD], dl[mt / DT][j / (2 * DT)]);
        }
        read(std::integral_constant<int, i + AHEAD>{});
        if constexpr (i % (4 / H) == 1 && i / (4 / H) < H * PW) issue_part(it + 1, i / (4 / H));
        if constexpr (i == 4 * PW) issue_stats(it + 1);
        if constexpr (i == 4 * PW + 1) issued();
        if constexpr (i == KS - 1) stats(l4, 0, 0);
        if constexpr (i == N1 + N2 - 1) stats(d4, 0, 2);
        if constexpr (i >= KS && i < N1) {   // out of the matrix cores' registers before dP needs them
          constexpr int e0 = 16 * (i - KS) / KS, e1 = 16 * (i - KS + 1) / KS;
#pragma unroll
          for (int e = e0; e < e1; ++e) {
            if (e % 4 == 0) stats(l4, e + 4, 0);
            s[0][e] = fmaf(s[0][e], sc, -part4(l4[(e / 4) & 1], e));
          }
        }
        if constexpr (i >= N1 && i < N1 + N2) {
          constexpr int e0 = 32 * (i - N1) / N2, e1 = 32 * (i - N1 + 1) / N2;
#pragma unroll
          for (int e = e0; e < e1; ++e) {
            const int m = e / 16, x = e % 16;
            if (m == 1 && e % 4 == 0) stats(l4, e + 4, 0);
            float p = fast_exp2(m == 0 ? s[0][x] : fmaf(s[1][x], sc, -part4(l4[(e / 4) & 1], e)));
            if constexpr (DIAG) p = q0 + 2 * (x & ~3) + 4 * h + (x & 3) < key ? 0.f : p;
            s[m][x] = p;
            w[x] = m ? fmaf(-lam, p, w[x]) : p;
          }
        }
        if constexpr (i == N1 + N2 - 1) {
          operand<FINE>(w, wf, wl);
        }
        if constexpr (i >= N1 + N2 && i < N1 + N2 + N3) {
          constexpr int e0 = 32 * (i - N1 - N2) / N3, e1 = 32 * (i - N1 - N2 + 1) / N3;
#pragma unroll
          for (int e = e0; e < e1; ++e) {
            if (e % 4 == 0) stats(d4, e + 4, 2);
            s[e / 16][e % 16] *= dp[e % 16] - part4(d4[(e / 4) & 1], e);
            if constexpr (DIAG && e0 % 16 == 0)   // the first query reads the first key alone
              if (e % 16 == 0 && q0 + 4 * h == 0) s[e / 16][0] = 0.f;
          }
        }
        if constexpr (i == N1 + N2 + N3 - 1) {
#pragma unroll
          for (int m = 0; m < 2; ++m) operand<FINE>(s[m], df[m], dl[m]);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    for (int n = 0; n < nh; ++n) {
      int j = 0;
      if (a.causal) {             // tiles before this wave's keys, and the diagonal
        for (; H * j + half < rb && j < ns; ++j, ++it) {
          arrive();
          issue_next(it + 1);
        }
        if (H * j + half < ntile) {
          arrive();
          tile((t0 + H * j + half) * 32, std::true_type{});
          ++j;
          ++it;
        }
      }
      for (; H * j + half < ntile; ++j, ++it) {
        arrive();
        tile((t0 + H * j + half) * 32, std::false_type{});
      }
      for (; j < ns; ++j, ++it) {
        arrive();
        issue_next(it + 1);
      }
    }
    wait_vm<0>();
  }
  // the two waves of a key block: the first ends with the sum of dV, the second of dK
  lds_barrier();                  // the tiles are read by none
  if constexpr (H == 2) {
    static_assert(4 * NT * 4096 <= (int)sizeof(smem), "the halves fit");
    unsigned char* const mine = smem + wave * NT * 4096;
    unsigned char* const other = smem + (wave ^ 1) * NT * 4096;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (half) put_acc(dv[m], mine + m * DT * 4096, lane);
      else put_acc(dk[m], mine + m * DT * 4096, lane);
    }
    lds_barrier();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (half) add_acc(dk[m], other + m * DT * 4096, lane);
      else add_acc(dv[m], other + m * DT * 4096, lane);
    }
    lds_barrier();                // the sums are read
  }
  // results by rows through LDS: both maps' halves of dV, then dK's, in bf16 or
  // (parts) one half at a time in fp32
  constexpr int P2 = 4 * D + 16;
  static_assert(4 * 32 * P2 <= (int)sizeof(smem), "the staged results fit");
  unsigned char* const st = smem + wave * 32 * P2;
  const int row0 = k0 + rb * 32, rows = a.L - row0 < 32 ? a.L - row0 : 32;
  const long long roff = (tok0 + row0) * ldk + g * 2 * a.hd, poff = (long long)part * a.B * a.L * ldk + roff;
  auto put = [&](const f32x16 (&x)[DT], int m, float f, bool ok, bf16* out, float* parts, bool last) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int d = 32 * t + 2 * i + 4 * h;
        if (d >= a.hd) continue;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = ok ? x[t][i + e] * f : 0.f;
        if (a.split > 1) store4<float>(reinterpret_cast<float*>(st + c * P2) + d, y[0], y[1], y[2], y[3]);
        else store4<bf16>(reinterpret_cast<bf16*>(st + c * P2) + m * a.hd + d, y[0], y[1], y[2], y[3]);
      }
    if (a.split > 1) store_rows(st, P2, parts + poff + m * a.hd, ldk * 4, 4 * a.hd, rows, lane);
    else if (last) store_rows(st, P2, out + roff, ldk * 2, 4 * a.hd, rows, lane);
  };
  bf16* const dko = reinterpret_cast<bf16*>(a.dk);
  bf16* const dvo = reinterpret_cast<bf16*>(a.dv);
  // V's tile has D columns per half: its first DT accumulators are the first
  if (H == 1 || half == 0) {
    put(dv[0], 0, 1.f, kok, dvo, a.dv_part, false);
    put(dv[1], 1, 1.f, kok, dvo, a.dv_part, true);
  }
  if (H == 1 || half == 1) {
    put(dk[0], 0, a.scale, kok && len > 1, dko, a.dk_part, false);
    put(dk[1], 1, -lam * a.scale, kok && len > 1, dko, a.dk_part, true);
  }
}

void launch_diff_bwd_bf16(const DiffArgs& a, hipStream_t s) {
  auto blocks = [&](int rows) { return (a.L + rows - 1) / rows * a.B; };
  by_width(a.hd, [&](auto d) {
    constexpr int D = decltype(d)::value;
    const dim3 dq((unsigned)(blocks(a.dq_rows) * a.hp)), dkv((unsigned)(blocks(a.dkv_rows) * a.gp * a.split + 1));
    if (a.dq_rows == 64) hipLaunchKernelGGL((diff_dq_lds<D, 2>), dq, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((diff_dq_lds<D, 1>), dq, dim3(256), 0, s, a);
    if (a.fine) {
      if (a.dkv_rows == 64) hipLaunchKernelGGL((diff_dkv_lds<D, 2, true>), dkv, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((diff_dkv_lds<D, 1, true>), dkv, dim3(256), 0, s, a);
    } else {
      if (a.dkv_rows == 64) hipLaunchKernelGGL((diff_dkv_lds<D, 2, false>), dkv, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((diff_dkv_lds<D, 1, false>), dkv, dim3(256), 0, s, a);
    }
  });
  if (a.split > 1) {
    const long long n = 2 * ((long long)a.B * a.L * a.gp * 2 * a.hd / 4);
    hipLaunchKernelGGL(diff_dkv_sum<bf16>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  }
}

}  // namespace sl
