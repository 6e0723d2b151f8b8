// Differential attention: checks of arguments, buffers, entry points.
#include "sl_diffattn.hpp"

namespace sl {

// ---------------------------------------------------------------------------
// host side
struct DiffPlan {
  size_t lse, lam, fix, rsc, o2, res, saved;    // offsets and size of the saved buffer
  size_t dsum, dlam, part, ws;             // of the workspace
  int split;
  long long part_elems;                    // of one part of dK or dV
};

// bf16: up to so many rows the weights and the score gradients of dK enter their
// products as the sum of two bf16 values (2^-16) instead of one (2^-8).  With one the
// results are off by 1.3 (O), 1.42 (dV) and 1.44 times (dK) their own rounding to bf16 where
// many terms are summed, and by up to 2.2 times where few are (2 rows; 1.5 at 33); with two
// by 1.00 times.  Two cost half as many products again of dV and dK and two thirds of
// the forward's: 8 x 32 tokens of 16 + 8 heads of 64 forward 23 -> 24 us, backward 46 -> 46, 4 x
// 128 of 32 + 8 of 128 33 -> 35 and 83 -> 88, 8 x 256 of 32 of 128 46 -> 51 and 102 -> 108, but
// 1 x 4096 of 32 + 8 219 -> 304 and 628 -> 724.
constexpr int kFineRows = 256;

// Work of the bf16 backward's workgroups: 128 rows (or keys) each, every wave 32
// of them, or 64 with two waves to a row taking turns at the tiles, which doubles
// the workgroups and halves their length but loads each tile for half the rows.
// The second kind is taken where the first leaves CUs idle: while there are not
// more than 256 of the second; and, of causal workgroups, whose lengths differ so
// that the longest decides, where one round of the first is to end early, up to 256
// of them in long sequences and fewer in short ones, whose set-up weighs more.
// Measured, 128 / 64 rows for dQ, dK and dV together, heads of 128, 128-row
// workgroups in brackets.  Not causal: 1 x 1024 (128) 163 / 133 us, 1 x 1280 (160)
// 191 / 249.  Causal: 16 x 128 (192) 85 / 118, 4 x 256 (96) 91 / 83, 8 x 256 (192) 96 / 122,
// 2 x 512 (128) 115 / 99, 4 x 512 (192) 116 / 131, 2 x 768 (168) 142 / 137 and (216) 143 /
// 151, 2 x 1024 (192) 162 / 152, (224) 166 / 165, (256) 166 / 171, 1 x 1200 (250) 188 / 190,
// 1 x 1536 (240) 216 / 202 and (264) 221 / 248, 1 x 2048 (256) 263 / 232 and (272) 274 /
// 294, 1 x 4096 (256) 460 / 361, (288) 480 / 463 and (384) 508 / 564.  Narrower heads lean to
// the second: 2 x 1024 (256) of 64, 115 / 105.
static int bwd_rows(const DiffArgs& a, int n) {   // n workgroups per block of rows
  const int most = a.L < 1280 ? 96 + a.L / 8 : 256;
  return filled(a, 64) * n <= 256 || (a.causal && filled(a, 128) * n <= most) ? 64 : 128;
}

// Parts that a kv group's heads are cut into for dK and dV: while there are fewer
// workgroups than one round of 256, or, of causal ones (their lengths differ), two;
// not where all tiles of the group are so few (fp32: one for each of the four waves)
// that the launch which adds the parts costs what they save.  Padding counts as rows,
// since the workspace's size does not know the lengths.
// Measured, the whole backward with 1 / 2 / 4 parts, 32 + 8 heads of 128 (workgroups
// with one part in brackets, bf16 of 128 keys):
//   bf16 causal 1 x 128 (4) 82 / 78 / 76 us, 4 x 128 (16) 83 / 83 / 81, 16 x 128 of 64 (64)
//   64 / 67 / 71, 1 x 1024 (32) 206 / 158 / 135, 2 x 1024 (64) 230 / 188 / 183, 1 x 4096 (128)
//   786 / 640 / 622, 2 x 4096 (256) 1200 / 1176 / 1231; not causal 1 x 2048 (64) 416 / 334 / 326,
//   4 x 1024 of 64 (128) 212 / 215 / 232
//   fp32 causal 1 x 32 (4) 86 / 88 / 89, 1 x 64 (8) 104 / 89 / 89, 4 x 128 (64) 143 / 113 / 100,
//   1 x 1024 (128) 771 / 497 / 385, 2 x 1024 (256) 926 / 690 / 747; not causal 1 x 1024 (128)
//   878 / 599 / 615, 2 x 1024 (256) 1132 / 1161 / 1202
static int dkv_split(sl_dtype dt, int B, int L, int hp, int gp, bool causal) {
  const int rows = dt == SL_F32 ? 32 : 128, grp = hp / gp;
  const long long n = (long long)((L + rows - 1) / rows) * B * gp;
  int s = 1;
  if (grp * ((L + 31) / 32) <= (dt == SL_F32 ? 4 : 16)) return s;
  while (s < grp && n * s < (causal ? 512 : 256)) {
    ++s;
    while (grp % s) ++s;
  }
  return s;
}

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
  const long long stats = (long long)lay->batch * hq * (lay->seq_len + 1);   // two rows per head pair
  Bump s, w;
  pl.lse = s.take(stats * 4);
  pl.lam = s.take(16);
  pl.fix = s.take(dt == SL_BF16 ? stats * 2 : 0);
  pl.rsc = s.take(dt == SL_BF16 ? stats * 4 : 0);
  pl.o2 = s.take(T * hq * hd * (dt == SL_BF16 ? 2 : 4));
  pl.res = s.take(dt == SL_BF16 ? T * hq * hd : 0);
  pl.saved = s.off;
  pl.dsum = w.take(stats * 4);
  // a partial sum of dlambda per wave, 4 to a workgroup of 32 rows or more
  pl.dlam = w.take(4 * (size_t)((lay->seq_len + 31) / 32) * lay->batch * (hq / 2) * 8);
  pl.split = dkv_split(dt, lay->batch, lay->seq_len, hq / 2, hkv / 2, true);   // the most parts
  pl.part_elems = T * hkv * hd;
  pl.part = w.take(pl.split > 1 ? 2 * (size_t)pl.split * pl.part_elems * 4 : 0);
  pl.ws = w.off;
  return SL_OK;
}

static sl_status diff_args(DiffArgs& a, const sl_layout* lay, const sl_diff_attn* p) {
  a = DiffArgs{};
  a.B = lay->batch;
  a.L = lay->seq_len;
  a.ls = a.L + 1;
  a.hp = p->heads.n_q_heads / 2;
  a.gp = p->heads.n_kv_heads / 2;
  a.hd = p->heads.head_dim;
  a.causal = p->causal != 0;
  a.fine = a.L <= kFineRows;
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
    if (a.lens[b] != a.lens[0]) a.mix = 1;
  }
  return SL_OK;
}

static void saved_args(DiffArgs& a, const DiffPlan& pl, void* saved) {
  char* p = reinterpret_cast<char*>(saved);
  a.lse = reinterpret_cast<float*>(p + pl.lse);
  a.lam = reinterpret_cast<float*>(p + pl.lam);
  a.fix = reinterpret_cast<float*>(p + pl.fix);
  a.rsc = reinterpret_cast<float*>(p + pl.rsc);
  a.o2 = p + pl.o2;
  a.res = reinterpret_cast<signed char*>(p + pl.res);
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
  if ((ws || ws_bytes) && (!ws || ws_bytes < pl.ws))   // none of it is used here
    SL_FAIL(SL_ERR_WORKSPACE, "workspace too small: %zu of %zu bytes", ws_bytes, pl.ws);
  st = check_arch();
  if (st != SL_OK) return st;
  a.q = q; a.k = k; a.v = v; a.o = o;
  saved_args(a, pl, saved);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dt == SL_BF16) launch_diff_fwd_bf16(a, s);
  else launch_diff_fwd_f32(a, s);
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
  saved_args(a, pl, const_cast<void*>(saved));
  a.dsum = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + pl.dsum);
  a.dlam_part = reinterpret_cast<double*>(reinterpret_cast<char*>(ws) + pl.dlam);
  a.split = dkv_split(dt, a.B, a.L, a.hp, a.gp, a.causal != 0);
  a.dq_rows = dt == SL_F32 ? 32 : bwd_rows(a, a.hp);
  a.dkv_rows = dt == SL_F32 ? 32 : bwd_rows(a, a.gp * a.split);
  a.npart = 4 * ((a.L + a.dq_rows - 1) / a.dq_rows) * a.B * a.hp;
  a.dk_part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + pl.part);
  a.dv_part = a.dk_part + a.split * pl.part_elems;
  a.dlq1 = g->dlq1; a.dlk1 = g->dlk1; a.dlq2 = g->dlq2; a.dlk2 = g->dlk2;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dt == SL_BF16) launch_diff_bwd_bf16(a, s);
  else launch_diff_bwd_f32(a, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}
