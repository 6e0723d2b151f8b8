// Token embedding: Y[t] = scale * E[id_t], and the table's gradient
// dE[v] = scale * (sum of dY[t] over the tokens t with id_t = v).
//
// Lookup: a row's vectors are read and written once (32768 rows of 4096 bf16 92 us, 5.8 TB/s;
// 2048 rows 9 us, of which 5 are the chain from the id to the row to its store).
//
// Gradient: the tokens are sorted by (id, place) first, so that the rows of one
// id stand in a run whose sum is taken in one fixed order, with no atomics on
// values.
//   1. Chunks of kChunk tokens are sorted by counting: a token's place is the
//      number of tokens of its chunk that sort before it, 16 tokens to a block.
//   2. Up to 16 sorted lists are merged at a time: a token's place is its place
//      in its own list plus the number of smaller ones in each other list.
//   3. The sorted list is cut into pieces of 64.  A block sums the rows of one piece over
//      1 KB of columns, in fp32, eight rows to a wave, which loads them together; the
//      waves' sums of one run are added through LDS.  A run that lies inside its
//      piece goes to the table; of one that crosses a border the partial sum is kept.
//   4. The partial sums of every crossing run are added in order.
// The table is zeroed beside step 1, every row of it: that needs no word of the ids, and
// runs as fast as memory takes it where a block writes 4 KB, a vector a thread (524 MB: 77 us; in
// 64 KB a block 98, which a search for the rows without a token needs to pay).
//
// Measured: 2048 tokens, 32000 x 4096 fp32: sort and zeros 81 us, sums 14.5, join 4.8; 32768 tokens,
// 128256 x 4096 bf16: 156, 8 for the merge, 76 (356 MB with what it writes: 4.7 TB/s) and 10.  What
// bounds it: the table's writes; then the sums' chain from the sorted list to the rows to the
// waves' exchange, two rounds of memory latency where there are few tokens.
#include "sl_rows.hpp"

namespace sl {

constexpr int kChunk = 2048;       // tokens sorted by counting
constexpr int kRankTokens = 16;    // of them in one block
constexpr int kLists = 16;         // sorted lists merged at a time
constexpr int kJoinWaves = 8;      // waves that add a run's partial sums
constexpr int kPieceWaves = 8, kWaveRows = 8, kPiece = kPieceWaves * kWaveRows;   // sorted tokens of a block
constexpr int kJoinSlice = 512;    // and columns of them, 8 a lane
constexpr uint32_t kNoKey = 0xFFFFFFFEu;

// ids outside the vocabulary are no tokens: they sort behind every id
__device__ inline uint32_t token_key(int id, uint32_t V) { return (uint32_t)id < V ? (uint32_t)id : V; }

template <typename T, int U>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const T* __restrict__ E, const int* __restrict__ ids, uint32_t V,
                                                        int nvec, int ntok, int lanes_log2, float scale,
                                                        T* __restrict__ Y) {
  constexpr int W = 16 / sizeof(T);
  using VT = Vec<T, W>;
  const int lanes = 1 << lanes_log2, col = blockIdx.y * lanes + (threadIdx.x & (lanes - 1));
  const int rows = 256 >> lanes_log2;
  if (col >= nvec) return;
  for (long long t0 = (long long)blockIdx.x * rows * U; t0 < ntok; t0 += (long long)gridDim.x * rows * U) {
    VT v[U];
    uint32_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = t0 + u * rows + (threadIdx.x >> lanes_log2);
      id[u] = t < ntok ? token_key(ids[t], V) : V;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (id[u] < V) v[u] = reinterpret_cast<const VT*>(E)[(long long)id[u] * nvec + col];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = t0 + u * rows + (threadIdx.x >> lanes_log2);
      VT o;
#pragma unroll
      for (int j = 0; j < W; ++j) o.v[j] = f2el<T>(id[u] < V ? el2f<T>(v[u].v[j]) * scale : 0.f);
      if (t < ntok) reinterpret_cast<VT*>(Y)[t * nvec + col] = o;
    }
  }
}

// 1. sid, stok of every chunk in order of (id, token); the blocks behind those zero the
// table's vectors
__global__ void __launch_bounds__(256) embed_rank_kernel(const int* __restrict__ ids, uint32_t V, int ntok,
                                                         uint32_t* __restrict__ sid, int* __restrict__ stok,
                                                         uint4* __restrict__ table, long long nvec) {
  constexpr int kGroups = kChunk / kRankTokens, N = kChunk / 256;
  __shared__ int part[4][kRankTokens];
  const unsigned rank_blocks = (unsigned)(ntok + kRankTokens - 1) / kRankTokens;
  if (blockIdx.x >= rank_blocks) {
    const long long step = (long long)(gridDim.x - rank_blocks) * 256;
    for (long long i = (long long)(blockIdx.x - rank_blocks) * 256 + threadIdx.x; i < nvec; i += step)
      table[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int base = (int)(blockIdx.x / kGroups) * kChunk, g0 = (int)(blockIdx.x % kGroups) * kRankTokens;
  const int n = ntok - base < kChunk ? ntok - base : kChunk;
  if (g0 >= n) return;
  const int tid = threadIdx.x, own = g0 / 256;   // the tokens of the block stand in this 256
  // a key at a place behind the block's tokens counts where it is smaller, one
  // before where it is not larger: key + 1 or key, against the token's key + 1
  uint32_t key[N], kown = kNoKey;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int p = i * 256 + tid;
    uint32_t k = p < n ? token_key(ids[base + p], V) : kNoKey;
    if (i == own) {
      kown = k;
      k = kNoKey;
    }
    key[i] = i > own ? k + 1 : k;
  }
  uint32_t above[kRankTokens];
  int count[kRankTokens];
#pragma unroll
  for (int g = 0; g < kRankTokens; ++g) {
    const int p = g0 + g;
    above[g] = (p < n ? token_key(ids[base + p], V) : 0) + 1;
    count[g] = kown + (own * 256 + tid >= p) < above[g];
  }
#pragma unroll
  for (int g = 0; g < kRankTokens; ++g)
#pragma unroll
    for (int i = 0; i < N; ++i) count[g] += key[i] < above[g];
#pragma unroll
  for (int g = 0; g < kRankTokens; g += 2) {      // two counts of at most kChunk / 4 in a register
    const int c = wave_count(count[g] | count[g + 1] << 16);
    if ((tid & 63) == 0) {
      part[tid >> 6][g] = c & 0xFFFF;
      part[tid >> 6][g + 1] = c >> 16;
    }
  }
  __syncthreads();
  if (tid < kRankTokens && g0 + tid < n) {
    const int at = base + part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
    sid[at] = token_key(ids[base + g0 + tid], V);
    stok[at] = base + g0 + tid;
  }
}

// 2. lists of `len` sorted tokens -> lists of kLists * len.  A block takes 64 neighbours of
// a list, one a lane, and each of its waves searches a quarter of the other lists, four at
// once: the lanes' searches run side by side through the same few lines.
__global__ void __launch_bounds__(256) embed_merge_kernel(const uint32_t* __restrict__ sid, const int* __restrict__ stok,
                                                          int ntok, int len, uint32_t* __restrict__ osid,
                                                          int* __restrict__ ostok) {
  constexpr int N = kLists / 4;
  __shared__ int counts[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i0 = blockIdx.x * 64, i = i0 + lane, list = i0 / len, mine = list % kLists;
  const long long first = (long long)(list - mine) * len;
  const uint32_t id = i < ntok ? sid[i] : 0;
  long long start[N];
  int lo[N], hi[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int l = wave * N + k;
    start[k] = first + (long long)l * len;
    lo[k] = 0;
    hi[k] = l == mine || start[k] >= ntok ? 0 : (int)(ntok - start[k] < len ? ntok - start[k] : len);
  }
  for (int rest = len; rest; rest >>= 1) {
    uint32_t at[N];
#pragma unroll
    for (int k = 0; k < N; ++k) at[k] = lo[k] < hi[k] ? sid[start[k] + ((lo[k] + hi[k]) >> 1)] : 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (lo[k] < hi[k]) {
        const int mid = (lo[k] + hi[k]) >> 1;
        if (at[k] < id + (wave * N + k < mine)) lo[k] = mid + 1;   // tokens of an earlier list go first
        else hi[k] = mid;
      }
  }
  counts[wave][lane] = (lo[0] + lo[1]) + (lo[2] + lo[3]);
  __syncthreads();
  if (wave == 0 && i < ntok) {
    const long long at = first + (i - list * (long long)len) + ((counts[0][lane] + counts[1][lane]) + (counts[2][lane] + counts[3][lane]));
    osid[at] = id;
    ostok[at] = stok[i];
  }
}

struct EmbedGradArgs {
  const void* dY;
  void* dE;
  const uint32_t* sid;   // sorted ids, V behind the last token
  const int* stok;       // their rows
  float* part;           // [pieces][2][D]: the sums of a piece's first and last run that cross its borders
  uint32_t V;
  int ntok, D, pieces, slices;
  float scale;
};

// N columns of a table row, or of a partial sum
template <int N, typename GT> __device__ inline void store_grad(GT* p, const float* acc, float scale) {
  constexpr int W = N * sizeof(GT) < 16 ? N : 16 / sizeof(GT);
  struct alignas(W * sizeof(GT)) Part { GT v[W]; };
#pragma unroll
  for (int e = 0; e < N / W; ++e) {
    Part o;
#pragma unroll
    for (int j = 0; j < W; ++j) o.v[j] = f2el<GT>(acc[e * W + j] * scale);
    *reinterpret_cast<Part*>(p + e * W) = o;
  }
}

// 3.  PAST: rows of dY past the caches.
template <typename T, typename GT, bool PAST>
__global__ void __launch_bounds__(64 * kPieceWaves) embed_grad_kernel(const EmbedGradArgs a) {
  constexpr int W = Pack<T>::W, R = kWaveRows;     // columns of a lane, rows of a wave
  __shared__ float left[kPieceWaves][64][W], right[kPieceWaves][64][W];   // sums of a wave's run that crosses its ends
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long units = (long long)a.pieces * a.slices;
  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int piece = (int)(unit / a.slices), col = ((int)(unit % a.slices) * 64 + lane) * W;
    const bool on = col < a.D;
    const int p0 = piece * kPiece, n = a.ntok - p0 < kPiece ? a.ntok - p0 : kPiece;
    const uint32_t kid = lane < n ? a.sid[p0 + lane] : a.V;
    // (a row of dY whatever a workspace holds that another stream has written over)
    const int tok = lane < n ? (int)min((uint32_t)a.stok[p0 + lane], (uint32_t)(a.ntok - 1)) : 0;
    const uint32_t before = p0 > 0 ? a.sid[p0 - 1] : a.V + 1, behind = p0 + n < a.ntok ? a.sid[p0 + n] : a.V + 1;
    auto id_at = [&](int i) -> uint32_t {          // of the piece's places and the two beside it
      return i < 0 ? before : i < n ? (uint32_t)__builtin_amdgcn_readlane(kid, i) : behind;
    };
    const int i0 = wave * R, i1 = i0 + R < n ? i0 + R : n;
    Pack<T> v[R];
#pragma unroll
    for (int u = 0; u < R; ++u)
      if (i0 + u < i1) {
        const long long row = __builtin_amdgcn_readlane(tok, i0 + u);
        const Pack<T>* const p = reinterpret_cast<const Pack<T>*>(reinterpret_cast<const T*>(a.dY) + row * a.D + col);
        const bool token = id_at(i0 + u) < a.V;
        if (on && token) {
          if constexpr (PAST) v[u].r = __builtin_nontemporal_load(&p->r);
          else v[u] = *p;
        }
      }
    float acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = 0.f;
    bool crosses = i0 < i1 && id_at(i0 - 1) == id_at(i0);   // the run began before this wave's rows
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int i = i0 + u;
      if (i >= i1) break;
      const uint32_t id = id_at(i);
      if (id >= a.V) break;                        // no tokens behind
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] += v[u].get(j);
      const bool ends = id_at(i + 1) != id;
      if (ends || i + 1 == i1) {
        if (ends && !crosses) {
          if (on) store_grad<W>(reinterpret_cast<GT*>(a.dE) + (long long)id * a.D + col, acc, a.scale);
        } else {
          float* const to = crosses ? left[wave][lane] : right[wave][lane];
#pragma unroll
          for (int j = 0; j < W; ++j) to[j] = acc[j];
        }
        crosses = false;
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = 0.f;
      }
    }
    __syncthreads();
    // The wave in whose rows a run begins adds it up, the first wave also the one that
    // began in an earlier piece.
    auto finish = [&](uint32_t id, bool inside, int w) __attribute__((always_inline)) {
      const int end = 63 - __builtin_clzll(__ballot(kid == id));
      for (; w * R <= end; ++w)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] += left[w][lane][j];
      const bool whole = inside && id_at(end + 1) != id;
      if (!on) return;
      if (whole) store_grad<W>(reinterpret_cast<GT*>(a.dE) + (long long)id * a.D + col, acc, a.scale);
      else store_grad<W>(a.part + ((long long)piece * 2 + inside) * a.D + col, acc, 1.f);
    };
    if (wave == 0 && id_at(0) == before && before < a.V) {
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = 0.f;
      finish(before, false, 0);
    }
    if (i0 < i1) {
      const uint32_t id = id_at(i1 - 1);
      // its last run goes on behind its rows and did not begin before them
      if (id < a.V && id_at(i1) == id && !(id_at(i0) == id && id_at(i0 - 1) == id)) {
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = right[wave][lane][j];
        finish(id, true, wave + 1);
      }
    }
    __syncthreads();                               // the sums have been read
  }
}

// 4. the runs that begin in a piece and go on behind it
template <typename GT>
__global__ void __launch_bounds__(64 * kJoinWaves) embed_join_kernel(const EmbedGradArgs a) {
  __shared__ float sum[kJoinWaves - 1][64][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slices = (a.D + kJoinSlice - 1) / kJoinSlice;
  const long long units = (long long)(a.pieces - 1) * slices;
  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int piece = (int)(unit / slices), col = (int)(unit % slices) * kJoinSlice + lane * 8;
    const int p0 = piece * kPiece, p1 = p0 + kPiece;
    const uint32_t id = a.sid[p1 - 1];
    if (id >= a.V || a.sid[p1] != id || (p0 > 0 && a.sid[p0] == id && a.sid[p0 - 1] == id)) continue;
    int end = piece + 1;                     // the piece in which the run ends
    for (;;) {
      const long long q = (long long)(end + lane + 1) * kPiece;   // the lane's piece goes on behind its end?
      const unsigned long long over = __ballot(q < a.ntok && a.sid[q < a.ntok ? q : 0] == id);
      if (~over) {
        end += __builtin_ctzll(~over);
        break;
      }
      end += 64;
    }
    const bool on = col < a.D;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    auto add = [&](long long slot) __attribute__((always_inline)) {
      const float* s = a.part + slot * a.D + col;
      const Vec<float, 4> x = *reinterpret_cast<const Vec<float, 4>*>(s);
      const Vec<float, 4> y = *reinterpret_cast<const Vec<float, 4>*>(s + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j] += x.v[j];
        acc[j + 4] += y.v[j];
      }
    };
    if (on) {
      if (wave == 0) add(2LL * piece + 1);
#pragma unroll 4
      for (int p = piece + 1 + wave; p <= end; p += kJoinWaves) add(2LL * p);
    }
    __syncthreads();                         // the last unit's sums have been read
    if (wave > 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[wave - 1][lane][j] = acc[j];
    __syncthreads();
    if (wave == 0 && on) {
#pragma unroll
      for (int w = 0; w < kJoinWaves - 1; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += sum[w][lane][j];
      store_grad<8>(reinterpret_cast<GT*>(a.dE) + (long long)id * a.D + col, acc, a.scale);
    }
  }
}

struct EmbedWs {
  size_t sid[2], stok[2], part, bytes;
  EmbedWs(int T, long long D) {
    Bump b;
    for (int i = 0; i < (T > kChunk ? 2 : 1); ++i) {
      sid[i] = b.take((size_t)T * 4);
      stok[i] = b.take((size_t)T * 4);
    }
    part = b.take((size_t)ceil_div(T, kPiece) * 2 * D * 4);
    bytes = b.off;
  }
};

static sl_status check_embed(const sl_layout* lay, int64_t D) {
  sl_status st = check_tokens(lay);
  if (st != SL_OK) return st;
  if (lay->batch * (long long)lay->seq_len > (1LL << 26)) SL_FAIL(SL_ERR_RANGE, "more than 2^26 tokens");
  if (D < 8 || D % 8 || D > 65536) SL_FAIL(SL_ERR_SHAPE, "d_model %lld must be a multiple of 8 in [8, 65536]", (long long)D);
  return SL_OK;
}

static sl_status check_embed_call(sl_dtype dt, const sl_layout* lay, int64_t V, int64_t D, float scale) {
  sl_status st = check_dtype(dt);
  if (st == SL_OK) st = check_embed(lay, D);
  if (st != SL_OK) return st;
  if (V < 1 || V > (1LL << 30)) SL_FAIL(SL_ERR_RANGE, "vocabulary of %lld outside [1, 2^30]", (long long)V);
  if (!(scale - scale == 0.f)) SL_FAIL(SL_ERR_RANGE, "scale is not finite");
  return SL_OK;
}

template <typename T>
static void launch_fwd(const void* E, const int32_t* ids, int64_t V, int64_t D, int ntok, float scale, void* Y,
                       hipStream_t s) {
  const int nvec = (int)(D * sizeof(T) / 16);
  int lg = 0;
  while (lg < 8 && (1 << lg) < nvec) ++lg;
  const int cols = ceil_div(nvec, 1 << lg), rows = 256 >> lg;
  // four rows in flight a thread where that leaves 16 blocks to a CU (one row, four in us: 2048 rows of
  // 4096 bf16 7.4, 8.2, 4096 13.5, 14.4, 8192, where they do, 27.3, 26.9; of 1000 fp32 4096 7.2, 7.9,
  // 16384 28.3, 27.2)
  if ((long long)ceil_div(ntok, rows * 4) * cols >= 4096)
    hipLaunchKernelGGL((embed_fwd_kernel<T, 4>), dim3(walk_grid(ceil_div(ntok, rows * 4), (1 << 23) / cols).x, cols), dim3(256), 0, s,
                       (const T*)E, ids, (uint32_t)V, nvec, ntok, lg, scale, (T*)Y);
  else
    hipLaunchKernelGGL((embed_fwd_kernel<T, 1>), dim3(walk_grid(ceil_div(ntok, rows), (1 << 23) / cols).x, cols), dim3(256), 0, s,
                       (const T*)E, ids, (uint32_t)V, nvec, ntok, lg, scale, (T*)Y);
}

template <typename T, typename GT>
static void launch_grad(const EmbedGradArgs& a, hipStream_t s) {
  // Rows of 32 MiB and more go past the caches, each read once (in us, through them and past, tokens of 4096
  // columns in bf16: 2048 tokens and 32000 rows in fp32 99, 102, 4096 116, 114, 8192 142, 132; with the
  // kernel before it that writes the rows 109, 109, 133, 128, 169, 163; 32768 tokens, 128256 rows in bf16 282, 266).
  const dim3 grid = walk_grid((long long)a.pieces * a.slices), block(64 * kPieceWaves);
  if ((long long)a.ntok * a.D * (long long)sizeof(T) >= 32LL << 20)
    hipLaunchKernelGGL((embed_grad_kernel<T, GT, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((embed_grad_kernel<T, GT, false>), grid, block, 0, s, a);
  if (a.pieces > 1)
    hipLaunchKernelGGL(embed_join_kernel<GT>, walk_grid((long long)(a.pieces - 1) * ceil_div(a.D, kJoinSlice)),
                       dim3(64 * kJoinWaves), 0, s, a);
}

}  // namespace sl

using namespace sl;

extern "C" sl_status sl_embed_fwd(sl_dtype dt, const sl_layout* lay, int64_t vocab, int64_t d_model, float scale,
                                  const void* E, const int32_t* ids, void* Y, void* stream) {
  if (!E || !ids || !Y) SL_FAIL(SL_ERR_NULL, "E, ids and Y required");
  sl_status st = check_embed_call(dt, lay, vocab, d_model, scale);
  if (st != SL_OK) return st;
  if (!aligned16(E) || !aligned16(ids) || !aligned16(Y)) SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  st = check_arch();
  if (st != SL_OK) return st;
  const int T = lay->batch * lay->seq_len;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dt == SL_BF16) launch_fwd<bf16>(E, ids, vocab, d_model, T, scale, Y, s);
  else launch_fwd<float>(E, ids, vocab, d_model, T, scale, Y, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}

extern "C" size_t sl_embed_workspace_bytes(const sl_layout* lay, int64_t d_model) {
  if (check_embed(lay, d_model) != SL_OK) return 0;
  return EmbedWs(lay->batch * lay->seq_len, d_model).bytes;
}

extern "C" sl_status sl_embed_bwd(sl_dtype dt, const sl_layout* lay, int64_t vocab, int64_t d_model, float scale,
                                  const int32_t* ids, const void* dY, sl_dtype grad_dt, void* dE, void* ws,
                                  size_t ws_bytes, void* stream) {
  if (!ids || !dY || !dE) SL_FAIL(SL_ERR_NULL, "ids, dY and dE required");
  sl_status st = check_embed_call(dt, lay, vocab, d_model, scale);
  if (st == SL_OK) st = check_dtype(grad_dt);
  if (st != SL_OK) return st;
  if (!aligned16(ids) || !aligned16(dY) || !aligned16(dE) || !aligned16(ws))
    SL_FAIL(SL_ERR_ALIGN, "every pointer must be 16-byte aligned");
  const int T = lay->batch * lay->seq_len;
  const EmbedWs at(T, d_model);
  if (!ws || ws_bytes < at.bytes)
    SL_FAIL(SL_ERR_WORKSPACE, "embedding workspace too small (%zu bytes, %zu needed)", ws_bytes, at.bytes);
  st = check_arch();
  if (st != SL_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* const w = reinterpret_cast<char*>(ws);
  auto sid = [&](int i) { return reinterpret_cast<uint32_t*>(w + at.sid[i]); };
  auto stok = [&](int i) { return reinterpret_cast<int*>(w + at.stok[i]); };
  const uint32_t V = (uint32_t)vocab;
  const long long nvec = vocab * d_model / (grad_dt == SL_BF16 ? 8 : 4);
  hipLaunchKernelGGL(embed_rank_kernel, dim3((unsigned)ceil_div(T, kRankTokens) + walk_grid((nvec + 255) / 256, 1 << 22).x),
                     dim3(256), 0, s, ids, V, T, sid(0), stok(0), reinterpret_cast<uint4*>(dE), nvec);
  int cur = 0;
  for (long long len = kChunk; len < T; len *= kLists, cur ^= 1)
    hipLaunchKernelGGL(embed_merge_kernel, dim3((unsigned)ceil_div(T, 64)), dim3(256), 0, s, sid(cur), stok(cur),
                       T, (int)len, sid(cur ^ 1), stok(cur ^ 1));
  EmbedGradArgs a{};
  a.dY = dY; a.dE = dE; a.sid = sid(cur); a.stok = stok(cur);
  a.part = reinterpret_cast<float*>(w + at.part);
  a.V = V; a.ntok = T; a.D = (int)d_model; a.scale = scale;
  a.pieces = ceil_div(T, kPiece);
  a.slices = ceil_div(d_model, dt == SL_BF16 ? 512 : 256);
  if (dt == SL_BF16 && grad_dt == SL_BF16) launch_grad<bf16, bf16>(a, s);
  else if (dt == SL_BF16) launch_grad<bf16, float>(a, s);
  else if (grad_dt == SL_BF16) launch_grad<float, bf16>(a, s);
  else launch_grad<float, float>(a, s);
  SL_HIP(hipGetLastError());
  return SL_OK;
}
