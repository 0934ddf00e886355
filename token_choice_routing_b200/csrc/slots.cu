// Slots sorted by expert from any routing (moe_sort_slots), and rows moved to that order and
// back (moe_permute, moe_unpermute) with their gradients.
//
// A slot s = t K + k carries the expert id its token chose, or an id outside [0, N) when it
// takes no expert. The sorted order is the stable one, (expert, slot): a slot's row is
//   offsets[id] + #{s' < s : id_s' = id}.
// unpermute: y[t] = base[t] + sum_k w[t,k] ys[row(t,k)], and its gradient
//   dys[row(t,k)] = w[t,k] dy[t],  dw[t,k] = <dy[t], ys[row(t,k)]>.
// Every slot has a row of its own, so all of them are gathers or one-to-one copies: no
// floating-point atomics, and results that do not depend on the order of execution.
#include "rows.cuh"

#include <algorithm>
#include <climits>

namespace moe {

// ---------------------------------------------------------------------------------------
// Sort. A counting sort over contiguous chunks of slots, one chunk per CTA: sort_count_kernel
// writes each chunk's slots per expert, sort_place_kernel adds up the chunks below its own,
// ranks its slots and writes their rows. Integer sums only, so the result is exact whatever
// the order.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxChunks = 148;
constexpr int kSortMinChunk = 4096;   // slots per CTA below which more CTAs are not worth it

struct SortShape {
  long long S;
  int chunks;
  long long per_chunk;  // a multiple of kSortThreads: every warp's share is a multiple of 32
};

static SortShape sort_shape(int T, int K) {
  SortShape s;
  s.S = (long long)T * K;
  long long n = std::max<long long>(1, std::min<long long>(kSortMaxChunks, (s.S + kSortMinChunk - 1) / kSortMinChunk));
  s.per_chunk = std::max<long long>(1, ((s.S + n - 1) / n + kSortThreads - 1) / kSortThreads) * kSortThreads;
  s.chunks = (int)std::max<long long>(1, (s.S + s.per_chunk - 1) / s.per_chunk);
  return s;
}

size_t sort_workspace_bytes(int T, int K, int N) {
  return 256 + align_up(sizeof(int32_t) * (size_t)N * sort_shape(T, K).chunks, 256);
}

struct SortArgs {
  const void* ids;
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm_tok;
  int32_t* slot_row;
  uint32_t* status;
  int32_t* table;  // [chunks][N] slots per expert of each chunk
  long long S, per_chunk;
  int K, N, chunks;
};

template <typename Id>
__device__ __forceinline__ int sort_id(const SortArgs& a, long long s, long long end) {
  if (s >= end) return -1;
  const Id v = __ldg(static_cast<const Id*>(a.ids) + s);
  return (v >= 0 && v < (Id)a.N) ? (int)v : -1;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  pdl_wait_then_release();
  extern __shared__ int s_hist[];
  for (int g = threadIdx.x; g < a.N; g += kSortThreads) s_hist[g] = 0;
  __syncthreads();
  const long long begin = a.per_chunk * blockIdx.x, end = min(a.S, begin + a.per_chunk);
  for (long long s = begin + threadIdx.x; s < end; s += kSortThreads) {
    const int id = sort_id<Id>(a, s, end);
    if (id >= 0) atomicAdd(&s_hist[id], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < a.N; g += kSortThreads) a.table[(size_t)blockIdx.x * a.N + g] = s_hist[g];
}

// Shared memory: whist [warps][N] (a warp's slots per expert, then its first row per expert),
// tot [N] and pre [N] (all chunks, and the chunks below this one), part [32].
template <typename Id>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
  pdl_wait_then_release();
  extern __shared__ int s_mem[];
  const int N = a.N, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int* whist = s_mem;
  int* tot = whist + kSortWarps * N;
  int* pre = tot + N;
  int* part = pre + N;
  for (int i = tid; i < kSortWarps * N + 2 * N; i += kSortThreads) s_mem[i] = 0;
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  __syncthreads();
  const long long per_warp = a.per_chunk / kSortWarps;
  const long long begin = a.per_chunk * blockIdx.x + per_warp * w;
  const long long end = min(a.S, begin + per_warp);
  int* mine = whist + w * N;
  for (long long s = begin + lane; s < end; s += 32) {
    const int id = sort_id<Id>(a, s, end);
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  if (a.chunks > 1) {
    // column sums of the table: consecutive threads take consecutive entries, so each thread's
    // expert changes with its step; integer atomics make the sums exact in any order
    for (int i = tid; i < a.chunks * N; i += kSortThreads) {
      const int c = i / N, g = i - c * N;
      const int v = __ldg(a.table + i);
      if (v) {
        atomicAdd(&tot[g], v);
        if (c < (int)blockIdx.x) atomicAdd(&pre[g], v);
      }
    }
  }
  __syncthreads();
  // first row of each warp's slots per expert, relative to the chunk's first row of that expert
  int total = 0;
  if (tid < N) {
    int run = 0;
    for (int ww = 0; ww < kSortWarps; ++ww) {
      const int v = whist[ww * N + tid];
      whist[ww * N + tid] = run;
      run += v;
    }
    total = a.chunks > 1 ? tot[tid] : run;
  }
  // exclusive scan of the totals over the experts (N <= kSortThreads)
  int scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) part[w] = scan;
  __syncthreads();
  if (w == 0) {
    int v = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    part[lane] = v;
  }
  __syncthreads();
  const int first = scan - total + (w > 0 ? part[w - 1] : 0);  // offsets[tid]
  if (tid < N) {
    if (blockIdx.x == 0) {
      a.counts[tid] = total;
      a.offsets[tid] = first;
      if (tid == N - 1) a.offsets[N] = first + total;
    }
    const int base = first + pre[tid];
    for (int ww = 0; ww < kSortWarps; ++ww) whist[ww * N + tid] += base;
  }
  __syncthreads();
  for (long long s0 = begin; s0 < end; s0 += 32) {  // warp-uniform trip count
    const long long s = s0 + lane;
    const int id = sort_id<Id>(a, s, end);
    const unsigned peers = __match_any_sync(0xffffffffu, id);
    int row = -1;
    if (id >= 0) row = mine[id] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && lane == 31 - __clz(peers)) mine[id] += __popc(peers);
    __syncwarp();
    if (s < end) {
      a.slot_row[s] = row;
      if (row >= 0) a.perm_tok[row] = (int)((unsigned)s / (unsigned)a.K);
    }
  }
}

template <typename Id>
static int sort_run(const SortArgs& a, cudaStream_t st) {
  const size_t count_smem = sizeof(int) * (size_t)a.N;
  const size_t place_smem = sizeof(int) * ((size_t)(kSortWarps + 2) * a.N + 32);
  if (place_smem > 48 * 1024 &&
      cudaFuncSetAttribute(sort_place_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)place_smem) !=
          cudaSuccess)
    return MOE_ERR_CUDA;
  if (a.chunks > 1) {
    const int r = launch_pdl(sort_count_kernel<Id>, dim3(a.chunks), dim3(kSortThreads), count_smem, st, a);
    if (r != MOE_OK) return r;
  }
  return launch_pdl(sort_place_kernel<Id>, dim3(a.chunks), dim3(kSortThreads), place_smem, st, a);
}

int launch_sort_slots(int T, int K, int N, const void* ids, int id_bytes, int32_t* counts, int32_t* offsets,
                      int32_t* perm_tok, int32_t* slot_row, void* ws, cudaStream_t st) {
  const SortShape sh = sort_shape(T, K);
  SortArgs a{};
  a.ids = ids;
  a.counts = counts;
  a.offsets = offsets;
  a.perm_tok = perm_tok;
  a.slot_row = slot_row;
  a.status = ws_ptr<uint32_t>(ws, 0);
  a.table = ws_ptr<int32_t>(ws, 256);
  a.S = sh.S;
  a.per_chunk = sh.per_chunk;
  a.K = K;
  a.N = N;
  a.chunks = sh.chunks;
  return id_bytes == 8 ? sort_run<long long>(a, st) : sort_run<int>(a, st);
}

// ---------------------------------------------------------------------------------------
// Row movement. Rows are read and written in pieces of V elements, consecutive pieces by
// consecutive lanes: 16 bytes where the layout allows it, single elements otherwise. A warp
// takes one token's columns [c0, c0 + 32 V NV), NV pieces a lane, and its lanes hold the token's
// slots (lane k: slot k), compacted four at a time so that all their pieces are in flight
// together.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
// Pieces a lane holds of each row (NV) and CTAs a multiprocessor (at most 64 registers a thread). With
// four slots at a time a lane has 8 row pieces and 2 of the token in flight: 32 warps x 5 KB cover
// the latency of HBM. Measured at T = 65536, d = 2048, K = 8, bf16 (unpermute): NV 2 with 4 CTAs
// 245 us (6.6 TB/s, the copy rate), NV 1 with 6 or 8 CTAs 271 and 248 us, NV 2 with 3 CTAs 266 us.
constexpr int kVecPieces = 2;
constexpr int kRowCtas = 4;
// Single elements (odd widths, unaligned rows): 8 a lane; 4 a lane measured 122 against 97 us
// (T = 16384, d = 1537, K = 8, bf16).
constexpr int kElemPieces = 8;

// The slot's row, -1 for none. A row past the buffer is skipped and recorded.
__device__ __forceinline__ int slot_row_checked(const int32_t* slot_row, long long t, int k, int K, long long rows,
                                                uint32_t* status) {
  if (k >= K) return -1;
  const int row = __ldg(slot_row + t * K + k);
  if (row >= rows) {
    if (status) atomicOr(status, kStatusBounds);
    return -1;
  }
  return row < 0 ? -1 : row;
}

struct RowArgs {
  const void* tok;     // token-side input [T, d] (x, dy) or base, ldt
  const void* rows_in; // row-side input [rows, d] (ys, dxs), ldr
  const uint8_t* scales;  // 8-bit rows: one scale byte per 32 columns (rows_in holds the codes)
  void* tok_out;       // token-side output, ldto
  void* rows_out;      // row-side output, ldro
  const float* w;      // [T, K], or null for weights of one
  float* dw;           // [T, K], or null
  const int32_t* slot_row;
  uint32_t* status;
  long long ldt, ldr, ldto, ldro, rows;
  int T, K, d;
  int items;           // T * chunks: a warp's work is one chunk of one token
  FastDiv chunks;      // chunks of a token: ceil(d / (32 V NV))
};

// The next (up to four) slots with a row, from the mask m: their rows (-1 past the end) and weights.
__device__ __forceinline__ void next_slots(unsigned& m, int row, float w, int (&r)[4], float (&wk)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = m ? __ffs(m) - 1 : 0;
    r[u] = __shfl_sync(0xffffffffu, row, k);
    wk[u] = __shfl_sync(0xffffffffu, w, k);
    if (m == 0u) r[u] = -1;
    m &= m - 1u;
  }
}

// tok_out[t] = tok[t] + sum_k w[t,k] rows_in[slot_row[t,k]], fp32 sums in slot order.
template <typename E, int V, int NV>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) collect_kernel(RowArgs a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (item >= (uint32_t)a.items) return;
  const long long t = a.chunks.quotient(item);
  const int c0 = (int)(item - (uint32_t)t * a.chunks.d) * (32 * V * NV) + lane * V;
  const int row = slot_row_checked(a.slot_row, t, lane, a.K, a.rows, a.status);
  const float w = (a.w && lane < a.K) ? __ldg(a.w + t * a.K + lane) : 1.f;
  const E* base = static_cast<const E*>(a.tok) + t * a.ldt;
  const E* rows_in = static_cast<const E*>(a.rows_in);
  float acc[NV][V];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = c0 + v * 32 * V;
    Piece<E, V> b;
    b.zero();
    if (a.tok && c < a.d) b.load_own(base + c);
    b.get(acc[v]);
  }
  unsigned m = __ballot_sync(0xffffffffu, row >= 0);
  while (m) {
    int r[4];
    float wk[4];
    next_slots(m, row, w, r, wk);
    Piece<E, V> p[4][NV];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const E* src = rows_in + (long long)r[u] * a.ldr;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = c0 + v * 32 * V;
        p[u][v].zero();
        if (r[u] >= 0 && c < a.d) p[u][v].load(src + c);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (r[u] < 0) continue;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[V];
        p[u][v].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[v][j] = fmaf(wk[u], f[j], acc[v][j]);
      }
    }
  }
  E* out = static_cast<E*>(a.tok_out) + t * a.ldto;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = c0 + v * 32 * V;
    if (c >= a.d) continue;
    Piece<E, V> o;
    o.set(acc[v]);
    o.store(out + c);
  }
}

// rows_out[slot_row[t,k]] = w[t,k] tok[t] (w null: a copy).
template <typename E, int V, int NV>
__global__ void __launch_bounds__(kRowThreads) spread_kernel(RowArgs a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (item >= (uint32_t)a.items) return;
  const long long t = a.chunks.quotient(item);
  const int c0 = (int)(item - (uint32_t)t * a.chunks.d) * (32 * V * NV) + lane * V;
  const int row = slot_row_checked(a.slot_row, t, lane, a.K, a.rows, a.status);
  const float w = (a.w && lane < a.K) ? __ldg(a.w + t * a.K + lane) : 1.f;
  unsigned m = __ballot_sync(0xffffffffu, row >= 0);
  if (m == 0u) return;
  const E* src = static_cast<const E*>(a.tok) + t * a.ldt;
  Piece<E, V> p[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = c0 + v * 32 * V;
    p[v].zero();
    if (c < a.d) p[v].load(src + c);
  }
  for (; m; m &= m - 1u) {
    const int k = __ffs(m) - 1;
    const float wk = __shfl_sync(0xffffffffu, w, k);
    E* dst = static_cast<E*>(a.rows_out) + (long long)__shfl_sync(0xffffffffu, row, k) * a.ldro;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = c0 + v * 32 * V;
      if (c >= a.d) continue;
      Piece<E, V> o = p[v];
      if (a.w) {
        float f[V];
        p[v].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] *= wk;
        o.set(f);
      }
      o.store(dst + c);
    }
  }
}

// rows_out[slot_row[t,k]] = w[t,k] tok[t] (rows_out null: not written) and dw[t,k] = <tok[t],
// rows_in[slot_row[t,k]]>, 0 for a slot without a row. WPT warps share a token, each every
// WPT-th chunk of its columns; a dot product is summed in fp32 per lane, over the lanes by a
// fixed shuffle tree and over the warps in order, so it does not depend on timing.
template <typename E, int V, int NV, bool CODES>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) spread_dot_kernel(RowArgs a, int wpt) {
  pdl_wait_then_release();
  __shared__ float part[kRowWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % wpt;
  const long long t = (long long)blockIdx.x * (kRowWarps / wpt) + warp / wpt;
  const int nb = (a.d + 31) / 32;
  float mydw = 0.f;
  if (t < a.T) {
    const int row = slot_row_checked(a.slot_row, t, lane, a.K, a.rows, a.status);
    const float w = (a.w && lane < a.K) ? __ldg(a.w + t * a.K + lane) : 1.f;
    const E* src = static_cast<const E*>(a.tok) + t * a.ldt;
    unsigned m = __ballot_sync(0xffffffffu, row >= 0);
    while (m) {
      const unsigned these = m;
      int r[4];
      float wk[4], dot[4] = {0.f, 0.f, 0.f, 0.f};
      next_slots(m, row, w, r, wk);
      for (int c0 = sub * 32 * V * NV + lane * V; c0 - lane * V < a.d; c0 += wpt * 32 * V * NV) {
        Piece<E, V> g[NV], p[4][NV];
        CodePiece<V> q[4][NV];
        uint32_t sb[4][NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = c0 + v * 32 * V;
          g[v].zero();
          if (c < a.d) g[v].load(src + c);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (r[u] < 0) continue;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int c = c0 + v * 32 * V;
            const long long at = (long long)r[u] * a.ldr + c;
            if constexpr (CODES) {
              sb[u][v] = 0;
              if (c < a.d) {
                q[u][v] = load_codes<V>(static_cast<const int8_t*>(a.rows_in) + at);
                sb[u][v] = __ldg(a.scales + (long long)r[u] * nb + (c >> 5));
              }
            } else {
              p[u][v].zero();
              if (c < a.d) p[u][v].load(static_cast<const E*>(a.rows_in) + at);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (r[u] < 0) continue;
          E* dst = static_cast<E*>(a.rows_out) + (long long)r[u] * a.ldro;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int c = c0 + v * 32 * V;
            if (c >= a.d) continue;
            float gf[V];
            g[v].get(gf);
            if constexpr (CODES) {
              float s = 0.f;  // the sum over a piece, then its scale: a power of two, exact
#pragma unroll
              for (int j = 0; j < V; j += 4) {
                float f[4];
                codes_to_float(q[u][v].word[j / 4], f);
#pragma unroll
                for (int i = 0; i < (V < 4 ? V : 4); ++i) s = fmaf(gf[j + i], f[i], s);
              }
              dot[u] = fmaf(s, scale_value(sb[u][v]), dot[u]);
            } else {
              float pf[V];
              p[u][v].get(pf);
#pragma unroll
              for (int j = 0; j < V; ++j) dot[u] = fmaf(gf[j], pf[j], dot[u]);
            }
            if (a.rows_out) {
              Piece<E, V> o;
#pragma unroll
              for (int j = 0; j < V; ++j) gf[j] *= wk[u];
              o.set(gf);
              o.store(dst + c);
            }
          }
        }
      }
      unsigned left = these;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float s = dot[u];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (left && lane == __ffs(left) - 1) mydw = s;
        left &= left - 1u;
      }
    }
  }
  if (wpt > 1) {
    part[warp][lane] = mydw;
    __syncthreads();
    if (sub == 0)
      for (int i = 1; i < wpt; ++i) mydw += part[warp + i][lane];
  }
  if (sub == 0 && t < a.T && lane < a.K) a.dw[t * a.K + lane] = mydw;
}

// Chunks per token and the grid over them; false when the index space is too large for any
// buffer of this GPU's memory.
static bool row_items(RowArgs& a, int chunk) {
  const int n = (int)(((long long)a.d + chunk - 1) / chunk);
  if ((long long)a.T * n >= (long long)INT_MAX) return false;
  a.chunks = FastDiv((uint32_t)n);
  a.items = a.T * n;
  return true;
}

template <typename E, int V, int NV>
static int collect_go(RowArgs a, cudaStream_t st) {
  if (!row_items(a, 32 * V * NV)) return MOE_ERR_UNSUPPORTED;
  return launch_pdl(collect_kernel<E, V, NV>, dim3((a.items + kRowWarps - 1) / kRowWarps), dim3(kRowThreads), 0, st, a);
}

template <typename E>
static int collect_run(const RowArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool vec = a.d % V == 0 && rows_aligned16(a.rows_in, a.ldr, sizeof(E)) &&
                   (!a.tok || rows_aligned16(a.tok, a.ldt, sizeof(E))) && rows_aligned16(a.tok_out, a.ldto, sizeof(E));
  return vec ? collect_go<E, V, kVecPieces>(a, st) : collect_go<E, 1, kElemPieces>(a, st);
}

template <typename E, int V, int NV>
static int spread_go(RowArgs a, cudaStream_t st) {
  if (!row_items(a, 32 * V * NV)) return MOE_ERR_UNSUPPORTED;
  return launch_pdl(spread_kernel<E, V, NV>, dim3((a.items + kRowWarps - 1) / kRowWarps), dim3(kRowThreads), 0, st, a);
}

template <typename E, int V, int NV, bool CODES>
static int spread_dot_go(const RowArgs& a, cudaStream_t st) {
  // more warps a token while the tokens alone do not fill the GPU and the row has chunks for them
  int wpt = 1;
  while (wpt < kRowWarps && (long long)a.T * wpt < (long long)sm_count() * 16 && a.d > wpt * 32 * V * NV) wpt *= 2;
  const long long per_block = kRowWarps / wpt;
  const dim3 grid((unsigned)((a.T + per_block - 1) / per_block));
  return launch_pdl(spread_dot_kernel<E, V, NV, CODES>, grid, dim3(kRowThreads), 0, st, a, wpt);
}

template <typename E>
static int spread_run(const RowArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool codes = a.scales != nullptr;
  const bool vec = a.d % V == 0 && rows_aligned16(a.tok, a.ldt, sizeof(E)) &&
                   (!a.rows_out || rows_aligned16(a.rows_out, a.ldro, sizeof(E))) &&
                   (!a.rows_in || (codes ? reinterpret_cast<uintptr_t>(a.rows_in) % V == 0
                                         : rows_aligned16(a.rows_in, a.ldr, sizeof(E))));
  if (!a.dw) return vec ? spread_go<E, V, kVecPieces>(a, st) : spread_go<E, 1, kElemPieces>(a, st);
  if (codes) return vec ? spread_dot_go<E, V, kVecPieces, true>(a, st) : spread_dot_go<E, 1, kElemPieces, true>(a, st);
  return vec ? spread_dot_go<E, V, kVecPieces, false>(a, st) : spread_dot_go<E, 1, kElemPieces, false>(a, st);
}

int launch_collect(int T, int K, long long rows, int d, int dtype, const void* rows_in, long long ldr, const float* w,
                   const int32_t* slot_row, const void* base, long long ldb, void* out, long long ldo,
                   uint32_t* status, cudaStream_t st) {
  RowArgs a{};
  a.tok = base;
  a.ldt = ldb;
  a.rows_in = rows_in;
  a.ldr = ldr;
  a.tok_out = out;
  a.ldto = ldo;
  a.w = w;
  a.slot_row = slot_row;
  a.status = status;
  a.rows = rows;
  a.T = T;
  a.K = K;
  a.d = d;
  return dtype == MOE_DTYPE_BF16 ? collect_run<__nv_bfloat16>(a, st)
         : dtype == MOE_DTYPE_F16 ? collect_run<__half>(a, st)
                                  : collect_run<float>(a, st);
}

int launch_spread(int T, int K, long long rows, int d, int dtype, const void* tok, long long ldt, const void* rows_in,
                  long long ldr, const uint8_t* scales, const float* w, const int32_t* slot_row, void* rows_out,
                  long long ldro, float* dw, uint32_t* status, cudaStream_t st) {
  RowArgs a{};
  a.tok = tok;
  a.ldt = ldt;
  a.rows_in = rows_in;
  a.ldr = ldr;
  a.scales = scales;
  a.w = w;
  a.dw = dw;
  a.rows_out = rows_out;
  a.ldro = ldro;
  a.slot_row = slot_row;
  a.status = status;
  a.rows = rows;
  a.T = T;
  a.K = K;
  a.d = d;
  return dtype == MOE_DTYPE_BF16 ? spread_run<__nv_bfloat16>(a, st)
         : dtype == MOE_DTYPE_F16 ? spread_run<__half>(a, st)
                                  : spread_run<float>(a, st);
}

}  // namespace moe
