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
// Row movement. One warp per token; its lanes hold the token's slots (lane k: slot k).
constexpr int kRowThreads = 256;

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
};

// tok_out[t] = tok[t] + sum_k w[t,k] rows_in[slot_row[t,k]], fp32 sums in slot order.
template <typename E, int V>
__global__ void __launch_bounds__(kRowThreads) collect_kernel(RowArgs a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int wpb = kRowThreads / 32;
  for (long long t = (long long)blockIdx.x * wpb + (threadIdx.x >> 5); t < a.T; t += (long long)gridDim.x * wpb) {
    const int row = slot_row_checked(a.slot_row, t, lane, a.K, a.rows, a.status);
    const float w = (a.w && lane < a.K) ? __ldg(a.w + t * a.K + lane) : 1.f;
    const unsigned has = __ballot_sync(0xffffffffu, row >= 0);
    const E* base = static_cast<const E*>(a.tok);
    E* out = static_cast<E*>(a.tok_out) + t * a.ldto;
    for (int c0 = 0; c0 < a.d; c0 += 32 * V) {  // warp-uniform trip count
      const int c = c0 + lane * V;
      const bool ok = c < a.d;
      float acc[V];
      const Piece<E, V> b = (base && ok) ? load_piece<E, V>(base + t * a.ldt + c) : zero_piece<E, V>();
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = elem_to_float<E>(b.e[j]);
      for (unsigned m = has; m; m &= m - 1u) {
        const int k = __ffs(m) - 1;
        const long long r = __shfl_sync(0xffffffffu, row, k);
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (ok) {
          const Piece<E, V> v = load_piece<E, V>(static_cast<const E*>(a.rows_in) + r * a.ldr + c);
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] = fmaf(wk, elem_to_float<E>(v.e[j]), acc[j]);
        }
      }
      if (ok) {
        Piece<E, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.e[j] = float_to_elem<E>(acc[j]);
        store_piece<E, V>(out + c, o);
      }
    }
  }
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// rows_out[slot_row[t,k]] = w[t,k] tok[t], and with dw, dw[t,k] = <tok[t], rows_in[slot_row[t,k]]>
// (fp32 sums per lane, then a fixed shuffle tree; 0 for a slot without a row).
template <typename E, int V, bool DOT, bool CODES>
__global__ void __launch_bounds__(kRowThreads) spread_kernel(RowArgs a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int wpb = kRowThreads / 32;
  const int nb = (a.d + 31) / 32;
  for (long long t = (long long)blockIdx.x * wpb + (threadIdx.x >> 5); t < a.T; t += (long long)gridDim.x * wpb) {
    const int row = slot_row_checked(a.slot_row, t, lane, a.K, a.rows, a.status);
    const float w = (a.w && lane < a.K) ? __ldg(a.w + t * a.K + lane) : 1.f;
    const E* src = static_cast<const E*>(a.tok) + t * a.ldt;
    float mydw = 0.f;
    for (unsigned m = __ballot_sync(0xffffffffu, row >= 0); m; m &= m - 1u) {
      const int k = __ffs(m) - 1;
      const long long r = __shfl_sync(0xffffffffu, row, k);
      const float wk = __shfl_sync(0xffffffffu, w, k);
      float dot = 0.f;
      for (int c = lane * V; c < a.d; c += 32 * V) {
        const Piece<E, V> v = load_piece<E, V>(src + c);
        if (a.rows_out) {
          Piece<E, V> o = v;
          if (a.w) {
#pragma unroll
            for (int j = 0; j < V; ++j) o.e[j] = float_to_elem<E>(wk * elem_to_float<E>(v.e[j]));
          }
          store_piece<E, V>(static_cast<E*>(a.rows_out) + r * a.ldro + c, o);
        }
        if (DOT) {
          if (CODES) {
            const int8_t* q = static_cast<const int8_t*>(a.rows_in) + r * a.ldr + c;
            const float sc = scale_value(__ldg(a.scales + r * nb + (c >> 5)));  // V divides 32
#pragma unroll
            for (int j = 0; j < V; ++j) dot = fmaf(elem_to_float<E>(v.e[j]), (float)q[j] * sc, dot);
          } else {
            const Piece<E, V> u = load_piece<E, V>(static_cast<const E*>(a.rows_in) + r * a.ldr + c);
#pragma unroll
            for (int j = 0; j < V; ++j) dot = fmaf(elem_to_float<E>(v.e[j]), elem_to_float<E>(u.e[j]), dot);
          }
        }
      }
      if (DOT) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == k) mydw = dot;
      }
    }
    if (DOT && lane < a.K) a.dw[t * a.K + lane] = mydw;
  }
}

static int row_grid(int T) {
  const int wpb = kRowThreads / 32;
  return (int)std::max<long long>(1, std::min<long long>(((long long)T + wpb - 1) / wpb, (long long)sm_count() * 8));
}

template <typename E>
static int collect_run(const RowArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool vec = a.d % V == 0 && rows_aligned16(a.rows_in, a.ldr, sizeof(E)) &&
                   (!a.tok || rows_aligned16(a.tok, a.ldt, sizeof(E))) && rows_aligned16(a.tok_out, a.ldto, sizeof(E));
  auto kern = vec ? collect_kernel<E, V> : collect_kernel<E, 1>;
  return launch_pdl(kern, dim3(row_grid(a.T)), dim3(kRowThreads), 0, st, a);
}

template <typename E, bool DOT, bool CODES>
static int spread_run(const RowArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool vec = a.d % V == 0 && rows_aligned16(a.tok, a.ldt, sizeof(E)) &&
                   (!a.rows_out || rows_aligned16(a.rows_out, a.ldro, sizeof(E))) &&
                   (!DOT || CODES || rows_aligned16(a.rows_in, a.ldr, sizeof(E)));
  auto kern = vec ? spread_kernel<E, V, DOT, CODES> : spread_kernel<E, 1, DOT, CODES>;
  return launch_pdl(kern, dim3(row_grid(a.T)), dim3(kRowThreads), 0, st, a);
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

template <bool DOT, bool CODES>
static int spread_types(int dtype, const RowArgs& a, cudaStream_t st) {
  return dtype == MOE_DTYPE_BF16 ? spread_run<__nv_bfloat16, DOT, CODES>(a, st)
         : dtype == MOE_DTYPE_F16 ? spread_run<__half, DOT, CODES>(a, st)
                                  : spread_run<float, DOT, CODES>(a, st);
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
  if (!dw) return spread_types<false, false>(dtype, a, st);
  return scales ? spread_types<true, true>(dtype, a, st) : spread_types<true, false>(dtype, a, st);
}

}  // namespace moe
