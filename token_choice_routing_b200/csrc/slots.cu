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
// writes each chunk's slots per expert, sort_place_kernel ranks its chunk's slots, adds up the
// chunks below its own and writes the rows. Integer sums only, so the result is exact whatever the
// order. With one chunk the placing kernel does it alone.
//
// What bounds it is the chain of dependent steps, not the 12 bytes a slot. So the ids are read once
// and stay in registers with their ranks, and with two kernels the ranking runs before the wait for
// the first one's table (the ids were complete before that kernel let this one start). 64 experts:
// 256 slots 2.8 us, 16k 4.9, 256k 6.8, 1M 12.8; in the last the counting takes 2.0 us, the ranking 2.8,
// the table's sums 1.8 and the rows, 4-byte stores all over perm_tok, 2.3 to 3.6. Ranks written by a
// first kernel and only offset by a second one took 14.3 us, and 10.2 at 256k slots.
// A warp takes 32 slots at a time; lanes of the same id find each other by one ballot per bit of the
// ids (a match instruction, which goes value by value, took 13 against 5 us for 16k slots; counters of
// a byte per lane and expert, summed by multiplication, were no faster at 1M slots and slower at fewer).
constexpr int kSortItems = 8;  // slots a thread holds; a CTA ranks 256 a warp at a time
constexpr int kCountThreads = 512;
constexpr int kSortMaxChunks = 148;
// One CTA does up to kSortOneChunk slots alone; more are cut into chunks of 1024 slots, or more once
// there are kSortMaxChunks of them (64 experts: 8192 slots 4.7 us; in chunks of 4096 10.2 us).
constexpr int kSortOneChunk = 2048;
// 16 warps a CTA while they rank a chunk in one pass, 32 beyond (a single step of 256 slots 3.0 us
// against 3.7 with 32 warps; 1M slots, 512 experts 28 against 43 with 16).
constexpr int kSortFewWarps = 4096;

struct SortShape {
  long long S;
  int chunks;
  long long per_chunk;  // a multiple of 1024
  int warps;            // of a CTA: 16 or 32
};

static SortShape sort_shape(int T, int K) {
  SortShape s;
  s.S = (long long)T * K;
  const long long n = s.S <= kSortOneChunk ? 1 : std::min<long long>(kSortMaxChunks, (s.S + 1023) / 1024);
  s.per_chunk = std::max<long long>(1, ((s.S + n - 1) / n + 1023) / 1024) * 1024;
  s.chunks = (int)std::max<long long>(1, (s.S + s.per_chunk - 1) / s.per_chunk);
  s.warps = s.per_chunk <= kSortFewWarps ? 16 : 32;
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
  FastDiv K;
  int N, chunks;
};

// The slot's expert, -1 for none. Read past the L1 cache: the placing kernel reads the ids before it
// waits for its predecessor.
template <typename Id>
__device__ __forceinline__ int sort_id(const SortArgs& a, long long s, long long end) {
  if (s >= end) return -1;
  const Id v = __ldcg(static_cast<const Id*>(a.ids) + s);
  return (v >= 0 && v < (Id)a.N) ? (int)v : -1;
}

template <typename Id>
__global__ void __launch_bounds__(kCountThreads) sort_count_kernel(SortArgs a) {
  constexpr int kThreads = kCountThreads, kPass = kThreads * kSortItems;
  pdl_wait_then_release();
  extern __shared__ int s_mem[];
  int* hist = s_mem;
  for (int g = threadIdx.x; g < a.N; g += kThreads) hist[g] = 0;
  __syncthreads();
  const long long begin = a.per_chunk * blockIdx.x, end = min(a.S, begin + a.per_chunk);
  for (long long s0 = begin + threadIdx.x; s0 < end; s0 += kPass) {
    int id[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) id[i] = sort_id<Id>(a, s0 + i * kThreads, end);
#pragma unroll
    for (int i = 0; i < kSortItems; ++i)
      if (id[i] >= 0) atomicAdd(&hist[id[i]], 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < a.N; g += kThreads) a.table[(size_t)blockIdx.x * a.N + g] = hist[g];
}

// Shared memory of the placing kernel: whist [warps][N + 1] (a warp's slots per expert, then the
// row of its first one; padded so that a column is free of bank conflicts), tot [N] (this pass's
// slots), base [N] (the row of the next slot), pre [N] (slots in the chunks below), part [32].
struct SortShared {
  int *whist, *tot, *base, *pre, *part;
  int ld;
  __device__ __forceinline__ SortShared(int* mem, int N, int warps) {
    ld = N + 1;
    whist = mem;
    tot = whist + warps * ld;
    base = tot + N;
    pre = base + N;
    part = pre + N;
  }
};
static size_t sort_smem(int N, int warps) { return sizeof(int) * ((size_t)warps * (N + 1) + 3 * (size_t)N + 32); }

// First pass of a chunk: base [e] = the row of this chunk's first slot of expert e, from the table
// (one chunk: from tot); CTA 0 writes counts and offsets. tot and whist are complete and synced.
template <int WARPS>
__device__ __forceinline__ void sort_first_rows(const SortArgs& a, const SortShared& m) {
  constexpr int kThreads = WARPS * 32;
  constexpr int kBatch = 10;  // loads in flight: 148 rows of 64 experts by 1024 threads at once
  const int N = a.N, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (a.chunks > 1) {
    // column sums: a thread takes expert g in every (kThreads / width)-th row. Not the
    // read-only path: the table is written while this kernel runs.
    const int width = min(kThreads, max(32, 1 << (32 - __clz(N - 1)))), rows = kThreads / width;
    for (int g = tid & (width - 1); g < N; g += width) {
      int all = 0, below = 0;
      for (int c0 = tid / width; c0 < a.chunks; c0 += rows * kBatch) {
        int v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int c = c0 + i * rows;
          v[i] = c < a.chunks ? __ldcg(a.table + (size_t)c * N + g) : 0;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          all += v[i];
          below += c0 + i * rows < (int)blockIdx.x ? v[i] : 0;
        }
      }
      atomicAdd(&m.base[g], all);
      atomicAdd(&m.pre[g], below);
    }
  } else {
    for (int e = tid; e < N; e += kThreads) m.base[e] = m.tot[e];
  }
  __syncthreads();
  // exclusive scan of the totals over the experts, two a thread (N <= 1024 <= 2 threads)
  const int e0 = 2 * tid, t0 = e0 < N ? m.base[e0] : 0, t1 = e0 + 1 < N ? m.base[e0 + 1] : 0;
  int scan = t0 + t1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) m.part[w] = scan;
  __syncthreads();
  if (w == 0) {
    int v = lane < WARPS ? m.part[lane] : 0;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    m.part[lane] = v;
  }
  __syncthreads();
  const int first = scan - t0 - t1 + (w > 0 ? m.part[w - 1] : 0);  // offsets[e0]
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = e0 + j;
    if (e >= N) continue;
    const int at = first + j * t0;
    if (blockIdx.x == 0) {
      a.counts[e] = j ? t1 : t0;
      a.offsets[e] = at;
      if (e == N - 1) a.offsets[N] = first + t0 + t1;
    }
    m.base[e] = at + m.pre[e];
  }
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  __syncthreads();
}

// whist: a warp's slots per expert -> the slots of the warps before it; tot: of all warps. WARPS
// lanes take an expert, lane l of them the l-th warp's slots.
template <int WARPS>
__device__ __forceinline__ void sort_warp_scan(const SortShared& m, int N) {
  constexpr int kPerWarp = 32 / WARPS;  // experts a warp takes at a time
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int e0 = kPerWarp * w; e0 < N; e0 += kPerWarp * WARPS) {
    const int e = e0 + lane / WARPS, l = lane % WARPS;
    const int v = e < N ? m.whist[l * m.ld + e] : 0;
    int scan = v;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, scan, o, WARPS);
      if (l >= o) scan += u;
    }
    if (e < N) {
      m.whist[l * m.ld + e] = scan - v;
      if (l == WARPS - 1) m.tot[e] = scan;
    }
  }
}

// One pass's steps between a warp's ranks and the rows; returns with base + whist in place.
template <int WARPS>
__device__ __forceinline__ void sort_join(const SortArgs& a, const SortShared& m, bool first_pass) {
  __syncthreads();
  sort_warp_scan<WARPS>(m, a.N);
  if (first_pass && a.chunks > 1) pdl_wait_then_release();  // the table is complete
  __syncthreads();
  if (first_pass) sort_first_rows<WARPS>(a, m);
}

// The warp's lanes with the same id, below 2^BITS.
template <int BITS>
__device__ __forceinline__ unsigned same_id(int id) {
  unsigned peers = __ballot_sync(0xffffffffu, id >= 0);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool bit = (id >> b) & 1;
    const unsigned set = __ballot_sync(0xffffffffu, bit);
    peers &= bit ? set : ~set;
  }
  return peers;
}

// Its registers have to leave room for a CTA of the counting kernel (512 threads of 32), so that the
// ranking starts while that one still runs: two CTAs' worth with 16 warps; 32 warps take 43 registers
// as they are (bounded to 64 14.1 us at 1M slots, to 48 13.7, this 12.8; 16 warps unbounded 8.4 against
// 6.8 us at 256k).
template <typename Id, int WARPS, int BITS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 16 ? 2 : 0) sort_place_kernel(SortArgs a) {
  constexpr int kThreads = WARPS * 32, kPass = kThreads * kSortItems;
  extern __shared__ int s_mem[];
  const SortShared m(s_mem, a.N, WARPS);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (a.chunks == 1) pdl_wait_then_release();  // this is the call's first kernel
  for (int i = tid; i < a.N; i += kThreads) m.base[i] = m.pre[i] = 0;
  const long long begin = a.per_chunk * blockIdx.x, end = min(a.S, begin + a.per_chunk);
  bool first_pass = true;
  for (long long p0 = begin; first_pass || p0 < end; p0 += kPass) {
    // an equal number of 32-slot groups for each warp
    const int items = (int)min((long long)kSortItems, (end - p0 + kThreads - 1) / kThreads);
    const long long mine0 = p0 + (long long)w * 32 * items + lane;
    int id[kSortItems], rank[kSortItems];
    unsigned peers[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) id[i] = i < items ? sort_id<Id>(a, mine0 + i * 32, end) : -1;
    for (int i = tid; i < WARPS * m.ld; i += kThreads) m.whist[i] = 0;
    __syncthreads();
    int* mine = m.whist + w * m.ld;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) peers[i] = i < items ? same_id<BITS>(id[i]) : 0u;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      if (i >= items) break;
      if (id[i] >= 0) rank[i] = mine[id[i]] + __popc(peers[i] & ((1u << lane) - 1u));
      __syncwarp();
      if (id[i] >= 0 && lane == 31 - __clz(peers[i])) mine[id[i]] += __popc(peers[i]);
      __syncwarp();
    }
    sort_join<WARPS>(a, m, first_pass);
    first_pass = false;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const long long s = mine0 + i * 32;
      if (i >= items || s >= end) break;
      const int row = id[i] >= 0 ? m.base[id[i]] + mine[id[i]] + rank[i] : -1;
      a.slot_row[s] = row;
      if (row >= 0) a.perm_tok[row] = (int)a.K.quotient((uint32_t)s);
    }
    __syncthreads();
    for (int e = tid; e < a.N; e += kThreads) m.base[e] += m.tot[e];
  }
}

template <typename Id, int WARPS, int BITS>
static int sort_go(const SortArgs& a, cudaStream_t st) {
  auto place = sort_place_kernel<Id, WARPS, BITS>;
  // the limit belongs to the kernel, not to the call (another thread's may be between this and its
  // launch): what 2^BITS experts need, set once for a device
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sort_smem(1 << BITS, WARPS));
    if (e != cudaSuccess) return cuda_status(e);
    attr_set[dev] = true;
  }
  const dim3 grid(a.chunks), block(WARPS * 32);
  if (a.chunks > 1) {
    const int r = launch_pdl(sort_count_kernel<Id>, grid, dim3(kCountThreads), sizeof(int) * (size_t)a.N, st, a);
    if (r != MOE_OK) return r;
  }
  return launch_pdl(place, grid, block, sort_smem(a.N, WARPS), st, a);
}

template <typename Id, int WARPS>
static int sort_bits(const SortArgs& a, cudaStream_t st) {
  return a.N <= 64 ? sort_go<Id, WARPS, 6>(a, st) : sort_go<Id, WARPS, 10>(a, st);
}

template <typename Id>
static int sort_run(const SortArgs& a, int warps, cudaStream_t st) {
  return warps == 16 ? sort_bits<Id, 16>(a, st) : sort_bits<Id, 32>(a, st);
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
  a.K = FastDiv((uint32_t)K);
  a.N = N;
  a.chunks = sh.chunks;
  return id_bytes == 8 ? sort_run<long long>(a, sh.warps, st) : sort_run<int>(a, sh.warps, st);
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
  int items;           // T * chunks of a launch: a warp's (narrow rows: a thread's) work is one chunk of one token
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

// tok_out[t] = tok[t] + sum_k w[t,k] rows_in[slot_row[t,k]], fp32 sums in slot order. FULL: all
// columns of the chunk are in the row.
template <typename E, int V, int NV, bool FULL>
__device__ __forceinline__ void collect_chunk(const RowArgs& a, long long t, int c0, int row, float w) {
  const E* base = static_cast<const E*>(a.tok) + t * a.ldt + c0;
  float acc[NV][V];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    Piece<E, V> b;
    b.zero();
    if (a.tok && (FULL || c0 + v * 32 * V < a.d)) b.load_own(base + v * 32 * V);
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
      const E* src = static_cast<const E*>(a.rows_in) + (long long)r[u] * a.ldr;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = c0 + v * 32 * V;
        p[u][v].zero();
        if (r[u] >= 0 && (FULL || c < a.d)) p[u][v].load(src + c);
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
  E* out = static_cast<E*>(a.tok_out) + t * a.ldto + c0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!FULL && c0 + v * 32 * V >= a.d) continue;
    Piece<E, V> o;
    o.set(acc[v]);
    o.store(out + v * 32 * V);
  }
}

template <typename E, int V, int NV>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) collect_kernel(RowArgs a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (item >= (uint32_t)a.items) return;
  const long long t = a.chunks.quotient(item);
  const int c0 = (int)(item - (uint32_t)t * a.chunks.d) * (32 * V * NV);
  const int row = slot_row_checked(a.slot_row, t, lane, a.K, a.rows, a.status);
  const float w = (a.w && lane < a.K) ? __ldg(a.w + t * a.K + lane) : 1.f;
  // whole chunks apart only for single elements, where the kernel is bound by instructions
  // (T = 16384, d = 1537, K = 8, bf16: 97 -> 86 us); with 16-byte pieces both paths together spill
  if (V == 1 && c0 + 32 * V * NV <= a.d)
    collect_chunk<E, V, NV, true>(a, t, c0 + lane * V, row, w);
  else
    collect_chunk<E, V, NV, false>(a, t, c0 + lane * V, row, w);
}

// rows_out[slot_row[t,k]] = w[t,k] tok[t] (w null: a copy). The row is read once and stays in
// registers. Bound by HBM's writes: T = 65536, d = 2048, K = 8, half the slots null, bf16 205 us
// (6.5 TB/s); T = 16384, d = 1024, K = 4 17.8 us (5.7 TB/s).
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

// s + the dot product of a piece with codes of scale sc. The values code * sc are exact; scaling the
// sum instead would save a multiplication an element (1 to 2% of the kernel) and overflow where
// the scaled products do not.
template <int V>
__device__ __forceinline__ float dot_codes(const float (&g)[V], const CodePiece<V>& q, float sc, float s) {
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    float f[4];
    codes_to_float(q.word[j / 4], f);
#pragma unroll
    for (int i = 0; i < (V < 4 ? V : 4); ++i) s = fmaf(g[j + i], f[i] * sc, s);
  }
  return s;
}

// rows_out[slot_row[t,k]] = w[t,k] tok[t] (rows_out null: not written) and dw[t,k] = <tok[t],
// rows_in[slot_row[t,k]]>, 0 for a slot without a row. wpt warps share a token, each every
// wpt-th chunk of its columns. A dot product is summed in fp32 per lane, over the lanes by a fixed
// shuffle tree and over the warps in order, so it does not depend on timing.
// Bound by HBM: T = 65536, d = 2048, K = 8, half the slots null, bf16 375 us (6.5 TB/s), from codes
// 319 us (6.0 TB/s); T = 16384 102 us; from codes at d = 1024, K = 4 29 us (4.7 TB/s), where a token
// has two rows and a warp's chain of lookup, loads and stores is not covered. A persistent grid
// that looks the next token's slots up ahead measured slower (375 -> 401 us and more).
// Eight single elements of five rows a lane need more registers than four CTAs leave (T = 16384,
// d = 1001, K = 4, bf16: 58 us with three CTAs, 94 with four; from codes 79 us with two, 231 with four).
template <typename E, int V, int NV, bool CODES>
__global__ void __launch_bounds__(kRowThreads, V == 1 && NV == kElemPieces ? (CODES ? 2 : 3) : kRowCtas)
    spread_dot_kernel(RowArgs a, int wpt) {
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
        uint32_t sb[V == 1 ? 1 : 4][NV];
        float lane_scale = 0.f;
        if constexpr (CODES && V == 1) {
          // 32 single elements are one block: lane u NV + v fetches slot u's scale of block v
          const int u = lane / NV, blk = (c0 - lane) / 32 + lane % NV;
          const int ru = u == 0 ? r[0] : u == 1 ? r[1] : u == 2 ? r[2] : r[3];
          if (u < 4 && ru >= 0 && blk < nb) lane_scale = scale_value(__ldg(a.scales + (long long)ru * nb + blk));
        }
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
            if constexpr (CODES && V == 1) {
              q[u][v].word[0] = c < a.d ? (uint32_t)(int)__ldg(static_cast<const int8_t*>(a.rows_in) + at) : 0u;
            } else if constexpr (CODES) {
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
            float gf[V];
            g[v].get(gf);
            if constexpr (CODES && V == 1)  // before any lane leaves; columns past the row hold zeros
              dot[u] = fmaf(gf[0], (float)(int)q[u][v].word[0] * __shfl_sync(0xffffffffu, lane_scale, u * NV + v), dot[u]);
            if (c >= a.d) continue;
            if constexpr (CODES && V == 1) {
            } else if constexpr (CODES) {
              dot[u] = dot_codes<V>(gf, q[u][v], scale_value(sb[u][v]), dot[u]);
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

// Narrow rows, of fewer pieces than a warp has lanes: a thread takes one piece of one token and
// reads the token's slots itself, four at a time. (chunks: pieces of a row.)
__device__ __forceinline__ void thread_slots(const RowArgs& a, long long t, int k0, int (&r)[4], float (&wk)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    r[u] = slot_row_checked(a.slot_row, t, k0 + u, a.K, a.rows, a.status);
    wk[u] = (a.w && k0 + u < a.K) ? __ldg(a.w + t * a.K + k0 + u) : 1.f;
  }
}

template <typename E, int V>
__global__ void __launch_bounds__(kRowThreads) collect_narrow_kernel(RowArgs a) {
  pdl_wait_then_release();
  const uint32_t item = blockIdx.x * kRowThreads + threadIdx.x;
  if (item >= (uint32_t)a.items) return;
  const long long t = a.chunks.quotient(item);
  const int c = (int)(item - (uint32_t)t * a.chunks.d) * V;
  Piece<E, V> b;
  b.zero();
  if (a.tok) b.load_own(static_cast<const E*>(a.tok) + t * a.ldt + c);
  float acc[V];
  b.get(acc);
  for (int k0 = 0; k0 < a.K; k0 += 4) {
    int r[4];
    float wk[4];
    thread_slots(a, t, k0, r, wk);
    Piece<E, V> p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      p[u].zero();
      if (r[u] >= 0) p[u].load(static_cast<const E*>(a.rows_in) + (long long)r[u] * a.ldr + c);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (r[u] < 0) continue;
      float f[V];
      p[u].get(f);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(wk[u], f[j], acc[j]);
    }
  }
  b.set(acc);
  b.store(static_cast<E*>(a.tok_out) + t * a.ldto + c);
}

template <typename E, int V>
__device__ __forceinline__ Piece<E, V> scaled(const Piece<E, V>& p, float w) {
  float f[V];
  p.get(f);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] *= w;
  Piece<E, V> o;
  o.set(f);
  return o;
}

template <typename E, int V>
__global__ void __launch_bounds__(kRowThreads) spread_narrow_kernel(RowArgs a) {
  pdl_wait_then_release();
  const uint32_t item = blockIdx.x * kRowThreads + threadIdx.x;
  if (item >= (uint32_t)a.items) return;
  const long long t = a.chunks.quotient(item);
  const int c = (int)(item - (uint32_t)t * a.chunks.d) * V;
  Piece<E, V> p;
  p.load(static_cast<const E*>(a.tok) + t * a.ldt + c);
  for (int k0 = 0; k0 < a.K; k0 += 4) {
    int r[4];
    float wk[4];
    thread_slots(a, t, k0, r, wk);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (r[u] >= 0)
        (a.w ? scaled<E, V>(p, wk[u]) : p).store(static_cast<E*>(a.rows_out) + (long long)r[u] * a.ldro + c);
  }
}

// A group of G lanes a token, a piece each.
template <typename E, int V, bool CODES>
__global__ void __launch_bounds__(kRowThreads) spread_dot_narrow_kernel(RowArgs a, int G) {
  pdl_wait_then_release();
  const int j = threadIdx.x & (G - 1), c = j * V;
  const long long t = (long long)blockIdx.x * (kRowThreads / G) + threadIdx.x / G;
  const bool token = t < a.T, mine = token && c < a.d;
  const int nb = (a.d + 31) / 32;
  Piece<E, V> g;
  g.zero();
  if (mine) g.load(static_cast<const E*>(a.tok) + t * a.ldt + c);
  float gf[V];
  g.get(gf);
  for (int k0 = 0; k0 < a.K; k0 += 4) {  // uniform trip count: the shuffles below are the warp's
    int r[4] = {-1, -1, -1, -1};
    float wk[4], dot[4];
    if (token) thread_slots(a, t, k0, r, wk);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      dot[u] = 0.f;
      if (!mine || r[u] < 0) continue;
      const long long at = (long long)r[u] * a.ldr + c;
      if constexpr (CODES) {
        const CodePiece<V> q = load_codes<V>(static_cast<const int8_t*>(a.rows_in) + at);
        const float sc = scale_value(__ldg(a.scales + (long long)r[u] * nb + (c >> 5)));
        dot[u] = dot_codes<V>(gf, q, sc, 0.f);
      } else {
        Piece<E, V> p;
        p.load(static_cast<const E*>(a.rows_in) + at);
        float f[V];
        p.get(f);
#pragma unroll
        for (int i = 0; i < V; ++i) dot[u] = fmaf(gf[i], f[i], dot[u]);
      }
      if (a.rows_out) scaled<E, V>(g, wk[u]).store(static_cast<E*>(a.rows_out) + (long long)r[u] * a.ldro + c);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      for (int o = G >> 1; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
      if (token && j == 0 && k0 + u < a.K) a.dw[t * a.K + k0 + u] = dot[u];
    }
  }
}

static unsigned blocks_for(long long n, int per_block) { return (unsigned)((n + per_block - 1) / per_block); }

template <typename P>
static P* past(P* p, long long n) { return p ? p + n : p; }
template <typename E>
static void past_rows(const void*& p, long long n) { p = past(static_cast<const E*>(p), n); }
template <typename E>
static void past_rows(void*& p, long long n) { p = past(static_cast<E*>(p), n); }

// Launches a kernel over the chunks of all tokens. They are numbered in 32 bits, so tokens with 2^31
// chunks and more (narrow rows reach that: 34M tokens of 63 single elements) come in parts.
template <typename E, typename Launch>
static int over_tokens(RowArgs a, int chunk, Launch launch) {
  const int n = (int)(((long long)a.d + chunk - 1) / chunk), most = INT_MAX / n;
  a.chunks = FastDiv((uint32_t)n);
  for (int left = a.T;;) {
    a.T = std::min(left, most);
    a.items = a.T * n;
    const int r = launch(a);
    left -= a.T;
    if (r != MOE_OK || left == 0) return r;
    past_rows<E>(a.tok, a.T * a.ldt);
    past_rows<E>(a.tok_out, a.T * a.ldto);
    a.w = past(a.w, (long long)a.T * a.K);
    a.slot_row += (long long)a.T * a.K;
  }
}

// Rows of at most this many pieces go to the narrow kernels, where a warp would leave half of its
// lanes idle and do a token's slot lookup for little (T = 65536, K = 8, bf16, unpermute: d = 64
// 53 -> 17 us, 256 60 -> 53 us; 512, beyond, 80 against 98 us). Single elements: d = 33 50 -> 27 us,
// 127, beyond, 56 against 94 us.
template <int V>
constexpr int kNarrow = V == 1 ? 64 : 32 * V;

template <typename E, int V, int NV>
static int collect_go(const RowArgs& a, cudaStream_t st) {
  if (a.d <= kNarrow<V>) {
    return over_tokens<E>(a, V, [&](const RowArgs& p) {
      return launch_pdl(collect_narrow_kernel<E, V>, dim3(blocks_for(p.items, kRowThreads)), dim3(kRowThreads), 0, st,
                        p);
    });
  }
  return over_tokens<E>(a, 32 * V * NV, [&](const RowArgs& p) {
    return launch_pdl(collect_kernel<E, V, NV>, dim3(blocks_for(p.items, kRowWarps)), dim3(kRowThreads), 0, st, p);
  });
}

template <typename E>
static int collect_run(const RowArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool vec = a.d % V == 0 && rows_aligned16(a.rows_in, a.ldr, sizeof(E)) &&
                   (!a.tok || rows_aligned16(a.tok, a.ldt, sizeof(E))) && rows_aligned16(a.tok_out, a.ldto, sizeof(E));
  if (vec) return collect_go<E, V, kVecPieces>(a, st);
  return a.d <= 128 ? collect_go<E, 1, 4>(a, st) : collect_go<E, 1, kElemPieces>(a, st);
}

template <typename E, int V, int NV>
static int spread_go(const RowArgs& a, cudaStream_t st) {
  if (a.d <= (V == 1 ? 32 : kNarrow<V>)) {  // single elements: d = 63 39 us this way, about 23 by warps
    return over_tokens<E>(a, V, [&](const RowArgs& p) {
      return launch_pdl(spread_narrow_kernel<E, V>, dim3(blocks_for(p.items, kRowThreads)), dim3(kRowThreads), 0, st,
                        p);
    });
  }
  return over_tokens<E>(a, 32 * V * NV, [&](const RowArgs& p) {
    return launch_pdl(spread_kernel<E, V, NV>, dim3(blocks_for(p.items, kRowWarps)), dim3(kRowThreads), 0, st, p);
  });
}

template <typename E, int V, int NV, bool CODES>
static int spread_dot_go(const RowArgs& a, cudaStream_t st) {
  if (a.d <= 32 * V) {  // a lane a piece
    int G = 1;
    while (G * V < a.d) G *= 2;
    const int per_block = kRowThreads / G;
    return launch_pdl(spread_dot_narrow_kernel<E, V, CODES>, dim3(blocks_for(a.T, per_block)), dim3(kRowThreads),
                      0, st, a, G);
  }
  // more warps a token while the tokens alone do not fill the GPU and the row has chunks for them
  int wpt = 1;
  // (T = 64, d = 2048, K = 8: 3.9 us)
  while (wpt < kRowWarps && (long long)a.T * wpt < (long long)sm_count() * 16 && a.d > wpt * 32 * V * NV) wpt *= 2;
  return launch_pdl(spread_dot_kernel<E, V, NV, CODES>, dim3(blocks_for(a.T, kRowWarps / wpt)), dim3(kRowThreads), 0,
                    st, a, wpt);
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
  if (vec)
    return codes ? spread_dot_go<E, V, kVecPieces, true>(a, st) : spread_dot_go<E, V, kVecPieces, false>(a, st);
  if (a.d <= 64) return codes ? spread_dot_go<E, 1, 2, true>(a, st) : spread_dot_go<E, 1, 2, false>(a, st);
  if (a.d <= 128) return codes ? spread_dot_go<E, 1, 4, true>(a, st) : spread_dot_go<E, 1, 4, false>(a, st);
  return codes ? spread_dot_go<E, 1, kElemPieces, true>(a, st) : spread_dot_go<E, 1, kElemPieces, false>(a, st);
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
