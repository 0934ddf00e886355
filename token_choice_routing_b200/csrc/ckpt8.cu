// Activations stored in 8 bits (moe_checkpoint8, moe_restore8) and SwiGLU's backward from
// pre-activations stored that way (moe_swiglu_backward8).
//
// A row is cut into blocks of 32 columns (the last one may be shorter). With m the block's
// largest magnitude, E = max(floor(log2 m) - 6, -126): its elements are held as
//   q = clamp(rint(x 2^-E), -127, 127),   value q 2^E,
// and E as the byte E + 127. A power of two as the scale makes the product x 2^-E and the
// value q 2^E exact, so the only rounding is rint's (half to even), and the value has at most
// 7 significant bits: exact again in bf16, fp16 and fp32. m 2^-E lies in [64, 128), so the
// error is at most 2^(E-1), except above 127.5 2^E (a bf16 block reaches exactly 127.5), where
// the clamp leaves less than 2^E. A block with an infinity or a NaN gets byte 255 and is
// restored as NaN throughout, so that an overflow in the forward shows in the gradient.
//
// All three are one pass over HBM and bound by it at the layer's sizes (bf16, copy rate 6.5 TB/s):
//   store   32768 x 1536  25.2 us  6.1 TB/s      131072 x 1536  96 us  6.3 TB/s
//   restore 32768 x 1536  26.9 us  5.7 TB/s      131072 x 1536 106 us  5.7 TB/s
//   SwiGLU  32768 x 768   45.0 us  5.6 TB/s      104857 x 1024 175 us  6.2 TB/s
// The two that write more than they read stay further from the copy rate, which reads as much.
// Getting there took the integer instructions out (68% of the ALU pipe at first): maxima, clamps
// and packing on two or four values at a time, no index arithmetic for dense tensors. Rows that no
// 16-byte access fits take one element a lane and stay bound by instructions: 60000 x 1001 store
// and restore 137 us (2.6 TB/s), SwiGLU's backward of 60000 x 499 90 us (3.4 TB/s).
#include "rows.cuh"

#include <algorithm>

namespace moe {

constexpr int kCkptThreads = 256;
constexpr int kCkptCtas = 8;     // CTAs of the grid a multiprocessor
constexpr int kSwigluCtas = 16;

// Rows in use: *used clamped to [0, rows] (recorded when it lies outside), or all of them.
__device__ __forceinline__ long long rows_in_use(const int32_t* used, long long rows, uint32_t* status) {
  if (!used) return rows;
  const long long u = __ldg(used);
  if (u < 0 || u > rows) {
    if (status && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kStatusBounds);
    return u < 0 ? 0 : rows;
  }
  return u;
}

// N consecutive elements in 16-byte pieces.
template <typename E, int N>
struct Run {
  static constexpr int V = 16 / sizeof(E), W = N / V;
  Piece<E, V> w[W];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i].load(p + i * V);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i].zero();
  }
  __device__ __forceinline__ void store(E* p) const {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i].store(p + i * V);
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float f[V];
      w[i].get(f);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i * V + j] = f[j];
    }
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = v[i * V + j];
      w[i].set(f);
    }
  }
};

// Work items (fixed pieces of a row) are taken in tiles of consecutive ones. A CTA starts at
// tile blockIdx.x and goes on in steps of the whole grid; the row and the item in it follow by
// addition, so that no 64-bit division is left in the loop.
struct ItemPos {
  long long row;
  uint32_t i;
};
__device__ __forceinline__ ItemPos at(const ItemPos& s, uint32_t off, const FastDiv& per_row) {
  const uint32_t n = s.i + off, q = per_row.quotient(n);
  return {s.row + q, n - q * per_row.d};
}
struct Walk {
  FastDiv per_row;    // items of a row
  uint32_t tile;      // items of a tile
  uint32_t step_rows, step_items;  // gridDim.x * tile items, as rows and items
  __device__ __forceinline__ ItemPos begin() const { return at({0, 0u}, blockIdx.x * tile, per_row); }
  __device__ __forceinline__ void next(ItemPos& s) const {
    s.row += step_rows;
    s.i += step_items;
    if (s.i >= per_row.d) {
      s.i -= per_row.d;
      ++s.row;
    }
  }
};

struct Ckpt8Args {
  const void* x;
  void* out;
  int8_t* codes;
  uint8_t* scales;
  const int32_t* used;
  uint32_t* status;
  long long rows, ld;
  int cols, nb;  // nb: blocks (scale bytes) of a row
  Walk walk;
};

// Where an item of N columns lies. FLAT: dense rows of whole blocks, the tensor one long row, so
// nothing is left to compute but the item's number; otherwise by its row.
template <bool FLAT, int N>
struct Spot {
  long long x, code, scale;  // element offsets of its columns, its codes and its block's scale
  uint32_t col;
  __device__ __forceinline__ Spot(const Ckpt8Args& a, long long first, const ItemPos& s, uint32_t off) {
    if constexpr (FLAT) {
      x = code = (first + off) * N;
      scale = (first + off) / (32 / N);
      col = 0;
    } else {
      const ItemPos p = at(s, off, a.walk.per_row);
      col = p.i * N;
      x = p.row * a.ld + col;
      code = p.row * a.cols + col;
      scale = p.row * a.nb + p.i / (32 / N);
    }
  }
};

// Store, rows of 16-byte pieces: an item is half a block, two neighbouring lanes a block (a row
// has 2 nb items; columns past its end stand for zeros). kUnroll items a thread are loaded before
// any is used: four with two CTAs a multiprocessor 25.1 us for 32768 x 1536, two 25.6, one 29.2; a
// quarter of a block an item 37 us.
constexpr int kItem = 16;
constexpr int kUnroll = 4;
template <typename E, bool FLAT>
__global__ void __launch_bounds__(kCkptThreads, 2) checkpoint8_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  constexpr int kTile = kCkptThreads * kUnroll, V = 16 / sizeof(E), W = kItem / V;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.walk.per_row.d;
  ItemPos s = a.walk.begin();
  for (long long first = (long long)blockIdx.x * kTile; first < n;
       first += (long long)gridDim.x * kTile, a.walk.next(s)) {
    const uint32_t left = (uint32_t)min((long long)kTile, n - first);
    Run<E, kItem> x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      const Spot<FLAT, kItem> p(a, first, s, off);
      x[u].zero();
      if (off < left) {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (FLAT || p.col + i * V < (uint32_t)a.cols) x[u].w[i].load(static_cast<const E*>(a.x) + p.x + i * V);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      const Spot<FLAT, kItem> p(a, first, s, off);
      uint32_t top = top_of<E, V>(x[u].w[0]);
#pragma unroll
      for (int i = 1; i < W; ++i) top = top_join<E, V>(top, top_of<E, V>(x[u].w[i]));
      top = top_join<E, V>(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const uint32_t byte = scale_byte(top_bits<E, V>(top));
      const float inv = scale_inverse(byte);
      float v[kItem];
      x[u].get(v);
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[j] = pack4(quantise(v[4 * j], inv), quantise(v[4 * j + 1], inv), quantise(v[4 * j + 2], inv),
                     quantise(v[4 * j + 3], inv));
        if (byte == kByteNan) q[j] = 0u;
      }
      if (off < left) {
        if (FLAT) {
          *reinterpret_cast<uint4*>(a.codes + p.code) = make_uint4(q[0], q[1], q[2], q[3]);
        } else {
          if (p.col < (uint32_t)a.cols) *reinterpret_cast<uint2*>(a.codes + p.code) = make_uint2(q[0], q[1]);
          if (p.col + 8 < (uint32_t)a.cols) *reinterpret_cast<uint2*>(a.codes + p.code + 8) = make_uint2(q[2], q[3]);
        }
        if ((threadIdx.x & 1u) == 0u) a.scales[p.scale] = (uint8_t)byte;
      }
    }
  }
}

// Rows of any width and alignment: a warp takes kElemBlocks blocks (an item), a lane one element of
// each: NB = 8 consecutive ones of a row, or of rows with fewer the NB (1, 2 or 4) of each of
// 8 / NB consecutive rows, so that all addresses are one base plus constants. What is the same for
// a whole block (its scale) is computed by one lane and handed round: the kernel is bound by integer
// instructions (37 a block before that, at 77% of the ALU pipe: 93 us for 60000 x 1001 in bf16).
constexpr int kElemBlocks = 8;
constexpr int kCkptWarps = kCkptThreads / 32;

// An item's place: its first row and column, the rows and columns that are left from there.
struct ElemSpot {
  long long row;
  int c0, rows, cols;
  template <int NB>
  __device__ __forceinline__ bool has(int u, int lane) const {  // block u has an element for this lane
    return (NB == kElemBlocks || u / NB < rows) && (u % NB) * 32 + lane < cols;
  }
};
template <int NB>
__device__ __forceinline__ ElemSpot elem_spot(const Ckpt8Args& a, const ItemPos& p, long long used) {
  constexpr int kRows = kElemBlocks / NB;
  ElemSpot s;
  s.row = p.row * kRows;
  s.c0 = (int)p.i * (32 * NB);
  s.rows = (int)min((long long)kRows, used - s.row);
  s.cols = a.cols - s.c0;
  return s;
}

// One item; FULL: all its elements are there.
template <typename E, int NB, bool FULL>
__device__ __forceinline__ void store_item(const Ckpt8Args& a, const ElemSpot& s) {
  const int lane = threadIdx.x & 31;
  const E* x = static_cast<const E*>(a.x) + s.row * a.ld + s.c0 + lane;
  int8_t* codes = a.codes + s.row * a.cols + s.c0 + lane;
  float v[kElemBlocks];
#pragma unroll
  for (int u = 0; u < kElemBlocks; ++u)
    v[u] = FULL || s.has<NB>(u, lane) ? elem_to_float<E>(__ldg(x + (u / NB) * a.ld + (u % NB) * 32)) : 0.f;
  uint32_t top = 0;  // lane u: of block u
#pragma unroll
  for (int u = 0; u < kElemBlocks; ++u) {
    const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(v[u]) & 0x7fffffffu);
    if (lane == u) top = t;
  }
  const uint32_t byte = scale_byte(top);
  const float inv = scale_inverse(byte);
  const unsigned bad = __ballot_sync(0xffffffffu, byte == kByteNan);
#pragma unroll
  for (int u = 0; u < kElemBlocks; ++u) {
    const uint32_t q = clamp2(quantise(v[u], __shfl_sync(0xffffffffu, inv, u)));
    if (FULL || s.has<NB>(u, lane))
      codes[(u / NB) * a.cols + (u % NB) * 32] = (int8_t)(((bad >> u) & 1u) ? 0u : q);
  }
  if (lane < kElemBlocks && s.has<NB>(lane, 0))
    a.scales[(s.row + lane / NB) * a.nb + s.c0 / 32 + lane % NB] = (uint8_t)byte;
}

template <typename E, int NB, bool FULL>
__device__ __forceinline__ void restore_item(const Ckpt8Args& a, const ElemSpot& s) {
  const int lane = threadIdx.x & 31;
  E* x = static_cast<E*>(a.out) + s.row * a.ld + s.c0 + lane;
  const int8_t* codes = a.codes + s.row * a.cols + s.c0 + lane;
  int q[kElemBlocks];
#pragma unroll
  for (int u = 0; u < kElemBlocks; ++u)
    q[u] = FULL || s.has<NB>(u, lane) ? (int)__ldg(codes + (u / NB) * a.cols + (u % NB) * 32) : 0;
  const bool mine = lane < kElemBlocks && s.has<NB>(lane, 0);
  const float sc =
      scale_value(mine ? (uint32_t)__ldg(a.scales + (s.row + lane / NB) * a.nb + s.c0 / 32 + lane % NB) : 0u);
#pragma unroll
  for (int u = 0; u < kElemBlocks; ++u) {
    const float v = (float)q[u] * __shfl_sync(0xffffffffu, sc, u);
    if (FULL || s.has<NB>(u, lane)) x[(u / NB) * a.ld + (u % NB) * 32] = float_to_elem<E>(v);
  }
}

template <typename E, int NB, bool STORE>
__global__ void __launch_bounds__(kCkptThreads) ckpt8_elem_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  constexpr int kRows = kElemBlocks / NB;
  const long long used = rows_in_use(a.used, a.rows, a.status);
  const long long n = (used + kRows - 1) / kRows * a.walk.per_row.d;
  ItemPos p = at(a.walk.begin(), threadIdx.x >> 5, a.walk.per_row);  // this warp's item
  for (long long i = (long long)blockIdx.x * kCkptWarps + (threadIdx.x >> 5); i < n;
       i += (long long)gridDim.x * kCkptWarps, a.walk.next(p)) {
    const ElemSpot s = elem_spot<NB>(a, p, used);
    if (s.rows == kRows && s.cols >= 32 * NB) {
      if (STORE) store_item<E, NB, true>(a, s);
      else restore_item<E, NB, true>(a, s);
    } else {
      if (STORE) store_item<E, NB, false>(a, s);
      else restore_item<E, NB, false>(a, s);
    }
  }
}

// Restore, rows of 16-byte pieces: an item is one of them, so that a warp's stores are whole
// sectors (half a block a lane, as in the store, leaves 16 of every 32 bytes to a second
// instruction: 28.8 us for 32768 x 1536). Eight items a thread 26.0 us, four 27.2, two 30.3.
constexpr int kRestoreUnroll = 8;
template <typename E, bool FLAT>
__global__ void __launch_bounds__(kCkptThreads) restore8_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  constexpr int V = 16 / sizeof(E), kTile = kCkptThreads * kRestoreUnroll;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.walk.per_row.d;
  ItemPos s = a.walk.begin();
  for (long long first = (long long)blockIdx.x * kTile; first < n;
       first += (long long)gridDim.x * kTile, a.walk.next(s)) {
    const uint32_t left = (uint32_t)min((long long)kTile, n - first);
    CodePiece<V> q[kRestoreUnroll];
    uint32_t byte[kRestoreUnroll];
#pragma unroll
    for (int u = 0; u < kRestoreUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      if (off >= left) continue;
      const Spot<FLAT, V> p(a, first, s, off);
      q[u] = load_codes<V>(a.codes + p.code);
      byte[u] = __ldg(a.scales + p.scale);
    }
#pragma unroll
    for (int u = 0; u < kRestoreUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      if (off >= left) continue;
      const Spot<FLAT, V> p(a, first, s, off);
      const float sc = scale_value(byte[u]);
      float v[V];
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        float f[4];
        codes_to_float(q[u].word[j], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * j + i] = f[i] * sc;
      }
      Piece<E, V> o;
      o.set(v);
      o.store(static_cast<E*>(a.out) + p.x);
    }
  }
}

struct Swiglu8Args {
  const int8_t* codes;
  const uint8_t* scales;
  const void* dh;
  void* dz;
  void* h;
  const int32_t* used;
  uint32_t* status;
  long long rows, ldh, lddz, ldo;  // row strides of dh, dz and h
  int F, nb, packed;
  Walk walk;
};

// da = dh b s (1 + a (1 - s)), db = dh a s, h = a s b with s = 1 / (1 + exp(-a)); fp32, one
// rounding per output. expf is within 2 ulp and the approximate reciprocal within 1; it gives 0
// where exp(-a) passes 2^126, as s is below fp32's normal range there. dh comes last in da: dh b
// alone may overflow where a small s leaves the gradient finite.
struct SwigluOut {
  float da, db, h;
};
__device__ __forceinline__ SwigluOut swiglu_grad(float a, float b, float g) {
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + expf(-a)));
  const float as = a * s;
  return {g * (b * (s * (1.f + a * (1.f - s)))), g * as, as * b};
}

// Rows of 16-byte pieces: an item is eight pairs. FLAT: dense rows in the packed order, where the
// pair's number over the whole tensor gives all offsets; otherwise by its row. Two items a thread
// with three CTAs a multiprocessor 45 us for 32768 x 768; one with five 49, two with five 52.
constexpr int kSwigluUnroll = 2;
constexpr int kPairs = 8;
template <bool FLAT>
struct PairSpot {
  long long a, b, sa, sb, dh, da, db, h;  // offsets of its codes, scales, dh, dz and h
  __device__ __forceinline__ PairSpot(const Swiglu8Args& g, long long first, const ItemPos& s, uint32_t off) {
    if constexpr (FLAT) {
      dh = h = (first + off) * kPairs;
      a = da = 2 * dh - (dh & 63);  // (dh / 64) * 128 + dh % 64
      b = db = a + 64;
      sa = a >> 5;
      sb = sa + 2;
    } else {
      const ItemPos p = at(s, off, g.walk.per_row);
      const int f = (int)p.i * kPairs;
      const int ca = g.packed ? (f >> 6) * 128 + (f & 63) : f, cb = g.packed ? ca + 64 : f + g.F;
      const long long q = p.row * 2 * g.F, sc = p.row * g.nb, z = p.row * g.lddz;
      a = q + ca;
      b = q + cb;
      sa = sc + (ca >> 5);
      sb = sc + (cb >> 5);
      dh = p.row * g.ldh + f;
      h = p.row * g.ldo + f;
      da = z + ca;
      db = z + cb;
    }
  }
};
template <typename E, bool FLAT>
__global__ void __launch_bounds__(kCkptThreads, 3) swiglu_backward8_kernel(Swiglu8Args a) {
  pdl_wait_then_release();
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.walk.per_row.d;
  constexpr int kTile = kCkptThreads * kSwigluUnroll;
  ItemPos s = a.walk.begin();
  for (long long first = (long long)blockIdx.x * kTile; first < n;
       first += (long long)gridDim.x * kTile, a.walk.next(s)) {
    const uint32_t left = (uint32_t)min((long long)kTile, n - first);
    uint2 qa[kSwigluUnroll], qb[kSwigluUnroll];
    uint32_t ba[kSwigluUnroll], bb[kSwigluUnroll];
    Run<E, kPairs> g[kSwigluUnroll];
#pragma unroll
    for (int u = 0; u < kSwigluUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      const PairSpot<FLAT> p(a, first, s, off);
      if (off < left) {
        qa[u] = __ldg(reinterpret_cast<const uint2*>(a.codes + p.a));
        qb[u] = __ldg(reinterpret_cast<const uint2*>(a.codes + p.b));
        ba[u] = __ldg(a.scales + p.sa);
        bb[u] = __ldg(a.scales + p.sb);
        g[u].load(static_cast<const E*>(a.dh) + p.dh);
      }
    }
#pragma unroll
    for (int u = 0; u < kSwigluUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      if (off >= left) continue;
      const PairSpot<FLAT> p(a, first, s, off);
      float va[2][4], vb[2][4], gv[kPairs], da[kPairs], db[kPairs], hv[kPairs];
      codes_to_float(qa[u].x, va[0]);
      codes_to_float(qa[u].y, va[1]);
      codes_to_float(qb[u].x, vb[0]);
      codes_to_float(qb[u].y, vb[1]);
      g[u].get(gv);
      const float sa = scale_value(ba[u]), sb = scale_value(bb[u]);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const SwigluOut o = swiglu_grad(va[j / 4][j % 4] * sa, vb[j / 4][j % 4] * sb, gv[j]);
        da[j] = o.da;
        db[j] = o.db;
        hv[j] = o.h;
      }
      Run<E, kPairs> o;
      o.set(da);
      o.store(static_cast<E*>(a.dz) + p.da);
      o.set(db);
      o.store(static_cast<E*>(a.dz) + p.db);
      if (a.h) {
        o.set(hv);
        o.store(static_cast<E*>(a.h) + p.h);
      }
    }
  }
}

// Rows of any width and alignment: a warp takes 32 kElemPairs consecutive pairs of one row, a lane
// every 32nd. Lane u (and kElemPairs + u, ...) holds the scales that the u-th group of 32 pairs needs.
// In the packed order a group's gate and up columns are each within one block; in halves the gate
// columns are, and the up columns, F further on, may spread over two.
constexpr int kElemPairs = 4;
template <typename E, bool PACKED, bool FULL>
__device__ __forceinline__ void swiglu_item(const Swiglu8Args& g, long long row, int f0, int left) {
  const int lane = threadIdx.x & 31, f = f0 + lane;
  const int8_t* codes = g.codes + row * 2 * g.F;
  const uint8_t* scales = g.scales + row * g.nb;
  const E* dh = static_cast<const E*>(g.dh) + row * g.ldh + f;
  // columns of the u-th pair: f0 is a multiple of 128, so in the packed order it is 2 f0 + ...
  auto col_a = [&](int u) { return PACKED ? 2 * f0 + (u >> 1) * 128 + (u & 1) * 32 + lane : f + 32 * u; };
  auto col_b = [&](int u) { return PACKED ? col_a(u) + 64 : f + 32 * u + g.F; };
  int qa[kElemPairs], qb[kElemPairs];
  float gv[kElemPairs];
#pragma unroll
  for (int u = 0; u < kElemPairs; ++u) {
    const bool ok = FULL || 32 * u < left;
    qa[u] = ok ? (int)__ldg(codes + col_a(u)) : 0;
    qb[u] = ok ? (int)__ldg(codes + col_b(u)) : 0;
    gv[u] = ok ? elem_to_float<E>(__ldg(dh + 32 * u)) : 0.f;
  }
  // lanes 0 .. kElemPairs-1: the gate blocks; from lane 16: the up blocks in order
  const int first_a = PACKED ? 2 * f0 / 32 : f0 / 32, first_b = PACKED ? first_a + 2 : (f0 + g.F) / 32;
  const int l = lane & 15;
  const int blk = (lane < 16 ? first_a : first_b) + (PACKED ? (l >> 1) * 4 + (l & 1) : l);
  const float sc = (l <= kElemPairs && blk < g.nb) ? scale_value(__ldg(scales + blk)) : 0.f;
  const int over = PACKED ? 0 : (((f0 + g.F) & 31) + lane) >> 5;  // 1: the lane's up columns lie in the next block
  E* dz = static_cast<E*>(g.dz) + row * g.lddz;
  E* h = g.h ? static_cast<E*>(g.h) + row * g.ldo + f : nullptr;
#pragma unroll
  for (int u = 0; u < kElemPairs; ++u) {
    const float sa = __shfl_sync(0xffffffffu, sc, u), sb = __shfl_sync(0xffffffffu, sc, 16 + u + over);
    const SwigluOut o = swiglu_grad((float)qa[u] * sa, (float)qb[u] * sb, gv[u]);
    if (FULL || 32 * u < left) {
      dz[col_a(u)] = float_to_elem<E>(o.da);
      dz[col_b(u)] = float_to_elem<E>(o.db);
      if (h) h[32 * u] = float_to_elem<E>(o.h);
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kCkptThreads) swiglu_backward8_elem_kernel(Swiglu8Args a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.walk.per_row.d;
  ItemPos p = at(a.walk.begin(), threadIdx.x >> 5, a.walk.per_row);
  for (long long i = (long long)blockIdx.x * kCkptWarps + (threadIdx.x >> 5); i < n;
       i += (long long)gridDim.x * kCkptWarps, a.walk.next(p)) {
    const int f0 = (int)p.i * 32 * kElemPairs;
    const int left = a.F - f0 - lane;
    const bool full = a.F - f0 >= 32 * kElemPairs;
    if (a.packed) {
      if (full) swiglu_item<E, true, true>(a, p.row, f0, left);
      else swiglu_item<E, true, false>(a, p.row, f0, left);
    } else {
      if (full) swiglu_item<E, false, true>(a, p.row, f0, left);
      else swiglu_item<E, false, false>(a, p.row, f0, left);
    }
  }
}

// The walk over rows of per_row items in tiles, and its grid: at most `ctas` CTAs a
// multiprocessor, each looping over its tiles.
static Walk make_walk(long long rows, long long per_row, int tile, int ctas, unsigned* grid) {
  const long long tiles = (rows * per_row + tile - 1) / tile;
  *grid = (unsigned)std::max<long long>(1, std::min<long long>(tiles, (long long)sm_count() * ctas));
  const long long step = (long long)*grid * tile;
  Walk w;
  w.per_row = FastDiv((uint32_t)per_row);
  w.tile = (uint32_t)tile;
  w.step_rows = (uint32_t)(step / per_row);
  w.step_items = (uint32_t)(step % per_row);
  return w;
}

static Ckpt8Args ckpt8_args(long long rows, int cols, const int32_t* used, uint32_t* status) {
  Ckpt8Args a{};
  a.used = used;
  a.status = status;
  a.rows = rows;
  a.cols = cols;
  a.nb = (cols + 31) / 32;
  return a;
}

// Rows whose columns lie in 16-byte pieces and whose codes in 8-byte ones; `flat`: dense rows of
// whole blocks besides, codes in 16-byte pieces.
static bool ckpt8_vec(const Ckpt8Args& a, const void* x, int bytes, bool* flat) {
  const uintptr_t codes = reinterpret_cast<uintptr_t>(a.codes);
  *flat = a.ld == a.cols && a.cols % 32 == 0 && codes % 16 == 0;
  return a.cols % 8 == 0 && rows_aligned16(x, a.ld, bytes) && codes % 8 == 0;
}

template <typename E, int NB, bool STORE>
static int ckpt8_elem_go(Ckpt8Args a, cudaStream_t st) {
  constexpr int kRows = kElemBlocks / NB;
  unsigned grid;
  a.walk = make_walk((a.rows + kRows - 1) / kRows, (a.nb + NB - 1) / NB, kCkptWarps, kCkptCtas, &grid);
  return launch_pdl(ckpt8_elem_kernel<E, NB, STORE>, dim3(grid), dim3(kCkptThreads), 0, st, a);
}

template <typename E, bool STORE>
static int ckpt8_elem_run(const Ckpt8Args& a, cudaStream_t st) {
  // several rows an item while a row has at most half the blocks of one (262144 x 7, store and
  // restore: 30 us, 128 with one row an item)
  if (a.nb == 1) return ckpt8_elem_go<E, 1, STORE>(a, st);
  if (a.nb == 2) return ckpt8_elem_go<E, 2, STORE>(a, st);
  return a.nb <= 4 ? ckpt8_elem_go<E, 4, STORE>(a, st) : ckpt8_elem_go<E, 8, STORE>(a, st);
}

template <typename E>
static int checkpoint8_run(Ckpt8Args a, cudaStream_t st) {
  bool flat;
  if (!ckpt8_vec(a, a.x, sizeof(E), &flat)) return ckpt8_elem_run<E, true>(a, st);
  unsigned grid;
  a.walk = make_walk(a.rows, 2 * a.nb, kCkptThreads * kUnroll, kCkptCtas, &grid);
  auto kern = flat ? checkpoint8_kernel<E, true> : checkpoint8_kernel<E, false>;
  return launch_pdl(kern, dim3(grid), dim3(kCkptThreads), 0, st, a);
}

template <typename E>
static int restore8_run(Ckpt8Args a, cudaStream_t st) {
  bool flat;
  if (!ckpt8_vec(a, a.out, sizeof(E), &flat)) return ckpt8_elem_run<E, false>(a, st);
  unsigned grid;
  a.walk = make_walk(a.rows, (long long)a.cols * sizeof(E) / 16, kCkptThreads * kRestoreUnroll, kCkptCtas, &grid);
  auto kern = flat ? restore8_kernel<E, true> : restore8_kernel<E, false>;
  return launch_pdl(kern, dim3(grid), dim3(kCkptThreads), 0, st, a);
}

template <typename E>
static int swiglu_backward8_run(Swiglu8Args a, cudaStream_t st) {
  const bool vec = a.F % 8 == 0 && rows_aligned16(a.dh, a.ldh, sizeof(E)) && rows_aligned16(a.dz, a.lddz, sizeof(E)) &&
                   (!a.h || rows_aligned16(a.h, a.ldo, sizeof(E))) && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  const bool flat = a.packed && a.ldh == a.F && a.lddz == 2 * a.F && (!a.h || a.ldo == a.F);
  unsigned grid;
  a.walk = make_walk(a.rows, vec ? a.F / kPairs : (a.F + 32 * kElemPairs - 1) / (32 * kElemPairs),
                     vec ? kCkptThreads * kSwigluUnroll : kCkptWarps, kSwigluCtas, &grid);
  auto kern = !vec ? swiglu_backward8_elem_kernel<E>
              : flat ? swiglu_backward8_kernel<E, true>
                     : swiglu_backward8_kernel<E, false>;
  return launch_pdl(kern, dim3(grid), dim3(kCkptThreads), 0, st, a);
}

int launch_checkpoint8(long long rows, int cols, int dtype, const void* x, long long ldx, const int32_t* used,
                       int8_t* codes, uint8_t* scales, uint32_t* status, cudaStream_t st) {
  Ckpt8Args a = ckpt8_args(rows, cols, used, status);
  a.x = x;
  a.ld = ldx;
  a.codes = codes;
  a.scales = scales;
  return dtype == MOE_DTYPE_BF16 ? checkpoint8_run<__nv_bfloat16>(a, st)
         : dtype == MOE_DTYPE_F16 ? checkpoint8_run<__half>(a, st)
                                  : checkpoint8_run<float>(a, st);
}

int launch_restore8(long long rows, int cols, int dtype, const int8_t* codes, const uint8_t* scales,
                    const int32_t* used, void* x, long long ldx, uint32_t* status, cudaStream_t st) {
  Ckpt8Args a = ckpt8_args(rows, cols, used, status);
  a.out = x;
  a.ld = ldx;
  a.codes = const_cast<int8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  return dtype == MOE_DTYPE_BF16 ? restore8_run<__nv_bfloat16>(a, st)
         : dtype == MOE_DTYPE_F16 ? restore8_run<__half>(a, st)
                                  : restore8_run<float>(a, st);
}

int launch_swiglu_backward8(long long rows, int F, int packed, int dtype, const int8_t* codes, const uint8_t* scales,
                            const void* dh, long long lddh, const int32_t* used, void* dz, long long lddz, void* h,
                            long long ldh, uint32_t* status, cudaStream_t st) {
  Swiglu8Args a{};
  a.codes = codes;
  a.scales = scales;
  a.dh = dh;
  a.dz = dz;
  a.h = h;
  a.used = used;
  a.status = status;
  a.rows = rows;
  a.ldh = lddh;
  a.lddz = lddz;
  a.ldo = ldh;
  a.F = F;
  a.nb = (2 * F + 31) / 32;
  a.packed = packed;
  return dtype == MOE_DTYPE_BF16 ? swiglu_backward8_run<__nv_bfloat16>(a, st)
         : dtype == MOE_DTYPE_F16 ? swiglu_backward8_run<__half>(a, st)
                                  : swiglu_backward8_run<float>(a, st);
}

}  // namespace moe
