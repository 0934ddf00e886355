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
#include "rows.cuh"

#include <algorithm>

#ifndef KU
#define KU 4
#endif
#ifndef KUS
#define KUS 2
#endif
#ifndef KMB
#define KMB 1
#endif
#ifndef KSB
#define KSB 1
#endif
#ifndef KG
#define KG 8
#endif
namespace moe {

constexpr int kCkptThreads = 256;
constexpr uint32_t kByteNan = 255u;

// Scale byte of a block from its largest magnitude's fp32 bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  const uint32_t e = top_bits >> 23;
  return e == 255u ? kByteNan : max((int)e - 6, 1);
}
// 2^-E (finite blocks: bytes 1 .. 248).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }

// rint(x 2^-E) clamped to +-127, as the low byte of 1.5 2^23 + code: the product is exact, so the
// addition's rounding to nearest even is the only one (|x 2^-E| < 128).
constexpr float kRoundBias = 12582912.f;
__device__ __forceinline__ uint32_t quantise(float x, float inv) {
  const float q = fmaf(x, inv, kRoundBias);
  return __float_as_uint(fminf(fmaxf(q, kRoundBias - 127.f), kRoundBias + 127.f));
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

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

// Eight consecutive elements as fp32, by 16-byte accesses.
template <typename E>
struct Eight {
  static constexpr int V = 16 / sizeof(E), W = 8 / V;
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
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float f[V];
      w[i].get(f);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i * V + j] = f[j];
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = v[i * V + j];
      w[i].set(f);
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
  int cols, nb;     // nb: blocks (scale bytes) of a row
  FastDiv per_row;  // work items of a row
};

// Work items are cut into tiles of consecutive ones, a CTA's step. tile_start gives the row
// and the item in it of a tile's first item; at() adds a thread's offset.
struct ItemPos {
  long long row;
  uint32_t i;
};
__device__ __forceinline__ ItemPos tile_start(long long first, const FastDiv& per_row) {
  const long long row = first / per_row.d;
  return {row, (uint32_t)(first - row * per_row.d)};
}
__device__ __forceinline__ ItemPos at(const ItemPos& s, uint32_t off, const FastDiv& per_row) {
  const uint32_t n = s.i + off, q = per_row.quotient(n);
  return {s.row + q, n - q * per_row.d};
}

// Store, rows of 16-byte pieces: an item is eight columns, four neighbouring lanes a block (a
// row has 4 nb items; those past its end stand for zeros). kUnroll items a thread are loaded
// before any is used.
constexpr int kUnroll = KU;
template <typename E>
__global__ void __launch_bounds__(kCkptThreads, KMB) checkpoint8_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.per_row.d;
  constexpr int kTile = kCkptThreads * kUnroll;
  for (long long first = (long long)blockIdx.x * kTile; first < n; first += (long long)gridDim.x * kTile) {
    const ItemPos s = tile_start(first, a.per_row);
    const uint32_t left = (uint32_t)min((long long)kTile, n - first);
    Eight<E> x[kUnroll];
    ItemPos p[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      p[u] = at(s, off, a.per_row);
      if (off < left && p[u].i * 8 < (uint32_t)a.cols)
        x[u].load(static_cast<const E*>(a.x) + p[u].row * a.ld + p[u].i * 8);
      else
        x[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[8];
      x[u].get(v);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t byte = scale_byte(top);
      const float inv = scale_inverse(byte);
      uint2 q = make_uint2(pack4(quantise(v[0], inv), quantise(v[1], inv), quantise(v[2], inv), quantise(v[3], inv)),
                           pack4(quantise(v[4], inv), quantise(v[5], inv), quantise(v[6], inv), quantise(v[7], inv)));
      if (byte == kByteNan) q = make_uint2(0u, 0u);
      if (u * kCkptThreads + threadIdx.x < left) {
        if (p[u].i * 8 < (uint32_t)a.cols)
          *reinterpret_cast<uint2*>(a.codes + p[u].row * a.cols + p[u].i * 8) = q;
        if ((p[u].i & 3u) == 0u) a.scales[p[u].row * a.nb + (p[u].i >> 2)] = (uint8_t)byte;
      }
    }
  }
}

// Rows of any width and alignment: a warp takes kElemBlocks consecutive blocks of one row (an
// item), a lane one element of each, so that all addresses are one base plus constants.
constexpr int kElemBlocks = 8;
constexpr int kElemCols = 32 * kElemBlocks;
constexpr int kCkptWarps = kCkptThreads / 32;
template <typename E>
__global__ void __launch_bounds__(kCkptThreads) checkpoint8_elem_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.per_row.d;
  for (long long first = (long long)blockIdx.x * kCkptWarps; first < n; first += (long long)gridDim.x * kCkptWarps) {
    if (first + (threadIdx.x >> 5) >= n) break;  // warp-uniform
    const ItemPos p = at(tile_start(first, a.per_row), threadIdx.x >> 5, a.per_row);
    const int c0 = (int)p.i * kElemCols;
    const int left = a.cols - c0 - lane;  // this lane's element of block u is in the row if 32 u < left
    const E* x = static_cast<const E*>(a.x) + p.row * a.ld + c0 + lane;
    int8_t* codes = a.codes + p.row * a.cols + c0 + lane;
    float v[kElemBlocks];
#pragma unroll
    for (int u = 0; u < kElemBlocks; ++u) v[u] = 32 * u < left ? elem_to_float<E>(__ldg(x + 32 * u)) : 0.f;
    uint32_t mine = 0;  // lane u: the scale byte of block u
#pragma unroll
    for (int u = 0; u < kElemBlocks; ++u) {
      const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v[u]) & 0x7fffffffu));
      const uint32_t q = quantise(v[u], scale_inverse(byte));
      if (32 * u < left) codes[32 * u] = byte == kByteNan ? 0 : (int8_t)q;
      if (lane == u) mine = byte;
    }
    const int blk = (int)p.i * kElemBlocks + lane;
    if (lane < kElemBlocks && blk < a.nb) a.scales[p.row * a.nb + blk] = (uint8_t)mine;
  }
}

// Restore, rows of 16-byte pieces: an item is eight columns.
template <typename E>
__global__ void __launch_bounds__(kCkptThreads, KMB) restore8_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.per_row.d;
  constexpr int kTile = kCkptThreads * kUnroll;
  for (long long first = (long long)blockIdx.x * kTile; first < n; first += (long long)gridDim.x * kTile) {
    const ItemPos s = tile_start(first, a.per_row);
    const uint32_t left = (uint32_t)min((long long)kTile, n - first);
    uint2 q[kUnroll];
    uint32_t byte[kUnroll];
    ItemPos p[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      p[u] = at(s, off, a.per_row);
      if (off < left) {
        q[u] = __ldg(reinterpret_cast<const uint2*>(a.codes + p[u].row * a.cols + p[u].i * 8));
        byte[u] = __ldg(a.scales + p[u].row * a.nb + (p[u].i >> 2));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (u * kCkptThreads + threadIdx.x >= left) continue;
      float lo[4], hi[4], v[8];
      codes_to_float(q[u].x, lo);
      codes_to_float(q[u].y, hi);
      const float sc = scale_value(byte[u]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = lo[j] * sc;
        v[4 + j] = hi[j] * sc;
      }
      Eight<E> o;
      o.set(v);
      o.store(static_cast<E*>(a.out) + p[u].row * a.ld + p[u].i * 8);
    }
  }
}

template <typename E>
__global__ void __launch_bounds__(kCkptThreads) restore8_elem_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.per_row.d;
  for (long long first = (long long)blockIdx.x * kCkptWarps; first < n; first += (long long)gridDim.x * kCkptWarps) {
    if (first + (threadIdx.x >> 5) >= n) break;
    const ItemPos p = at(tile_start(first, a.per_row), threadIdx.x >> 5, a.per_row);
    const int c0 = (int)p.i * kElemCols;
    const int left = a.cols - c0 - lane;
    E* x = static_cast<E*>(a.out) + p.row * a.ld + c0 + lane;
    const int8_t* codes = a.codes + p.row * a.cols + c0 + lane;
    const uint8_t* scales = a.scales + p.row * a.nb + p.i * kElemBlocks;
    int q[kElemBlocks];
    uint32_t byte[kElemBlocks];
#pragma unroll
    for (int u = 0; u < kElemBlocks; ++u) {
      q[u] = 32 * u < left ? (int)__ldg(codes + 32 * u) : 0;
      byte[u] = 32 * u < left ? (uint32_t)__ldg(scales + u) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kElemBlocks; ++u)
      if (32 * u < left) x[32 * u] = float_to_elem<E>((float)q[u] * scale_value(byte[u]));
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
  FastDiv per_row;
};

// da = dh b s (1 + a (1 - s)), db = dh a s, h = a s b with s = 1 / (1 + exp(-a)); fp32, one
// rounding per output. expf and the fast division are within 2 ulp each; the division gives 0
// where exp(-a) passes 2^126, as s is below fp32's normal range there.
struct SwigluOut {
  float da, db, h;
};
__device__ __forceinline__ SwigluOut swiglu_grad(float a, float b, float g) {
  const float s = __fdividef(1.f, 1.f + expf(-a));
  const float as = a * s;
  return {g * b * s * (1.f + a * (1.f - s)), g * as, as * b};
}

// Rows of 16-byte pieces: an item is eight pairs of pre-activations.
constexpr int kSwigluUnroll = KUS;
template <typename E>
__global__ void __launch_bounds__(kCkptThreads, KSB) swiglu_backward8_kernel(Swiglu8Args a) {
  pdl_wait_then_release();
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.per_row.d;
  constexpr int kTile = kCkptThreads * kSwigluUnroll;
  for (long long first = (long long)blockIdx.x * kTile; first < n; first += (long long)gridDim.x * kTile) {
    const ItemPos s = tile_start(first, a.per_row);
    const uint32_t left = (uint32_t)min((long long)kTile, n - first);
    uint2 qa[kSwigluUnroll], qb[kSwigluUnroll];
    uint32_t ba[kSwigluUnroll], bb[kSwigluUnroll];
    Eight<E> g[kSwigluUnroll];
    ItemPos p[kSwigluUnroll];
    int ca[kSwigluUnroll], cb[kSwigluUnroll];
#pragma unroll
    for (int u = 0; u < kSwigluUnroll; ++u) {
      const uint32_t off = u * kCkptThreads + threadIdx.x;
      p[u] = at(s, off, a.per_row);
      const int f = (int)p[u].i * 8;
      ca[u] = a.packed ? (f >> 6) * 128 + (f & 63) : f;
      cb[u] = a.packed ? ca[u] + 64 : f + a.F;
      if (off < left) {
        const int8_t* q = a.codes + p[u].row * 2 * a.F;
        const uint8_t* sc = a.scales + p[u].row * a.nb;
        qa[u] = __ldg(reinterpret_cast<const uint2*>(q + ca[u]));
        qb[u] = __ldg(reinterpret_cast<const uint2*>(q + cb[u]));
        ba[u] = __ldg(sc + (ca[u] >> 5));
        bb[u] = __ldg(sc + (cb[u] >> 5));
        g[u].load(static_cast<const E*>(a.dh) + p[u].row * a.ldh + f);
      }
    }
#pragma unroll
    for (int u = 0; u < kSwigluUnroll; ++u) {
      if (u * kCkptThreads + threadIdx.x >= left) continue;
      float va[2][4], vb[2][4], gv[8], da[8], db[8], hv[8];
      codes_to_float(qa[u].x, va[0]);
      codes_to_float(qa[u].y, va[1]);
      codes_to_float(qb[u].x, vb[0]);
      codes_to_float(qb[u].y, vb[1]);
      g[u].get(gv);
      const float sa = scale_value(ba[u]), sb = scale_value(bb[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const SwigluOut o = swiglu_grad(va[j / 4][j % 4] * sa, vb[j / 4][j % 4] * sb, gv[j]);
        da[j] = o.da;
        db[j] = o.db;
        hv[j] = o.h;
      }
      Eight<E> o;
      E* dz = static_cast<E*>(a.dz) + p[u].row * a.lddz;
      o.set(da);
      o.store(dz + ca[u]);
      o.set(db);
      o.store(dz + cb[u]);
      if (a.h) {
        o.set(hv);
        o.store(static_cast<E*>(a.h) + p[u].row * a.ldo + p[u].i * 8);
      }
    }
  }
}

// Rows of any width and alignment: a warp takes 32 kElemPairs consecutive pairs of one row.
constexpr int kElemPairs = 4;
template <typename E>
__global__ void __launch_bounds__(kCkptThreads) swiglu_backward8_elem_kernel(Swiglu8Args a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.per_row.d;
  for (long long first = (long long)blockIdx.x * kCkptWarps; first < n; first += (long long)gridDim.x * kCkptWarps) {
    if (first + (threadIdx.x >> 5) >= n) break;
    const ItemPos p = at(tile_start(first, a.per_row), threadIdx.x >> 5, a.per_row);
    const int f0 = (int)p.i * 32 * kElemPairs + lane;
    const int left = a.F - f0;
    const int8_t* codes = a.codes + p.row * 2 * a.F;
    const uint8_t* scales = a.scales + p.row * a.nb;
    const E* dh = static_cast<const E*>(a.dh) + p.row * a.ldh + f0;
    E* dz = static_cast<E*>(a.dz) + p.row * a.lddz;
    int qa[kElemPairs], qb[kElemPairs];
    uint32_t ba[kElemPairs], bb[kElemPairs];
    float g[kElemPairs];
#pragma unroll
    for (int u = 0; u < kElemPairs; ++u) {
      if (32 * u >= left) continue;
      const int f = f0 + 32 * u;
      const int ca = a.packed ? (f >> 6) * 128 + (f & 63) : f, cb = a.packed ? ca + 64 : f + a.F;
      qa[u] = __ldg(codes + ca);
      qb[u] = __ldg(codes + cb);
      ba[u] = __ldg(scales + (ca >> 5));
      bb[u] = __ldg(scales + (cb >> 5));
      g[u] = elem_to_float<E>(__ldg(dh + 32 * u));
    }
#pragma unroll
    for (int u = 0; u < kElemPairs; ++u) {
      if (32 * u >= left) continue;
      const int f = f0 + 32 * u;
      const int ca = a.packed ? (f >> 6) * 128 + (f & 63) : f, cb = a.packed ? ca + 64 : f + a.F;
      const SwigluOut o = swiglu_grad((float)qa[u] * scale_value(ba[u]), (float)qb[u] * scale_value(bb[u]), g[u]);
      dz[ca] = float_to_elem<E>(o.da);
      dz[cb] = float_to_elem<E>(o.db);
      if (a.h) static_cast<E*>(a.h)[p.row * a.ldo + f] = float_to_elem<E>(o.h);
    }
  }
}

// CTAs for `items` in tiles: at most eight a multiprocessor, each looping over its tiles.
static unsigned tile_grid(long long rows, long long per_row, int tile) {
  const long long tiles = (rows * per_row + tile - 1) / tile;
  return (unsigned)std::max<long long>(1, std::min<long long>(tiles, (long long)sm_count() * KG));
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

template <typename E>
static int checkpoint8_run(Ckpt8Args a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && rows_aligned16(a.x, a.ld, sizeof(E)) &&
                   reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  a.per_row = FastDiv((uint32_t)(vec ? 4 * a.nb : (a.cols + kElemCols - 1) / kElemCols));
  const int tile = vec ? kCkptThreads * kUnroll : kCkptWarps;
  return launch_pdl(vec ? checkpoint8_kernel<E> : checkpoint8_elem_kernel<E>, dim3(tile_grid(a.rows, a.per_row.d, tile)),
                    dim3(kCkptThreads), 0, st, a);
}

template <typename E>
static int restore8_run(Ckpt8Args a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && rows_aligned16(a.out, a.ld, sizeof(E)) &&
                   reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  a.per_row = FastDiv((uint32_t)(vec ? a.cols / 8 : (a.cols + kElemCols - 1) / kElemCols));
  const int tile = vec ? kCkptThreads * kUnroll : kCkptWarps;
  return launch_pdl(vec ? restore8_kernel<E> : restore8_elem_kernel<E>, dim3(tile_grid(a.rows, a.per_row.d, tile)),
                    dim3(kCkptThreads), 0, st, a);
}

template <typename E>
static int swiglu_backward8_run(Swiglu8Args a, cudaStream_t st) {
  const bool vec = a.F % 8 == 0 && rows_aligned16(a.dh, a.ldh, sizeof(E)) && rows_aligned16(a.dz, a.lddz, sizeof(E)) &&
                   (!a.h || rows_aligned16(a.h, a.ldo, sizeof(E))) && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  a.per_row = FastDiv((uint32_t)(vec ? a.F / 8 : (a.F + 32 * kElemPairs - 1) / (32 * kElemPairs)));
  const int tile = vec ? kCkptThreads * kSwigluUnroll : kCkptWarps;
  return launch_pdl(vec ? swiglu_backward8_kernel<E> : swiglu_backward8_elem_kernel<E>,
                    dim3(tile_grid(a.rows, a.per_row.d, tile)), dim3(kCkptThreads), 0, st, a);
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
