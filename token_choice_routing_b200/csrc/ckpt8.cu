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

namespace moe {

constexpr int kCkptThreads = 256;
constexpr uint32_t kByteNan = 255u;

// Scale byte of a block from its largest magnitude's fp32 bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  const uint32_t e = top_bits >> 23;
  return e == 255u ? kByteNan : max((int)e - 6, 1);
}
// 2^-E and 2^E of a scale byte (finite blocks: bytes 1 .. 248).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); }
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == kByteNan ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}
__device__ __forceinline__ int quantise(float x, float inv, uint32_t byte) {
  const float q = fminf(fmaxf(rintf(x * inv), -127.f), 127.f);
  return byte == kByteNan ? 0 : (int)q;
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

struct Ckpt8Args {
  const void* x;
  void* out;
  int8_t* codes;
  uint8_t* scales;
  const int32_t* used;
  uint32_t* status;
  long long rows, ld;
  int cols, nb;
};

// One warp per block of 32 columns, a lane per element.
template <typename E>
__global__ void __launch_bounds__(kCkptThreads) checkpoint8_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.nb;
  for (long long i = (long long)blockIdx.x * (kCkptThreads / 32) + (threadIdx.x >> 5); i < n;
       i += (long long)gridDim.x * (kCkptThreads / 32)) {
    const long long row = i / a.nb;
    const int c = (int)(i - row * a.nb) * 32 + lane;
    const float x = c < a.cols ? elem_to_float<E>(static_cast<const E*>(a.x)[row * a.ld + c]) : 0.f;
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu);
    const uint32_t byte = scale_byte(top);
    if (c < a.cols) a.codes[row * a.cols + c] = (int8_t)quantise(x, scale_inverse(byte), byte);
    if (lane == 0) a.scales[i] = (uint8_t)byte;
  }
}

template <typename E>
__global__ void __launch_bounds__(kCkptThreads) restore8_kernel(Ckpt8Args a) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.nb;
  for (long long i = (long long)blockIdx.x * (kCkptThreads / 32) + (threadIdx.x >> 5); i < n;
       i += (long long)gridDim.x * (kCkptThreads / 32)) {
    const long long row = i / a.nb;
    const int c = (int)(i - row * a.nb) * 32 + lane;
    if (c < a.cols)
      static_cast<E*>(a.out)[row * a.ld + c] =
          float_to_elem<E>((float)a.codes[row * a.cols + c] * scale_of(a.scales[i]));
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
  int F, packed;
};

// da = dh b s (1 + a (1 - s)), db = dh a s, h = a s b with s = 1 / (1 + exp(-a)); fp32, one
// rounding per output.
struct SwigluOut {
  float da, db, h;
};
__device__ __forceinline__ SwigluOut swiglu_grad(float a, float b, float g) {
  const float s = 1.f / (1.f + expf(-a));
  const float as = a * s;
  return {g * b * s * (1.f + a * (1.f - s)), g * as, as * b};
}

// One thread per pair of pre-activations.
template <typename E>
__global__ void __launch_bounds__(kCkptThreads) swiglu_backward8_kernel(Swiglu8Args a) {
  pdl_wait_then_release();
  const long long n = rows_in_use(a.used, a.rows, a.status) * a.F;
  const int nb = (2 * a.F + 31) / 32;
  for (long long i = (long long)blockIdx.x * kCkptThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kCkptThreads) {
    const long long row = i / a.F;
    const int f = (int)(i - row * a.F);
    const int ca = a.packed ? (f >> 6) * 128 + (f & 63) : f;
    const int cb = a.packed ? ca + 64 : f + a.F;
    const int8_t* q = a.codes + row * 2 * a.F;
    const uint8_t* sc = a.scales + row * nb;
    const SwigluOut o = swiglu_grad((float)q[ca] * scale_of(sc[ca >> 5]), (float)q[cb] * scale_of(sc[cb >> 5]),
                                    elem_to_float<E>(static_cast<const E*>(a.dh)[row * a.ldh + f]));
    E* dz = static_cast<E*>(a.dz) + row * a.lddz;
    dz[ca] = float_to_elem<E>(o.da);
    dz[cb] = float_to_elem<E>(o.db);
    if (a.h) static_cast<E*>(a.h)[row * a.ldo + f] = float_to_elem<E>(o.h);
  }
}

static int ckpt_grid(long long items, int per_block) {
  return (int)std::max<long long>(1, std::min<long long>((items + per_block - 1) / per_block, (long long)sm_count() * 8));
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

int launch_checkpoint8(long long rows, int cols, int dtype, const void* x, long long ldx, const int32_t* used,
                       int8_t* codes, uint8_t* scales, uint32_t* status, cudaStream_t st) {
  Ckpt8Args a = ckpt8_args(rows, cols, used, status);
  a.x = x;
  a.ld = ldx;
  a.codes = codes;
  a.scales = scales;
  auto kern = dtype == MOE_DTYPE_BF16 ? checkpoint8_kernel<__nv_bfloat16>
              : dtype == MOE_DTYPE_F16 ? checkpoint8_kernel<__half>
                                       : checkpoint8_kernel<float>;
  return launch_pdl(kern, dim3(ckpt_grid(rows * a.nb, kCkptThreads / 32)), dim3(kCkptThreads), 0, st, a);
}

int launch_restore8(long long rows, int cols, int dtype, const int8_t* codes, const uint8_t* scales,
                    const int32_t* used, void* x, long long ldx, uint32_t* status, cudaStream_t st) {
  Ckpt8Args a = ckpt8_args(rows, cols, used, status);
  a.out = x;
  a.ld = ldx;
  a.codes = const_cast<int8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  auto kern = dtype == MOE_DTYPE_BF16 ? restore8_kernel<__nv_bfloat16>
              : dtype == MOE_DTYPE_F16 ? restore8_kernel<__half>
                                       : restore8_kernel<float>;
  return launch_pdl(kern, dim3(ckpt_grid(rows * a.nb, kCkptThreads / 32)), dim3(kCkptThreads), 0, st, a);
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
  a.packed = packed;
  auto kern = dtype == MOE_DTYPE_BF16 ? swiglu_backward8_kernel<__nv_bfloat16>
              : dtype == MOE_DTYPE_F16 ? swiglu_backward8_kernel<__half>
                                       : swiglu_backward8_kernel<float>;
  return launch_pdl(kern, dim3(ckpt_grid(rows * F, kCkptThreads)), dim3(kCkptThreads), 0, st, a);
}

}  // namespace moe
