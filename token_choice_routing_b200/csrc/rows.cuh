// Row access shared by the slot-sorting and 8-bit checkpoint kernels: a lane's piece of a row
// in bf16, fp16 or fp32 as fp32 values, by 16-byte accesses where the row layout allows them
// and by single elements otherwise.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

// Bytes of one element of a moe_dtype_t (0: not one).
inline int dtype_bytes(int dtype) {
  return dtype == MOE_DTYPE_F32 ? 4 : (dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16) ? 2 : 0;
}

// Whether rows at p, ld elements of `bytes` apart, all start on a 16-byte boundary.
inline bool rows_aligned16(const void* p, int64_t ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ((uint64_t)ld * (uint64_t)bytes) % 16u == 0;
}

// Division of n < 2^31 by a fixed 1 <= d < 2^31 as a multiplication (Granlund and Montgomery):
// with 2^(l-1) < d <= 2^l and m = ceil(2^(31+l) / d), floor(n / d) = floor(n m / 2^(31+l)).
struct FastDiv {
  uint32_t d, m, shift;
  FastDiv() : d(1), m(0), shift(0) {}
  explicit FastDiv(uint32_t div) : d(div), m(0), shift(0) {
    int l = 0;
    while ((1ull << l) < div) ++l;
    if (l > 0) {
      m = (uint32_t)(((1ull << (31 + l)) + div - 1) / div);
      shift = (uint32_t)(l - 1);
    }
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return d == 1u ? n : __umulhi(n, m) >> shift; }
#endif
};

#ifdef __CUDACC__

template <typename T>
__device__ __forceinline__ float elem_to_float(T v);
template <>
__device__ __forceinline__ float elem_to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float elem_to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float elem_to_float<float>(float v) { return v; }

// The rounding to an output's type, to nearest even, of a value computed in fp32.
template <typename T>
__device__ __forceinline__ T float_to_elem(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 float_to_elem<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half float_to_elem<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float float_to_elem<float>(float v) { return v; }

// V consecutive elements as they lie in memory: four words by one 16-byte access, or one element
// (V = 1). The words stay whole until they are used: element arrays made the compiler split and
// rejoin them, at twice the kernel's time for the 16-bit types.
template <typename T, int V>
struct Piece {
  static_assert(V * sizeof(T) == 16, "a piece is 16 bytes or one element");
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_own(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void get(float (&v)[V]) const;
  __device__ __forceinline__ void set(const float (&v)[V]);
};
template <typename T>
struct Piece<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(p); }
  __device__ __forceinline__ void load_own(const T* p) { w = *p; }  // p may be written by this kernel
  __device__ __forceinline__ void zero() { w = float_to_elem<T>(0.f); }
  __device__ __forceinline__ void store(T* p) const { *p = w; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = elem_to_float<T>(w); }
  __device__ __forceinline__ void set(const float (&v)[1]) { w = float_to_elem<T>(v[0]); }
};

// Two 16-bit elements of a word as fp32 and back.
template <typename T>
__device__ __forceinline__ float2 word_to_float2(uint32_t w);
template <>
__device__ __forceinline__ float2 word_to_float2<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16lo(w), bf16hi(w));
}
template <>
__device__ __forceinline__ float2 word_to_float2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t float2_to_word(float a, float b);
template <>
__device__ __forceinline__ uint32_t float2_to_word<__nv_bfloat16>(float a, float b) { return pack_bf16x2(a, b); }
template <>
__device__ __forceinline__ uint32_t float2_to_word<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int V>
__device__ __forceinline__ void Piece<T, V>::get(float (&v)[V]) const {
  if constexpr (V == 4) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  } else {
    const float2 a = word_to_float2<T>(w.x), b = word_to_float2<T>(w.y), c = word_to_float2<T>(w.z),
                 d = word_to_float2<T>(w.w);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
  }
}
template <typename T, int V>
__device__ __forceinline__ void Piece<T, V>::set(const float (&v)[V]) {
  if constexpr (V == 4)
    w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    w = make_uint4(float2_to_word<T>(v[0], v[1]), float2_to_word<T>(v[2], v[3]), float2_to_word<T>(v[4], v[5]),
                   float2_to_word<T>(v[6], v[7]));
}

// Four int8 codes of a word as fp32: each byte, its sign bit flipped, becomes the low mantissa
// byte of 2^23 + (code + 128), from which 2^23 + 128 is taken off exactly. One byte permute and
// one addition a code, where the integer conversion runs at a fraction of that rate.
__device__ __forceinline__ void codes_to_float(uint32_t word, float (&v)[4]) {
  const uint32_t u = word ^ 0x80808080u;
  v[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)) - 8388736.f;
  v[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541)) - 8388736.f;
  v[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)) - 8388736.f;
  v[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543)) - 8388736.f;
}

// A piece of a row held in 8 bits, without its scale (V divides 32: one scale byte a piece).
template <int V>
struct CodePiece {
  uint32_t word[V >= 4 ? V / 4 : 1];
};
template <int V>
__device__ __forceinline__ CodePiece<V> load_codes(const int8_t* p) {
  CodePiece<V> r;
  if constexpr (V == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    r.word[0] = v.x;
    r.word[1] = v.y;
  } else if constexpr (V == 4) {
    r.word[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else {
    static_assert(V == 1, "8, 4 or 1 codes");
    r.word[0] = (uint8_t)__ldg(p);
  }
  return r;
}

// 2^E of a scale byte, NaN for byte 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// ---- 8-bit blocks: 32 columns with one power-of-two scale (the format is described in ckpt8.cu)
constexpr uint32_t kByteNan = 255u;

// Scale byte of a block from its largest magnitude's fp32 bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  const uint32_t e = top_bits >> 23;
  return e == 255u ? kByteNan : max((int)e - 6, 1);
}
// 2^-E (finite blocks: bytes 1 .. 248).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __uint_as_float((254u - min(byte, 253u)) << 23);
}

// rint(x 2^-E) as the low 16 bits of 1.5 2^23 + code: the product is exact, so the addition's
// rounding to nearest even is the only one. |x 2^-E| < 128: the code is in [-128, 128] before the
// clamp, which is taken on two 16-bit codes at a time.
constexpr float kRoundBias = 12582912.f;
__device__ __forceinline__ uint32_t quantise(float x, float inv) { return __float_as_uint(fmaf(x, inv, kRoundBias)); }
__device__ __forceinline__ uint32_t clamp2(uint32_t two) {
  return __vmaxs2(__vmins2(two, 0x007f007fu), 0xff81ff81u);
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(clamp2(__byte_perm(a, b, 0x5410)), clamp2(__byte_perm(c, d, 0x5410)), 0x6420);
}

// Bits of the largest magnitude among the elements of a piece, as fp32 bits. The 16-bit types are
// compared as bits, two at a time: magnitudes order as their bits do, infinity and NaN on top.
template <typename E, int V>
__device__ __forceinline__ uint32_t top_of(const Piece<E, V>& p) {
  if constexpr (V == 4) {
    return max(max(p.w.x & 0x7fffffffu, p.w.y & 0x7fffffffu), max(p.w.z & 0x7fffffffu, p.w.w & 0x7fffffffu));
  } else {
    return __vmaxu2(__vmaxu2(p.w.x & 0x7fff7fffu, p.w.y & 0x7fff7fffu),
                    __vmaxu2(p.w.z & 0x7fff7fffu, p.w.w & 0x7fff7fffu));
  }
}
template <typename E, int V>
__device__ __forceinline__ uint32_t top_join(uint32_t a, uint32_t b) {
  return V == 4 ? max(a, b) : __vmaxu2(a, b);
}
template <typename E, int V>
__device__ __forceinline__ uint32_t top_bits(uint32_t t) {
  if constexpr (V == 4) {
    return t;
  } else {
    return __float_as_uint(word_to_float2<E>(max(t & 0xffffu, t >> 16)).x);
  }
}

// One block from 32 bf16 values in 16 words: its codes to a 16-byte boundary; returns the scale byte.
__device__ __forceinline__ uint32_t store_block8(const uint32_t (&w)[16], int8_t* codes) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
  const uint32_t byte = scale_byte(max(top & 0xffffu, top >> 16) << 16);
  const float inv = scale_inverse(byte);
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = pack4(quantise(bf16lo(w[2 * j]), inv), quantise(bf16hi(w[2 * j]), inv), quantise(bf16lo(w[2 * j + 1]), inv),
                 quantise(bf16hi(w[2 * j + 1]), inv));
    if (byte == kByteNan) q[j] = 0u;
  }
  reinterpret_cast<uint4*>(codes)[0] = make_uint4(q[0], q[1], q[2], q[3]);
  reinterpret_cast<uint4*>(codes)[1] = make_uint4(q[4], q[5], q[6], q[7]);
  return byte;
}

#endif  // __CUDACC__

}  // namespace moe
