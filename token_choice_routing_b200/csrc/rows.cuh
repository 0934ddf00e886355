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

#ifdef __CUDACC__

template <typename T>
__device__ __forceinline__ float elem_to_float(T v);
template <>
__device__ __forceinline__ float elem_to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float elem_to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float elem_to_float<float>(float v) { return v; }

// One rounding to nearest even, the only one an output of these kernels takes.
template <typename T>
__device__ __forceinline__ T float_to_elem(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 float_to_elem<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half float_to_elem<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float float_to_elem<float>(float v) { return v; }

// V consecutive elements: one 16-byte access when V fills it, an element access when V = 1.
template <typename T, int V>
struct Piece {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* p) {
  Piece<T, V> r;
  if constexpr (V * sizeof(T) == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    memcpy(r.e, &v, 16);
  } else {
    static_assert(V == 1, "a piece is 16 bytes or one element");
    r.e[0] = *p;
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ Piece<T, V> zero_piece() {
  Piece<T, V> r;
  memset(r.e, 0, sizeof(r.e));
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, V>& r) {
  if constexpr (V * sizeof(T) == 16) {
    uint4 v;
    memcpy(&v, r.e, 16);
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    *p = r.e[0];
  }
}

#endif  // __CUDACC__

}  // namespace moe
