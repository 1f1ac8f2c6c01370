// Element types and vector accesses of the row operators (route.cu, rows.cu,
// mx_quant.cu): fp32, bf16 and fp16 elements in memory, fp32 in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "internal.h"

namespace mm {

template <typename T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// N elements moved by one access, aligned to its own size.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// Vec's loads and stores: one access of up to 32 bytes, kept out of L1 (each row passes through once).
template <typename V>
__device__ __forceinline__ V load_once(const V* p) {
  V v;
  if constexpr (sizeof(V) == 32) {
    uint32_t w[8];
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
    memcpy(&v, w, 32);
  } else if constexpr (sizeof(V) == 16) {
    uint32_t w[4];
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
    memcpy(&v, w, 16);
  } else {
    v = *p;
  }
  return v;
}
template <typename V>
__device__ __forceinline__ void store_once(V* p, const V& v) {
  if constexpr (sizeof(V) == 32) {
    uint32_t w[8];
    memcpy(w, &v, 32);
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *p = v;
  }
}

inline int dtype_size(int dtype) { return dtype == MM_MOE_DTYPE_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) { return dtype >= MM_MOE_DTYPE_F32 && dtype <= MM_MOE_DTYPE_F16; }

// The widest access (32, 16, 8, 4 or 2 bytes) that every given address and row
// pitch is a multiple of; the bits of all of them are or-ed into `bits`.
inline int access_bytes(uint64_t bits) {
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
}

// f(T{}) with the element type a dtype names
template <typename F>
cudaError_t with_dtype(int dtype, F f) {
  switch (dtype) {
    case MM_MOE_DTYPE_F32: return f(float{});
    case MM_MOE_DTYPE_BF16: return f(__nv_bfloat16{});
    case MM_MOE_DTYPE_F16: return f(__half{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mm
