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

// `bytes` (1 to 16) bytes from any address, and zeros or neighbouring bytes after them. Only 16-byte granules that
// hold one of these bytes are read.
__device__ __forceinline__ uint4 load16_any(const void* p, int bytes) {
  const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
  const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - m);
  const uint4 lo = __ldg(g);
  if (m == 0) return lo;
  uint4 hi = make_uint4(0, 0, 0, 0);
  if (m + bytes > 16) hi = __ldg(g + 1);
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (m & 8u) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (m & 4u) ? w[i + 1] : w[i];
  const uint32_t b = (m & 3u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], b), __funnelshift_r(w[1], w[2], b), __funnelshift_r(w[2], w[3], b),
                    __funnelshift_r(w[3], w[4], b));
}

// The i-th of the 16-byte granules of memory that a row of H elements at `row` touches: the elements [first, first + n)
// it holds. Rows on no 16-byte boundary are taken by the granules of what is written, so that all stores but a row's
// first and last are whole.
template <typename T>
struct Granule {
  static constexpr int kWhole = 16 / sizeof(T);
  int first, n;
  __device__ __forceinline__ Granule(const T* row, int H, int i) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / static_cast<int>(sizeof(T));
    const int e = i * kWhole - off;
    first = e < 0 ? 0 : e;
    n = min(e + kWhole, H) - first;
  }
  // granules that a row touches, at most
  __host__ __device__ static int most(int H) { return (H + 2 * kWhole - 2) / kWhole; }
  __device__ __forceinline__ Vec<T, kWhole> load(const T* row) const {
    const uint4 w = load16_any(row + first, n * static_cast<int>(sizeof(T)));
    Vec<T, kWhole> v;
    memcpy(&v, &w, 16);
    return v;
  }
  __device__ __forceinline__ void store(T* row, const Vec<T, kWhole>& v) const {
    if (n == kWhole) {
      *reinterpret_cast<Vec<T, kWhole>*>(row + first) = v;
    } else {
#pragma unroll
      for (int i = 0; i < kWhole; ++i)
        if (i < n) row[first + i] = v.v[i];
    }
  }
};

inline int dtype_size(int dtype) { return dtype == MM_MOE_DTYPE_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) { return dtype >= MM_MOE_DTYPE_F32 && dtype <= MM_MOE_DTYPE_F16; }

// The widest access (32 or 16 bytes, else 0) that every given address and row pitch is a multiple of; the bits of
// all of them are or-ed into `bits`.
inline int access_bytes(uint64_t bits) { return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0; }

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
