// What the training-pass operators share: element access in groups of eight, argument checks, launch counting.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "dp_device.cuh"
#include "dp_internal.h"
#include "dp_launch.h"
#include "dpops.h"

namespace dp {

typedef uint16_t bf16_t;  // bit pattern

template <typename T>
struct Elem;
template <>
struct Elem<bf16_t> {
  static __device__ __forceinline__ float get(bf16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ bf16_t put(float v) { return bf16_rn(v); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// Packed pairs of fp32 beside dp_device.cuh's.
__device__ __forceinline__ f2_t f2_fma(f2_t a, f2_t b, f2_t c) {
  f2_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2_t f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float f2_sum(f2_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}
__device__ __forceinline__ uint32_t f2_to_bf16x2(f2_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return bf16x2_rn(a, b);
}

// Eight elements as they lie in memory: one 16-byte word of bf16, two of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  uint4 a;
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  }
  __device__ __forceinline__ void unpack2(f2_t (&v)[4]) const {
    v[0] = bf16x2_to_f2(a.x); v[1] = bf16x2_to_f2(a.y); v[2] = bf16x2_to_f2(a.z); v[3] = bf16x2_to_f2(a.w);
  }
  __device__ __forceinline__ void pack2(const f2_t (&v)[4]) {
    a = make_uint4(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]), f2_to_bf16x2(v[2]), f2_to_bf16x2(v[3]));
  }
  __device__ __forceinline__ void pack(const float (&v)[8]) {
    a.x = bf16x2_rn(v[0], v[1]); a.y = bf16x2_rn(v[2], v[3]);
    a.z = bf16x2_rn(v[4], v[5]); a.w = bf16x2_rn(v[6], v[7]);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void unpack2(f2_t (&v)[4]) const {
    v[0] = f2_pack(a.x, a.y); v[1] = f2_pack(a.z, a.w); v[2] = f2_pack(b.x, b.y); v[3] = f2_pack(b.z, b.w);
  }
  __device__ __forceinline__ void pack2(const f2_t (&v)[4]) {
    f2_unpack(v[0], a.x, a.y);
    f2_unpack(v[1], a.z, a.w);
    f2_unpack(v[2], b.x, b.y);
    f2_unpack(v[3], b.z, b.w);
  }
  __device__ __forceinline__ void pack(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// 16-byte aligned access to eight elements, once-read and once-written data past L1.
__device__ __forceinline__ Raw8<bf16_t> load_raw8(const bf16_t* p) {
  Raw8<bf16_t> r;
  r.a = __ldcs(reinterpret_cast<const uint4*>(p));
  return r;
}
__device__ __forceinline__ Raw8<float> load_raw8(const float* p) {
  Raw8<float> r;
  r.a = __ldcs(reinterpret_cast<const float4*>(p));
  r.b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  return r;
}
__device__ __forceinline__ void store_raw8(bf16_t* p, const Raw8<bf16_t>& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
}
// Eight fp32 as one 32-byte store where the address allows it: two 16-byte stores touch every sector twice.
__device__ __forceinline__ void store_raw8(float* p, const Raw8<float>& r) {
  if (((uintptr_t)p & 31) == 0) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(r.a.x), "f"(r.a.y), "f"(r.a.z),
                 "f"(r.a.w), "f"(r.b.x), "f"(r.b.y), "f"(r.b.z), "f"(r.b.w)
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = r.a;
    reinterpret_cast<float4*>(p)[1] = r.b;
  }
}

// How many of the eight elements from c on a row of dim has.
__device__ __forceinline__ int there8(int64_t c, int64_t dim) { return dim - c < 0 ? 0 : dim - c > 8 ? 8 : (int)(dim - c); }

// ---- eight elements at any address
//
// Rows that are not 16-byte aligned (an odd width, a slice at an odd offset) would otherwise go element by element: eight
// instructions for eight elements, each over every sector of the warp's piece, a quarter of the aligned path's rate.

// Words i + by/4 .. of w, moved down by `by` bytes in all (0 <= by <= 16, a multiple of two).
template <int N, int OUT>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N], uint32_t by, uint32_t (&out)[OUT]) {
  if (by & 16) {
#pragma unroll
    for (int i = 0; i + 4 < N; ++i) w[i] = w[i + 4];
  }
  if (by & 8) {
#pragma unroll
    for (int i = 0; i + 2 < N; ++i) w[i] = w[i + 2];
  }
  if (by & 4) {
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) w[i] = w[i + 1];
  }
#pragma unroll
  for (int i = 0; i < OUT; ++i) out[i] = __funnelshift_r(w[i], i + 1 < N ? w[i + 1] : 0u, (by & 2) * 8);
}

// The first n (0..8) elements from byte `by` on of words that hold them, zeros behind them.
template <typename T, int N>
__device__ __forceinline__ Raw8<T> take8(uint32_t (&w)[N], uint32_t by, int n) {
  constexpr int WORDS = sizeof(T) * 2;  // 32-bit words of eight elements
  uint32_t out[WORDS];
  shift_words(w, by, out);
  if (n < 8) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      const int left = n * (int)sizeof(T) - 4 * i;  // bytes of this word that count
      out[i] &= left >= 4 ? 0xffffffffu : left == 2 ? 0xffffu : 0u;
    }
  }
  Raw8<T> r;
  uint32_t* to = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < WORDS; ++i) to[i] = out[i];
  return r;
}

// The first n (0..8) elements at p, zeros behind them.  Whole 16-byte words are read where they lie inside [lo, hi), the
// tensor; the others' elements one by one.
template <typename T>
__device__ __forceinline__ Raw8<T> load_any8(const T* p, int n, const T* lo, const T* hi) {
  constexpr int WORDS = sizeof(T) * 2;
  const uint32_t s = (uint32_t)(uintptr_t)p & 15u;
  const char* first = reinterpret_cast<const char*>(p) - s;
  const uint32_t need = s + (uint32_t)n * sizeof(T);  // bytes from `first`
  const uint32_t whole = (need + 15u) & ~15u;
  uint32_t w[WORDS + 4];
#pragma unroll
  for (int i = 0; i < WORDS + 4; ++i) w[i] = 0;
  if (n > 0 && first >= reinterpret_cast<const char*>(lo) && first + whole <= reinterpret_cast<const char*>(hi)) {
#pragma unroll
    for (int q = 0; q <= WORDS / 4; ++q) {
      if (need <= 16u * q) continue;
      const uint4 x = *(reinterpret_cast<const uint4*>(first) + q);  // L1 has it for the next lane
      w[4 * q] = x.x; w[4 * q + 1] = x.y; w[4 * q + 2] = x.z; w[4 * q + 3] = x.w;
    }
    return take8<T>(w, s, n);
  }
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < 2 * WORDS; ++i)
    if (i * 2 < n * (int)sizeof(T)) w[i >> 1] |= (uint32_t)h[i] << (16 * (i & 1));
  return take8<T>(w, 0, n);
}

// Writes the first n (0..8) elements of r to p; called by whole warps.  Where the next lane's elements follow this lane's in
// memory, the 16-byte word that the two share is put together and written by the next lane; what no whole word covers is
// written in halves of a word.
template <typename T>
__device__ __forceinline__ void store_any8(T* p, int n, const Raw8<T>& r) {
  constexpr int WORDS = sizeof(T) * 2;
  constexpr bool TWO = WORDS == 8;
  const int lane = threadIdx.x & 31, bytes = n * (int)sizeof(T);
  const uint32_t at = (uint32_t)(uintptr_t)p;
  const int s = (int)(at & 15u), cut = 16 - s;  // aligned words begin at bytes -s, cut, cut + 16 of this lane's
  uint32_t w[4 + WORDS], out[WORDS];
  const uint32_t* from = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < WORDS; ++i) w[4 + i] = from[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, from[WORDS - 4 + i], 1);  // the previous lane's last 16 bytes
  const uint32_t next_at = __shfl_down_sync(0xffffffffu, at, 1);
  const int next_bytes = __shfl_down_sync(0xffffffffu, bytes, 1);
  const bool gives = lane < 31 && n == 8 && next_at == at + 4 * WORDS && next_bytes >= cut;  // its bytes behind the last whole word
  const bool takes = __shfl_up_sync(0xffffffffu, (int)gives, 1) != 0 && lane > 0;
  shift_words(w, (uint32_t)cut, out);
  char* first = reinterpret_cast<char*>(p) - s;
  const bool word0 = (s == 0 || takes) && bytes >= cut, word1 = TWO && bytes >= cut + 16;
  if (word0) *reinterpret_cast<uint4*>(first) = make_uint4(out[0], out[1], out[2], out[3]);
  if (word1) *reinterpret_cast<uint4*>(first + 16) = make_uint4(out[WORDS - 4], out[WORDS - 3], out[WORDS - 2], out[WORDS - 1]);
  const int tail = TWO ? cut + 16 : cut;
  if (bytes > 0 && (!word0 || (TWO && !word1) || (bytes > tail && !gives))) {
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 2 * WORDS; ++i) {
      const int b = 2 * i;
      const bool written = b < cut ? word0 : b < tail ? word1 : gives;
      if (b < bytes && !written) h[i] = (uint16_t)(from[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// A parameter of either type, at any element offset; NULL stands for `none`.
__device__ __forceinline__ float param_at(const void* p, int64_t i, int dtype, float none) {
  if (!p) return none;
  return dtype == DP_BF16 ? bf16_to_f32(__ldg(static_cast<const uint16_t*>(p) + i))
                          : __ldg(static_cast<const float*>(p) + i);
}
// Writes v to (or adds it to) element i of a gradient of either type.
__device__ __forceinline__ void grad_put(void* p, int64_t i, int dtype, int accumulate, float v) {
  if (dtype == DP_BF16) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    *q = bf16_rn(accumulate ? __fadd_rn(bf16_to_f32(*q), v) : v);
  } else {
    float* q = static_cast<float*>(p) + i;
    *q = accumulate ? __fadd_rn(*q, v) : v;
  }
}

// Kernels of one call may be launched so that each is set up before the one ahead of it has ended: grid_wait waits for that end
// (and its writes), grid_go lets the next one be set up.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- host side

template <typename K, typename P>
cudaError_t launch_after(K kernel, int64_t ctas, dim3 threads, cudaStream_t stream, const P& params) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)ctas);
  c.blockDim = threads;
  c.stream = stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, params);
}

inline dp_status_t op_fail(dp_status_t s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return report_error(s, msg);
}
inline dp_status_t op_launched(const char* what, int n) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return op_fail(DP_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  add_launches((uint64_t)n);
  return DP_OK;
}
inline int elem_size(int dtype) { return dtype == DP_F32 ? 4 : 2; }
inline bool is_aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline dp_status_t check_dtype(int dtype, const char* name) {
  if (dtype != DP_BF16 && dtype != DP_F32) return op_fail(DP_ERR_INVALID_ARG, "%s: element type %d unknown", name, dtype);
  return DP_OK;
}
// A device pointer to elements of `size` bytes; needed: NULL is refused.
inline dp_status_t check_dev(const void* p, size_t size, bool needed, const char* name) {
  if (!p) return needed ? op_fail(DP_ERR_INVALID_ARG, "%s is NULL", name) : DP_OK;
  if (!is_aligned(p, size)) return op_fail(DP_ERR_ALIGNMENT, "%s is not %d-byte aligned", name, (int)size);
  return DP_OK;
}

}  // namespace dp

#define DP_TRY(expr)                        \
  do {                                      \
    const dp_status_t try_status_ = (expr); \
    if (try_status_ != DP_OK) return try_status_; \
  } while (0)
