// What the paged attention kernels share: the requests' ranges and small conversions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "cache_layout.cuh"
#include "mxattn_internal.h"
#include "sm100_ptx.cuh"

namespace mxattn {

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ldg8(const uint8_t* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t ldg4(const uint8_t* p) {
  uint32_t r;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf162(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t word_of(const uint2& v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ uint32_t word_of(uint32_t v, int) { return v; }

// Where a request's rows and keys are, read once per CTA.
struct RequestRange {
  int start, n;            // first row of q, rows
  int64_t kv, cap;         // kv_len as given (>= 0), and how many keys may be visited at all
};
__device__ __forceinline__ RequestRange request_range(const PagedParams& p, int r) {
  RequestRange q;
  const int T = static_cast<int>(p.T);
  q.start = max(0, min(p.q_start[r], T));
  q.n = max(0, min(p.q_start[r + 1], T) - q.start);
  q.kv = max(p.kv_len[r], 0);
  q.cap = min(min(q.kv, static_cast<int64_t>(0x7FFFFF00)), min(static_cast<int64_t>(p.table_width) << p.page_shift, p.max_kv));
  return q;
}

}  // namespace mxattn
