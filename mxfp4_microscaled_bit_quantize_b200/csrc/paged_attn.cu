// Attention of new tokens over the paged MXFP4 KV cache: the simplest form, one warp per (token,
// query head), one key at a time, all arithmetic in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cmath>
#include <cstdint>

#include "cache_layout.cuh"
#include "mxattn_internal.h"
#include "sm100_ptx.cuh"

namespace mxattn {

// Value of channel c of a row (K: which = 0).
template <int D>
__device__ __forceinline__ float cache_value(const uint8_t* chunk, uint32_t off, uint32_t c, int which, int page_shift) {
  constexpr uint32_t NB = D / 32;
  const uint32_t b = c >> 5, e = c & 31u;
  const uint32_t byte = which == 0 ? (e >> 3) * (4 * NB) + 4 * b + ((e & 7u) >> 1)
                                   : (e >> 2) * (2 * NB) + 2 * b + ((e & 3u) >> 1);
  const uint32_t raw = chunk[off * (D / 2) + byte];
  const uint32_t code = (c & 1u) ? raw >> 4 : raw & 15u;
  const uint32_t i = off & 15u;
  const uint32_t srow = off - i + (which ? v_scale_row(i) : k_scale_row(i));
  const uint32_t s = chunk[((D / 2u) << page_shift) + srow * NB + b];
  uint32_t h[4];
  e2m1x8_to_half2(code, h);
  return __half2float(__low2half(*reinterpret_cast<const __half2*>(&h[0]))) * pow2_from_byte(s);
}

template <int D>
__global__ void __launch_bounds__(128) paged_simple_kernel(const PagedParams p) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t per_request = static_cast<int64_t>(p.max_new) * p.Hq;
  const int r = static_cast<int>(unit / per_request);
  if (r >= p.R) return;
  const int i = static_cast<int>((unit - r * per_request) / p.Hq), h = static_cast<int>(unit % p.Hq);
  const int start = max(0, min(p.q_start[r], static_cast<int>(p.T)));
  const int n = min(min(p.q_start[r + 1], static_cast<int>(p.T)) - start, p.max_new);
  if (i >= n) return;
  const int raw_kv = p.kv_len[r];
  const int64_t cap = min(static_cast<int64_t>(p.table_width) << p.page_shift, p.max_kv);
  int64_t last = p.causal ? static_cast<int64_t>(raw_kv) - n + i : static_cast<int64_t>(raw_kv) - 1;
  last = min(last, cap - 1);
  const int head = h / (p.Hq / p.Hkv);
  const int64_t row = static_cast<int64_t>(start + i);
  float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    q[c] = __bfloat162float(p.q[row * p.q_token_stride + h * p.q_head_stride + lane * C + c]) * p.scale_log2;
    o[c] = 0.f;
  }
  const int64_t chunk = cache_chunk_bytes(D, 1u << p.page_shift);
  for (int64_t j = 0; j <= last; ++j) {
    const int page = p.block_table[static_cast<int64_t>(r) * p.table_width + (j >> p.page_shift)];
    if (page < 0 || page >= p.n_pages) continue;            // a page that is not there: its keys are masked
    const uint8_t* kc = p.cache + (static_cast<int64_t>(page) * p.Hkv + head) * 2 * chunk;
    const uint32_t off = static_cast<uint32_t>(j & ((1ll << p.page_shift) - 1));
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s += q[c] * cache_value<D>(kc, off, lane * C + c, 0, p.page_shift);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    l = l * a + w;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = o[c] * a + w * cache_value<D>(kc + chunk, off, lane * C + c, 1, p.page_shift);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) p.out[(row * p.Hq + h) * D + lane * C + c] = __float2bfloat16_rn(o[c] * inv);
  if (p.lse && lane == 0) p.lse[row * p.Hq + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

cudaError_t launch_paged(const PagedParams& p, int d, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.R) * p.max_new * p.Hq;
  const unsigned grid = static_cast<unsigned>((units + 3) / 4);
  if (d == 128) paged_simple_kernel<128><<<grid, 128, 0, stream>>>(p);
  else paged_simple_kernel<64><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mxattn
