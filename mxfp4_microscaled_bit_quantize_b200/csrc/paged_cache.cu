// Kernels around the paged MXFP4 KV cache (layout: cache_layout.cuh):
//  * plan_kernel: block tables and slot maps of a batch from its requests' lengths,
//  * append_kernel: bf16 K and V rows of new tokens -> MXFP4 in their slots,
//  * read_kernel: the values that slots hold, as bf16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "cache_layout.cuh"
#include "mxattn_internal.h"
#include "sm100_ptx.cuh"

namespace mxattn {

// ------------------------------------------------------------------ plan
//
// Request r holds ctx tokens in held = ceil(ctx / P) pages and gets n more, so it needs
// ceil((ctx + n) / P) - held pages, handed out from the free list in the order of the requests: two
// prefix sums, over the tokens and over the pages. Every CTA computes both sums over all requests
// (kPlanThreads at a time, carrying the totals), since a sum over some thousand L2-resident integers
// costs less than a second launch or a wait between CTAs; the CTAs then share the writing of the
// slots and of the new table entries, each found by a binary search in the sums. Slots are computed
// from the free list, never from table entries that this launch writes. Where kv_len is written over ctx_len the
// CTAs are one cluster, which waits between reading a chunk's lengths and writing them. Bound: launch and memory latency (a
// decoding step of 256 requests reads and writes 7 KB, a prefill of 64 ragged prompts 0.55 MB): 5.1 and 6.6 us on
// the device, 15 us as a Python call, which is its host side.
constexpr int kPlanThreads = 512;
constexpr unsigned kPlanCluster = 8;    // CTAs of a call in place (65536 tokens: 17 us, 7 with buffers of their own)

struct PlanPair { int64_t tok; int64_t pages; };

__device__ __forceinline__ int64_t warp_scan_incl(int64_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Inclusive sum over the CTA; *total receives the sum of all. `part` has one entry per warp.
__device__ __forceinline__ int64_t cta_scan_incl(int64_t v, int64_t* part, int64_t* total) {
  const int warp = threadIdx.x >> 5;
  v = warp_scan_incl(v);
  if ((threadIdx.x & 31) == 31) part[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return v + before;
}

// Last index i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int64_t* a, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ int64_t part[kPlanThreads / 32];
  __shared__ int64_t tok0[kPlanThreads], page0[kPlanThreads];   // exclusive sums of this chunk
  __shared__ int ctx_s[kPlanThreads], held_s[kPlanThreads];     // ctx < 0: the request is refused
  __shared__ int64_t taken_s;
  const int tid = threadIdx.x;
  const int shift = p.page_shift;
  const int64_t P = 1ll << shift;
  int64_t tok_carry = 0, page_carry = 0, taken = 0;
  int refused = 0;
  if (tid == 0) taken_s = 0;
  for (int r0 = 0; r0 < p.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    const bool in = r < p.R;
    const int64_t ctx = in ? p.ctx_len[r] : 0;
    const int64_t n = in ? max(p.new_len[r], 0) : 0;
    int64_t tok_all, page_all;
    const int64_t tok = tok_carry + cta_scan_incl(n, part, &tok_all) - n;
    const int64_t held = (ctx + P - 1) >> shift, full = (ctx + n + P - 1) >> shift;
    // refused: bad lengths, tokens past the slot map, more pages than the table's row holds
    bool ok = in && ctx >= 0 && p.new_len[r] >= 0 && tok + n <= p.max_tokens && full <= p.table_width && ctx + n <= 0x7FFFFFFF;
    const int64_t need = ok ? full - held : 0;
    const int64_t first = page_carry + cta_scan_incl(need, part, &page_all) - need;
    if (need > 0 && first + need > p.n_free) ok = false;    // ... or too few free pages
    tok0[tid] = tok;
    page0[tid] = first;
    ctx_s[tid] = ok ? static_cast<int>(ctx) : -1;
    held_s[tid] = static_cast<int>(held);
    if (p.in_place) {                                       // every CTA of the cluster has read this chunk's lengths
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (in && blockIdx.x == 0) {
      p.q_start[r] = static_cast<int>(min(tok, p.max_tokens));
      p.kv_len[r] = static_cast<int>(ok ? ctx + n : max(ctx, static_cast<int64_t>(0)));
    }
    if (ok && need > 0) atomicMax(reinterpret_cast<unsigned long long*>(&taken_s), static_cast<unsigned long long>(first + need));
    refused += __syncthreads_count(in && !ok);              // also: the chunk's sums are in shared memory
    taken = taken_s;
    const int cnt = min(p.R - r0, kPlanThreads);
    const int64_t tok_end = min(tok_carry + tok_all, p.max_tokens);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    for (int64_t t = tok_carry + mine; t < tok_end; t += step) {
      const int i = last_not_above(tok0, cnt, t);
      int64_t slot = -1;
      if (ctx_s[i] >= 0) {
        const int64_t pos = ctx_s[i] + (t - tok0[i]);
        const int64_t pg = pos >> shift;
        const int page = pg >= held_s[i] ? p.free_pages[page0[i] + pg - held_s[i]]
                                         : p.block_table[static_cast<int64_t>(r0 + i) * p.table_width + pg];
        if (page >= 0) slot = static_cast<int64_t>(page) * P + (pos & (P - 1));
      }
      p.slots[t] = slot;
    }
    const int64_t page_end = min(page_carry + page_all, static_cast<int64_t>(p.n_free));
    for (int64_t f = page_carry + mine; f < page_end; f += step) {
      const int i = last_not_above(page0, cnt, f);
      if (ctx_s[i] >= 0) p.block_table[static_cast<int64_t>(r0 + i) * p.table_width + held_s[i] + (f - page0[i])] = p.free_pages[f];
    }
    tok_carry += tok_all;
    page_carry += page_all;
    __syncthreads();                                        // before the next chunk overwrites the sums
  }
  const int64_t total = min(tok_carry, p.max_tokens);
  for (int64_t t = total + static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; t < p.max_tokens;
       t += static_cast<int64_t>(gridDim.x) * kPlanThreads)
    p.slots[t] = -1;                                        // rows behind the last request
  if (blockIdx.x == 0 && tid == 0) {
    p.q_start[p.R] = static_cast<int>(total);
    p.info[0] = static_cast<int>(total);
    p.info[1] = static_cast<int>(taken);
    p.info[2] = refused;
    p.info[3] = 0;
  }
}

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
  const int64_t want = (p.max_tokens + kPlanThreads - 1) / kPlanThreads;
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want > 148 ? 148 : want);
  if (!p.in_place || grid == 1) {
    PlanParams apart = p;
    apart.in_place = 0;                                      // one CTA: each length is read and written by the same thread
    plan_kernel<<<grid, kPlanThreads, 0, stream>>>(apart);
    return cudaGetLastError();
  }
  cudaLaunchAttribute one{};
  one.id = cudaLaunchAttributeClusterDimension;
  one.val.clusterDim.x = kPlanCluster;
  one.val.clusterDim.y = one.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPlanCluster);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cfg.attrs = &one;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, p);
}

// ------------------------------------------------------------------ append

__device__ __forceinline__ void bf16x8_to_float(const uint4& raw, float* v) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// One thread quantizes one 32-element block; the nb threads of a row exchange words so that each
// stores 16 contiguous bytes of the interleaved row. Bound: HBM, 2 + 17/32 bytes a value. 32768 tokens of 8 heads
// of 128 channels, appended (170 MB): 34 us, 5.0 TB/s, 76 % of the copy bandwidth; read back: 32 us.
template <int NB>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  const int64_t per_token = static_cast<int64_t>(p.Hkv) * NB;
  const int64_t total = 2 * p.T * per_token;                 // K blocks, then V blocks
  const int64_t rounded = (total + 31) / 32 * 32;            // whole warps: the exchange needs all lanes
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; g < rounded;
       g += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const bool in = g < total;
    const int64_t half = p.T * per_token;
    const int which = in && g >= half ? 1 : 0;
    const int64_t gg = in ? g - which * half : 0;
    const int64_t tok = gg / per_token;
    const int rest = static_cast<int>(gg - tok * per_token);
    const int head = rest / NB, b = rest % NB;
    const int64_t slot = in ? p.slots[tok] : -1;
    const bool live = slot >= 0 && slot < p.n_slots;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
    if (live) {
      const __nv_bfloat16* src = (which ? p.v + tok * p.v_token_stride + head * p.v_head_stride
                                        : p.k + tok * p.k_token_stride + head * p.k_head_stride) + b * 32;
      if (which ? p.v_vec : p.k_vec) {
#pragma unroll
        for (int c = 0; c < 4; ++c) bf16x8_to_float(*reinterpret_cast<const uint4*>(src + 8 * c), v + 8 * c);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __bfloat162float(src[i]);
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
    const uint32_t byte = e8m0_scale_byte(amax, p.mode);
    const float inv = inv_pow2_from_byte(byte);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= inv;                // exact: power of two
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt_e2m1x8(v + 8 * i);
    // q: the 16-byte piece b of the row in K's order (words p of blocks 0 .. nb - 1)
    uint32_t q[4];
    if (NB == 4) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int mine = b ^ s;
        const uint32_t send = mine & 2 ? (mine & 1 ? w[3] : w[2]) : (mine & 1 ? w[1] : w[0]);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, send, s);   // block b ^ s, word b
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j == mine) q[j] = got;
      }
    } else {
      const uint32_t s0 = b ? w[0] : w[2], s1 = b ? w[1] : w[3];
      const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 1), r1 = __shfl_xor_sync(0xffffffffu, s1, 1);
      q[0] = b ? r0 : w[0];
      q[1] = b ? w[2] : r0;
      q[2] = b ? r1 : w[1];
      q[3] = b ? w[3] : r1;
    }
    if (!live) continue;
    const int64_t page = slot >> p.page_shift;
    const uint32_t off = static_cast<uint32_t>(slot & ((1ll << p.page_shift) - 1));
    const uint32_t chunk = (static_cast<uint32_t>(NB) * 17u) << p.page_shift;
    uint8_t* base = p.cache + ((page * p.Hkv + head) * 2 + which) * static_cast<int64_t>(chunk);
    uint4 o;
    if (which == 0) o = make_uint4(q[0], q[1], q[2], q[3]);
    else if (NB == 4) o = make_uint4(lo16x2(q[0], q[1]), lo16x2(q[2], q[3]), hi16x2(q[0], q[1]), hi16x2(q[2], q[3]));
    else o = make_uint4(lo16x2(q[0], q[1]), hi16x2(q[0], q[1]), lo16x2(q[2], q[3]), hi16x2(q[2], q[3]));
    *reinterpret_cast<uint4*>(base + off * (NB * 16) + b * 16) = o;
    const uint32_t i = off & 15u;
    const uint32_t srow = off - i + (which ? v_scale_row(i) : k_scale_row(i));
    base[((static_cast<uint32_t>(NB) * 16u) << p.page_shift) + srow * NB + b] = static_cast<uint8_t>(byte);
  }
}

cudaError_t launch_append(const AppendParams& p, int d, cudaStream_t stream) {
  const int64_t total = 2 * p.T * p.Hkv * (d / 32);
  const int64_t want = (total + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want > 148 * 8 ? 148 * 8 : want);
  if (d == 128) append_kernel<4><<<grid, 256, 0, stream>>>(p);
  else append_kernel<2><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ read

// One thread decodes one 16-byte piece of a row: NB / 4 * 4 words of 8 codes.
template <int NB>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams p) {
  const int64_t per_token = static_cast<int64_t>(p.Hkv) * NB;
  const int64_t half = p.T * per_token, total = 2 * half;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int which = g >= half ? 1 : 0;
    const int64_t gg = g - which * half;
    const int64_t tok = gg / per_token;
    const int rest = static_cast<int>(gg - tok * per_token);
    const int head = rest / NB, pc = rest % NB;
    const int64_t slot = p.slots[tok];
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    uint32_t scales = 0;
    if (slot >= 0 && slot < p.n_slots) {
      const int64_t page = slot >> p.page_shift;
      const uint32_t off = static_cast<uint32_t>(slot & ((1ll << p.page_shift) - 1));
      const uint32_t chunk = (static_cast<uint32_t>(NB) * 17u) << p.page_shift;
      const uint8_t* base = p.cache + ((page * p.Hkv + head) * 2 + which) * static_cast<int64_t>(chunk);
      o = *reinterpret_cast<const uint4*>(base + off * (NB * 16) + pc * 16);
      const uint32_t i = off & 15u;
      const uint32_t srow = off - i + (which ? v_scale_row(i) : k_scale_row(i));
      const uint8_t* sp = base + ((static_cast<uint32_t>(NB) * 16u) << p.page_shift) + srow * NB;
      scales = NB == 4 ? *reinterpret_cast<const uint32_t*>(sp) : *reinterpret_cast<const uint16_t*>(sp);
    }
    uint32_t q[4];
    if (which == 0) { q[0] = o.x; q[1] = o.y; q[2] = o.z; q[3] = o.w; }
    else if (NB == 4) { q[0] = lo16x2(o.x, o.z); q[1] = hi16x2(o.x, o.z); q[2] = lo16x2(o.y, o.w); q[3] = hi16x2(o.y, o.w); }
    else { q[0] = lo16x2(o.x, o.y); q[1] = hi16x2(o.x, o.y); q[2] = lo16x2(o.z, o.w); q[3] = hi16x2(o.z, o.w); }
    __nv_bfloat16* dst = (which ? p.v : p.k) + (tok * p.Hkv + head) * (NB * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // NB = 4: word pc of block j; NB = 2: word 2 pc + j / 2 of block j % 2
      const int b = NB == 4 ? j : (j & 1), word = NB == 4 ? pc : 2 * pc + (j >> 1);
      const float s = pow2_from_byte((scales >> (8 * b)) & 0xFFu);
      uint32_t h[4], r[4];
      e2m1x8_to_half2(q[j], h);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[x]));
        const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * s, f.y * s);   // exact in the normal range
        r[x] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(dst + b * 32 + word * 8) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

cudaError_t launch_read(const ReadParams& p, int d, cudaStream_t stream) {
  const int64_t total = 2 * p.T * p.Hkv * (d / 32);
  const int64_t want = (total + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want > 148 * 8 ? 148 * 8 : want);
  if (d == 128) read_kernel<4><<<grid, 256, 0, stream>>>(p);
  else read_kernel<2><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mxattn
