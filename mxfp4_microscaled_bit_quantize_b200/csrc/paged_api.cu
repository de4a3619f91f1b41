// Host side of the paged KV cache's entry points: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mxattn.h"
#include "cache_layout.cuh"
#include "mxattn_internal.h"

using namespace mxattn;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// log2 of a supported page size (a power of two from 16 to 256), -1 for any other.
int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// Checks shared by the calls that touch the cache; *shift receives log2(page_size).
mxattn_status check_cache(const void* cache, int Hkv, int d, int page_size, int64_t n_pages, int* shift) {
  if (Hkv < 1 || d < 1 || page_size < 1 || n_pages < 0) return MXATTN_ERR_INVALID_ARG;
  *shift = page_shift_of(page_size);
  if ((d != 64 && d != 128) || *shift < 0 || n_pages >= (1ll << 31) || Hkv > 65535) return MXATTN_ERR_UNSUPPORTED;
  if (n_pages > 0 && (!cache || !aligned(cache, 16))) return MXATTN_ERR_INVALID_ARG;
  return MXATTN_OK;
}

struct Span { const void* at; uint64_t bytes; };
bool overlap(const Span& a, const Span& b) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < a.bytes : x - y < b.bytes);
}

// The ranges in which rows and units of work are counted.
bool countable(int R, int Hq, int Hkv, int max_new) {
  return static_cast<int64_t>(max_new) * (Hq / Hkv) < (1ll << 30) && static_cast<int64_t>(max_new) * Hq < (1ll << 31) / (R > 0 ? R : 1);
}

// Status area, then the partial rows of split requests.
size_t paged_workspace(const SplitPlan& s, int d) {
  return 256 + static_cast<size_t>(s.part_rows) * (d + 1) * sizeof(float);
}

}  // namespace

extern "C" {

size_t mxattn_cache_page_bytes(int Hkv, int page_size, int d) {
  if (Hkv < 1 || (d != 64 && d != 128) || page_shift_of(page_size) < 0) return 0;
  return static_cast<size_t>(Hkv) * 2 * cache_chunk_bytes(static_cast<uint32_t>(d), static_cast<uint32_t>(page_size));
}

mxattn_status mxattn_cache_plan(const int32_t* ctx_len, const int32_t* new_len, int R, int32_t* block_table,
                                int table_width, const int32_t* free_pages, int n_free, int page_size,
                                int32_t* q_start, int32_t* kv_len, int64_t* slots, int64_t max_tokens, int32_t* info,
                                void* stream) {
  if (R < 0 || table_width < 0 || n_free < 0 || max_tokens < 0 || page_size < 1) return MXATTN_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || max_tokens >= (1ll << 31)) return MXATTN_ERR_UNSUPPORTED;
  if (!q_start || !info || (R > 0 && (!ctx_len || !new_len || !kv_len))) return MXATTN_ERR_INVALID_ARG;
  if ((R > 0 && table_width > 0 && !block_table) || (n_free > 0 && !free_pages) || (max_tokens > 0 && !slots))
    return MXATTN_ERR_INVALID_ARG;
  if (!aligned(ctx_len, 4) || !aligned(new_len, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(slots, 8) || !aligned(info, 4))
    return MXATTN_ERR_INVALID_ARG;
  // Every CTA reads the inputs while others write, so nothing may be both, but for kv_len over ctx_len.
  const uint64_t lens = 4ull * R;
  const Span ins[] = {{ctx_len, lens}, {new_len, lens}, {free_pages, 4ull * n_free}};
  const Span outs[] = {{kv_len, lens}, {q_start, lens + 4}, {slots, 8ull * max_tokens}, {info, 16},
                       {block_table, static_cast<uint64_t>(R) * table_width >= 1ull << 61 ? ~0ull : lens * table_width}};
  const bool in_place = R > 0 && kv_len == ctx_len;
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 3; ++i)
      if (!(in_place && o == 0 && i == 0) && overlap(outs[o], ins[i])) return MXATTN_ERR_INVALID_ARG;
    for (int x = 0; x < o; ++x)
      if (overlap(outs[o], outs[x])) return MXATTN_ERR_INVALID_ARG;
  }
  PlanParams p{};
  p.in_place = in_place ? 1 : 0;
  p.ctx_len = ctx_len;
  p.new_len = new_len;
  p.R = R;
  p.block_table = block_table;
  p.table_width = table_width;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.page_shift = shift;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.slots = slots;
  p.max_tokens = max_tokens;
  p.info = info;
  return launch_plan(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXATTN_OK : MXATTN_ERR_CUDA;
}

mxattn_status mxattn_cache_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                  int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots, int64_t T,
                                  int Hkv, int d, int page_size, int64_t n_pages, int scale_mode, uint8_t* cache,
                                  void* stream) {
  if (scale_mode != MXATTN_SCALE_OCP && scale_mode != MXATTN_SCALE_UOS) return MXATTN_ERR_INVALID_ARG;
  int shift;
  const mxattn_status st = check_cache(cache, Hkv, d, page_size, n_pages, &shift);
  if (st != MXATTN_OK) return st;
  if (T < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
    return MXATTN_ERR_INVALID_ARG;
  if (T >= (1ll << 31)) return MXATTN_ERR_UNSUPPORTED;
  if (T == 0) return MXATTN_OK;
  if (!k || !v || !slots || !aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8)) return MXATTN_ERR_INVALID_ARG;
  AppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_token_stride = k_token_stride;
  p.k_head_stride = k_head_stride;
  p.v_token_stride = v_token_stride;
  p.v_head_stride = v_head_stride;
  p.slots = slots;
  p.T = T;
  p.n_slots = n_pages << shift;
  p.Hkv = Hkv;
  p.page_shift = shift;
  p.mode = scale_mode;
  p.k_vec = aligned(k, 16) && k_token_stride % 8 == 0 && k_head_stride % 8 == 0;
  p.v_vec = aligned(v, 16) && v_token_stride % 8 == 0 && v_head_stride % 8 == 0;
  p.cache = cache;
  return launch_append(p, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXATTN_OK : MXATTN_ERR_CUDA;
}

mxattn_status mxattn_cache_read(const uint8_t* cache, const int64_t* slots, int64_t T, int Hkv, int d, int page_size,
                                int64_t n_pages, void* k, void* v, void* stream) {
  int shift;
  const mxattn_status st = check_cache(cache, Hkv, d, page_size, n_pages, &shift);
  if (st != MXATTN_OK) return st;
  if (T < 0) return MXATTN_ERR_INVALID_ARG;
  if (T >= (1ll << 31)) return MXATTN_ERR_UNSUPPORTED;
  if (T == 0) return MXATTN_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return MXATTN_ERR_INVALID_ARG;
  ReadParams p{};
  p.cache = cache;
  p.slots = slots;
  p.T = T;
  p.n_slots = n_pages << shift;
  p.Hkv = Hkv;
  p.page_shift = shift;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  return launch_read(p, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXATTN_OK : MXATTN_ERR_CUDA;
}

size_t mxattn_paged_workspace_size(int64_t T, int R, int Hq, int Hkv, int d, int max_new, int64_t max_kv) {
  if (T < 0 || R < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (d != 64 && d != 128) || max_new < 0 || max_kv < 0 ||
      !countable(R, Hq, Hkv, max_new))
    return 0;
  return paged_workspace(plan_splits(R, Hq, Hkv, d, max_new, max_kv), d);
}

mxattn_status mxattn_paged_forward(const void* q, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* cache,
                                   const int32_t* block_table, int table_width, const int32_t* q_start,
                                   const int32_t* kv_len, void* out, float* lse, int64_t T, int R, int Hq, int Hkv,
                                   int d, int page_size, int64_t n_pages, int max_new, int64_t max_kv, int causal,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || T < 0 || R < 0 || table_width < 0 || max_new < 0 || max_kv < 0)
    return MXATTN_ERR_INVALID_ARG;
  if (q_token_stride < 0 || q_head_stride < 0) return MXATTN_ERR_INVALID_ARG;
  int shift;
  const mxattn_status st = check_cache(cache, Hkv, d, page_size, n_pages, &shift);
  if (st != MXATTN_OK) return st;
  if (T >= (1ll << 31)) return MXATTN_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256)) return MXATTN_ERR_INVALID_ARG;
  if (!countable(R, Hq, Hkv, max_new)) return MXATTN_ERR_UNSUPPORTED;
  const SplitPlan plan = plan_splits(R, Hq, Hkv, d, max_new, max_kv);
  if (plan.units >= (1ll << 31)) return MXATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < paged_workspace(plan, d)) return MXATTN_ERR_WORKSPACE;
  if (T == 0 || R == 0 || max_new == 0) return MXATTN_OK;
  if (!q || !out || !q_start || !kv_len || (table_width > 0 && !block_table)) return MXATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4))
    return MXATTN_ERR_INVALID_ARG;
  PagedParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.cache = cache;
  p.block_table = block_table;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.T = T;
  p.n_pages = n_pages;
  p.max_kv = max_kv;
  p.R = R;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.table_width = table_width;
  p.page_shift = shift;
  p.max_new = max_new;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  p.status = static_cast<unsigned int*>(workspace);
  return launch_paged(p, plan, static_cast<uint8_t*>(workspace) + 256, d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MXATTN_OK : MXATTN_ERR_CUDA;
}

}  // extern "C"
