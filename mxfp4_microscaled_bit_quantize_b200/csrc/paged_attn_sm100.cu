// Attention of many new tokens over the paged MXFP4 KV cache (chunks of prompts, cross attention): tcgen05
// products in bf16 with K and V tiles made from the pages on the way to shared memory.
//
//   S = Q K^T;  m' = max(m, rowmax S c),  c = log2(e) / sqrt(d);  P = 2^(S c - m');
//   O = 2^(m - m') O + P V;  l = 2^(m - m') l + rowsum P;  out = O / l
//
// Bound: 4 d FLOP per (query head, key) on the tensor cores, next to one exponential (MUFU: 16 per clock and SM)
// per (query head, key): for d = 128 and 256 query rows both need about 2100 clocks per 128 keys. The conversion
// of the 128 keys (E2M1 times a power of two is exact in bf16) costs about 1000 issue slots per SM sub-partition,
// half of them on the half-rate ALU pipe, so a CTA owns 256 query rows to share it.
//
// Work unit: one CTA (one per SM: it takes all 512 TMEM columns) owns 256 consecutive rows (token, query head of
// the group) of one request and KV head, as two tiles A and B of 128, and visits the keys of one split in tiles
// of 128. 896 threads:
//   warps 0, 1    issue the products of tile A, B (one thread each): S(t) into TMEM, then P V(t) with P as the
//                 TMEM operand, then S(t + 1) over the same columns, each after the commit of the one before
//   warps 4-11    convert: page lookups and code loads one tile ahead in registers, then K(t) and V(t) as bf16
//                 into a two-stage ring (128-byte swizzle: K is K-major, V MN-major)
//   warps 12-27   softmax of tiles A and B, two threads per row; the tiles' exponentials take turns, so that one
//                 tile's products run under the other's; O is rescaled in TMEM where a row's maximum has grown
// P is rounded to bf16 (8 bits) for the product: the TMEM operand has V's type, and V needs bf16's range (fp16 tiles with
// references of their own took 1.40 instead of 1.25 ms); the row sum is taken before the rounding, in fp32. The key that
// dominates a row enters without a rounding, as P = 1, if the reference follows every larger score. With references that
// move only past 2^8 it is rounded too, and the error against 64 bits was 1.35e-3 instead of 1.13e-3 (fp32 arithmetic
// rounded once: 1.12e-3) for 2048 tokens over 30720, 1.05e-3 instead of 0.91e-3 (0.90e-3) for ragged chunks over 3001;
// following costs 1 to 5 % of the time (1208 -> 1218 us, 123 -> 127 us, 32760 rows over 512 keys 634 -> 670 us).
//
// Measured (d = 128): 2048 tokens over 30720 keys, 32 query and 8 KV heads: 1.22 ms, 874 TFLOP/s, 63 % of the
// bf16 rate sustained under the power limit; 32760 rows x 40 heads over 512 keys: 0.67 ms, 513 TFLOP/s (four key
// tiles per CTA: set-up, first loads and output are half of its 19 us). A pair of tiles takes about 4300 clocks
// per 128 keys: a row tile's own chain (load S and maxima 900, exponentials 1500, hand-over 350, P V 650, S 1050)
// is what bounds it. Tried and slower: one S buffer for both tiles with P in columns of its own, 64-key steps
// with two S buffers a tile (M = 128, N = 64 products take as long as N = 128), fp16 tiles with the codes
// converted by cvt (half the conversion, but a softmax that spills), several pairs of row tiles per CTA.
#include <cuda_bf16.h>
#include <cstdint>

#include "paged_common.cuh"

namespace mxattn {

namespace {

constexpr int kTcThreads = 896, kTcLaunchRegs = 72;
constexpr int kIssueRegs = 40, kConvRegs = 56, kRowRegs = 88;
static_assert(kIssueRegs + 2 * kConvRegs + 4 * kRowRegs <= 7 * kTcLaunchRegs, "register split");
constexpr int kConvWarp0 = 4, kRowWarp0 = 12;    // warps 0-3 issue, 4-11 convert, 12-27 softmax
constexpr uint32_t kTcCols = 512, kColSx = 0, kColOx = 256;   // S / P of tile X at 128 X, O at 256 + 128 X
constexpr uint32_t kSw128 = 2;                                // descriptor code of the 128-byte swizzle
constexpr int kTcStages = 2;
constexpr uint32_t kPlaces = 148;                             // CTAs that run at the same time, one per SM
template <int D>
struct __align__(1024) TcSmem {
  static_assert(D == 64 || D == 128, "Q and the output stage are laid out for these");
  static constexpr int kTile = 128 * D * 2;      // 128 rows of D bf16, as D / 64 slabs of 128 x 128 bytes
  uint8_t q[2][32768];                           // the tile's Q, and 128 rows x 256 bytes of output at the end
  uint8_t k[kTcStages][kTile];
  uint8_t v[kTcStages][kTile];
  uint64_t bar_q;
  uint64_t bar_k_full[kTcStages], bar_v_full[kTcStages], bar_k_empty[kTcStages], bar_v_empty[kTcStages];
  uint64_t bar_s_full[2], bar_p_full[2], bar_pv[2], bar_drain[2], bar_turn[2];
  uint32_t tmem_base;
  int abort_flag;
};

// Instruction descriptor, kind::f16: bf16 operands, fp32 accumulator, M = 128; B MN-major or K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t n, uint32_t b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// mbar_wait whose loop is a bare try_wait: the abort flag and the clock are looked at every 64th time,
// since the instructions of the waiting warps are taken from the working ones.
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* status, unsigned int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      *abort_flag = 1;
      atomicCAS(status, 0u, code);
      return false;
    }
  }
}
__device__ __forceinline__ bool warp_wait_tc(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* status, unsigned int code) {
  return __all_sync(0xffffffffu, mbar_poll(bar, parity, abort_flag, status, code));
}
// The same for the issuing warps, whose waits lie on the critical path: test_wait returns at once, where
// try_wait sleeps and wakes late.
__device__ __forceinline__ bool warp_spin_tc(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* status, unsigned int code) {
  bool ok = mbar_test_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
      for (int i = 0; i < 64 && !ok; ++i) ok = mbar_test_wait(bar, parity);
      if (ok || *abort_flag) break;
      if (global_timer_ns() - t0 > kWaitTimeoutNs) {
        *abort_flag = 1;
        atomicCAS(status, 0u, code);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void drain_wait_tc(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 200ull * 1000ull * 1000ull) break;
}

// 16 TMEM lanes, two halves of the warp, the upper one kOff columns on: 16 columns each.
template <int kOff>
__device__ __forceinline__ void tmem_ld16x2_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr), "n"(kOff));
}
template <int kOff>
__device__ __forceinline__ void tmem_st16x2_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, {%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17};" ::"r"(taddr), "n"(kOff), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}

// Eight codes times 2^(s - 127) as bf16, in the order e0 e4 e1 e5 e2 e6 e3 e7. A nibble (s eem) shifted
// to the sign and to the three bits at the border of bf16's exponent and mantissa is the code's value
// times 2^-126, exactly (code 1, E2M1's subnormal, becomes a bf16 subnormal), so one product by
// 2^(s - 1) finishes it; scales above 2 need a second one, since 2^(s - 1) leaves bf16's range there.
template <bool LARGE>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t s, uint32_t (&r)[4]) {
  const uint32_t mul = ((LARGE ? min(s, 128u) : s) + 126u) * 0x00800080u;
  const uint32_t t[4] = {w << 12, w << 8, w << 4, w};
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = mul_bf162(((t[j] >> 6) & 0x01C001C0u) | (t[j] & 0x80008000u), mul);
  if (LARGE) {
    const uint32_t more = (max(s, 128u) - 1u) * 0x00800080u;             // 2^(s - 128), or 1
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = mul_bf162(r[j], more);
  }
}

// What a converting lane holds of a tile's K or V: piece (lane & 3) of rows (lane >> 2) and
// (lane >> 2) + 8 of its warp's 16, and those rows' scale bytes.
template <int D> struct Raw;
template <> struct Raw<128> { uint4 w[2]; uint32_t s[2]; };
template <> struct Raw<64> { uint2 w[2]; uint32_t s[2]; };

__device__ __forceinline__ void clear(uint4& v) { v = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void clear(uint2& v) { v = make_uint2(0u, 0u); }
__device__ __forceinline__ void load_piece(uint4& v, const uint8_t* p) { v = ldg16(p); }
__device__ __forceinline__ void load_piece(uint2& v, const uint8_t* p) { v = ldg8(p); }
template <int D>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p) {
  if constexpr (D == 128) return ldg4(p);
  uint16_t r;
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
  return r;
}

// Word c of each block of a row, from the row's piece c.
template <int W>
__device__ __forceinline__ void block_words(const uint4& o, uint32_t (&q)[4]) {
  if (W == 0) { q[0] = o.x; q[1] = o.y; q[2] = o.z; q[3] = o.w; }
  else { q[0] = lo16x2(o.x, o.z); q[1] = hi16x2(o.x, o.z); q[2] = lo16x2(o.y, o.w); q[3] = hi16x2(o.y, o.w); }
}
template <int W>
__device__ __forceinline__ void block_words(const uint2& o, uint32_t (&q)[2]) {
  if (W == 0) { q[0] = o.x; q[1] = o.y; }
  else { q[0] = lo16x2(o.x, o.y); q[1] = hi16x2(o.x, o.y); }
}

// Rows of a tile into shared memory: 16-byte column j of row r in slab j / 8 at (j % 8) ^ (r % 8).
// Lanes of odd rows take the blocks of a pair in the other order, so that the eight lanes of a store
// phase (two rows, four pieces) cover all banks.
template <int D, int W, bool LARGE>
__device__ __forceinline__ void store_rows_as(const Raw<D>& raw, uint32_t tile, uint32_t row0, uint32_t lane) {
  constexpr int NB = D / 32;
  const uint32_t c = lane & 3u, odd = (lane >> 2) & 1u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t row = row0 + 8u * i + (lane >> 2);
    uint32_t q[NB];
    block_words<W>(raw.w[i], q);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t bx = static_cast<uint32_t>(b) ^ odd;
      const uint32_t w = odd ? q[b ^ 1] : q[b];
      uint32_t r[4];
      codes_to_bf16<LARGE>(w, (raw.s[i] >> (8u * bx)) & 0xFFu, r);
      const uint32_t col = 4u * bx + c;
      st_shared_v4(tile + (col >> 3) * (128u * 128u) + row * 128u + (((col ^ row) & 7u) << 4), r[0], r[1], r[2], r[3]);
    }
  }
}

// One choice for the warp's rows: any scale byte of 128 or more takes the form with two products.
template <int D, int W>
__device__ __forceinline__ void store_rows(const Raw<D>& raw, uint32_t tile, uint32_t row0, uint32_t lane) {
  if (__any_sync(0xffffffffu, ((raw.s[0] | raw.s[1]) & 0x80808080u) != 0u))
    store_rows_as<D, W, true>(raw, tile, row0, lane);
  else
    store_rows_as<D, W, false>(raw, tile, row0, lane);
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) paged_tc_kernel(const PagedParams p, const SplitParams sp) {
  constexpr int NB = D / 32;
  using Sm = TcSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // uniform: descriptors in uniform registers

  // ---- set-up by a warp that has nothing else to do
  if (warp == 3 && lane == 0) {
    mbar_init(&s.bar_q, 16);
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(&s.bar_k_full[i], 8);
      mbar_init(&s.bar_v_full[i], 8);
      mbar_init(&s.bar_k_empty[i], 2);
      mbar_init(&s.bar_v_empty[i], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s.bar_s_full[x], 1);
      mbar_init(&s.bar_p_full[x], 8);
      mbar_init(&s.bar_pv[x], 1);
      mbar_init(&s.bar_turn[x], 8);
      mbar_init(&s.bar_drain[x], 1);
    }
    s.abort_flag = 0;
    fence_mbar_init();
  }

  // ---- work unit
  const int G = p.Hq / p.Hkv;
  uint32_t u = blockIdx.x;
  const int split = static_cast<int>(u % sp.splits);
  u /= sp.splits;
  const int pair = static_cast<int>(sp.row_tiles - 1 - u % sp.row_tiles);   // causal: longest first
  u /= sp.row_tiles;
  const int head = static_cast<int>(u % p.Hkv), r = static_cast<int>(u / p.Hkv);
  const RequestRange rq = request_range(p, r);
  const int n_used = min(rq.n, p.max_new);
  const int rows_all = n_used * G;
  const int used_splits = max(1, static_cast<int>((rq.cap + sp.chunk - 1) / sp.chunk));
  if (pair * 256 >= rows_all || split >= used_splits) return;
  auto limit_of = [&](int row) -> int64_t {                   // keys j < limit are visible to the row
    const int64_t l = p.causal ? rq.kv - rq.n + row / G + 1 : rq.kv;
    return max(min(l, rq.cap), static_cast<int64_t>(0));
  };
  const int64_t key_begin = split * sp.chunk;
  int n_x[2];
  int64_t lim_all = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int first = pair * 256 + x * 128, last = min(rows_all, first + 128) - 1;
    const int64_t lim = first < rows_all ? min(limit_of(last), key_begin + sp.chunk) : 0;
    n_x[x] = lim > key_begin ? static_cast<int>((lim - key_begin + 127) >> 7) : 0;
    lim_all = max(lim_all, lim);
  }
  const int n_max = max(n_x[0], n_x[1]);

  if (warp == 0) {
    tmem_alloc(&s.tmem_base, kTcCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;

  if (warp < 4) {
    regs_dec<kIssueRegs>();
    if (warp < 2) {
      // ======================= products of tile x =======================
      const int x = warp;
      const int n_own = x == 0 ? n_x[0] : n_x[1], n_other = x == 0 ? n_x[1] : n_x[0];
      const bool leader = elect_one_sync();
      const uint64_t d_k = smem_desc(0, 0, 1024, kSw128);                 // K-major: 8 rows are 1 KB
      const uint64_t d_v = smem_desc(0, 128 * 128, 1024, kSw128);         // MN-major: slabs 16 KB apart, 8 keys 1 KB
      const uint32_t a_q = smem_u32(s.q[x]) >> 4, a_k = smem_u32(s.k[0]) >> 4, a_v = smem_u32(s.v[0]) >> 4;
      const uint32_t t_s = tmem + kColSx + 128 * x, t_o = tmem + kColOx + 128 * x;
      bool ok = n_own == 0 || warp_spin_tc(&s.bar_q, 0, abort_flag, p.status, kStatusTimeoutQ);
      auto wait_k = [&](int t) -> bool {
        return warp_spin_tc(&s.bar_k_full[t % kTcStages], (t / kTcStages) & 1, abort_flag, p.status, kStatusTimeoutKV | (t % kTcStages));
      };
      auto issue_s = [&](int t) {
        const int st = t % kTcStages;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (kk >> 2) * 1024u + (kk & 3) * 2u;         // slab, 32 bytes per 16 channels
            tc_mma_ss(t_s, d_k | (a_q + at), d_k | (a_k + st * (Sm::kTile >> 4) + at), idesc_bf16(128, 0), kk > 0);
          }
          tc_commit(&s.bar_s_full[x]);
          tc_commit(&s.bar_k_empty[st]);
          if (t >= n_other) mbar_arrive(&s.bar_k_empty[st]);               // the other tile has no product here
        }
        __syncwarp();
      };
      if (ok && n_own > 0) {
        ok = wait_k(0);
        if (ok) issue_s(0);
      }
      for (int t = 0; ok && t < n_own; ++t) {
        const int st = t % kTcStages;
        ok = warp_spin_tc(&s.bar_v_full[st], (t / kTcStages) & 1, abort_flag, p.status, kStatusTimeoutKV | 8 | st) &&
             warp_spin_tc(&s.bar_p_full[x], t & 1, abort_flag, p.status, kStatusTimeoutP | x);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(t_o, t_s + 8 * kk, d_v | (a_v + st * (Sm::kTile >> 4) + kk * 128u), idesc_bf16(D, 1), t > 0 || kk > 0);
          tc_commit(&s.bar_pv[x]);
          tc_commit(&s.bar_v_empty[st]);
          if (t >= n_other) mbar_arrive(&s.bar_v_empty[st]);
        }
        __syncwarp();
        if (t + 1 < n_own) {
          // S(t + 1) overwrites the columns that hold P(t)
          ok = wait_k(t + 1) && warp_spin_tc(&s.bar_pv[x], t & 1, abort_flag, p.status, kStatusTimeoutPV | x);
          if (ok) issue_s(t + 1);
        }
      }
      // everything issued above must complete before TMEM is released
      if (leader) {
        tc_commit(&s.bar_drain[x]);
        drain_wait_tc(&s.bar_drain[x], 0);
      }
      __syncwarp();
    }
  } else if (warp < kRowWarp0) {
    regs_dec<kConvRegs>();
    // ======================= conversion: pages -> bf16 tiles =======================
    const uint32_t row0 = static_cast<uint32_t>(warp - kConvWarp0) * 16u, g8 = static_cast<uint32_t>(lane) >> 2, c = lane & 3;
    const uint32_t shift = p.page_shift, page_mask = (1u << shift) - 1u, n_pages = static_cast<uint32_t>(p.n_pages);
    const uint32_t codes = static_cast<uint32_t>(D / 2) << shift;         // bytes of codes in a chunk
    const uint32_t chunk = codes + (static_cast<uint32_t>(NB) << shift);
    const uint64_t page_stride = static_cast<uint64_t>(p.Hkv) * 2u * chunk;
    const uint8_t* base = p.cache + static_cast<uint64_t>(head) * 2u * chunk;
    const int32_t* table = p.block_table + static_cast<int64_t>(r) * p.table_width;
    // table entry of this warp's 16 keys in tile t (-1: none). It is looked at when the codes are loaded,
    // a tile later: a comparison here would wait for it.
    auto page_of = [&](int t) -> int {
      const int64_t key = key_begin + t * 128ll + row0;
      return t < n_max && key < lim_all ? __ldg(table + (key >> shift)) : -1;
    };
    const uint32_t lane_code = c * (D / 8) + g8 * (D / 2);
    auto load = [&](Raw<D>& raw, int t, int pg, int which) {
      const int64_t key0 = key_begin + t * 128ll + row0;
      const bool there = static_cast<uint32_t>(pg) < n_pages;
      const uint32_t off = static_cast<uint32_t>(key0) & page_mask;
      const uint8_t* ch = base + static_cast<uint32_t>(pg) * page_stride + (which ? chunk : 0u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        clear(raw.w[i]);
        raw.s[i] = 0;
        if (there && key0 + 8 * i + g8 < lim_all) {
          load_piece(raw.w[i], ch + off * (D / 2) + 8 * i * (D / 2) + lane_code);
          raw.s[i] = load_scales<D>(ch + codes + (off + (which ? v_scale_row(g8 + 8 * i) : k_scale_row(g8 + 8 * i))) * NB);
        }
      }
    };
    Raw<D> rk, rv;
    int pg = page_of(0), pg_next = page_of(1);
    if (n_max > 0) {
      load(rk, 0, pg, 0);
      load(rv, 0, pg, 1);
    }
    bool ok = true;
    for (int t = 0; ok && t < n_max; ++t) {
      const int st = t % kTcStages;
      const uint32_t par = ((t / kTcStages) & 1) ^ 1;
      const int pg_after = page_of(t + 2);
      if (t >= kTcStages) ok = warp_wait_tc(&s.bar_k_empty[st], par, abort_flag, p.status, kStatusTimeoutEmpty | st);
      if (!ok) break;
      store_rows<D, 0>(rk, smem_u32(s.k[st]), row0, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.bar_k_full[st]);
      if (t + 1 < n_max) load(rk, t + 1, pg_next, 0);
      if (t >= kTcStages) ok = warp_wait_tc(&s.bar_v_empty[st], par, abort_flag, p.status, kStatusTimeoutEmpty | 8 | st);
      if (!ok) break;
      store_rows<D, 1>(rv, smem_u32(s.v[st]), row0, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.bar_v_full[st]);
      if (t + 1 < n_max) load(rv, t + 1, pg_next, 1);
      pg_next = pg_after;
    }
  } else {
    regs_inc<kRowRegs>();
    // ======================= softmax: two threads per row =======================
    // A warp owns 16 rows of its lane quarter; lanes 0-15 take keys 0 .. 63 of a tile, lanes 16-31 keys
    // 64 .. 127 of the same rows (tcgen05.ld 16x32bx2), and of O the two halves of the channels.
    const int sw = warp - kRowWarp0, x = sw >> 3, quarter = warp & 3, kh = lane >> 4;
    const int r0 = quarter * 32 + ((sw >> 2) & 1) * 16;
    const int in_tile = r0 + (lane & 15);
    const int row = pair * 256 + x * 128 + in_tile;
    const int i = row / G, h = row - i * G;
    const bool live = row < rows_all;
    const int n = x == 0 ? n_x[0] : n_x[1], n_other = x == 0 ? n_x[1] : n_x[0];
    // The warp's 16 Q rows into shared memory, each 8 channels in the order of the converted codes. A load
    // instruction covers whole rows (256 bytes for d = 128), found by the lanes that own them: a lane that reads its
    // own row alone touches a line per lane and instruction, which took 3.7 us of a CTA's 20.
    if (n > 0) {
      constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;               // 16-byte pieces of a row, rows per instruction
      const int64_t at = (rq.start + i) * p.q_token_stride + (head * G + h) * p.q_head_stride;
      const uint32_t tile = smem_u32(s.q[x]);
      const int pc = lane % kPieces;
      const uint32_t live_mask = __ballot_sync(0xffffffffu, live);
      uint4 w[16 / kAtOnce];                // all loads in flight before the first store
#pragma unroll
      for (int j = 0; j < 16 / kAtOnce; ++j) {
        const int rr = j * kAtOnce + lane / kPieces;
        const int64_t from = __shfl_sync(0xffffffffu, at, rr);
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if ((live_mask >> rr) & 1u) w[j] = *reinterpret_cast<const uint4*>(p.q + from + pc * 8);
      }
#pragma unroll
      for (int j = 0; j < 16 / kAtOnce; ++j) {
        const int rr = r0 + j * kAtOnce + lane / kPieces;
        st_shared_v4(tile + (pc >> 3) * (128u * 128u) + rr * 128u + (((pc ^ rr) & 7) << 4), lo16x2(w[j].x, w[j].z), hi16x2(w[j].x, w[j].z),
                     lo16x2(w[j].y, w[j].w), hi16x2(w[j].y, w[j].w));
      }
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.bar_q);
    // the Q rows of a CTA that will run when this one's place is free, on their way to L2 (a seventieth of the
    // time with four key tiles per CTA)
    uint32_t nu = blockIdx.x + kPlaces;
    if (nu < gridDim.x) {
      nu /= sp.splits;
      const int next_row = static_cast<int>(sp.row_tiles - 1 - nu % sp.row_tiles) * 256 + x * 128 + in_tile;
      nu /= sp.row_tiles;
      if (static_cast<int>(nu / p.Hkv) == r && next_row < rows_all) {
        const __nv_bfloat16* next = p.q + (rq.start + next_row / G) * p.q_token_stride + (static_cast<int>(nu % p.Hkv) * G + next_row % G) * p.q_head_stride;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(next + kh * (D / 2)));
      }
    }

    const uint32_t lane_addr = static_cast<uint32_t>(r0) << 16;
    const uint32_t t_s = tmem + lane_addr + kColSx + 128 * x, t_o = tmem + lane_addr + kColOx + 128 * x;
    const float c = p.scale_log2;
    const int lim = live ? static_cast<int>(max(limit_of(row) - key_begin, static_cast<int64_t>(0))) : 0;   // in the split
    const uint32_t shift = p.page_shift;
    const int32_t* table = p.block_table + static_cast<int64_t>(r) * p.table_width;
    // lane j < 8 looks after keys 16 j .. 16 j + 15 of a tile: their table entry, one tile ahead
    const uint32_t n_pages = static_cast<uint32_t>(p.n_pages);
    auto entry_of = [&](int t) -> int {
      const int64_t key = key_begin + t * 128ll + lane * 16;
      return t < n && lane < 8 && key < lim_all ? __ldg(table + (key >> shift)) : 0;
    };
    float m = -INFINITY, mu = 0.f, l0 = 0.f, l1 = 0.f;
    int entry = entry_of(0);
    bool ok = true;
    for (int t = 0; ok && t < n; ++t) {
      const uint32_t gone = __ballot_sync(0xffffffffu, static_cast<uint32_t>(entry) >= n_pages && lane < 8 && key_begin + t * 128ll + lane * 16 < lim_all);
      entry = entry_of(t + 1);
      ok = warp_wait_tc(&s.bar_s_full[x], t & 1, abort_flag, p.status, kStatusTimeoutS | x);
      if (!ok) break;
      tc_fence_after();
      float v[64];                         // keys 64 kh .. of the tile
      {
        uint32_t raw[64];
        tmem_ld16x2_32<64>(t_s, *reinterpret_cast<uint32_t(*)[32]>(raw));
        tmem_ld16x2_32<64>(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(raw + 32));
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = __uint_as_float(raw[j]);
      }
      const int left = lim - t * 128 - 64 * kh;
      if (__any_sync(0xffffffffu, left < 64) || gone) {
        const uint32_t gone_h = gone >> (4 * kh);
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = (j < left && !((gone_h >> (j >> 4)) & 1u)) ? v[j] : -INFINITY;
      }
      float a0 = fmax3(v[0], v[1], v[2]), a1 = fmax3(v[3], v[4], v[5]), a2 = fmaxf(v[6], v[7]), a3 = fmaxf(v[8], v[9]);
#pragma unroll
      for (int j = 10; j < 58; j += 8) {
        a0 = fmax3(a0, v[j], v[j + 1]);
        a1 = fmax3(a1, v[j + 2], v[j + 3]);
        a2 = fmax3(a2, v[j + 4], v[j + 5]);
        a3 = fmax3(a3, v[j + 6], v[j + 7]);
      }
      a0 = fmax3(a0, v[58], v[59]);
      a1 = fmax3(a1, v[60], v[61]);
      a2 = fmax3(a2, v[62], v[63]);
      float top = fmaxf(fmax3(a0, a1, a2), a3);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) * c;
      const bool up = top > m;
      if (__any_sync(0xffffffffu, up)) {
        const float mn = up ? top : m;
        const float mun = mn == -INFINITY ? 0.f : mn;
        const float alpha = m == -INFINITY ? 0.f : ex2(m - mun);
        l0 *= alpha;
        l1 *= alpha;
        if (t > 0) {                       // P V(t - 1) is complete: S(t) was issued after it
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[16];
            tmem_ld16x2_16<D / 2>(t_o + 16 * q, o);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st16x2_16<D / 2>(t_o + 16 * q, o);
          }
        }
        m = mn;
        mu = mun;
      }
      // the tiles' exponentials take turns, so that one tile's products run under the other's softmax
      const int before = x == 0 ? t - 1 : t;
      if (before >= 0 && before < n_other) ok = warp_wait_tc(&s.bar_turn[x], before & 1, abort_flag, p.status, kStatusTimeoutS | 4 | x);
      if (!ok) break;
#pragma unroll
      for (int q = 0; q < 2; ++q) {        // 32 scores of each half become 16 columns of P, over S columns that are in registers
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float e0, e1;
          ffma2_bc(e0, e1, v[32 * q + j], v[32 * q + j + 1], c, -mu);
          e0 = ex2(e0);
          e1 = ex2(e1);
          fadd2(l0, l1, l0, l1, e0, e1);
          pk[j >> 1] = pack_bf162(e0, e1);
        }
        if (q == 1 && lane == 0) mbar_arrive(&s.bar_turn[x ^ 1]);
        tmem_st16x2_16<32>(t_s + 16 * q, pk);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.bar_p_full[x]);
    }
    // ---- out = O / l, or the split's part
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (ok && n > 0) ok = warp_wait_tc(&s.bar_pv[x], (n - 1) & 1, abort_flag, p.status, kStatusTimeoutPV | 4 | x);
    if (ok) {
      tc_fence_after();
      float sum = l0 + l1;
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse2 = sum == 0.f ? -INFINITY : mu + log2f(sum);   // NaN stays NaN
      int64_t orow = static_cast<int64_t>(rq.start + i) * p.Hq + head * G + h;
      const uint32_t live_rows = __popc(__ballot_sync(0xffffffffu, live) & 0xFFFFu);   // the warp's first rows
      // The rows leave through shared memory (Q's, which no product reads any more), so that a store
      // instruction covers whole lines: passes of up to 256 bytes of each of the warp's 16 rows, piece j
      // of row rr at j ^ (rr % 8). Columns 2 j, 2 j + 1 of each 8 hold channels j, j + 4.
      const uint32_t stage = smem_u32(s.q[x]) + static_cast<uint32_t>(r0) * 256u;
      const uint32_t my_row = stage + (lane & 15) * 256u, sw7 = static_cast<uint32_t>(lane) & 7u;
      auto put = [&](uint32_t piece, uint32_t a, uint32_t b, uint32_t cc, uint32_t d) { st_shared_v4(my_row + ((piece ^ sw7) << 4), a, b, cc, d); };
      auto flush = [&](uint32_t pieces, uint8_t* dst, int64_t row_bytes) {    // pieces of 16 bytes per row: 8 or 16
        __syncwarp();
        const uint32_t per = 32u / pieces, pc = static_cast<uint32_t>(lane) % pieces;
#pragma unroll 4
        for (uint32_t rr0 = 0; rr0 < 16u; rr0 += per) {
          const uint32_t rr = rr0 + static_cast<uint32_t>(lane) / pieces;
          const int64_t to = __shfl_sync(0xffffffffu, orow, rr);
          const uint4 val = ld_shared_v4(stage + rr * 256u + ((pc ^ (rr & 7u)) << 4));
          if (rr < live_rows) *reinterpret_cast<uint4*>(dst + to * row_bytes + pc * 16u) = val;
        }
        __syncwarp();
      };
      const bool direct = used_splits == 1;
      // parts are indexed by request and token, which bounds them by what the plan laid out
      if (!direct) orow = (static_cast<int64_t>(r) * p.max_new + i) * p.Hq + head * G + h;
      // fp32 parts: 64 channels a pass; with d = 128 a pass takes one half of the lanes' channels
      const int passes = direct ? 1 : D / 64;
#pragma unroll 1
      for (int pp = 0; pp < passes; ++pp) {
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld16x2_32<D / 2>(t_o + 32 * q, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
          }
          const uint32_t col8 = (kh * (D / 2) + 32 * q) / 8;                  // first of the lane's four groups of 8 channels
          if (direct || D == 64 || kh == pp) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              float e[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) e[(j >> 1) + 4 * (j & 1)] = __uint_as_float(o[8 * w + j]) * inv;
              if (direct) {
                put(col8 + w, pack_bf162(e[0], e[1]), pack_bf162(e[2], e[3]), pack_bf162(e[4], e[5]), pack_bf162(e[6], e[7]));
              } else {
                const uint32_t piece = 2u * ((col8 + w) & 7u);
                put(piece, __float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
                put(piece + 1, __float_as_uint(e[4]), __float_as_uint(e[5]), __float_as_uint(e[6]), __float_as_uint(e[7]));
              }
            }
          }
        }
        if (direct) flush(D / 8, reinterpret_cast<uint8_t*>(p.out), D * 2);
        else flush(16, reinterpret_cast<uint8_t*>(sp.part_o + static_cast<int64_t>(split) * D + 64 * pp), static_cast<int64_t>(sp.splits) * D * 4);
      }
      if (live && kh == 0) {
        if (used_splits > 1) sp.part_lse[orow * sp.splits + split] = lse2;
        else if (p.lse) p.lse[orow] = lse2 * 0.6931471805599453f;
      }
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcCols);
  }
}

template <int D>
cudaError_t launch_tc_d(const PagedParams& p, const SplitParams& sp, int64_t units, cudaStream_t stream) {
  // the softmax warps' registers come from the block's launch allocation: a build with fewer registers
  // per thread than the split assumes would make them wait forever
  static int regs = -1;
  if (regs < 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, paged_tc_kernel<D>);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs != kTcLaunchRegs) return cudaErrorInvalidConfiguration;
  const int smem = static_cast<int>(sizeof(TcSmem<D>) + 1024);
  const cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_tc_kernel<D><<<static_cast<unsigned>(units), kTcThreads, smem, stream>>>(p, sp);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, const SplitParams& sp, int d, int64_t units, cudaStream_t stream) {
  // a timeout is reported in the status word, which no CTA can clear for the others
  const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(unsigned int), stream);
  if (e != cudaSuccess) return e;
  return d == 128 ? launch_tc_d<128>(p, sp, units, stream) : launch_tc_d<64>(p, sp, units, stream);
}

}  // namespace mxattn
