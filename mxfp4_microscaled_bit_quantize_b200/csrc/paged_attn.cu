// Attention of few new tokens over the paged MXFP4 KV cache (decoding, drafted tokens to verify).
//
//   x_j = (q . k_j) log2(e) / sqrt(d),  out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
//
// Bound: 17/16 d bytes of K and V per key and KV head have to come from HBM once, for all query heads of the
// group and all new tokens. At 6.5 TB/s an SM may spend about 90 clocks on 16 keys of d = 128, and E2M1 codes
// have to become numbers in that time, so the kernel keeps the instructions per key down rather than the FLOPs:
//   * a warp takes 16 keys at a time in the order of the mma fragments (the cache's layout does the gather, see
//     cache_layout.cuh) from a ring of its own in shared memory, into which it copies four groups ahead; the four
//     warps of a CTA take turns on the groups and meet once, at the end;
//   * S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16: the keys (or channels) are the 16 rows, the queries
//     (tokens x heads of the group) the 8 columns, so that decoding wastes no half tile. tcgen05's smallest tile
//     has 128 rows; here there are up to 16;
//   * E2M1 codes become fp16 by cvt (exact); no scale is ever multiplied into K or V: a K block's scale
//     multiplies its 32-channel partial score in fp32, a V block's scale its fp16 probability, four
//     multiplications each for 8 queries instead of 16;
//   * Q is fp16 after a power of two per row that brings its largest element to [2^7, 2^8) (bf16's 8 bits fit,
//     elements 2^-21 below the largest and smaller lose bits below 2^-32 of it);
//   * the reference m of a column moves only when a score passes it by 7, so that the maximum over the warp's
//     lanes is rarely taken; p = 2^(x - m + 7) <= 2^14 is summed in fp32 and rounded to fp16 (11 bits) for the
//     product;
//   * V's block scales enter relative to r_b, the largest exponent so far of channel block b, as 2^(s - r_b) in
//     fp16, where s is at most 6 below r_b: with p's rounding and that of the product, both at steps of 2^-24 when
//     they are subnormal, a probability is off by half a step of 8 bits or by (1 + 2^6) 2^-32 < 2^-25 of the row's
//     largest, whichever is more (with 14 instead of 6, 2^-18: small probabilities vanished behind one outlier of V).
//     A group with a block further below takes a path with bf16 operands, whose 8 bits need no such care (64 requests
//     of 8192 keys, 32 query and 8 KV heads, d = 128: 156 us, 211 where every group takes it).
// A long context is split over CTAs (chunk keys each); their results meet in paged_combine_kernel.
//
// Measured (d = 128, 32 query and 8 KV heads, pages of 16): 64 requests of up to 8192 keys, one token each, 89 us
// (267 MB: 3.0 TB/s, 45 % of the copy bandwidth); 2 x 131072 keys, four tokens each, pages of 64: 117 us (285 MB:
// 2.4 TB/s). The copies alone take 56 us of the 89; the rest is arithmetic that they do not hide: the ALU pipe,
// which cvt shares with the logic on nibbles and scale bytes, is 58 % busy, the schedulers issue 65 % of the time
// with 16 warps of 128 registers. Fragments loaded to registers one group ahead instead of the ring took 94 us, two
// groups a turn, deeper rings or 12 warps of 168 registers the same as now.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cmath>
#include <cstdint>

#include "paged_common.cuh"

namespace mxattn {

constexpr int kSmallWarps = 4;
constexpr int kMaxSplits = 128;
constexpr int kRingGroups = 4;          // groups of 16 keys in a warp's ring
constexpr uint32_t kNear = 6;           // V scales this far below their reference stay in fp16; kNear + 1 is a mask of bits
static_assert(((kNear + 1) & (kNear + 2)) == 0, "differences 0 .. kNear + 1 are told by their upper bits");

template <int NB> struct Frag;          // what a lane holds of 16 keys
template <> struct Frag<4> { uint4 k0, k1; uint2 ks; };
template <> struct Frag<2> { uint2 k0, k1; uint32_t ks; };
template <int NB> struct VFrag;
template <> struct VFrag<4> { uint2 v[4]; uint4 vs; };
template <> struct VFrag<2> { uint32_t v[4]; uint2 vs; };

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// 16 keys in a warp's ring: K codes, V codes, K scales, V scales as they lie in the page (17 d bytes), but
// for d = 128 the 16-byte pieces of V row t are at piece ^ (t / 2 % 4): a lane reads 8 bytes of rows 2c and
// their neighbours, whose 64-byte rows would otherwise share banks four ways.
template <int NB> constexpr uint32_t kGroupBytes = 16u * 17u * 2u * NB;

// A lane's constants for copying groups into the ring and reading them back (byte offsets in the page's two
// chunks of this head, and in a slot).
template <int NB>
struct GroupLane {
  uint32_t from_row, from_v, from_sc;         // K codes; V codes behind them; scales
  uint32_t to_v, to_sc, k, v, ks, vs;
  bool has_sc;                                // NB lanes copy K's scales, the next NB lanes V's
  __device__ __forceinline__ GroupLane(uint32_t lane, int page_shift) {
    constexpr uint32_t kRow = 16u * NB, kCodes = 16u * kRow;
    const uint32_t g = lane >> 2, c = lane & 3u;
    const uint32_t codes = kRow << page_shift, chunk = codes + (static_cast<uint32_t>(NB) << page_shift);
    from_row = lane * 16u;
    from_v = chunk;
    has_sc = lane < 2u * NB;
    from_sc = lane < NB ? codes + lane * 16u : chunk + codes + (lane - NB) * 16u;
    to_v = kCodes + (NB == 4 ? (lane ^ ((lane >> 3) & 3u)) << 4 : lane << 4);   // row lane / 4, piece (lane & 3) ^ (row / 2 % 4)
    to_sc = 2u * kCodes + lane * 16u;
    k = lane * (4u * NB);
    v = kCodes + (NB == 4 ? c * 128u + (((g >> 1) ^ c) << 4) + (g & 1u) * 8u : c * 64u + g * 4u);   // rows 2c, 2c + 1, 2c + 8, 2c + 9
    ks = 2u * kCodes + g * (2u * NB);
    vs = 2u * kCodes + 16u * NB + c * (4u * NB);
  }
};
// Copies 16 tokens into ring slot `dst`; kc: the page's K chunk of this head, off: the first token in the page.
template <int NB>
__device__ __forceinline__ void fetch_group(uint32_t dst, uint32_t lane, const GroupLane<NB>& at, const uint8_t* kc, uint32_t off) {
  const uint8_t* row = kc + (off * (16u * NB) + at.from_row);
  const uint8_t* vrow = row + at.from_v;
  copy16(dst + lane * 16u, row);
  copy16(dst + at.to_v, vrow);
  if (NB == 4) {
    copy16(dst + 512u + lane * 16u, row + 512);
    copy16(dst + at.to_v + 512u, vrow + 512);
  }
  if (at.has_sc) copy16(dst + at.to_sc, kc + (off * NB + at.from_sc));
}
__device__ __forceinline__ void read_k(Frag<4>& f, uint32_t src, const GroupLane<4>& at) {
  f.k0 = ld_shared_v4(src + at.k);
  f.k1 = ld_shared_v4(src + at.k + 512u);
  f.ks = ld_shared_v2(src + at.ks);
}
__device__ __forceinline__ void read_k(Frag<2>& f, uint32_t src, const GroupLane<2>& at) {
  f.k0 = ld_shared_v2(src + at.k);
  f.k1 = ld_shared_v2(src + at.k + 256u);
  f.ks = ld_shared_u32(src + at.ks);
}
__device__ __forceinline__ void read_v(VFrag<4>& f, uint32_t src, const GroupLane<4>& at) {
  f.vs = ld_shared_v4(src + at.vs);
  f.v[0] = ld_shared_v2(src + at.v);
  f.v[1] = ld_shared_v2(src + at.v + 64u);
  f.v[2] = ld_shared_v2(src + at.v + 512u);
  f.v[3] = ld_shared_v2(src + at.v + 576u);
}
__device__ __forceinline__ void read_v(VFrag<2>& f, uint32_t src, const GroupLane<2>& at) {
  f.vs = ld_shared_v2(src + at.vs);
  f.v[0] = ld_shared_u32(src + at.v);
  f.v[1] = ld_shared_u32(src + at.v + 32u);
  f.v[2] = ld_shared_u32(src + at.v + 256u);
  f.v[3] = ld_shared_u32(src + at.v + 288u);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Scale bytes of block b for the lane's keys g and g + 8 as fp32 powers of two (byte 0 becomes 0).
__device__ __forceinline__ float pow2_bits(uint32_t w, int b) {
  const uint32_t x = b < 3 ? w << (23 - 8 * b) : w >> 1;
  return __uint_as_float(x & 0x7F800000u);
}
__device__ __forceinline__ void k_scales(const Frag<4>& f, int b, float& s0, float& s1) {
  s0 = pow2_bits(f.ks.x, b);
  s1 = pow2_bits(f.ks.y, b);
}
__device__ __forceinline__ void k_scales(const Frag<2>& f, int b, float& s0, float& s1) {
  s0 = pow2_bits(f.ks, b);
  s1 = pow2_bits(f.ks, b + 2);
}

// V scale bytes of the lane's keys (2c, 2c + 1) [h = 0] or (2c + 8, 2c + 9) [h = 1] as 16-bit pairs, block b.
__device__ __forceinline__ void v_scale_pairs(const VFrag<4>& f, uint32_t (&s)[4][2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = h ? f.vs.z : f.vs.x, b = h ? f.vs.w : f.vs.y;
    const uint32_t lo = __byte_perm(a, b, 0x5410), hi = __byte_perm(a, b, 0x7632);
    s[0][h] = lo & 0x00FF00FFu;
    s[1][h] = (lo >> 8) & 0x00FF00FFu;
    s[2][h] = hi & 0x00FF00FFu;
    s[3][h] = (hi >> 8) & 0x00FF00FFu;
  }
}
__device__ __forceinline__ void v_scale_pairs(const VFrag<2>& f, uint32_t (&s)[2][2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = h ? f.vs.y : f.vs.x;      // halves: keys 2c, 2c + 1; bytes: blocks 0, 1
    s[0][h] = a & 0x00FF00FFu;
    s[1][h] = (a >> 8) & 0x00FF00FFu;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kSmallWarps * 32, NT == 1 ? 4 : 2) paged_small_kernel(const PagedParams p, const SplitParams sp) {
  constexpr int NB = D / 32, kRows = 8 * NT, kPad = D + 4;
  // the warps' rings; at the end the warps' results take their place
  constexpr uint32_t kRing = kRingGroups * kGroupBytes<NB>, kRingBytes = kSmallWarps * kRing, kOutBytes = kSmallWarps * kRows * kPad * 4u;
  __shared__ __align__(128) uint8_t ring[kRingBytes > kOutBytes ? kRingBytes : kOutBytes];
  float (*so)[kRows][kPad] = reinterpret_cast<float (*)[kRows][kPad]>(ring);
  __shared__ float sm[kSmallWarps][kRows], sl[kSmallWarps][kRows], su[kSmallWarps][NB];   // reference, sum of p; unit of a block of V
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3u;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

  const int G = p.Hq / p.Hkv;
  uint32_t u = blockIdx.x;
  const int split = static_cast<int>(u % sp.splits);
  u /= sp.splits;
  const int rt = static_cast<int>(u % sp.row_tiles);
  u /= sp.row_tiles;
  const int head = static_cast<int>(u % p.Hkv), r = static_cast<int>(u / p.Hkv);
  const RequestRange rq = request_range(p, r);
  const int n_used = min(rq.n, p.max_new);
  const int used_splits = max(1, static_cast<int>((rq.cap + sp.chunk - 1) / sp.chunk));
  if (rt * kRows >= n_used * G || split >= used_splits) return;

  // ---- which keys: the copies go out before anything else is loaded
  auto limit_of = [&](int i) -> int {        // keys j < limit are visible to token i (it grows with i)
    return static_cast<int>(max(min(p.causal ? rq.kv - rq.n + i + 1 : rq.kv, rq.cap), static_cast<int64_t>(0)));
  };
  const int lim_min = limit_of(rt * kRows / G), lim_max = limit_of((min((rt + 1) * kRows, n_used * G) - 1) / G);
  const int first = static_cast<int>(split * sp.chunk) >> 4;
  const int stop = (min(lim_max, static_cast<int>(min((split + 1) * sp.chunk, static_cast<int64_t>(0x7FFFFFFF)))) + 15) >> 4;
  const int32_t* table = p.block_table + static_cast<int64_t>(r) * p.table_width;
  const uint32_t n_pages = static_cast<uint32_t>(p.n_pages), page_mask = (1u << p.page_shift) - 1u;
  const uint32_t head_bytes = 2u * cache_chunk_bytes(D, 1u << p.page_shift);
  const uint32_t page_bytes = static_cast<uint32_t>(p.Hkv) * head_bytes;      // below 2^32 for every supported shape
  const GroupLane<NB> at(lane, p.page_shift);
  const uint8_t* base = p.cache + static_cast<uint64_t>(head) * head_bytes;

  auto page_of = [&](int grp) -> int {
    return grp < stop ? __ldg(table + ((grp << 4) >> p.page_shift)) : -1;     // looked at when it is used: a comparison would wait
  };
  // The ring holds the next kRingGroups groups of this warp, copied asynchronously; their pages are looked up
  // one turn before the copy. `there` remembers, newest group in bit 0, which of them have a page.
  const uint32_t my_ring = smem_u32(ring) + warp * kRing;
  uint32_t there = 0u;
  auto fetch = [&](uint32_t dst, int grp, int page) {
    const bool ok = static_cast<uint32_t>(page) < n_pages;
    there = (there << 1) | (ok ? 1u : 0u);
    if (ok) fetch_group<NB>(dst, lane, at, base + static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_bytes, (static_cast<uint32_t>(grp) << 4) & page_mask);
    copies_commit();
  };
  int grp = first + static_cast<int>(warp);
  {
    int pages[kRingGroups];
#pragma unroll
    for (int i = 0; i < kRingGroups; ++i) pages[i] = page_of(grp + i * kSmallWarps);
#pragma unroll
    for (int i = 0; i < kRingGroups; ++i) fetch(my_ring + i * kGroupBytes<NB>, grp + i * kSmallWarps, pages[i]);
  }
  int page_ahead = page_of(grp + kRingGroups * kSmallWarps);

  // ---- Q: column nt * 8 + g of this lane, channels 32 b + 8 c .. + 7 as four fp16 pairs
  uint32_t qf[NT][NB][4];
  float qscale[NT][2];
  int lim[NT][2];          // keys j < lim are visible to columns 2c, 2c + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = rt * kRows + nt * 8 + static_cast<int>(g);
    const int i = row / G, h = row - i * G;
    const bool live = i < n_used;
    float amax = 0.f;
    uint4 raw[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      raw[b] = make_uint4(0u, 0u, 0u, 0u);
      if (live)
        raw[b] = *reinterpret_cast<const uint4*>(p.q + (rq.start + i) * p.q_token_stride + (head * G + h) * p.q_head_stride + b * 32 + c * 8);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = word_of(raw[b], w);
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x << 16)), fabsf(__uint_as_float(x & 0xFFFF0000u))));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100), 127);
    const float mul = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);      // 2^(7 - e)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = word_of(raw[b], w);
        qf[nt][b][w] = pack_half2(__uint_as_float(x << 16) * mul, __uint_as_float(x & 0xFFFF0000u) * mul);
      }
    const int mine = live ? limit_of(i) : 0;
    const float back = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int from = (2 * c + x) * 4;
      qscale[nt][x] = __shfl_sync(0xffffffffu, back, from);
      lim[nt][x] = __shfl_sync(0xffffffffu, mine, from);
    }
  }

  // Scores stay in units of the columns' qscale: thr is the raw score that moves a reference, mu7 = m - 7
  // (0 while the column has seen no key, so that 2^(-inf - mu7) is 0 and not NaN).
  float o[NT][2 * NB][4];
  float l[NT][2], m[NT][2], mu7[NT][2], thr[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[nt][t][x] = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) { l[nt][x] = 0.f; m[nt][x] = -INFINITY; mu7[nt][x] = 0.f; thr[nt][x] = -INFINITY; }
  }
  int rb[NB];                                 // reference exponent byte r of V's channel blocks, -1 before the first group
  uint32_t top[NB];                           // r + 1 in both halves
#pragma unroll
  for (int b = 0; b < NB; ++b) { rb[b] = -1; top[b] = 0xFFFFFFFFu; }   // the first group is above it

  auto step = [&](uint32_t slot, int grp, auto&& refill) {
    const int key0 = grp << 4;
    Frag<NB> f;
    read_k(f, slot, at);
    // ---- S^T: partial scores of each 32-channel block, times the block's scale
    float s[NT][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t a[4], a8[4];
      e2m1x8_to_half2(word_of(f.k0, b), a);
      e2m1x8_to_half2(word_of(f.k1, b), a8);
      float s0, s1;
      k_scales(f, b, s0, s1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4];
        mma_f16_zero(acc, a[0], a8[0], a[1], a8[1], qf[nt][b][0], qf[nt][b][1]);
        mma_f16(acc, a[2], a8[2], a[3], a8[3], qf[nt][b][2], qf[nt][b][3]);
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][x] = b == 0 ? acc[x] * (x < 2 ? s0 : s1) : fmaf(acc[x], x < 2 ? s0 : s1, s[nt][x]);
      }
    }
    if (key0 + 16 > lim_min) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (key0 + static_cast<int>(g) + (x >> 1) * 8 >= lim[nt][x & 1]) s[nt][x] = -INFINITY;
    }
    // ---- the columns' references: moved only when a score passes one by 7
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) up |= fmaxf(s[nt][x], s[nt][x + 2]) > thr[nt][x];
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float t = fmaxf(s[nt][x], s[nt][x + 2]);
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16)) * qscale[nt][x];
          const float mn = fmaxf(m[nt][x], t);
          const float alpha = m[nt][x] == -INFINITY ? 0.f : ex2(m[nt][x] - mn);
          m[nt][x] = mn;
          mu7[nt][x] = mn == -INFINITY ? 0.f : mn - 7.f;
          thr[nt][x] = (mn + 7.f) / qscale[nt][x];
          l[nt][x] *= alpha;
#pragma unroll
          for (int tt = 0; tt < 2 * NB; ++tt) { o[nt][tt][x] *= alpha; o[nt][tt][x + 2] *= alpha; }
        }
    }
    // ---- p = 2^(x - m + 7), summed in fp32
    float pv[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 4; ++x) pv[nt][x] = ex2(fmaf(s[nt][x], qscale[nt][x & 1], -mu7[nt][x & 1]));
      l[nt][0] += pv[nt][0] + pv[nt][2];
      l[nt][1] += pv[nt][1] + pv[nt][3];
    }
    // ---- V's scales relative to the reference exponents
    VFrag<NB> fv;
    read_v(fv, slot, at);
    refill();
    uint32_t vs[NB][2];                       // becomes r + 1 - s in both halves
    v_scale_pairs(fv, vs);
    // In range: s within [r - kNear, r + 1]. The subtraction in 16-bit halves of numbers up to 256 is exact: a half that
    // would borrow is itself negative and shows in its upper bits.
    uint32_t out_of_range = 0u;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      vs[b][0] = top[b] - vs[b][0];
      vs[b][1] = top[b] - vs[b][1];
      out_of_range |= vs[b][0] | vs[b][1];
    }
    // One far below takes the wide path; one above the reference, a negative half, moves it (O is scaled down).
    bool wide = __any_sync(0xffffffffu, (out_of_range & ~((kNear + 1u) * 0x00010001u)) != 0u);
    const bool tail = key0 + 16 > lim_max;
    if ((wide && __any_sync(0xffffffffu, (out_of_range & 0x80008000u) != 0u)) || tail) {
      wide = false;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        vs[b][0] = top[b] - vs[b][0];
        vs[b][1] = top[b] - vs[b][1];
        if (tail) {                           // tokens behind the end, whatever their bytes say: no scale at all
#pragma unroll
          for (int h = 0; h < 2; ++h)
            vs[b][h] &= (key0 + 8 * h + 2 * static_cast<int>(c) < lim_max ? 0xFFFFu : 0u) |
                        (key0 + 8 * h + 2 * static_cast<int>(c) + 1 < lim_max ? 0xFFFF0000u : 0u);
        }
        const int t = static_cast<int>(__reduce_max_sync(0xffffffffu, max(max(vs[b][0] & 0xFFFFu, vs[b][0] >> 16), max(vs[b][1] & 0xFFFFu, vs[b][1] >> 16))));
        const int r_new = max(rb[b], t);
        if (tail) {                           // ... and then the reference's, under p = 0
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (key0 + 8 * h + 2 * static_cast<int>(c) >= lim_max) vs[b][h] |= static_cast<uint32_t>(r_new);
            if (key0 + 8 * h + 2 * static_cast<int>(c) + 1 >= lim_max) vs[b][h] |= static_cast<uint32_t>(r_new) << 16;
          }
        }
        const int lo = static_cast<int>(__reduce_min_sync(0xffffffffu, min(min(vs[b][0] & 0xFFFFu, vs[b][0] >> 16), min(vs[b][1] & 0xFFFFu, vs[b][1] >> 16))));
        if (r_new > rb[b]) {
          const float down = rb[b] < 0 ? 0.f : exp2f(static_cast<float>(rb[b] - r_new));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[nt][2 * b + tt][x] *= down;
          rb[b] = r_new;
        }
        wide |= lo < rb[b] - static_cast<int>(kNear);
        top[b] = static_cast<uint32_t>(rb[b] + 1) * 0x00010001u;
        vs[b][0] = top[b] - vs[b][0];
        vs[b][1] = top[b] - vs[b][1];
      }
    }
    // ---- O^T += V^T P^T: P^T (key pairs of column g) by movmatrix. Words w of a key pair hold blocks 2w,
    //      2w + 1; nibbles of the two keys are brought together so that one cvt gives the pair of one channel:
    //      [key pair][2 (block & 1) + tile], rows g (even nibbles) and g + 8 (odd nibbles).
    auto v_pairs = [&](int w, uint32_t (&ev)[2][4], uint32_t (&od)[2][4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = word_of(fv.v[2 * h], w), y = word_of(fv.v[2 * h + 1], w);
        e2m1x8_to_half2((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[h]);
        e2m1x8_to_half2(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[h]);
      }
    };
    uint32_t pt[NT][2], ev[2][4], od[2][4];
    if (!wide) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pt[nt][0] = transpose8x8(pack_half2(pv[nt][0], pv[nt][1]));
        pt[nt][1] = transpose8x8(pack_half2(pv[nt][2], pv[nt][3]));
      }
#pragma unroll
      for (int w = 0; w < NB / 2; ++w) {
        v_pairs(w, ev, od);
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          const int b = 2 * w + bb;
          const uint32_t sc0 = 0x40004000u - vs[b][0] * 1024u, sc1 = 0x40004000u - vs[b][1] * 1024u;   // 2^(s - r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = hmul2(pt[nt][0], sc0), b1 = hmul2(pt[nt][1], sc1);
#pragma unroll
            for (int t = 0; t < 2; ++t)
              mma_f16(o[nt][2 * b + t], ev[0][2 * bb + t], od[0][2 * bb + t], ev[1][2 * bb + t], od[1][2 * bb + t], b0, b1);
          }
        }
      }
    } else {
      // bf16: an fp16 code's bits, moved to the places of bf16's exponent and mantissa, are the code times 2^-112, and P
      // (8 bits) takes 2^(s - r + 112). Exact for s down to r - 112 and p down to 2^-21 of the row's largest.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pt[nt][0] = transpose8x8(pack_bf162(pv[nt][0], pv[nt][1]));
        pt[nt][1] = transpose8x8(pack_bf162(pv[nt][2], pv[nt][3]));
      }
      auto as_bf16 = [](uint32_t h) { return ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u); };
#pragma unroll
      for (int w = 0; w < NB / 2; ++w) {
        v_pairs(w, ev, od);
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          const int b = 2 * w + bb;
          // exponent fields s - r + 112 + 127 in both halves, 0 (no weight) where that is negative
          const uint32_t sc0 = (__vmaxu2(0x01F001F0u - vs[b][0], 0x01000100u) - 0x01000100u) << 7;
          const uint32_t sc1 = (__vmaxu2(0x01F001F0u - vs[b][1], 0x01000100u) - 0x01000100u) << 7;
          uint32_t a[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            a[t][0] = as_bf16(ev[0][2 * bb + t]);
            a[t][1] = as_bf16(od[0][2 * bb + t]);
            a[t][2] = as_bf16(ev[1][2 * bb + t]);
            a[t][3] = as_bf16(od[1][2 * bb + t]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t b0 = mul_bf162(pt[nt][0], sc0), b1 = mul_bf162(pt[nt][1], sc1);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma_bf16(o[nt][2 * b + t], a[t][0], a[t][1], a[t][2], a[t][3], b0, b1);
          }
        }
      }
    }
  };
  uint32_t slot = my_ring;
  for (; grp < stop; grp += kSmallWarps) {
    copies_wait<kRingGroups - 1>();
    __syncwarp();
    const uint32_t now = slot;
    slot = slot == my_ring + (kRingGroups - 1) * kGroupBytes<NB> ? my_ring : slot + kGroupBytes<NB>;
    auto refill = [&]() {
      __syncwarp();                           // the slot is read by every lane before it is filled again
      fetch(now, grp + kRingGroups * kSmallWarps, page_ahead);
      page_ahead = page_of(grp + (kRingGroups + 1) * kSmallWarps);
    };
    if ((there >> (kRingGroups - 1)) & 1u) step(now, grp, refill);
    else refill();
  }
  copies_wait<0>();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();                            // the rings give way to the results

  // ---- the warps' results meet in shared memory. V's references join last, behind the division by the row's sum: p
  //      reaches 2^14, so the sums themselves in V's units would leave fp32's range for values that fit it.
#pragma unroll
  for (int b = 0; b < NB; ++b)
    if (lane == b) su[warp][b] = rb[b] < 0 ? 0.f : pow2_from_byte(static_cast<uint32_t>(rb[b]));
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float t = l[nt][x];
      t += __shfl_xor_sync(0xffffffffu, t, 4);
      t += __shfl_xor_sync(0xffffffffu, t, 8);
      t += __shfl_xor_sync(0xffffffffu, t, 16);
      const int row = nt * 8 + 2 * static_cast<int>(c) + x;
      if (g == 0) {
        sl[warp][row] = t;
        sm[warp][row] = m[nt][x];
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float4 v = make_float4(o[nt][2 * b][x], o[nt][2 * b][x + 2], o[nt][2 * b + 1][x], o[nt][2 * b + 1][x + 2]);
        *reinterpret_cast<float4*>(&so[warp][row][32 * b + 4 * g]) = v;
      }
    }
  }
  __syncthreads();
  constexpr int kPer = D / 32;
  for (int row = static_cast<int>(warp); row < kRows; row += kSmallWarps) {
    const int at = rt * kRows + row;
    const int i = at / G, h = at - i * G;
    if (i >= n_used) break;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) top = fmaxf(top, sm[w][row]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, k[kSmallWarps], acc[kPer];
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      k[w] = ex2(sm[w][row] - base);                     // 0 for a warp that saw no key
      sum = fmaf(k[w], sl[w][row], sum);
    }
    const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);   // 2^-22; nothing here waits for a division's slow path
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      const float unit = su[w][lane * kPer / 32];
#pragma unroll
      for (int x = 0; x < kPer; ++x) acc[x] = fmaf(k[w] * inv * so[w][row][lane * kPer + x], unit, acc[x]);
    }
    const float lse2 = sum == 0.f ? -INFINITY : base - 7.f + log2f(sum);   // NaN stays NaN
    const int64_t orow = static_cast<int64_t>(rq.start + i) * p.Hq + head * G + h;
    if (used_splits == 1) {
#pragma unroll
      for (int x = 0; x < kPer; x += 2)
        *reinterpret_cast<uint32_t*>(p.out + orow * D + lane * kPer + x) = pack_bf162(acc[x], acc[x + 1]);
      if (p.lse && lane == 0) p.lse[orow] = lse2 * 0.6931471805599453f;
    } else {
      const int64_t prow = ((static_cast<int64_t>(r) * p.max_new + i) * p.Hq + head * G + h) * sp.splits + split;
      float* po = sp.part_o + prow * D + lane * kPer;
#pragma unroll
      for (int x = 0; x < kPer; ++x) po[x] = acc[x];
      if (lane == 0) sp.part_lse[prow] = lse2;
    }
  }
}

// out = sum over the splits of a row of 2^(lse_s - lse) o_s: one warp per row.
template <int D>
__global__ void __launch_bounds__(128) paged_combine_kernel(const PagedParams p, const SplitParams sp) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t per_request = static_cast<int64_t>(p.max_new) * p.Hq;
  const bool any = unit < p.R * per_request;
  const int r = any ? static_cast<int>(unit / per_request) : 0;
  const int64_t rest = unit - r * per_request;
  const int i = static_cast<int>(rest / p.Hq), h = static_cast<int>(rest % p.Hq);
  const RequestRange rq = request_range(p, r);
  const int used = static_cast<int>((rq.cap + sp.chunk - 1) / sp.chunk);
  // Launched ahead of the parts' end, see launch_rows. Every warp waits for it, those with nothing to join too:
  // the launch behind this one relies on this one's end alone.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!any || i >= rq.n || used <= 1) return;
  const int64_t orow = static_cast<int64_t>(rq.start + i) * p.Hq + h;
  const int64_t prow = ((static_cast<int64_t>(r) * p.max_new + i) * p.Hq + h) * sp.splits;
  const float* lse = sp.part_lse + prow;
  const float* po = sp.part_o + prow * D + lane * kPer;
  static_assert(kMaxSplits <= 128, "four splits a lane");
  float w[4];                              // lane s % 32 has the weight of split s
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = lane + 32 * j < used ? lse[lane + 32 * j] : -INFINITY;
    top = fmaxf(top, w[j]);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float base = (top == -INFINITY ? 0.f : top) + 7.f;   // weights up to 2^-7: 128 of them times a value stay in fp32's range
  float sum = 0.f, acc[kPer];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = ex2(w[j] - base);
    sum += w[j];
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
#pragma unroll
  for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(used - 32 * j, 32);
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float k = __shfl_sync(0xffffffffu, w[j], s);
#pragma unroll
      for (int x = 0; x < kPer; ++x) acc[x] = fmaf(k, po[static_cast<int64_t>(32 * j + s) * D + x], acc[x]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int x = 0; x < kPer; x += 2)
    *reinterpret_cast<uint32_t*>(p.out + orow * D + lane * kPer + x) = pack_bf162(acc[x] * inv, acc[x + 1] * inv);
  if (p.lse && lane == 0) p.lse[orow] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
}

// Up to 16 rows (new tokens x heads of a group) go to the mma.sync kernel, whose time does not depend on
// rows that are not there; more rows share the tcgen05 kernel's conversion of the keys.
SplitPlan plan_splits(int R, int Hq, int Hkv, int d, int max_new, int64_t max_kv) {
  SplitPlan s{};
  const int64_t rows = static_cast<int64_t>(max_new) * (Hq / Hkv);
  if (max_kv > 0x7FFFFF00) max_kv = 0x7FFFFF00;              // as in request_range
  s.tc = rows > 16;
  s.nt = rows <= 8 ? 1 : 2;
  const int64_t per = s.tc ? 256 : 8 * s.nt;
  const int64_t unit = s.tc ? 128 : 64;                      // chunks are multiples of this many keys
  s.row_tiles = (rows + per - 1) / per;
  const int64_t units = static_cast<int64_t>(R) * Hkv * s.row_tiles;
  // A long batch is cut into this many CTAs: four for each of 148 x 4 places with one column tile, two for
  // each of 148 x 2 with two (64 ragged requests of up to 8192 keys: 88 us, 99 with half as many; 2 x 131072
  // keys and two column tiles: 115 us, 134 with twice or half as many).
  constexpr int64_t kSpread[3] = {0, 2368, 592};
  int64_t chunk;
  if (s.tc) {
    // CTAs run one to an SM and a CTA's set-up and output cost about as much as four tiles of 128 keys, so the
    // splits are chosen by waves x (4 + tiles of a split), joining the parts counted as four more. A split has to
    // gain a tenth: the bounds overstate ragged batches, and parts take workspace (device time; 32 query and 8 KV heads,
    // d = 128 but for the first: 7 requests of up to 777 tokens over 3001, 15/3 heads, d = 64: 126 us in one part, 137 in
    // three; 2048 over 8000: 389 us in one, 441 in two, 477 in four; 2048 over 14336: 622, 673, 684; 2048 over 30720: 1217,
    // 1275, 1214; 800 over 7392: 171, 194, 177; 1024 over 60000: 1133, 1175, 1215, 1144 in eight; 512 over 30000: 582, 317,
    // 333; 2 x 100 over 8000: 214, 119, 70, 78 in eight; 8 over 100000: 230 in nine, 131 in 18, 186 in 98).
    const int64_t tiles = (max_kv + 127) / 128;
    const int64_t whole = (units + 147) / 148 * (4 + tiles);
    int64_t best = 0, parts = 1;
    for (int64_t n = 1; n <= kMaxSplits && n * 2 <= (tiles > 2 ? tiles : 2) && (n == 1 || units * n <= 1184); ++n) {
      const int64_t cost = (units * n + 147) / 148 * (4 + (tiles + n - 1) / n) + (n > 1 ? 4 : 0);
      if (n == 1 || (cost < best && cost * 10 < 9 * whole)) { best = cost; parts = n; }
    }
    chunk = (tiles + parts - 1) / parts * 128;
  } else {
    chunk = (units * max_kv + kSpread[s.nt] - 1) / kSpread[s.nt];
  }
  chunk = (chunk + unit - 1) / unit * unit;
  if (chunk < unit) chunk = unit;
  int64_t splits = (max_kv + chunk - 1) / chunk;
  if (splits > kMaxSplits) {
    chunk = ((max_kv + kMaxSplits - 1) / kMaxSplits + unit - 1) / unit * unit;
    splits = (max_kv + chunk - 1) / chunk;
  }
  s.chunk = chunk;
  s.splits = splits < 1 ? 1 : splits;
  s.units = units * s.splits;
  s.part_rows = s.splits > 1 ? static_cast<int64_t>(R) * max_new * Hq * s.splits : 0;   // at most 1184 x 256
  return s;
}

template <int D>
static cudaError_t launch_rows(const PagedParams& p, const SplitParams& sp, const SplitPlan& s, cudaStream_t stream) {
  cudaError_t e;
  if (s.tc) {
    e = launch_paged_tc(p, sp, D, s.units, stream);
  } else {
    if (s.nt == 1) paged_small_kernel<D, 1><<<static_cast<unsigned>(s.units), kSmallWarps * 32, 0, stream>>>(p, sp);
    else paged_small_kernel<D, 2><<<static_cast<unsigned>(s.units), kSmallWarps * 32, 0, stream>>>(p, sp);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || s.splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(p.R) * p.max_new * p.Hq;
  // started while the last parts are still being made: it looks up its rows and then waits for their end
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D>, p, sp);
}

cudaError_t launch_paged(const PagedParams& p, const SplitPlan& s, void* part, int d, cudaStream_t stream) {
  SplitParams sp{};
  sp.chunk = s.chunk;
  sp.splits = static_cast<uint32_t>(s.splits);
  sp.row_tiles = static_cast<uint32_t>(s.row_tiles);
  sp.part_o = static_cast<float*>(part);
  sp.part_lse = sp.part_o + s.part_rows * d;
  return d == 128 ? launch_rows<128>(p, sp, s, stream) : launch_rows<64>(p, sp, s, stream);
}

}  // namespace mxattn
