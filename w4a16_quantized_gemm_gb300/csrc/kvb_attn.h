// Parameters shared by the kernels of the paged cache's attention.
#pragma once

#include "kvb_common.cuh"

namespace w4 {
namespace kvb {

constexpr int kFewRows = 64;  // most rows per (sequence, KV head) of the kernel for few rows (without weights, and of
                              // trees: half)

struct AttnParams {
  View V;
  const uint16_t* Q;
  long long q_stride;
  int Hq, G, bf16;
  float scale_log2;  // scale of the scores times log2(e)
  uint16_t* out;
  float* lse;
  const float* w_in;
  float* w_out;
  long long w_stride;
  int chunk, chunks;  // tokens per slice, slices (by max_len)
  int rows_per_cta;   // rows that share a CTA, and with it their slices
  int wpr;            // warps per row of the joining launch
  int split;          // CTAs that share a token tile's rows (kvb_weights.cu)
  float* part;        // [rows][Hq][chunks][D]
  float2* part_ml;    // [rows][Hq][chunks]: m, l
  float* scores;      // [Hkv][rows x G][score_stride], base-2 logarithms of the unnormalised weights
  long long score_stride;
  // A tree's masks, [rows][tree_stride] words of which the first tree_words count; NULL: causal.
  const uint32_t* tree;
  long long tree_stride;
  int tree_words;
};

// The tcgen05 kernel (kvb_prefill.cu): `pairs` pairs of 128-row tiles per
// (sequence, KV head); slices of P.chunk tokens, a multiple of 128.
tm_status launch_prefill_attn(const AttnParams& P, int format, int D, int pairs, cudaStream_t stream);

// The same for trees of up to 128 rows a KV head (kvb_tree.cu).
tm_status launch_tree_attn(const AttnParams& P, int format, int D, cudaStream_t stream);

// The weights that tokens drew from many rows, by their lse (kvb_weights.cu).
tm_status launch_row_weights(const AttnParams& P, int format, int D, cudaStream_t stream);

// Slices of `tiles` token tiles, each in a CTA of its own, for which waves of CTAs x (tiles of a slice + what starting
// one costs) is the least; `join` for joining several.  None shorter than four tiles, at most `most`.
inline long long slices_by_waves(long long ctas, long long tiles, int start, int join, long long most) {
  const long long sms = num_sms(current_device());
  long long best = 1, cost = -1;
  for (long long c = 1; c == 1 || (c <= most && tiles / c >= 4); ++c) {
    const long long t = (ctas * c + sms - 1) / sms * ((tiles + c - 1) / c + start) + (c > 1 ? join : 0);
    if (cost < 0 || t < cost) {
      best = c;
      cost = t;
    }
  }
  return best;
}

#if defined(__CUDACC__)
// What a tree's row sees of 32 tokens: bit x stands for new token `first` + x (below 0: a token before the tree).
__device__ __forceinline__ uint32_t tree_bits(const AttnParams& P, const uint32_t* mask, int first) {
  const int at = first >> 5;  // rounds down
  auto word = [&](int k) { return k < 0 ? 0xffffffffu : k < P.tree_words ? mask[k] : 0u; };
  return __funnelshift_r(word(at), word(at + 1), first & 31);
}

// What a tree's row sees of columns 32 c .. 32 c + 31 of a token tile: up to column `rel`, without holes (a bit per
// 16 columns), and of the new tokens, of which the tile's first is number `fresh`, those in its mask.
__device__ __forceinline__ uint32_t tree_columns(const AttnParams& P, const uint32_t* mask, int fresh, int rel,
                                                 uint32_t holes, int c) {
  const int x = rel - 32 * c;
  uint32_t see = x >= 31 ? 0xffffffffu : x < 0 ? 0u : (2u << x) - 1u;
  if ((holes >> (2 * c)) & 1u) see &= 0xffff0000u;
  if ((holes >> (2 * c)) & 2u) see &= 0x0000ffffu;
  if (fresh + 32 * c + 32 > 0 && x >= 0) see &= tree_bits(P, mask, fresh + 32 * c);
  return see;
}

// mbar_wait with a spin before the timer comes in.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, err);
}

// One lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}

// The framework's products and commits with a predicate in place of a branch:
// a converged warp computes the operands (they stay in uniform registers: under
// `if (lane == 0)` each product took 50 to 75 cycles to issue), one lane issues.
__device__ __forceinline__ void mma_ss_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// MN-major operand: rows of K (tokens) of 128 bytes, 128-byte swizzle, 8-row
// atoms 1024 bytes apart along K, 64-element panels `panel` bytes apart along N.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// 16 bytes, or zeros.
__device__ __forceinline__ uint4 ldg_or_zero(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)ok));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// Into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// One warp: pages and scales of the 16-token groups of N token tiles of 128 (from token j0 on, up to j1), a slot of
// META [SLOTS][8] x {ks, log2 vs, 1 / vs, group of the pool} and one of HOLES (bits) for each.  A page's number, then its
// scales: two loads that wait for each other, so that lane 8 i + g takes group g of tile i of four tiles at once, the
// scales four tiles ahead and the numbers eight (tile by tile they cost 3.2 k cycles each, more than all the rest of
// a tile of 128 rows).  The codes are requested into L2 on the way, four tiles ahead.
template <int D, int SLOTS>
__device__ __forceinline__ void publish_pages(const View& V, int b, int h, int j0, int j1, int N, uint32_t meta,
                                              uint32_t holes_at, uint32_t full, uint32_t empty,
                                              volatile int* abort_flag, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  const int* table = V.table + (size_t)b * V.table_stride;
  auto token = [&](int n) { return j0 + n * 128 + 16 * lane; };  // the lane's of tiles n .. n + 3
  auto entry = [&](int n) { return token(n) < j1 ? table[token(n) >> V.t_shift] : -1; };
  struct Group {
    float ks, vs;
    uint32_t at;
    bool hole;
  };
  auto scales = [&](int n, int page) {
    const int j = token(n);
    const bool there = (unsigned)page < (unsigned)V.pages && j < j1;
    Group g = {1.f, 1.f, 0xffffffffu, j < j1 && !there};
    if (there) {
      const size_t cell = (size_t)page * V.Hkv + h;
      g.at = (uint32_t)(((cell << V.t_shift) + (j & ((1 << V.t_shift) - 1))) >> 4);
      g.ks = V.ks[cell];
      g.vs = V.vs[cell];
    }
    return g;
  };
  // A page at a time: each of these copies takes its thread about 60 cycles.
  auto request = [&](int n, const Group& g) {
    if (g.at != 0xffffffffu && (token(n) & ((1 << V.t_shift) - 1)) == 0) {
      prefetch_l2(V.k + (size_t)g.at * (16 * D), D << V.t_shift);
      prefetch_l2(V.v + (size_t)g.at * (16 * D), D << V.t_shift);
    }
  };
  int page = entry(0);
  Group next = scales(0, page);
  page = entry(4);
#pragma unroll 1
  for (int n0 = 0; n0 < N; n0 += 4) {
    const Group g = next;
    next = scales(n0 + 4, page);  // past the end: nothing
    page = entry(n0 + 8);
    const float lv = __log2f(fmaxf(g.vs, kScaleFloor)), inv = ex2(-lv);
    const uint32_t holes = __ballot_sync(0xffffffffu, g.hole);
#pragma unroll 1
    for (int n = n0; n < N && n < n0 + 4; ++n) {
      const int slot = n % SLOTS;
      const bool alive = wait_bar(empty + 8 * slot, ((uint32_t)(n / SLOTS) & 1u) ^ 1u, abort_flag, err);
      if (!__all_sync(0xffffffffu, alive)) return;
      if (lane >> 3 == n - n0)
        sts128(meta + slot * 128 + (lane & 7) * 16, __float_as_uint(g.ks), __float_as_uint(lv), __float_as_uint(inv), g.at);
      if (lane == 0)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(holes_at + 4 * slot), "r"((holes >> (8 * (n - n0))) & 0xffu) : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * slot);
      if (lane >> 3 == n - n0) request(n0 + 4, next);
      __syncwarp();
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// tcgen05.wait::ld for a load into r: what reads r stays behind the wait.
__device__ __forceinline__ void tc_wait_ld_of(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Tensor memory: 32 lanes x 32 consecutive 32-bit columns, thread i to lane (base lane + i).
__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 lanes x 16 columns.
__device__ __forceinline__ void tc_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
#endif

}  // namespace kvb
}  // namespace w4
