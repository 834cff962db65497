// Parameters shared by the kernels of the paged cache's attention.
#pragma once

#include "kvb_common.cuh"

namespace w4 {
namespace kvb {

constexpr int kFewRows = 64;  // most rows per (sequence, KV head) of the kernel for few rows (without weights: half)

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

// The weights that tokens drew from many rows, by their lse (kvb_weights.cu).
tm_status launch_row_weights(const AttnParams& P, int format, int D, cudaStream_t stream);

#if defined(__CUDACC__)
// What a tree's row sees of 32 tokens: bit x stands for new token `first` + x (below 0: a token before the tree).
__device__ __forceinline__ uint32_t tree_bits(const AttnParams& P, const uint32_t* mask, int first) {
  const int at = first >> 5;  // rounds down
  auto word = [&](int k) { return k < 0 ? 0xffffffffu : k < P.tree_words ? mask[k] : 0u; };
  return __funnelshift_r(word(at), word(at + 1), first & 31);
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
#endif

}  // namespace kvb
}  // namespace w4
