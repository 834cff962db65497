// Parameters shared by the kernels of the paged cache's attention.
#pragma once

#include "kvb_common.cuh"

namespace w4 {
namespace kvb {

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
  float* part;        // [rows][Hq][chunks][D]
  float2* part_ml;    // [rows][Hq][chunks]: m, l
  float* scores;      // [rows][Hq][score_stride], base-2 logarithms of the unnormalised weights
  long long score_stride;
};

// The tcgen05 kernel (kvb_prefill.cu): `pairs` pairs of 128-row tiles per
// (sequence, KV head); slices of P.chunk tokens, a multiple of 128.
tm_status launch_prefill_attn(const AttnParams& P, int format, int D, int pairs, cudaStream_t stream);

}  // namespace kvb
}  // namespace w4
