// Append to the paged 8-bit KV cache: new keys and values quantised into their
// pages, one scale per page and head.
//
// One CTA per (page that new tokens fall into, head, K or V): the new values
// are read once and stay in registers (at most T D = 16384 of them, 64 per
// thread) across the maximum, taken on their bit patterns, and the rounding.  A page that already holds
// tokens keeps the larger of its scale and the one that the new tokens need;
// where it grows, the earlier codes are rounded anew (each page sees that a few
// times while it fills: the maximum of a growing set rises ever more rarely).
//
// Measured: 26.6 k tokens x 8 heads x 128, bf16 -> e4m3, 31 us: 0.78 of the HBM copy rate (the stream, and
// 15 instructions a value before the types were separated and e4m3 went by magnitude: 34 us; IEEE
// divisions: 77).  One token of 32 sequences: 5 us, a launch and two dependent loads.
#include "kvb_append.cuh"

namespace w4 {
namespace kvb {

template <int FMT, bool BF16, int VECS>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams P) {
  __shared__ uint32_t warp_max[kAppendThreads / 32];
  const View& V = P.V;
  const int b = blockIdx.z, h = blockIdx.y, sel = blockIdx.x & 1, tid = threadIdx.x;
  const Span s = span(V, b);
  const int T = 1 << V.t_shift;
  const int first = max(s.old, 0);
  const int blk = (first >> V.t_shift) + (int)(blockIdx.x >> 1);
  const int begin = blk << V.t_shift;
  if (blk >= V.table_stride) return;
  const int lo = max(first, begin), hi = min(s.old + s.n, begin + T);
  if (lo >= hi) return;
  if (sel == 0 && P.w)
    for (int t = lo + tid; t < hi && t < P.w_stride; t += kAppendThreads)
      P.w[((size_t)b * V.Hkv + h) * P.w_stride + t] = 0.f;
  const int page = page_of(V, V.table, b, V.table_stride, blk);
  if (page < 0) return;

  append_page<FMT, BF16, VECS>(V, s, h, page, begin, lo, hi, P.x[sel], P.stride[sel], P.d_shift, sel ? V.v : V.k,
                               sel ? V.vs : V.ks, warp_max);
}

template <int FMT, bool BF16>
void launch_append(const AppendParams& P, dim3 grid, int vecs, cudaStream_t s) {
  if (vecs <= 1)
    append_kernel<FMT, BF16, 1><<<grid, kAppendThreads, 0, s>>>(P);
  else if (vecs <= 2)
    append_kernel<FMT, BF16, 2><<<grid, kAppendThreads, 0, s>>>(P);
  else if (vecs <= 4)
    append_kernel<FMT, BF16, 4><<<grid, kAppendThreads, 0, s>>>(P);
  else
    append_kernel<FMT, BF16, 8><<<grid, kAppendThreads, 0, s>>>(P);
}

}  // namespace kvb
}  // namespace w4

using namespace w4;
using namespace w4::kvb;

extern "C" tm_status tm_kvb_append(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Kn,
                                   long long k_stride, const void* Vn, long long v_stride, int dtype, float* w,
                                   long long w_stride, void* stream) {
  AppendParams P;
  const tm_status st = check(cache, batch, true, &P.V);
  if (st != TM_OK) return st;
  if (dtype != TM_KVB_F16 && dtype != TM_KVB_BF16) return TM_ERR_INVALID_ARG;
  if (!batch->q_start && (batch->rows != batch->B || (batch->B > 0 && batch->max_q < 1))) return TM_ERR_INVALID_ARG;
  const View& V = P.V;
  if (V.B == 0 || V.rows == 0 || V.max_q == 0 || V.table_stride == 0) return TM_OK;
  const long long width = (long long)cache->Hkv * cache->D;
  if (!Kn || !Vn || k_stride < width || v_stride < width || w_stride < 0) return TM_ERR_INVALID_ARG;
  if (!aligned(Kn, 16) || !aligned(Vn, 16) || k_stride % 8 || v_stride % 8 || !aligned(w, 4)) return TM_ERR_ALIGNMENT;
  P.x[0] = static_cast<const uint16_t*>(Kn);
  P.x[1] = static_cast<const uint16_t*>(Vn);
  P.stride[0] = k_stride;
  P.stride[1] = v_stride;
  P.d_shift = cache->D == 64 ? 6 : 7;
  P.w = w;
  P.w_stride = w_stride;
  const dim3 grid((unsigned)(2 * append_pages(V)), (unsigned)V.Hkv, (unsigned)V.B);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int vecs = ((cache->T < V.max_q ? cache->T : V.max_q) * cache->D / 8 + kAppendThreads - 1) / kAppendThreads;
  const bool bf16 = dtype == TM_KVB_BF16;
  if (cache->format == TM_KVB_INT8)
    bf16 ? launch_append<TM_KVB_INT8, true>(P, grid, vecs, s) : launch_append<TM_KVB_INT8, false>(P, grid, vecs, s);
  else
    bf16 ? launch_append<TM_KVB_E4M3, true>(P, grid, vecs, s) : launch_append<TM_KVB_E4M3, false>(P, grid, vecs, s);
  if (cudaGetLastError() != cudaSuccess) return TM_ERR_CUDA;
  set_launch_count(1);
  return TM_OK;
}
