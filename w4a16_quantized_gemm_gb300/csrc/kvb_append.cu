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
#include <type_traits>

#include "kvb_common.cuh"

namespace w4 {
namespace kvb {

constexpr int kAppendThreads = 256;

struct AppendParams {
  View V;
  const uint16_t* x[2];  // keys, values
  long long stride[2];   // elements per token
  int d_shift;           // log2 D
  float* w;
  long long w_stride;
};

// NaN to 0, infinities to the type's largest finite value.
__device__ __forceinline__ float finite(float x, float top) {
  return x != x ? 0.f : fminf(fmaxf(x, -top), top);
}

// Codes of the four values of two words.  CLEAN: none is an infinity or NaN.
// e4m3 goes by magnitude: the signs are the high bits of the four high bytes.
template <int FMT, bool BF16, bool CLEAN>
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, const Divisor& by, float top) {
  const uint32_t signs = FMT == TM_KVB_E4M3 ? prmt(a, b, 0x7531u) & 0x80808080u : 0u;
  if (FMT == TM_KVB_E4M3) {
    a &= 0x7fff7fffu;
    b &= 0x7fff7fffu;
  }
  float2 x = unpack(a, BF16), y = unpack(b, BF16);
  if (!CLEAN) {
    x = make_float2(finite(x.x, top), finite(x.y, top));
    y = make_float2(finite(y.x, top), finite(y.y, top));
  }
  if (FMT == TM_KVB_INT8) return encode4<FMT>(f32x2(x.x, x.y), f32x2(y.x, y.y), by);
  return e4m3x4(f32x2_get(divide(f32x2(x.x, x.y), by)), f32x2_get(divide(f32x2(y.x, y.y), by))) | signs;
}

// VECS: vectors of 8 values per thread, enough for the new tokens of one page.
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

  const int vec_shift = P.d_shift - 3;  // vectors of 8 values per token
  const int total = (hi - lo) << vec_shift;
  const uint16_t* src = P.x[sel] + (s.row0 + (long long)(lo - s.old)) * P.stride[sel] + ((long long)h << P.d_shift);
  const float top = BF16 ? 3.3895313892515355e38f : 65504.f;
  uint4 x[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int v = tid + i * kAppendThreads;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < total)
      x[i] = *reinterpret_cast<const uint4*>(src + (v >> vec_shift) * P.stride[sel] +
                                             ((v & ((1 << vec_shift) - 1)) << 3));
  }
  // The largest magnitude as a bit pattern: those of 16-bit floats are ordered, and the pattern
  // of an infinity or NaN tells whether any value needs cleaning.
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    m2 = __vmaxu2(m2, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu));
    m2 = __vmaxu2(m2, __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
  if ((tid & 31) == 0) warp_max[tid >> 5] = m;
  const size_t cell = (size_t)page * V.Hkv + h;
  float* scale = (sel ? V.vs : V.ks) + cell;
  const bool continued = s.old > begin;
  const float was = continued ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) m = max(m, warp_max[i]);
  const bool clean = m < (BF16 ? 0x7f80u : 0x7c00u);
  float a = unpack(m, BF16).x;
  if (!clean) {  // uniform: the largest finite magnitude, an infinity counting as `top`
    float f = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const uint32_t wd[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = unpack(wd[k], BF16);
        f = fmaxf(f, fmaxf(fabsf(finite(v.x, top)), fabsf(finite(v.y, top))));
      }
    }
    m = __reduce_max_sync(0xffffffffu, __float_as_uint(f));
    __syncthreads();
    if ((tid & 31) == 0) warp_max[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) m = max(m, warp_max[i]);
    a = __uint_as_float(m);
  }
  const float now = fmaxf(scale_for<FMT>(a), was);
  const Divisor by = divisor(now);
  if (tid == 0) *scale = now;

  uint8_t* codes = (sel ? V.v : V.k) + ((cell << V.t_shift) << P.d_shift);
  uint8_t* dst = codes + ((size_t)(lo - begin) << P.d_shift);
  auto store = [&](auto is_clean) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int v = tid + i * kAppendThreads;
      if (v >= total) break;
      uint2 c;
      c.x = codes4<FMT, BF16, decltype(is_clean)::value>(x[i].x, x[i].y, by, top);
      c.y = codes4<FMT, BF16, decltype(is_clean)::value>(x[i].z, x[i].w, by, top);
      *reinterpret_cast<uint2*>(dst + ((size_t)v << 3)) = c;
    }
  };
  if (clean)
    store(std::true_type{});
  else
    store(std::false_type{});
  if (continued && now > was) {
    const int earlier = (lo - begin) << vec_shift;
    const uint64_t was2 = f32x2(was, was);
    for (int v = tid; v < earlier; v += kAppendThreads) {
      uint2* at = reinterpret_cast<uint2*>(codes + ((size_t)v << 3));
      uint2 c = *at;
      c.x = recode4<FMT>(c.x, was2, by);
      c.y = recode4<FMT>(c.y, was2, by);
      *at = c;
    }
  }
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
  // Pages that max_q consecutive tokens can touch.
  const long long pages = ((long long)V.max_q + cache->T - 2) / cache->T + 1;
  const dim3 grid((unsigned)(2 * pages), (unsigned)V.Hkv, (unsigned)V.B);
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
