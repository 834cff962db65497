// What the kernels that append to the paged 8-bit KV cache share: the codes of 16-bit values, and the
// quantisation of one head's new values into one page.
#pragma once

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

// One CTA of THREADS: the tokens of slots lo .. hi - 1 (all in the page of slots begin ..) of head h into
// `pool`.  VECS: vectors of 8 values per thread, enough for the new tokens of one page.
template <int FMT, bool BF16, int VECS, int THREADS = kAppendThreads>
__device__ __forceinline__ void append_page(const View& V, const Span& s, int h, int page, int begin, int lo, int hi,
                                            const uint16_t* x_in, long long stride, int d_shift, uint8_t* pool,
                                            float* scales, uint32_t* warp_max) {
  const int tid = threadIdx.x;
  const int vec_shift = d_shift - 3;  // vectors of 8 values per token
  const int total = (hi - lo) << vec_shift;
  const uint16_t* src = x_in + (s.row0 + (long long)(lo - s.old)) * stride + ((long long)h << d_shift);
  const float top = BF16 ? 3.3895313892515355e38f : 65504.f;
  uint4 x[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int v = tid + i * THREADS;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < total)
      x[i] = *reinterpret_cast<const uint4*>(src + (v >> vec_shift) * stride +
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
  float* scale = scales + cell;
  const bool continued = s.old > begin;
  const float was = continued ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) m = max(m, warp_max[i]);
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
    for (int i = 0; i < THREADS / 32; ++i) m = max(m, warp_max[i]);
    a = __uint_as_float(m);
  }
  const float now = fmaxf(scale_for<FMT>(a), was);
  const Divisor by = divisor(now);
  if (tid == 0) *scale = now;

  uint8_t* codes = pool + ((cell << V.t_shift) << d_shift);
  uint8_t* dst = codes + ((size_t)(lo - begin) << d_shift);
  auto store = [&](auto is_clean) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int v = tid + i * THREADS;
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
    for (int v = tid; v < earlier; v += THREADS) {
      uint2* at = reinterpret_cast<uint2*>(codes + ((size_t)v << 3));
      uint2 c = *at;
      c.x = recode4<FMT>(c.x, was2, by);
      c.y = recode4<FMT>(c.y, was2, by);
      *at = c;
    }
  }
}

// Pages that max_q consecutive tokens can touch.
inline long long append_pages(const View& V) {
  const long long T = 1ll << V.t_shift;
  return ((long long)V.max_q + T - 2) / T + 1;
}

}  // namespace kvb
}  // namespace w4
