// Shared pieces of the paged 8-bit KV cache (one scale per page and head):
// argument checks, the codes' conversions and asynchronous copies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "../../include/tm_kvb.h"
#include "tm_common.cuh"

namespace w4 {
namespace kvb {

constexpr float kScaleFloor = 9.31322574615478515625e-10f;  // 2^-30

// What a kernel needs of a cache and a batch.
struct View {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int* table;
  const int* kv_len;
  const int* q_start;
  int pages, Hkv, t_shift;  // T = 1 << t_shift
  int B, table_stride, max_q, max_len;
  int rows;
};

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Host checks that every call shares; fills `view`.  `pointers`: the device
// fields are checked too.
inline tm_status check(const tm_kvb_cache* c, const tm_kvb_batch* b, bool pointers, View* view) {
  if (!c || !b) return TM_ERR_INVALID_ARG;
  if (c->pages < 0 || c->Hkv < 1 || c->Hkv > 65535 || (c->T != 16 && c->T != 32 && c->T != 64 && c->T != 128) ||
      (c->D != 64 && c->D != 128) || (c->format != TM_KVB_INT8 && c->format != TM_KVB_E4M3))
    return TM_ERR_INVALID_ARG;
  if (b->B < 0 || b->B > 65535 || b->table_stride < 0 || b->max_q < 0 || b->max_len < 0 || b->rows < 0)
    return TM_ERR_INVALID_ARG;
  // Row and token indices are 32-bit in the kernels; products with sizes are 64-bit.
  const long long room = (long long)b->table_stride * c->T;
  if (room > 0x40000000ll || b->rows > 0x7fffff00ll || (long long)c->pages * c->Hkv > 0x7fffffffll)
    return TM_ERR_UNSUPPORTED;
  if (b->B > 0 && pointers) {
    if (!c->k || !c->v || !c->ks || !c->vs || !b->table || !b->kv_len) return TM_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->ks, 4) || !aligned(c->vs, 4) ||
        !aligned(b->table, 4) || !aligned(b->kv_len, 4) || !aligned(b->q_start, 4))
      return TM_ERR_ALIGNMENT;
  }
  int shift = 4;
  while ((1 << shift) < c->T) ++shift;
  long long len = b->max_len > 0 ? b->max_len : room;
  if (len > room) len = room;
  *view = {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->ks, c->vs, b->table, b->kv_len, b->q_start,
           c->pages, c->Hkv, shift, b->B, b->table_stride, b->max_q, (int)len, (int)b->rows};
  return TM_OK;
}

#if defined(__CUDACC__)

// Sequence b: its tokens, those that the call may read, its first row, the
// rows that the call computes, and the position of the first of them.
struct Span {
  int raw, len, row0, n, old;
};
__device__ __forceinline__ Span span(const View& V, int b) {
  Span s;
  s.raw = max(V.kv_len[b], 0);
  s.len = min(s.raw, V.max_len);
  const int lo = V.q_start ? min(max(V.q_start[b], 0), V.rows) : b;
  const int hi = V.q_start ? min(max(V.q_start[b + 1], 0), V.rows) : b + 1;
  s.row0 = lo;
  s.old = s.raw - max(hi - lo, 0);
  s.n = min(max(hi - lo, 0), V.max_q);
  return s;
}
// The page of block `blk`, or -1 for a hole.
__device__ __forceinline__ int page_of(const View& V, const int* table, int b, int stride, int blk) {
  const int p = table[(size_t)b * stride + blk];
  return (unsigned)p < (unsigned)V.pages ? p : -1;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Two e4m3 codes (low and high byte of a 16-bit word) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

// Four codes of a word as fp16 pairs (bytes 0, 1) and (2, 3), exactly.  int8:
// the byte with its sign bit flipped is b + 128; OR-ed into the mantissa of
// 1024.0 it gives 1152 + b.
template <int FMT>
__device__ __forceinline__ void codes_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == TM_KVB_INT8) {
    const uint32_t x = w ^ 0x80808080u;
    lo = hsub2_u32(prmt(x, 0x64646464u, 0x4140u), 0x64806480u);
    hi = hsub2_u32(prmt(x, 0x64646464u, 0x4342u), 0x64806480u);
  } else {
    lo = e4m3x2_half2((uint16_t)w);
    hi = e4m3x2_half2((uint16_t)(w >> 16));
  }
}

// Codes of two words as four fp16 pairs (byte i of a, byte i of b).
template <int FMT>
__device__ __forceinline__ void codes_half_pairs(uint32_t a, uint32_t b, uint32_t (&out)[4]) {
  codes_half<FMT>(prmt(a, b, 0x5140u), out[0], out[1]);
  codes_half<FMT>(prmt(a, b, 0x7362u), out[2], out[3]);
}

// Packed pairs of binary32 (one instruction for two).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 f32x2_get(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Four codes of a word as binary32, exactly, in two pairs.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, uint64_t& lo, uint64_t& hi) {
  uint32_t a, b;
  codes_half<FMT>(w, a, b);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  lo = f32x2(x.x, x.y);
  hi = f32x2(y.x, y.y);
}

// Division by a scale of many values: t = x i with i the rounded reciprocal,
// then one correction by the remainder x - t s (Markstein's), which gives the
// rounded quotient that the codes are defined by (the rounding to a code could
// only see a miss next to a tie, where the remainder decides).
struct Divisor {
  uint64_t s, i;
};
__device__ __forceinline__ Divisor divisor(float s) {
  const float i = __frcp_rn(s);
  return {f32x2(-s, -s), f32x2(i, i)};
}
__device__ __forceinline__ uint64_t divide(uint64_t x, const Divisor& d) {
  const uint64_t t = mul_f32x2(x, d.i);
  return fma_f32x2(fma_f32x2(t, d.s, x), d.i, t);
}

// To the nearest e4m3 codes, ties to even, saturating.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
}

// Codes of four quotients x / s with |x| at most the largest code times s (to
// its rounding): to the nearest, ties to even.  int8: adding 1.5 2^23 leaves the
// rounded integer in the low byte.  e4m3: of magnitudes (the correction loses a zero's sign).
template <int FMT>
__device__ __forceinline__ uint32_t encode4(uint64_t lo, uint64_t hi, const Divisor& d) {
  const uint64_t ql = divide(lo, d), qh = divide(hi, d);
  if (FMT == TM_KVB_INT8) {
    const uint64_t magic = f32x2(12582912.f, 12582912.f);
    const float2 a = f32x2_get(add_f32x2(ql, magic)), b = f32x2_get(add_f32x2(qh, magic));
    return prmt(prmt(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040u),
                prmt(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040u), 0x5410u);
  }
  return e4m3x4(f32x2_get(ql), f32x2_get(qh));
}

// Codes of (c s) / s' for the four codes c of a word: a page's new scale.  e4m3
// goes by magnitude, the signs stay.
template <int FMT>
__device__ __forceinline__ uint32_t recode4(uint32_t w, uint64_t s, const Divisor& d) {
  uint64_t lo, hi;
  decode4<FMT>(FMT == TM_KVB_INT8 ? w : w & 0x7f7f7f7fu, lo, hi);
  if (FMT == TM_KVB_INT8) return encode4<FMT>(mul_f32x2(lo, s), mul_f32x2(hi, s), d);
  const float2 a = f32x2_get(divide(mul_f32x2(lo, s), d)), b = f32x2_get(divide(mul_f32x2(hi, s), d));
  return e4m3x4(a, b) | (w & 0x80808080u);
}

// The scale that values up to `a` need: a times the binary32 reciprocal of the
// largest code, at least 2^-30.
template <int FMT>
__device__ __forceinline__ float scale_for(float a) {
  return fmaxf(__fmul_rn(a, FMT == TM_KVB_INT8 ? 1.f / 127.f : 1.f / 448.f), kScaleFloor);
}

// 16-byte asynchronous copy global -> shared; zeros where !ok.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

#endif  // __CUDACC__

}  // namespace kvb
}  // namespace w4
