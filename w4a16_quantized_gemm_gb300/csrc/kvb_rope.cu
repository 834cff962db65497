// Append to the paged 8-bit KV cache with the position rotation on the way: keys rotated and quantised into
// their pages, values quantised, queries rotated into a buffer, all in one launch.
//
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s
// in binary32, each product and each sum rounded (no fused multiply-add: the codes are then the same wherever they
// are computed).  Rotated keys are quantised from binary32, not from a 16-bit copy.
//
// One CTA per (page that new tokens fall into, KV head, role): keys, values as in the append without rotation, and the
// query heads of the group.  A thread works on units of 16 dimensions: two vectors of 8 that hold both halves of their
// pairs.  The rotated keys stay in registers (at most 64 a thread) across the maximum and the rounding.
//
// Bound by memory.  Measured: 26.6 k tokens, bf16, 32 query heads, 8 KV heads of 128 to e4m3: 99.6 us for 600 MB, 0.89 of
// the HBM copy rate (queries in the keys' CTAs of 256 threads, which then are two per SM: 141 us).  One token of 32
// sequences: 2.5 us, a launch and three dependent loads.
#include "kvb_append.cuh"

namespace w4 {
namespace kvb {

struct RopeParams {
  AppendParams A;
  const uint16_t* Q;
  uint16_t* q_out;
  long long q_stride, qo_stride;
  int G;
  const float* table;
  const int* pos;
  int positions, dims;
  int roles;  // CTAs of a page and KV head: keys, values, and queries where there are any
};

__device__ __forceinline__ void unpack8(const uint4& v, bool bf16, float* y) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack(w[k], bf16);
    y[2 * k] = f.x;
    y[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* y, bool bf16) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = bf16 ? pack_bf162(y[2 * k], y[2 * k + 1]) : pack_half2(y[2 * k], y[2 * k + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(const float* p, float* y) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w;
  y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}
// The 8 pairs of a unit: (y[e], y[8 + e]), or neighbours.
template <bool INTER>
__device__ __forceinline__ void turn16(float* y, const float* c, const float* s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (INTER)
      turn(y[2 * e], y[2 * e + 1], c[e], s[e]);
    else
      turn(y[e], y[8 + e], c[e], s[e]);
  }
}

// Codes of four finite values of at most the largest code times the scale.
template <int FMT>
__device__ __forceinline__ uint32_t codes_of(const float* y, const Divisor& by) {
  if (FMT == TM_KVB_INT8) return encode4<FMT>(f32x2(y[0], y[1]), f32x2(y[2], y[3]), by);
  const uint32_t signs = prmt(prmt(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x0073u),
                              prmt(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x0073u), 0x5410u) & 0x80808080u;
  return e4m3x4(f32x2_get(divide(f32x2(fabsf(y[0]), fabsf(y[1])), by)),
                f32x2_get(divide(f32x2(fabsf(y[2]), fabsf(y[3])), by))) | signs;
}

// UNITS: units of 16 dimensions per thread, enough for the new tokens of one page and head.
template <int FMT, bool BF16, int UNITS, bool INTER, int THREADS>
__global__ void __launch_bounds__(THREADS, (UNITS == 4 ? 2 : 3) * 256 / THREADS) append_rope_kernel(const RopeParams R) {
  __shared__ uint32_t warp_max[THREADS / 32];
  const AppendParams& P = R.A;
  const View& V = P.V;
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int nth = (int)(blockIdx.x / R.roles), role = (int)blockIdx.x - nth * R.roles;
  const Span s = span(V, b);
  const int T = 1 << V.t_shift;
  // Pages by slot; queries of rows without one (more rows than tokens: negative slots) are rotated all the same.
  const int end = s.old + s.n, pages = ((end - 1) >> V.t_shift) - (s.old >> V.t_shift);
  if (s.n == 0 || nth > pages) return;
  const int blk = (s.old >> V.t_shift) + nth;
  const int begin = blk * T;
  const int lo = max(s.old, begin), hi = nth == pages ? end : begin + T;  // lengths reach 2^31 - 1
  const int D = 1 << P.d_shift, unit_shift = P.d_shift - 4;
  const int total = (hi - lo) << unit_shift;
  const int turning = R.dims >> 4;  // units of a token that rotate
  // The first element of a unit's two vectors.
  auto places = [&](int p, int& d0, int& d1) {
    const bool halves = !INTER && p < turning;
    d0 = halves ? 8 * p : 16 * p;
    d1 = halves ? 8 * p + (R.dims >> 1) : 16 * p + 8;
  };
  auto angles = [&](long long row, int t, int p, float* c, float* sn) {
    const int at = min(max(R.pos ? R.pos[row] : t, 0), R.positions - 1);
    const float* cs = R.table + (size_t)at * R.dims + 8 * p;
    load8(cs, c);
    load8(cs + (R.dims >> 1), sn);
  };

  if (role == 2) {  // ---- queries: four heads of the group, so that angles serve them together
    const int fours = (R.G + 3) >> 2;
    for (int i = tid; i < total * fours; i += THREADS) {
      const int u = i / fours, g0 = 4 * (i - u * fours);
      const int t = lo + (u >> unit_shift), p = u & ((1 << unit_shift) - 1);
      const long long row = s.row0 + (long long)(t - s.old);
      int d0, d1;
      places(p, d0, d1);
      const uint16_t* src = R.Q + row * R.q_stride + (long long)(h * R.G + g0) * D;
      uint16_t* dst = R.q_out + row * R.qo_stride + (long long)(h * R.G + g0) * D;
      uint4 a[4], z[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (g0 + g < R.G) {
          a[g] = *reinterpret_cast<const uint4*>(src + g * D + d0);
          z[g] = *reinterpret_cast<const uint4*>(src + g * D + d1);
        }
      float c[8], sn[8];
      if (p < turning) angles(row, t, p, c, sn);
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (g0 + g < R.G) {
          if (p < turning) {
            float q[16];
            unpack8(a[g], BF16, q);
            unpack8(z[g], BF16, q + 8);
            turn16<INTER>(q, c, sn);
            a[g] = pack8(q, BF16);
            z[g] = pack8(q + 8, BF16);
          }
          *reinterpret_cast<uint4*>(dst + g * D + d0) = a[g];
          *reinterpret_cast<uint4*>(dst + g * D + d1) = z[g];
        }
    }
    return;
  }

  const bool slots = blk >= 0 && blk < V.table_stride;
  const int page = slots ? page_of(V, V.table, b, V.table_stride, blk) : -1;
  if (role == 1) {  // ---- values
    if (P.w && slots)
      for (int t = lo + tid; t < hi && t < P.w_stride; t += THREADS)
        P.w[((size_t)b * V.Hkv + h) * P.w_stride + t] = 0.f;
    if (page >= 0)
      append_page<FMT, BF16, 2 * UNITS, THREADS>(V, s, h, page, begin, lo, hi, P.x[1], P.stride[1], P.d_shift, V.v, V.vs, warp_max);
    return;
  }

  // ---- keys
  if (page < 0) return;  // a hole takes none
  const float top = BF16 ? 3.3895313892515355e38f : 65504.f;
  const uint16_t* keys = P.x[0] + (long long)h * D;
  float y[UNITS][16];
  // The rotated keys; clean: NaN and infinities replaced before and after.
  auto fetch = [&](int i, auto clean) {
    const int u = tid + i * THREADS;
#pragma unroll
    for (int e = 0; e < 16; ++e) y[i][e] = 0.f;
    if (u >= total) return;
    const int t = lo + (u >> unit_shift), p = u & ((1 << unit_shift) - 1);
    const long long row = s.row0 + (long long)(t - s.old);
    int d0, d1;
    places(p, d0, d1);
    const uint16_t* src = keys + row * P.stride[0];
    const uint4 a = *reinterpret_cast<const uint4*>(src + d0), z = *reinterpret_cast<const uint4*>(src + d1);
    unpack8(a, BF16, y[i]);
    unpack8(z, BF16, y[i] + 8);
    if (decltype(clean)::value)
#pragma unroll
      for (int e = 0; e < 16; ++e) y[i][e] = finite(y[i][e], top);
    if (p < turning) {
      float c[8], sn[8];
      angles(row, t, p, c, sn);
      turn16<INTER>(y[i], c, sn);
    }
    if (decltype(clean)::value)
#pragma unroll
      for (int e = 0; e < 16; ++e) y[i][e] = finite(y[i][e], 3.40282347e38f);
  };
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    fetch(i, std::false_type{});
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(y[i][e]) & 0x7fffffffu);
  }
  auto join = [&](uint32_t v) {  // over the CTA
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((tid & 31) == 0) warp_max[tid >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) v = max(v, warp_max[i]);
    return v;
  };
  const size_t cell = (size_t)page * V.Hkv + h;
  float* scale = V.ks + cell;
  const bool continued = s.old > begin;
  const float was = continued ? *scale : 0.f;
  m = join(m);
  if (m >= 0x7f800000u) {  // uniform: an infinity or NaN somewhere
    m = 0u;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      fetch(i, std::true_type{});
#pragma unroll
      for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(y[i][e]) & 0x7fffffffu);
    }
    m = join(m);
  }
  const float now = fmaxf(scale_for<FMT>(__uint_as_float(m)), was);
  const Divisor by = divisor(now);
  if (tid == 0) *scale = now;
  uint8_t* codes = V.k + ((cell << V.t_shift) << P.d_shift);
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int u = tid + i * THREADS;
    if (u >= total) break;
    const int t = lo + (u >> unit_shift), p = u & ((1 << unit_shift) - 1);
    int d0, d1;
    places(p, d0, d1);
    uint8_t* dst = codes + ((size_t)(t - begin) << P.d_shift);
    *reinterpret_cast<uint2*>(dst + d0) = make_uint2(codes_of<FMT>(y[i], by), codes_of<FMT>(y[i] + 4, by));
    *reinterpret_cast<uint2*>(dst + d1) = make_uint2(codes_of<FMT>(y[i] + 8, by), codes_of<FMT>(y[i] + 12, by));
  }
  if (continued && now > was) {  // earlier codes of the page, rounded anew
    const int earlier = (lo - begin) << (P.d_shift - 3);
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

template <int FMT, bool BF16, bool INTER>
static void launch_rope(const RopeParams& P, dim3 grid, int units, cudaStream_t s) {
  // Where the CTAs do not all start at once, smaller ones keep more pages in flight: 64 threads for up to 128 units, 128
  // for up to 512.  Four prompts of 8191 tokens (512 units) 99.6 us (256 threads: 106.6); 16 k tokens, 32/8 heads, pages
  // of 64 units 32 (83), of 128 units 30 and 52 (49 and 90; 128 threads: 33 and 57); 46 x 519, 256 units 13.6 (16.1; 64
  // threads: 16.3); one token of each of 32 sequences 2.5 (4.1).  Else more threads are done earlier: 26 nodes of each of
  // 16, 32/4 heads of 64: 2.9 (128 threads: 3.5).
  constexpr int kHalf = kAppendThreads / 2, kQuarter = kAppendThreads / 4;
  const bool waves = (long long)grid.x * grid.y * grid.z > 3ll * num_sms(current_device());
  if (waves && units <= kQuarter)
    append_rope_kernel<FMT, BF16, 1, INTER, kQuarter><<<grid, kQuarter, 0, s>>>(P);
  else if (waves && units <= 2 * kQuarter)
    append_rope_kernel<FMT, BF16, 2, INTER, kQuarter><<<grid, kQuarter, 0, s>>>(P);
  else if (waves && units <= 2 * kHalf)
    append_rope_kernel<FMT, BF16, 2, INTER, kHalf><<<grid, kHalf, 0, s>>>(P);
  else if (waves && units <= 4 * kHalf)
    append_rope_kernel<FMT, BF16, 4, INTER, kHalf><<<grid, kHalf, 0, s>>>(P);
  else if (units <= kAppendThreads)
    append_rope_kernel<FMT, BF16, 1, INTER, kAppendThreads><<<grid, kAppendThreads, 0, s>>>(P);
  else if (units <= 2 * kAppendThreads)
    append_rope_kernel<FMT, BF16, 2, INTER, kAppendThreads><<<grid, kAppendThreads, 0, s>>>(P);
  else
    append_rope_kernel<FMT, BF16, 4, INTER, kAppendThreads><<<grid, kAppendThreads, 0, s>>>(P);
}

template <int FMT, bool BF16>
static void launch_rope(const RopeParams& P, dim3 grid, int units, bool interleaved, cudaStream_t s) {
  interleaved ? launch_rope<FMT, BF16, true>(P, grid, units, s) : launch_rope<FMT, BF16, false>(P, grid, units, s);
}

}  // namespace kvb
}  // namespace w4

using namespace w4;
using namespace w4::kvb;

extern "C" tm_status tm_kvb_append_rope(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Kn,
                                        long long k_stride, const void* Vn, long long v_stride, const void* Q,
                                        long long q_stride, int Hq, void* q_out, long long qo_stride,
                                        const tm_kvb_rope* rope, int dtype, float* w, long long w_stride,
                                        void* stream) {
  RopeParams P = {};
  const tm_status st = check(cache, batch, true, &P.A.V);
  if (st != TM_OK) return st;
  const int D = cache->D;
  if (dtype != TM_KVB_F16 && dtype != TM_KVB_BF16) return TM_ERR_INVALID_ARG;
  if (!batch->q_start && (batch->rows != batch->B || (batch->B > 0 && batch->max_q < 1))) return TM_ERR_INVALID_ARG;
  if (!rope || rope->positions < 1 || rope->dims < 16 || rope->dims > D || rope->dims % 16) return TM_ERR_INVALID_ARG;
  if (Q && (Hq < 1 || Hq % cache->Hkv)) return TM_ERR_INVALID_ARG;
  const View& V = P.A.V;
  if (V.B == 0 || V.rows == 0 || V.max_q == 0) return TM_OK;
  const long long width = (long long)cache->Hkv * D;
  if (!Kn || !Vn || !rope->table || k_stride < width || v_stride < width || w_stride < 0) return TM_ERR_INVALID_ARG;
  if (Q && (!q_out || q_stride < (long long)Hq * D || qo_stride < (long long)Hq * D || (q_out == Q && qo_stride != q_stride)))
    return TM_ERR_INVALID_ARG;
  if (!aligned(Kn, 16) || !aligned(Vn, 16) || k_stride % 8 || v_stride % 8 || !aligned(w, 4) ||
      !aligned(rope->table, 16) || !aligned(rope->pos, 4))
    return TM_ERR_ALIGNMENT;
  if (Q && (!aligned(Q, 16) || !aligned(q_out, 16) || q_stride % 8 || qo_stride % 8)) return TM_ERR_ALIGNMENT;
  P.A.x[0] = static_cast<const uint16_t*>(Kn);
  P.A.x[1] = static_cast<const uint16_t*>(Vn);
  P.A.stride[0] = k_stride;
  P.A.stride[1] = v_stride;
  P.A.d_shift = D == 64 ? 6 : 7;
  P.A.w = w;
  P.A.w_stride = w_stride;
  P.Q = static_cast<const uint16_t*>(Q);
  P.q_out = static_cast<uint16_t*>(q_out);
  P.q_stride = q_stride;
  P.qo_stride = qo_stride;
  P.G = Q ? Hq / cache->Hkv : 0;
  P.table = rope->table;
  P.pos = rope->pos;
  P.positions = rope->positions;
  P.dims = rope->dims;
  P.roles = Q ? 3 : 2;
  const dim3 grid((unsigned)(P.roles * append_pages(V)), (unsigned)V.Hkv, (unsigned)V.B);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int units = (cache->T < V.max_q ? cache->T : V.max_q) * D / 16;  // of a page
  const bool bf16 = dtype == TM_KVB_BF16, inter = rope->interleaved != 0;
  if (cache->format == TM_KVB_INT8)
    bf16 ? launch_rope<TM_KVB_INT8, true>(P, grid, units, inter, s)
         : launch_rope<TM_KVB_INT8, false>(P, grid, units, inter, s);
  else
    bf16 ? launch_rope<TM_KVB_E4M3, true>(P, grid, units, inter, s)
         : launch_rope<TM_KVB_E4M3, false>(P, grid, units, inter, s);
  if (cudaGetLastError() != cudaSuccess) return TM_ERR_CUDA;
  set_launch_count(1);
  return TM_OK;
}
