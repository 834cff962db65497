// Accepted drafts of the paged 8-bit KV cache: a path through the new tokens of each sequence moves to their front.
//
// One CTA per (sequence, KV head, K or V).  Token path[i] goes to slot old + i.  The path ascends, so that a token
// never moves up: 128 slots at a time (whole pages) are read into registers, then written, and what later slots
// read has not been written yet.  Codes that stay in their page stay as they are; those from another page follow the
// append's rule, x = c s_src being the new value:
//   s = max(s_old, max |x| r) where the page keeps a token, else max |x| r;  codes Q(x / s), kept ones Q((c s_old) / s)
// Latency-bound: a few dependent loads (lengths, path, pages, scales and codes), a few KB a CTA.  Measured: 32
// sequences, paths of up to 6, 8 KV heads: 3.7 us; 64 sequences, paths of up to 40 through pages of 16: 8.3 us (1024
// CTAs, four on an SM: 1.7 waves, in which each of a thread's four vectors runs through its loads and the page's
// shared maximum before the next one starts).
#include "kvb_common.cuh"

namespace w4 {
namespace kvb {

constexpr int kAcceptThreads = 256;
constexpr int kAcceptSlots = 128;  // slots per pass: at most 8 pages of 16, at least one

struct AcceptParams {
  View V;
  const int* path;
  const int* count;
  int path_stride;
  float* w;
  long long w_stride;
  int* new_len;
};

// Largest magnitude of 16 codes, as a number.
template <int FMT>
__device__ __forceinline__ float largest16(const uint4& c) {
  uint32_t m;
  if (FMT == TM_KVB_INT8)
    m = __vmaxu4(__vmaxu4(__vabs4(c.x), __vabs4(c.y)), __vmaxu4(__vabs4(c.z), __vabs4(c.w)));
  else
    m = __vmaxu4(__vmaxu4(c.x & 0x7f7f7f7fu, c.y & 0x7f7f7f7fu), __vmaxu4(c.z & 0x7f7f7f7fu, c.w & 0x7f7f7f7fu));
  m = max(max(m & 0xffu, (m >> 8) & 0xffu), max((m >> 16) & 0xffu, m >> 24));
  if (FMT == TM_KVB_INT8) return (float)m;
  const uint32_t h = e4m3x2_half2((uint16_t)m);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptParams P) {
  constexpr int VPT = D / 16;                                     // 16-byte vectors per token
  constexpr int VECS = kAcceptSlots * VPT / kAcceptThreads;       // per thread and pass
  __shared__ int cut_s, page_s[8];
  __shared__ uint32_t need_s[8], away_s, stay_s;                  // bits: the page takes tokens from others, keeps some
  const View& V = P.V;
  const int b = blockIdx.y, h = blockIdx.x >> 1, sel = blockIdx.x & 1, tid = threadIdx.x;
  const int raw = max(V.kv_len[b], 0);
  // No row is read here, so that only the number of them counts.
  const int n = V.q_start ? max(max(V.q_start[b + 1], 0) - max(V.q_start[b], 0), 0) : 1;
  const int old = raw - n;
  const int* path = P.path + (size_t)b * P.path_stride;
  if (old < 0 || n == 0) {  // nothing to choose from: as it is
    if (blockIdx.x == 0 && tid == 0) P.new_len[b] = raw;
    return;
  }
  // The path ends before the first entry that is no new token or not above the one before it.
  const int most = min(min(max(P.count[b], 0), P.path_stride), n);
  if (tid == 0) cut_s = most;
  __syncthreads();
  for (unsigned i = tid; i < (unsigned)most; i += kAcceptThreads) {  // counts reach 2^31 - 1
    const int at = path[i];
    if (at < 0 || at >= n || (i > 0 && path[i - 1] >= at)) atomicMin(&cut_s, (int)i);
  }
  __syncthreads();
  const int count = cut_s;

  if (sel == 0) {
    if (blockIdx.x == 0 && tid == 0) P.new_len[b] = old + count;
    if (P.w) {  // the weights move along, the rest of the new ones are cleared
      float* w = P.w + ((size_t)b * V.Hkv + h) * P.w_stride;
      const unsigned room = (unsigned)max(min((long long)n, P.w_stride - old), 0ll);  // new tokens that have a weight
      for (unsigned i0 = 0; i0 < room; i0 += kAcceptThreads) {
        const unsigned i = i0 + tid;
        const long long src = i < (unsigned)count ? (long long)old + path[i] : P.w_stride;
        const float x = src < P.w_stride ? w[src] : 0.f;
        __syncthreads();
        if (i < room) w[old + i] = x;
      }
    }
  }

  uint8_t* pool = sel ? V.v : V.k;
  float* scales = sel ? V.vs : V.ks;
  const int T = 1 << V.t_shift;
  const int room = V.table_stride << V.t_shift;  // slots with a table entry: at most 2^30
  auto page_at = [&](int slot) {
    return slot < room ? page_of(V, V.table, b, V.table_stride, slot >> V.t_shift) : -1;
  };
  const int end = min(old + count, room);  // slots past the table hold nothing
  for (int base = old / kAcceptSlots * kAcceptSlots; base < end; base += kAcceptSlots) {
    if (tid < 8) {
      const int slot = base + tid * T;
      page_s[tid] = tid * T < kAcceptSlots && slot < end ? page_at(slot) : -1;
      need_s[tid] = 0u;
    }
    if (tid == 0) {
      away_s = 0u;
      stay_s = 0u;
    }
    __syncthreads();
    uint4 c[VECS];
    float from[VECS];  // the source's scale; -1: it stays in its page (or there is nothing)
    int take[VECS];    // 0: nothing to write, 1: to its slot as it is (or rounded anew), 2: from another page
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      const int v = tid + k * kAcceptThreads, t = v / VPT, slot = base + t;
      take[k] = 0;
      from[k] = -1.f;
      c[k] = make_uint4(0u, 0u, 0u, 0u);
      if (slot < old || slot >= end || page_s[t >> V.t_shift] < 0) continue;
      const int src = old + path[slot - old];
      const bool away = (src >> V.t_shift) != (slot >> V.t_shift);
      const int page = away ? page_at(src) : page_s[t >> V.t_shift];
      take[k] = away ? 2 : 1;
      const size_t cell = (size_t)max(page, 0) * V.Hkv + h;
      if (page >= 0)
        c[k] = *reinterpret_cast<const uint4*>(pool + (((cell << V.t_shift) + (src & (T - 1))) * D + (v % VPT) * 16));
      if (away) {
        from[k] = page >= 0 ? scales[cell] : 0.f;
        atomicMax(&need_s[t >> V.t_shift], __float_as_uint(__fmul_rn(largest16<FMT>(c[k]), from[k])));
        atomicOr(&away_s, 1u << (t >> V.t_shift));
      } else {
        atomicOr(&stay_s, 1u << (t >> V.t_shift));
      }
    }
    __syncthreads();
    // ---- every source of this pass is in registers
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      if (!take[k]) continue;
      const int v = tid + k * kAcceptThreads, t = v / VPT, p = t >> V.t_shift;
      const size_t cell = (size_t)page_s[p] * V.Hkv + h;
      const bool keeps = old > base + p * T || ((stay_s >> p) & 1u);
      if ((away_s >> p) & 1u) {
        const float need = scale_for<FMT>(__uint_as_float(need_s[p]));
        const float was = scales[cell], now = keeps ? fmaxf(was, need) : need;
        const Divisor by = divisor(now);
        const float s = take[k] == 2 ? from[k] : was;
        if (take[k] == 2 || now > was) {
          const uint64_t s2 = f32x2(s, s);
          c[k] = make_uint4(recode4<FMT>(c[k].x, s2, by), recode4<FMT>(c[k].y, s2, by), recode4<FMT>(c[k].z, s2, by),
                            recode4<FMT>(c[k].w, s2, by));
        }
      }
      *reinterpret_cast<uint4*>(pool + (((cell << V.t_shift) + (t & (T - 1))) * D + (v % VPT) * 16)) = c[k];
    }
    // Tokens before the new ones in the first page, where its scale grows.
    const int p0 = (old - base) >> V.t_shift;
    if (old >= base && old - base < kAcceptSlots && ((away_s >> p0) & 1u) && page_s[p0] >= 0) {
      const size_t cell = (size_t)page_s[p0] * V.Hkv + h;
      const float was = scales[cell], now = fmaxf(was, scale_for<FMT>(__uint_as_float(need_s[p0])));
      if (now > was) {
        const Divisor by = divisor(now);
        const uint64_t s2 = f32x2(was, was);
        uint4* at = reinterpret_cast<uint4*>(pool + (cell << V.t_shift) * D);
        for (int v = tid; v < (old & (T - 1)) * VPT; v += kAcceptThreads) {
          uint4 x = at[v];
          at[v] = make_uint4(recode4<FMT>(x.x, s2, by), recode4<FMT>(x.y, s2, by), recode4<FMT>(x.z, s2, by),
                             recode4<FMT>(x.w, s2, by));
        }
      }
    }
    __syncthreads();
    if (tid < 8 && ((away_s >> tid) & 1u)) {
      const size_t cell = (size_t)page_s[tid] * V.Hkv + h;
      const float need = scale_for<FMT>(__uint_as_float(need_s[tid]));
      const bool keeps = old > base + tid * T || ((stay_s >> tid) & 1u);
      scales[cell] = keeps ? fmaxf(scales[cell], need) : need;
    }
    __syncthreads();
  }
}

}  // namespace kvb
}  // namespace w4

using namespace w4;
using namespace w4::kvb;

extern "C" tm_status tm_kvb_accept(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const int* path,
                                   int path_stride, const int* count, float* w, long long w_stride, int* new_len,
                                   void* stream) {
  AcceptParams P = {};
  const tm_status st = check(cache, batch, true, &P.V);
  if (st != TM_OK) return st;
  const View& V = P.V;
  if (!batch->q_start && batch->rows != batch->B) return TM_ERR_INVALID_ARG;
  if (path_stride < 0 || w_stride < 0) return TM_ERR_INVALID_ARG;
  if (V.B == 0) return TM_OK;
  if ((!path && path_stride > 0) || !count || !new_len || new_len == batch->kv_len) return TM_ERR_INVALID_ARG;
  if (!aligned(path, 4) || !aligned(count, 4) || !aligned(new_len, 4) || !aligned(w, 4)) return TM_ERR_ALIGNMENT;
  P.path = path;
  P.count = count;
  P.path_stride = path_stride;
  P.w = w;
  P.w_stride = w_stride;
  P.new_len = new_len;
  const dim3 grid((unsigned)(2 * V.Hkv), (unsigned)V.B);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->format == TM_KVB_INT8)
    cache->D == 64 ? accept_kernel<TM_KVB_INT8, 64><<<grid, kAcceptThreads, 0, s>>>(P)
                   : accept_kernel<TM_KVB_INT8, 128><<<grid, kAcceptThreads, 0, s>>>(P);
  else
    cache->D == 64 ? accept_kernel<TM_KVB_E4M3, 64><<<grid, kAcceptThreads, 0, s>>>(P)
                   : accept_kernel<TM_KVB_E4M3, 128><<<grid, kAcceptThreads, 0, s>>>(P);
  if (cudaGetLastError() != cudaSuccess) return TM_ERR_CUDA;
  set_launch_count(1);
  return TM_OK;
}
