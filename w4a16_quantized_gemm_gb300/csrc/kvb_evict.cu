// Eviction from the paged 8-bit KV cache by accumulated attention weight.
//
// One thread-block cluster per (sequence, KV head).  Selection: a radix select
// of the count-th largest key over the head's weights, 8 bits a round, the
// histograms summed over the cluster through distributed shared memory; then
// each kept token's new slot is its rank among the kept ones, from counts of
// the tokens before it (no atomics on positions, so ties fall to the lowest
// index).  Move: a warp takes one (new page, K or V), gathers its tokens' codes
// into shared memory, finds the maximum, rounds them to the new scale, and
// writes them after a cluster barrier.
//
// In place: kept tokens move to lower slots in their order, so a new page reads
// only from pages at or after itself.  Pages go in waves of increasing index;
// within a wave every read comes before the barrier and every write after it,
// and no later wave reads what an earlier one wrote.  Into fresh
// pages nothing waits.  No workspace, one launch.
//
// Measured: 8 heads, 2304 -> 2048 tokens 18.6 us (a chain of latencies: key loads 1 us, four
// rounds of histogram and scan 5 us, gather 4 us, requantising 4 us on 64 SMs); 32 x 8 heads, up
// to 4001 -> 1000 tokens, e4m3, 51 us, 2.7 TB/s of what has to move (issue slots 62 %, DRAM 0.39 of the copy rate:
// neither is full; arithmetic on codes and the latencies of the selection in turn); 2 x 8 heads, 131072 -> 4096,
// 49 us (16 k keys per CTA through shared-memory histograms, barriers).  In place the same take 17, 56 and 48 us.
#include "kvb_common.cuh"

namespace w4 {
namespace kvb {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kStage = 65536;  // bytes of tokens staged per CTA: a warp per page (two CTAs fit an SM; 128 KB was slower)
// Every CTA of a cluster selects for itself up to half of this many tokens, a
// cluster of one up to all: that costs less than the cluster barriers of a shared selection (8 heads, to
// 2048 kept, alone against shared: 2304 tokens 18.7 / 20.7 us, 8192 tokens 22.8 / 20.8, 16000 tokens
// 28.8 / 22.8; 32 x 8 heads of 8000 tokens in clusters of one 55.6 / 58.3).
constexpr int kLocalKeys = 8192;
constexpr int kMaxCluster = 8;
constexpr int kKeyCap = 16384;  // most keys of a CTA's slice held in shared memory (64 KB); the rest are read again

static_assert(kKeyCap * 4 <= kStage, "the keys and the tokens share their place");

struct EvictParams {
  View V;
  const int* dst_table;
  int dst_stride;
  const float* w;
  long long w_stride;
  float* w_out;
  long long w_out_stride;
  int budget, first, recent;
  int* kept;
  int* new_len;
  int d_shift;
  int move_warps;
  int list_off;  // shared memory: the list of a local selection, behind the keys and the tokens
  int key_cap;     // keys of a slice held in shared memory
  int local_keys;  // tokens up to which a CTA selects alone
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_shared_rank(addr, rank)) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();  // the barrier's aligned form wants whole warps
  cluster_sync_all();
}
// Word `addr` of the first n CTAs of the cluster (n <= kMaxCluster), all requested before the first is used.
__device__ __forceinline__ uint32_t sum_cluster(uint32_t addr, int n) {
  uint32_t v[kMaxCluster], sum = 0u;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) v[r] = r < n ? ld_cluster(addr, r) : 0u;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) sum += v[r];
  return sum;
}

template <int FMT>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictParams P) {
  extern __shared__ __align__(16) uint8_t smem[];  // keys, then the warps' tokens
  __shared__ uint32_t hist[2][256], total[8];
  __shared__ uint32_t warp_gt[kEvictWarps], warp_eq[kEvictWarps], cta_count[2];
  __shared__ uint32_t found[3];
  __shared__ float row_scale[kEvictWarps][128];
  __shared__ uint32_t row_at[kEvictWarps][128];
  const View& V = P.V;
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int C = gridDim.x;
  const int T = 1 << V.t_shift, D = 1 << P.d_shift;
  const int L = min(max(V.kv_len[b], 0), V.max_len);
  const int count = min(L, P.budget);
  const size_t head = (size_t)b * V.Hkv + h;
  const float* w = P.w + head * P.w_stride;
  int* kept = P.kept + head * P.budget;

  const bool local = L <= P.local_keys;
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + P.list_off);  // the kept, of a local selection
  if (L > count) {
    // ---------------- selection ----------------
    const int SC = local ? 1 : C, sr = local ? 0 : (int)rank;  // CTAs that share the keys, and this one's place
    auto barrier = [&] { local ? __syncthreads() : cluster_barrier(); };
    const int per = ((L + SC - 1) / SC + kEvictThreads - 1) / kEvictThreads * kEvictThreads;
    const int s0 = min(L, sr * per), s1 = min(L, s0 + per);
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
    auto rank_of = [&](int j, float x, int page) -> uint32_t {
      if (j < P.first || j >= L - P.recent) return 0xFFFFFFFFu;
      x += 0.f;  // -0 counts as 0
      if ((unsigned)page >= (unsigned)V.pages || x != x) return 0u;
      const uint32_t u = __float_as_uint(x);
      return (u >> 31) ? ~u : (u | 0x80000000u);
    };
    const int* table = V.table + (size_t)b * V.table_stride;
    const int cached = min(s1, s0 + P.key_cap);
    for (int j0 = s0 + tid; j0 < cached; j0 += 8 * kEvictThreads) {
      float x[8];
      int page[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i * kEvictThreads;
        x[i] = j < cached ? w[j] : 0.f;
        page[i] = j < cached ? table[j >> V.t_shift] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i * kEvictThreads;
        if (j < cached) keys[j - s0] = rank_of(j, x[i], page[i]);
      }
    }
    // A slice's keys in shared memory first, then those that are computed again each time.
    auto far_key = [&](int j) { return rank_of(j, w[j], table[j >> V.t_shift]); };
    auto key = [&](int j) { return j < cached ? keys[j - s0] : far_key(j); };
    const bool near = cached == s1;  // all in shared memory
    uint32_t prefix = 0u, mask = 0u, want = (uint32_t)count;
    if (tid < 256) hist[0][tid] = hist[1][tid] = 0u;
    __syncthreads();
    for (int shift = 24; shift >= 0; shift -= 8) {
      uint32_t* mine = hist[(shift >> 3) & 1];
      auto count_key = [&](uint32_t k) {
        if ((k & mask) == prefix) atomicAdd(&mine[(k >> shift) & 255u], 1u);
      };
      const int whole = (cached - s0) / 4 * 4;
      for (int j = 4 * tid; j < whole; j += 4 * kEvictThreads) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + j);
        count_key(k.x);
        count_key(k.y);
        count_key(k.z);
        count_key(k.w);
      }
      for (int j = s0 + whole + tid; j < s1; j += kEvictThreads) count_key(key(j));
      barrier();
      // Thread t < 256 holds digit 255 - t: from the largest keys down.
      uint32_t n = 0u, upto = 0u;
      if (tid < 256) {
        n = upto = local ? mine[255 - tid] : sum_cluster(smem_u32(&mine[255 - tid]), C);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        if (lane == 31) total[warp] = upto;
        // The other histogram was last read, by the whole cluster, before this round's barrier.
        hist[1 - ((shift >> 3) & 1)][tid] = 0u;
      }
      __syncthreads();
      if (tid < 256) {
        for (int i = 0; i < warp; ++i) upto += total[i];
        if (upto - n < want && want <= upto) {
          found[0] = 255u - (uint32_t)tid;
          found[1] = want - (upto - n);
          found[2] = n;
        }
      }
      __syncthreads();
      prefix |= found[0] << shift;
      mask |= 255u << shift;
      want = found[1];
      if (want == found[2]) {  // all of these digits are kept: no further ones decide
        --prefix;
        want = 0u;
        break;
      }
    }
    // The kept: every key above `prefix`, and the first `want` equal to it.
    const int sub = per / kEvictWarps;
    const int w0 = min(s1, s0 + warp * sub), w1 = min(s1, w0 + sub);
    const uint32_t before = (1u << lane) - 1u;
    uint32_t gt = 0u, eq = 0u;
    auto tally = [&](int j, uint32_t k) {
      gt += __popc(__ballot_sync(0xffffffffu, j + lane < w1 && k > prefix));
      eq += __popc(__ballot_sync(0xffffffffu, j + lane < w1 && k == prefix));
    };
    if (near) {
#pragma unroll 4
      for (int j = w0; j < w1; j += 32) tally(j, j + lane < w1 ? keys[j + lane - s0] : 0u);
    } else {
      for (int j = w0; j < w1; j += 32) tally(j, j + lane < w1 ? key(j + lane) : 0u);
    }
    if (lane == 0) {
      warp_gt[warp] = gt;
      warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid < 2) {
      uint32_t v = 0u;
      for (int i = 0; i < kEvictWarps; ++i) v += tid ? warp_eq[i] : warp_gt[i];
      cta_count[tid] = v;
    }
    barrier();
    gt = sum_cluster(smem_u32(&cta_count[0]), sr);
    eq = sum_cluster(smem_u32(&cta_count[1]), sr);
    for (int i = 0; i < warp; ++i) {
      gt += warp_gt[i];
      eq += warp_eq[i];
    }
    auto emit = [&](int j, uint32_t k) {
      const bool in = j + lane < w1;
      const uint32_t mg = __ballot_sync(0xffffffffu, in && k > prefix);
      const uint32_t me = __ballot_sync(0xffffffffu, in && k == prefix);
      const uint32_t g = gt + __popc(mg & before), e = eq + __popc(me & before);
      if (in && (k > prefix || (k == prefix && e < want))) {
        const uint32_t pos = g + min(e, want);
        if (sr == (int)rank) kept[pos] = j + lane;
        if (local) list[pos] = (uint16_t)(j + lane);
      }
      gt += __popc(mg);
      eq += __popc(me);
    };
    if (near) {
#pragma unroll 4
      for (int j = w0; j < w1; j += 32) emit(j, j + lane < w1 ? keys[j + lane - s0] : 0u);
    } else {
      for (int j = w0; j < w1; j += 32) emit(j, j + lane < w1 ? key(j + lane) : 0u);
    }
  } else {
    for (int j = (int)rank * kEvictThreads + tid; j < L; j += C * kEvictThreads) kept[j] = j;
  }
  for (int j = count + (int)rank * kEvictThreads + tid; j < P.budget; j += C * kEvictThreads) kept[j] = -1;
  if (rank == 0 && h == 0 && tid == 0) P.new_len[b] = count;
  if (local)
    __syncthreads();
  else
    cluster_barrier();
  auto kept_at = [&](int pos) { return L == count ? pos : local ? (int)list[pos] : kept[pos]; };

  // ---------------- move ----------------
  const int chunk_shift = P.d_shift - 4;  // 16-byte chunks per token
  const int chunks = T << chunk_shift;
  uint8_t* stage = smem + ((size_t)(warp << V.t_shift) << P.d_shift);  // of the first move_warps warps
  const uint32_t stage_u = smem_u32(stage);
  float* rs = row_scale[warp];
  uint32_t* ra = row_at[warp];
  const int units = 2 * ((count + T - 1) >> V.t_shift), wave = C * P.move_warps;
  // In place: a new page that is the old page of its block, or the weights over themselves.  (A page that
  // serves another block of the call may not be a destination.)  Otherwise no wave has to wait.
  bool shared_place = P.w_out == P.w;
  for (int i = tid; i < units / 2 && i < V.table_stride; i += kEvictThreads)
    shared_place |= V.table[(size_t)b * V.table_stride + i] == P.dst_table[(size_t)b * P.dst_stride + i];
  shared_place = __syncthreads_or(shared_place);
  for (int u0 = 0; u0 < units; u0 += wave) {
    const int u = warp < P.move_warps ? u0 + (int)rank * P.move_warps + warp : units;
    const int blk = u >> 1, sel = u & 1;
    const int base = blk << V.t_shift;
    bool same = false;
    int from = -1, to = -1;
    float now = kScaleFloor;
    float kw[4];
    if (u < units) {
      const int last = min(count, base + T) - 1;
      same = kept_at(last) == last;
      from = page_of(V, V.table, b, V.table_stride, min(blk, V.table_stride - 1));
      to = page_of(V, P.dst_table, b, P.dst_stride, blk);
      const float* scales = sel ? V.vs : V.ks;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = lane + 32 * i;
        if (t < T) {
          const int pos = base + t;
          const int j = pos < count ? kept_at(pos) : -1;
          const int page = j >= 0 ? page_of(V, V.table, b, V.table_stride, j >> V.t_shift) : -1;
          const size_t cell = (size_t)max(page, 0) * V.Hkv + h;
          rs[t] = page >= 0 ? scales[cell] : 0.f;
          // the token's row of the pool (a pool of 2^32 rows of 64 bytes would be 256 GiB)
          ra[t] = page >= 0 ? (uint32_t)((cell << V.t_shift) + (j & (T - 1))) : 0xffffffffu;
          kw[i] = j >= 0 ? w[j] : 0.f;
        }
      }
      __syncwarp();
      const uint8_t* pool = sel ? V.v : V.k;
#pragma unroll 4
      for (int c = lane; c < chunks; c += 32) {
        const uint32_t at = ra[c >> chunk_shift];
        const bool there = at != 0xffffffffu;
        cp16(stage_u + 16 * c, pool + (there ? (size_t)at * D + ((c & ((1 << chunk_shift) - 1)) << 4) : 0), there);
      }
      cp_commit();
      cp_wait<0>();
      __syncwarp();
      if (same) {
        if (from >= 0) now = scales[(size_t)from * V.Hkv + h];
      } else {
        float a = 0.f;
#pragma unroll 4
        for (int c = lane; c < chunks; c += 32) {
          const uint4 q = *reinterpret_cast<const uint4*>(stage + 16 * c);
          const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
          __half2 m = __float2half2_rn(0.f);  // the codes are exact in fp16
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t x, y;
            codes_half<FMT>(wd[k], x, y);
            m = __hmax2(m, __hmax2(__habs2(*reinterpret_cast<__half2*>(&x)), __habs2(*reinterpret_cast<__half2*>(&y))));
          }
          a = fmaxf(a, __fmul_rn(fmaxf(__low2float(m), __high2float(m)), rs[c >> chunk_shift]));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        now = scale_for<FMT>(a);
        const Divisor by = divisor(now);
#pragma unroll 2
        for (int c = lane; c < chunks; c += 32) {
          uint4* at = reinterpret_cast<uint4*>(stage + 16 * c);
          const uint4 q = *at;
          uint32_t wd[4] = {q.x, q.y, q.z, q.w};
          const float s = rs[c >> chunk_shift];
          const uint64_t s2 = f32x2(s, s);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            wd[k] = recode4<FMT>(wd[k], s2, by);
          }
          *at = make_uint4(wd[0], wd[1], wd[2], wd[3]);
        }
      }
      __syncwarp();
    }
    if (shared_place) cluster_barrier();
    if (u < units) {
      if (sel == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = base + lane + 32 * i;
          if (lane + 32 * i < T && pos < count) P.w_out[head * P.w_out_stride + pos] = kw[i];
        }
      if (to >= 0 && !(same && to == from)) {
        const size_t cell = (size_t)to * V.Hkv + h;
        uint8_t* dst = (sel ? V.v : V.k) + ((cell << V.t_shift) << P.d_shift);
#pragma unroll 4
        for (int c = lane; c < chunks; c += 32)
          *reinterpret_cast<uint4*>(dst + 16 * c) = *reinterpret_cast<const uint4*>(stage + 16 * c);
        if (lane == 0) (sel ? V.vs : V.ks)[cell] = now;
      }
      __syncwarp();
    }
  }
  for (int j = count + (int)rank * kEvictThreads + tid; j < P.budget; j += C * kEvictThreads)
    P.w_out[head * P.w_out_stride + j] = 0.f;
  // No CTA leaves while another may still read its shared memory.
  cluster_barrier();
}

template <int FMT>
tm_status launch_evict(EvictParams P, cudaStream_t stream) {
  const View& V = P.V;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(evict_kernel<FMT>), kStage + 2 * kLocalKeys)) return TM_ERR_CUDA;
  // CTAs per cluster: as many as the pages or the keys can use, while two CTAs per SM hold all clusters
  // (32 x 8 heads of 4001 tokens: clusters of one 59 us, of two 66, of four 81 at the time).
  const long long T = 1ll << V.t_shift, heads = (long long)V.B * V.Hkv;
  const long long units = 2 * ((P.budget + T - 1) / T), room = 2ll * num_sms(current_device());
  const int page = (int)T << P.d_shift;
  P.move_warps = kStage / page < kEvictWarps ? kStage / page : kEvictWarps;
  int C = 1;
  while (C < kMaxCluster && heads * 2 * C <= room && (units > C * 8 || V.max_len > C * 4096ll)) C *= 2;
  if (units < P.move_warps * C) P.move_warps = (int)((units + C - 1) / C);
  P.local_keys = C == 1 ? kLocalKeys : kLocalKeys / 2;
  const long long slice = (V.max_len + C - 1) / C + kEvictThreads;
  const long long alone = V.max_len < P.local_keys ? V.max_len : P.local_keys;
  const long long most = V.max_len <= P.local_keys || slice < alone ? alone : slice;
  P.key_cap = (int)(most < kKeyCap ? most : kKeyCap);
  const size_t stage = (size_t)P.move_warps * page, keys = (size_t)P.key_cap * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C, (unsigned)V.Hkv, (unsigned)V.B);
  cfg.blockDim = dim3(kEvictThreads, 1, 1);
  P.list_off = (int)(stage > keys ? stage : (keys + 15) / 16 * 16);
  cfg.dynamicSmemBytes = P.list_off + 2 * (size_t)(P.budget < alone ? P.budget : alone);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<FMT>, P) == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

}  // namespace kvb
}  // namespace w4

using namespace w4;
using namespace w4::kvb;

extern "C" tm_status tm_kvb_evict(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const int* dst_table,
                                  int dst_stride, const float* w, long long w_stride, float* w_out,
                                  long long w_out_stride, int budget, int first, int recent, int* kept, int* new_len,
                                  void* stream) {
  EvictParams P;
  const tm_status st = check(cache, batch, true, &P.V);
  if (st != TM_OK) return st;
  const View& V = P.V;
  if (budget < 1 || first < 0 || recent < 0 || (long long)first + recent > budget) return TM_ERR_INVALID_ARG;
  if (V.B == 0) return TM_OK;
  if (!dst_table || !w || !w_out || !kept || !new_len || new_len == V.kv_len) return TM_ERR_INVALID_ARG;
  if ((long long)dst_stride * cache->T < budget || w_stride < V.max_len || w_out_stride < budget)
    return TM_ERR_INVALID_ARG;
  if (w == w_out && w_stride != w_out_stride) return TM_ERR_INVALID_ARG;
  if (!aligned(dst_table, 4) || !aligned(w, 4) || !aligned(w_out, 4) || !aligned(kept, 4) || !aligned(new_len, 4))
    return TM_ERR_ALIGNMENT;
  P.dst_table = dst_table;
  P.dst_stride = dst_stride;
  P.w = w;
  P.w_stride = w_stride;
  P.w_out = w_out;
  P.w_out_stride = w_out_stride;
  P.budget = budget;
  P.first = first;
  P.recent = recent;
  P.kept = kept;
  P.new_len = new_len;
  P.d_shift = cache->D == 64 ? 6 : 7;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const tm_status r =
      cache->format == TM_KVB_INT8 ? launch_evict<TM_KVB_INT8>(P, s) : launch_evict<TM_KVB_E4M3>(P, s);
  if (r == TM_OK) set_launch_count(1);
  return r;
}
