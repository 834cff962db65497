// The weight that each token of the paged 8-bit KV cache drew from many rows:
// w_j += sum over rows of 2^(s_j - lse), the scores once more, on tcgen05.
//
// The scores stand transposed: a cluster takes 2 x 128 tokens of one (sequence,
// KV head), their codes exact in fp16 (or bf16, after the queries' type) as the A
// operands in tensor memory, and all rows that see them, 128 at a time as the B
// operand in shared memory -- the queries' own bits, no scaling -- its CTAs
// taking the row tiles in turn.  A thread of the epilogue owns one token, so
// the sum needs no exchange but the cluster's at the end and has a fixed order;
// a compensated sum joins the row tiles (a long prompt adds tens of thousands of terms).
//   warps 0-3, 4-7: epilogue of the first and the second token tile;
//   warps 8-11: query rows by 16-byte asynchronous copies into a ring of three, and their lse;
//   warp 12: the products: one token tile's scores while the other's are summed.
//
// Measured: three prompts of up to 1499 tokens, 64 query and 8 KV heads: 62 us, tensor pipe 27 %, XU
// (exponentials) 35 %; one token tile per CTA 75 us (each row tile then comes from L2 twice as often: 5 TB/s).
#include "kvb_attn.h"

namespace w4 {
namespace kvb {

static __device__ uint32_t s_err_kvbw;

constexpr int kWtThreads = 416;
constexpr int kWtTile = 128;    // tokens per token tile, rows per row tile
constexpr int kWtTokens = 256;  // tokens per CTA: two tiles, so that a row tile is fetched for both
constexpr int kWtSlots = 3;
// CTAs that share a token tile's rows: early tokens are seen by all, late ones by few (one 201 us, two 197,
// four 217 for those prompts with their attention, one token tile per CTA; two 183, four 189 with two).
constexpr int kWtSplit = 2;

template <int D>
struct WtShape {
  static constexpr uint32_t PANEL = kWtTile * 128;
  static constexpr uint32_t TILE = D / 64 * PANEL;
  static constexpr uint32_t ROWS = kWtSlots * TILE;              // [slots][128] x -lse (base 2; -inf: no row)
  static constexpr uint32_t LAST = ROWS + kWtSlots * 128 * 4;    // [slots][128] x last visible token
  static constexpr uint32_t SUMS = LAST + kWtSlots * 128 * 4;    // [256]
  static constexpr uint32_t BARS = SUMS + kWtTokens * 4;
  static constexpr uint32_t SMEM = BARS + 128 + 1024;
};

template <int FMT, int D, bool BF16>
__global__ void __launch_bounds__(kWtThreads, 1) weights_kernel(const AttnParams P) {
  using SH = WtShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  const View& V = P.V;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int bh = blockIdx.x / P.split, b = bh / V.Hkv, h = bh - b * V.Hkv;
  const int share = blockIdx.x - bh * P.split;  // this CTA's place in its cluster
  const int tok0 = blockIdx.y * kWtTokens;
  const Span s = span(V, b);
  const int rows = s.n * P.G;
  const int first = max(tok0 - s.old, 0);  // the first query that sees a token of the tile
  const int r0 = first < s.n ? first * P.G : rows;
  const int tiles = tok0 < s.len && r0 < rows ? (rows - r0 + kWtTile - 1) / kWtTile : 0;
  const int N = (tiles - share + P.split - 1) / P.split;  // tiles share, share + split, ... are this CTA's
  auto first_row = [&](int n) { return r0 + (n * P.split + share) * kWtTile; };
  // Whether some row of tile n sees the second token tile at all; once it does, later ones do.
  auto second = [&](int n) {
    const int last_i = (min(first_row(n) + kWtTile, rows) - 1) / P.G;
    return tok0 + kWtTile < s.len && s.old + last_i >= tok0 + kWtTile;
  };

  const uint32_t bars = base + SH::BARS;
  auto q_full = [&](int i) { return bars + 8 * i; };
  auto q_empty = [&](int i) { return bars + 24 + 8 * i; };
  auto s_full = [&](int i) { return bars + 48 + 8 * i; };
  auto s_empty = [&](int i) { return bars + 64 + 8 * i; };
  const uint32_t a_full = bars + 80, done = bars + 88;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SH::BARS + 96);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::BARS + 100);
  const size_t out = ((size_t)b * V.Hkv + h) * P.w_stride;
  if (tiles == 0) {  // nothing is added here (the whole cluster leaves)
    const int j = tok0 + tid;
    if (share == 0 && tid < kWtTokens && j < P.w_stride) P.w_out[out + j] = P.w_in ? P.w_in[out + j] : 0.f;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kWtSlots; ++i) {
      mbar_init(q_full(i), 4);
      mbar_init(q_empty(i), 1 + 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_empty(i), 4);
    }
    mbar_init(a_full, 8);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // A_0, A_1 (D/2 columns each) from 0 and 64, scores from 128 and 256

  if (warp < 8) {
    // ---------------- one token per thread: warps 0-3 the first tile's, 4-7 the second's ----------------
    const int half = warp >> 2, j = tok0 + tid;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int page = j < s.len ? page_of(V, V.table, b, V.table_stride, j >> V.t_shift) : -1;
    const size_t cell = (size_t)max(page, 0) * V.Hkv + h;
    {
      const uint8_t* src = V.k + ((cell << V.t_shift) + (j & ((1 << V.t_shift) - 1))) * D;
#pragma unroll
      for (int c = 0; c < D; c += 64) {
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 x = page >= 0 ? *reinterpret_cast<const uint4*>(src + c + 16 * k) : make_uint4(0, 0, 0, 0);
          codes_half<FMT>(x.x, o[8 * k], o[8 * k + 1]);
          codes_half<FMT>(x.y, o[8 * k + 2], o[8 * k + 3]);
          codes_half<FMT>(x.z, o[8 * k + 4], o[8 * k + 5]);
          codes_half<FMT>(x.w, o[8 * k + 6], o[8 * k + 7]);
        }
        if (BF16)
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 f = unpack(o[k], false);
            o[k] = pack_bf162(f.x, f.y);
          }
        tc_st_32x32b_x32(tmem + lanes + 64 * half + c / 2, o);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full);
    }
    const float c = page >= 0 ? V.ks[cell] * P.scale_log2 : 0.f;
    const uint64_t c2 = f32x2(c, c);
    float sum = 0.f, lost = 0.f;
    int seen = 0;  // row tiles that this token tile took part in
    for (int n = 0; n < N; ++n) {
      const int slot = n % kWtSlots;
      bool alive = wait_bar(q_full(slot), (uint32_t)(n / kWtSlots) & 1u, abort_flag, &s_err_kvbw);
      const bool mine = half == 0 || second(n);
      if (mine) alive = alive && wait_bar(s_full(half), (uint32_t)seen & 1u, abort_flag, &s_err_kvbw);
      if (!__all_sync(0xffffffffu, alive)) break;
      if (!mine) {
        if (lane == 0) mbar_arrive(q_empty(slot));
        continue;
      }
      ++seen;
      tc_fence_after();
      const bool whole = s.old + first_row(n) / P.G >= tok0 + kWtTile * half + kWtTile - 1;  // every row sees every token
      uint64_t part[4] = {};
#pragma unroll 1
      for (int x0 = 0; x0 < 128; x0 += 64) {  // 64 rows at a time: 128 scores would not fit the registers
        uint32_t v[2][32];
        tc_ld_32x32b_x32(tmem + lanes + 128 + 128 * half + x0, v[0]);
        tc_ld_32x32b_x32(tmem + lanes + 128 + 128 * half + x0 + 32, v[1]);
        tc_wait_ld();
        if (x0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_empty(half));
        }
        const uint8_t* row = smem + SH::ROWS + slot * 512 + 4 * x0;
        if (whole) {
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(row + 4 * k);  // -lse of four rows
            const uint32_t* x = &v[k >> 5][k & 31];
            const float2 e0 = f32x2_get(fma_f32x2(f32x2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, l.x));
            const float2 e1 = f32x2_get(fma_f32x2(f32x2(__uint_as_float(x[2]), __uint_as_float(x[3])), c2, l.y));
            part[(k >> 1) & 2] = add_f32x2(part[(k >> 1) & 2], f32x2(ex2(e0.x), ex2(e0.y)));
            part[((k >> 1) & 2) + 1] = add_f32x2(part[((k >> 1) & 2) + 1], f32x2(ex2(e1.x), ex2(e1.y)));
          }
        } else {
          const uint8_t* last = smem + SH::LAST + slot * 512 + 4 * x0;
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const float2 l = *reinterpret_cast<const float2*>(row + 4 * k);
            const int2 see = *reinterpret_cast<const int2*>(last + 4 * k);
            const float p0 = ex2(fmaf(__uint_as_float(v[k >> 5][k & 31]), c, l.x));
            const float p1 = ex2(fmaf(__uint_as_float(v[k >> 5][(k & 31) + 1]), c, l.y));
            part[(k >> 1) & 3] = add_f32x2(part[(k >> 1) & 3], f32x2(j <= see.x ? p0 : 0.f, j <= see.y ? p1 : 0.f));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(slot));
      // sum += the tile's, with what rounding drops carried along (Kahan)
      const float2 all = f32x2_get(add_f32x2(add_f32x2(part[0], part[1]), add_f32x2(part[2], part[3])));
      const float y = __fadd_rn(__fadd_rn(all.x, all.y), -lost);
      const float t = __fadd_rn(sum, y);
      lost = __fadd_rn(__fadd_rn(t, -sum), -y);
      sum = t;
    }
    reinterpret_cast<float*>(smem + SH::SUMS)[tid] = sum;
    tc_fence_before();
  } else if (warp < 12) {
    // ---------------- query rows ----------------
    const int t = tid - 256;
    constexpr int CPR = D / 8;  // 16-byte chunks per row
    constexpr int RPP = 128 / CPR;
    const int c = t % CPR, rr = t / CPR;
    // A thread's rows are RPP apart: (query, head) and its address move by constants, with a carry.
    const int G = P.G, dq = RPP / G, dg = RPP - dq * G;
    const long long step = dq * P.q_stride + (long long)dg * D, carry = P.q_stride - (long long)G * D;
    int row = first_row(0) + rr, g = row % G;
    const uint16_t* src = P.Q + (long long)(s.row0 + row / G) * P.q_stride + (long long)(h * G + g) * D + 8 * c;
    int lrow = first_row(0) + t, li = lrow / G, lg = lrow - li * G;  // the row whose lse the thread fetches
    const int hop = P.split * kWtTile, ldq = hop / G, ldg = hop - ldq * G;
    const int jump = hop - kWtTile, jq = jump / G, jg = jump - jq * G;  // from a tile's end to the next one's start
    bool alive = true;
    auto issue = [&](int n) {
      if (n < N) {
        const int slot = n % kWtSlots;
        const float x = lrow < rows ? P.lse[(size_t)(s.row0 + li) * P.Hq + h * G + lg] : -INFINITY;
        const int last = lrow < rows ? min(s.old + li, s.len - 1) : -1;
        alive = alive && wait_bar(q_empty(slot), ((uint32_t)(n / kWtSlots) & 1u) ^ 1u, abort_flag, &s_err_kvbw);
        if (alive) {
          const uint32_t dst = base + slot * SH::TILE + (c >> 3) * SH::PANEL;
#pragma unroll
          for (int p = 0; p < kWtTile / RPP; ++p) {
            const int q = p * RPP + rr;
            cp16(dst + q * 128 + (((c & 7) ^ (q & 7)) << 4), row < rows ? src : P.Q, row < rows);
            row += RPP;
            g += dg;
            src += step;
            if (g >= G) {
              g -= G;
              src += carry;
            }
          }
          row += jump;
          g += jg;
          src += jq * P.q_stride + (long long)jg * D;
          if (g >= G) {
            g -= G;
            src += carry;
          }
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + SH::ROWS + slot * 512 + 4 * t),
                       "f"(x != -INFINITY ? x * -1.44269504088896f : -INFINITY)
                       : "memory");
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + SH::LAST + slot * 512 + 4 * t), "r"(last) : "memory");
        }
        lrow += hop;
        li += ldq;
        lg += ldg;
        if (lg >= G) {
          lg -= G;
          ++li;
        }
      }
      cp_commit();
    };
    issue(0);
    issue(1);
    for (int n = 0; n < N; ++n) {
      cp_wait<1>();
      fence_proxy_async_smem();
      if (!__all_sync(0xffffffffu, alive)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(n % kWtSlots));
      issue(n + 2);
    }
    cp_wait<0>();
  } else {
    // ---------------- products ----------------
    constexpr uint32_t id = idesc_f16_f32(128, 128) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
    const uint32_t lead = elect_one(), tm0 = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq = smem_desc_sw128(base);
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, &s_err_kvbw)) != 0;
    };
    bool alive = wait_all(a_full, 0);
    int seen[2] = {0, 0};
    for (int n = 0; n < N && alive; ++n) {
      const int slot = n % kWtSlots;
      alive = wait_all(q_full(slot), (uint32_t)(n / kWtSlots) & 1u);
      const uint64_t db = dq + (uint64_t)slot * (SH::TILE >> 4);
      const int tiles_here = second(n) ? 2 : 1;
      for (int i = 0; i < tiles_here && alive; ++i) {
        alive = wait_all(s_empty(i), ((uint32_t)seen[i] & 1u) ^ 1u);
        if (!alive) break;
        ++seen[i];
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts_if(lead, tm0 + 128 + 128 * i, tm0 + 64 * i + 8 * k,
                    db + (k >> 2) * (uint64_t)(SH::PANEL >> 4) + (uint64_t)((k & 3) * 2), id, k > 0);
        commit_if(lead, s_full(i));
      }
      if (!alive) break;
      commit_if(lead, q_empty(slot));
    }
    commit_if(lead, done);
    if (lead) {
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(done, 0)) {
        if (globaltimer() - t0 > kWaitLimitNs) {
          atomicOr(&s_err_kvbw, kErrTimeout);
          break;
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // ---- the cluster's sums, in order
  __syncwarp();
  cluster_sync_all();
  const int j = tok0 + tid;
  if (share == 0 && tid < kWtTokens && j < P.w_stride) {
    const bool there = j < s.len && page_of(V, V.table, b, V.table_stride, j >> V.t_shift) >= 0;
    float sum = 0.f;
    for (int c = 0; c < P.split; ++c) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(v)
                   : "r"(map_shared_rank(base + SH::SUMS + 4 * tid, c))
                   : "memory");
      sum += v;
    }
    P.w_out[out + j] = (P.w_in ? P.w_in[out + j] : 0.f) + (there ? sum : 0.f);
  }
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while its sums are read
}

template <int FMT, int D, bool BF16>
static tm_status launch(const AttnParams& P, cudaStream_t stream) {
  using SH = WtShape<D>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(weights_kernel<FMT, D, BF16>), SH::SMEM)) return TM_ERR_CUDA;
  AttnParams Q = P;
  Q.split = kWtSplit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.V.B * P.V.Hkv * Q.split), (unsigned)((P.w_stride + kWtTokens - 1) / kWtTokens), 1);
  cfg.blockDim = dim3(kWtThreads, 1, 1);
  cfg.dynamicSmemBytes = SH::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)Q.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_kernel<FMT, D, BF16>, Q) == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

template <int FMT, int D>
static tm_status launch(const AttnParams& P, cudaStream_t stream) {
  return P.bf16 ? launch<FMT, D, true>(P, stream) : launch<FMT, D, false>(P, stream);
}

tm_status launch_row_weights(const AttnParams& P, int format, int D, cudaStream_t stream) {
  if (format == TM_KVB_INT8) return D == 64 ? launch<TM_KVB_INT8, 64>(P, stream) : launch<TM_KVB_INT8, 128>(P, stream);
  return D == 64 ? launch<TM_KVB_E4M3, 64>(P, stream) : launch<TM_KVB_E4M3, 128>(P, stream);
}

}  // namespace kvb

cudaError_t kvb_weights_error_bits(uint32_t* bits, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, kvb::s_err_kvbw, sizeof(v));
  if (e != cudaSuccess) return e;
  if (clear && v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(kvb::s_err_kvbw, &zero, sizeof(zero));
  }
  *bits = v;
  return e;
}

}  // namespace w4
