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

// TREE: every row sees the tokens before the new ones, and of these those that its mask names.
template <int FMT, int D, bool BF16, bool TREE>
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
  const int first = TREE ? 0 : max(tok0 - s.old, 0);  // the first query that sees a token of the tile
  const int r0 = first < s.n ? first * P.G : rows;
  const int tiles = tok0 < s.len && r0 < rows ? (rows - r0 + kWtTile - 1) / kWtTile : 0;
  const int N = (tiles - share + P.split - 1) / P.split;  // tiles share, share + split, ... are this CTA's
  auto first_row = [&](int n) { return r0 + (n * P.split + share) * kWtTile; };
  // Whether some row of tile n sees the second token tile at all; once it does, later ones do.
  auto second = [&](int n) {
    const int last_i = (min(first_row(n) + kWtTile, rows) - 1) / P.G;
    return tok0 + kWtTile < s.len && (TREE || s.old + last_i >= tok0 + kWtTile);
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
        __syncwarp();  // lanes without a token took another way
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
      // whether every row sees every token
      const bool whole = s.old + (TREE ? -1 : first_row(n) / P.G) >= tok0 + kWtTile * half + kWtTile - 1;
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
            bool see0, see1;
            if constexpr (TREE) {
              const int node = j - s.old;  // its word is the same one for most of the warp: a broadcast
              auto sees = [&](int row) {
                return node < 0 || (row >= 0 && (node >> 5) < P.tree_words &&
                                    ((P.tree[row * P.tree_stride + (node >> 5)] >> (node & 31)) & 1u));
              };
              see0 = sees(see.x);
              see1 = sees(see.y);
            } else {
              see0 = j <= see.x;
              see1 = j <= see.y;
            }
            part[(k >> 1) & 3] = add_f32x2(part[(k >> 1) & 3], f32x2(see0 ? p0 : 0.f, see1 ? p1 : 0.f));
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
        // the row's last visible token (of a tree: its mask's row); none: -1
        const int last = lrow < rows ? (TREE ? s.row0 + li : min(s.old + li, s.len - 1)) : -1;
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

// Trees of up to 512 rows: the same row tiles for all tokens.  A CTA keeps its queries and takes a slice of the tokens
// in tiles of 128, which its two groups of four warps take in turn, a token per thread: convert the codes of the group's
// next tile into tensor memory, sum this one's scores, a row tile at a time.  16 sequences of 4096 tokens, 8 KV heads,
// 104 rows: 39 us (a new CTA for every 256 tokens 90, a pair of them, as above, 171; masks from global memory in place
// of shared 52); 160 rows 125 with the attention (238), 2 x 30000 tokens, 504 rows 198 (308).
constexpr int kRtThreads = 288;
constexpr int kRtTiles = 4;  // row tiles at most: 128 KB of queries, 32 KB of masks

template <int D>
struct RtShape {
  static constexpr uint32_t PANEL = kWtTile * 128;
  static constexpr uint32_t TILE = D / 64 * PANEL;
  static constexpr uint32_t BARS = 0;
  static constexpr uint32_t Q = 1024;  // [tiles]
  // behind them [tiles * 128] x -lse (base 2; -inf: no row), then [tiles * 128][words] of the masks
  static uint32_t smem(int tiles, int words) { return 1024 + Q + tiles * (TILE + kWtTile * (4 + 4 * words)); }
};

template <int FMT, int D, bool BF16>
__global__ void __launch_bounds__(kRtThreads, 1) tree_weights_kernel(const AttnParams P, int slice) {
  using SH = RtShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  const View& V = P.V;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int b = blockIdx.x / V.Hkv, h = blockIdx.x - b * V.Hkv;
  const Span s = span(V, b);
  const int rows = s.n * P.G, tiles = (rows + kWtTile - 1) / kWtTile;
  const long long j0 = (long long)blockIdx.y * slice, j1 = min(j0 + slice, P.w_stride);
  const int N = rows > 0 && j0 < s.len ? (int)((min(j1, (long long)s.len) - j0 + kWtTile - 1) / kWtTile) : 0;
  const size_t out = ((size_t)b * V.Hkv + h) * P.w_stride;
  // What no tile holds: nothing is added there.
  for (long long j = j0 + (long long)N * kWtTile + tid; j < j1; j += kRtThreads)
    P.w_out[out + j] = P.w_in ? P.w_in[out + j] : 0.f;
  if (N == 0) return;

  const uint32_t lse_at = SH::Q + tiles * SH::TILE, masks_at = lse_at + tiles * kWtTile * 4;
  const uint32_t bars = base + SH::BARS;
  auto a_full = [&](int i) { return bars + 8 * i; };
  auto s_full = [&](int i) { return bars + 16 + 8 * i; };
  const uint32_t done = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SH::BARS + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::BARS + 44);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(a_full(i), 4);
      mbar_init(s_full(i), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  } else {
    // The queries, 16 bytes a thread, a row by neighbouring lanes; their lse.
    constexpr int LANES = D / 8, STEP = 256 / LANES;
    const int c = tid % LANES;
#pragma unroll 4
    for (int row = tid / LANES; row < tiles * kWtTile; row += STEP) {
      const bool have = row < rows;
      const int q = have ? row / P.G : 0, head = h * P.G + (have ? row - q * P.G : 0);
      const uint4 x = ldg_or_zero(P.Q + (s.row0 + q) * P.q_stride + (long long)head * D + 8 * c, have);
      sts128(base + SH::Q + (row >> 7) * SH::TILE + (c >> 3) * SH::PANEL + (row & 127) * 128 +
                 (((c & 7) ^ (row & 7)) << 4), x.x, x.y, x.z, x.w);
    }
    for (int row = tid; row < tiles * kWtTile; row += 256) {
      const bool have = row < rows;
      const int q = have ? row / P.G : 0, head = h * P.G + (have ? row - q * P.G : 0);
      const float x = have ? P.lse[(size_t)(s.row0 + q) * P.Hq + head] : -INFINITY;
      reinterpret_cast<float*>(smem + lse_at)[row] = x != -INFINITY ? x * -1.44269504088896f : -INFINITY;
      const uint32_t* mask = P.tree + (s.row0 + q) * P.tree_stride;
      for (int k = 0; k < P.tree_words; ++k)
        reinterpret_cast<uint32_t*>(smem + masks_at)[row * P.tree_words + k] = have ? mask[k] : 0u;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // A of group i's even and odd tiles at 128 i and 128 i + 64, scores at 256 + 128 i

  if (warp < 8) {
    const int i = warp >> 2, t = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16, ts = tmem + lanes + 256 + 128 * i;
    auto token = [&](int n) { return (int)j0 + n * kWtTile + t; };
    auto page_for = [&](int n) {
      return n < N && token(n) < s.len ? page_of(V, V.table, b, V.table_stride, token(n) >> V.t_shift) : -1;
    };
    // The page of a tile is looked up three of the group's tiles ahead, its codes are fetched two ahead.
    uint4 x[D / 16];
    auto fetch = [&](int n, int page) {  // returns what multiplies the scores; 0: no token
      const size_t cell = (size_t)max(page, 0) * V.Hkv + h;
      const uint8_t* src = V.k + ((cell << V.t_shift) + (token(n) & ((1 << V.t_shift) - 1))) * D;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) x[c] = ldg_or_zero(src + 16 * c, page >= 0);
      return page >= 0 ? V.ks[cell] * P.scale_log2 : 0.f;
    };
    auto convert = [&](int odd) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          codes_half<FMT>(x[4 * c + k].x, o[8 * k], o[8 * k + 1]);
          codes_half<FMT>(x[4 * c + k].y, o[8 * k + 2], o[8 * k + 3]);
          codes_half<FMT>(x[4 * c + k].z, o[8 * k + 4], o[8 * k + 5]);
          codes_half<FMT>(x[4 * c + k].w, o[8 * k + 6], o[8 * k + 7]);
        }
        if (BF16)
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 f = unpack(o[k], false);
            o[k] = pack_bf162(f.x, f.y);
          }
        __syncwarp();  // lanes without a token took another way
        tc_st_32x32b_x32(tmem + lanes + 128 * i + 64 * odd + 32 * c, o);
      }
      tc_wait_st();
    };
    int page = page_for(i), page_next = page_for(i + 2);
    bool there = page >= 0, there_next = false;
    float scale = fetch(i, page), scale_next = 0.f;
    if (i < N) {
      convert(0);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full(i));
    }
    if (i + 2 < N) {
      there_next = page_next >= 0;
      scale_next = fetch(i + 2, page_next);
    }
    page_next = page_for(i + 4);
    bool alive = true;
    int unit = 0;  // row tiles of this group's tokens so far
#pragma unroll 1
    for (int n = i; n < N; n += 2) {
      const int turn = n >> 1;
      const float c = scale;
      const bool counts = there;
      scale = scale_next;
      there = there_next;
      if (n + 2 < N) {
        convert((turn + 1) & 1);
        if (n + 4 < N) {
          there_next = page_next >= 0;
          scale_next = fetch(n + 4, page_next);
          page_next = page_for(n + 6);
        }
      }
      const int j = token(n);
      const bool whole = (int)j0 + n * kWtTile + kWtTile <= s.old;  // every row sees every token
      const uint64_t c2 = f32x2(c, c);
      uint64_t part[4] = {};  // each at most 64 rows' sums
#pragma unroll 1
      for (int r = 0; r < tiles; ++r, ++unit) {
        alive = wait_bar(s_full(i), (uint32_t)unit & 1u, abort_flag, &s_err_kvbw);
        alive = __all_sync(0xffffffffu, alive);
        if (!alive) break;
        tc_fence_after();
#pragma unroll 1
        for (int x0 = 0; x0 < 128; x0 += 64) {
          uint32_t v[2][32];
          tc_ld_32x32b_x32(ts + x0, v[0]);
          tc_ld_32x32b_x32(ts + x0 + 32, v[1]);
          tc_wait_ld_of(v[0]);
          tc_wait_ld_of(v[1]);
          // The scores are read; after the last row tile's the next codes stand ready.
          if (x0 && (r + 1 < tiles || n + 2 < N)) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(a_full(i));
          }
          const int row0 = r * kWtTile + x0;
          const uint8_t* row = smem + lse_at + 4 * row0;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(row + 4 * k);  // -lse of four rows
              const uint32_t* y = &v[k >> 5][k & 31];
              const float2 e0 = f32x2_get(fma_f32x2(f32x2(__uint_as_float(y[0]), __uint_as_float(y[1])), c2, l.x));
              const float2 e1 = f32x2_get(fma_f32x2(f32x2(__uint_as_float(y[2]), __uint_as_float(y[3])), c2, l.y));
              part[(k >> 1) & 2] = add_f32x2(part[(k >> 1) & 2], f32x2(ex2(e0.x), ex2(e0.y)));
              part[((k >> 1) & 2) + 1] = add_f32x2(part[((k >> 1) & 2) + 1], f32x2(ex2(e1.x), ex2(e1.y)));
            }
          } else {
            const int node = j - s.old, words = P.tree_words, word = max(node, 0) >> 5;
            uint32_t mask = base + masks_at + 4 * (row0 * words + min(word, words - 1));
            // All rows see the tokens before the new ones, none the new ones that no word stands for.
            const uint32_t before = node < 0 ? 0xffffffffu : 0u, named = word < words ? 0xffffffffu : 0u;
#pragma unroll
            for (int k = 0; k < 64; k += 2, mask += 8 * words) {
              const float2 l = *reinterpret_cast<const float2*>(row + 4 * k);
              const float e0 = fmaf(__uint_as_float(v[k >> 5][k & 31]), c, l.x);
              const float e1 = fmaf(__uint_as_float(v[k >> 5][(k & 31) + 1]), c, l.y);
              const bool see0 = (((lds32(mask) & named) | before) >> (node & 31)) & 1u;
              const bool see1 = (((lds32(mask + 4 * words) & named) | before) >> (node & 31)) & 1u;
              part[(k >> 1) & 3] = add_f32x2(part[(k >> 1) & 3], f32x2(see0 ? ex2(e0) : 0.f, see1 ? ex2(e1) : 0.f));
            }
          }
        }
      }
      if (!alive) break;
      const float2 all = f32x2_get(add_f32x2(add_f32x2(part[0], part[1]), add_f32x2(part[2], part[3])));
      if (j < j1) P.w_out[out + j] = (P.w_in ? P.w_in[out + j] : 0.f) + (counts ? all.x + all.y : 0.f);
    }
    tc_fence_before();
  } else {
    // ---------------- products ----------------
    constexpr uint32_t id = idesc_f16_f32(128, 128) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
    const uint32_t lead = elect_one(), tm0 = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq = smem_desc_sw128(base + SH::Q);
    bool alive = true;
#pragma unroll 1
    for (int n0 = 0; n0 < N && alive; n0 += 2) {
#pragma unroll 1
      for (int x = 0; x < 2 * tiles && alive; ++x) {  // the two tiles' rows in turn
        const int i = x & 1, r = x >> 1, turn = n0 >> 1, unit = turn * tiles + r;
        if (n0 + i >= N) continue;
        alive = __all_sync(0xffffffffu, wait_bar(a_full(i), (uint32_t)unit & 1u, abort_flag, &s_err_kvbw));
        if (!alive) break;
        tc_fence_after();
        const uint64_t db = dq + (uint64_t)r * (SH::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts_if(lead, tm0 + 256 + 128 * i, tm0 + 128 * i + 64 * (turn & 1) + 8 * k,
                    db + (k >> 2) * (uint64_t)(SH::PANEL >> 4) + (uint64_t)((k & 3) * 2), id, k > 0);
        commit_if(lead, s_full(i));
      }
    }
    commit_if(lead, done);
    if (lead) {  // nothing is left in flight when tensor memory is freed, on an abort either
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
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int D, bool BF16>
static tm_status launch_tree(const AttnParams& P, cudaStream_t stream) {
  using SH = RtShape<D>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(tree_weights_kernel<FMT, D, BF16>), SH::smem(kRtTiles, 16)))
    return TM_ERR_CUDA;
  // A start costs about as much as ten tiles.
  const long long ctas = (long long)P.V.B * P.V.Hkv, tiles = ((long long)P.V.max_len + kWtTile - 1) / kWtTile;
  const long long slices = slices_by_waves(ctas, tiles, 10, 0, 64);
  const long long slice = ((tiles + slices - 1) / slices > 4 ? (tiles + slices - 1) / slices : 4) * kWtTile;
  const dim3 grid((unsigned)ctas, (unsigned)((P.w_stride + slice - 1) / slice));
  const uint32_t smem = SH::smem((P.V.max_q * P.G + kWtTile - 1) / kWtTile, P.tree_words);
  tree_weights_kernel<FMT, D, BF16><<<grid, kRtThreads, smem, stream>>>(P, (int)slice);
  return cudaGetLastError() == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

template <int FMT, int D, bool BF16, bool TREE>
static tm_status launch(const AttnParams& P, cudaStream_t stream) {
  using SH = WtShape<D>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(weights_kernel<FMT, D, BF16, TREE>), SH::SMEM)) return TM_ERR_CUDA;
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
  return cudaLaunchKernelEx(&cfg, weights_kernel<FMT, D, BF16, TREE>, Q) == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

template <int FMT, int D>
static tm_status launch(const AttnParams& P, cudaStream_t stream) {
  if (P.tree && (long long)P.V.max_q * P.G <= kRtTiles * kWtTile)
    return P.bf16 ? launch_tree<FMT, D, true>(P, stream) : launch_tree<FMT, D, false>(P, stream);
  if (P.tree) return P.bf16 ? launch<FMT, D, true, true>(P, stream) : launch<FMT, D, false, true>(P, stream);
  return P.bf16 ? launch<FMT, D, true, false>(P, stream) : launch<FMT, D, false, false>(P, stream);
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
