// Attention over the paged 8-bit KV cache for few rows (single tokens, drafts):
// memory-bound, on mma.m16n8k16 straight from the codes.
//
// With one scale per page and head, s_j = (q . c_j) a with a = ks scale log2(e),
// and the output sum_j p_j vs c'_j.  The codes enter the products as exact fp16
// numbers; ks multiplies the fp32 scores, and vs goes into the exponent:
//   w_j = 2^(s_j + log2 vs - m + 6),  out = sum_j w_j c'_j / sum_j w_j / vs,
// m the running maximum of s_j + log2 vs, so that the fp16 weights keep their
// precision whatever the pages' value scales are.  The 6 moves the weights away
// from fp16's subnormals; m only moves when the maximum has grown by more
// than 8, so w < 2^14 and the accumulators are rarely rescaled.
//
// A CTA takes one (sequence, KV head), up to 8, 16 or 32 rows (query token,
// query head of the group) and a slice of the tokens.  Its four warps take steps of 32
// tokens in turn, each with a running softmax and a TMA ring of its own (a
// 16-token group of a page and head is one swizzled box), so that no warp
// waits for another before the end.  All rows share the conversion of the codes,
// which is most of the arithmetic.  The slices' partial states go through a
// workspace, and a second launch joins them and sums the tokens' weights.
//
// Order of tokens and dimensions: the K fragment's column n holds token
// sigma(n) of an 8-token group, a lane's 16-byte chunk holds 16 dimensions that
// four k-steps take word by word (the queries are read in the same order), and
// the V fragment's column n holds dimension 16 n + i of n-tile i (D = 128; 8 n + i
// for 64).  sigma and the swizzle make all shared loads conflict-free.
//
// Measured: 32 x up to 4096 tokens, int8, 32 query and 8 KV heads, weights: 62 us for 217 MB of codes (first
// launch 50, 0.62 of the HBM copy rate); 2 x 131072 tokens, e4m3, 64 query heads: 90 us for 453 MB (first
// launch 80, 0.83).  No unit is full there (issue slots 52 and 45 %, ALU pipe 49 %): what counts is the latency
// of dependent instructions, 3.8 of a thread per byte of codes, at 12 warps an SM (by registers and shared
// memory).  16 rows in place of 8: 65.4 and 94.4 us; 16 tokens a step with 12 or 16 warps: 65 to 88 and 96 to 119.
// 13 x up to 1531 tokens, e4m3, 12 heads of 64 not shared, weights: 17 us for 23 MB, a launch of about 12 (624 CTAs,
// 37 % of the issue slots, waiting for memory) and one of 8 (15 %, chains of loads and barriers).
#include <cfloat>
#include <cmath>

#include "kvb_attn.h"
#include "kvb_ring.h"

namespace w4 {
namespace kvb {

static __device__ uint32_t s_err_kvbd;

constexpr int kFewWarps = 4;
constexpr int kStep = 32;                      // tokens per step of a warp
constexpr int kTile = kFewWarps * kStep;       // tokens per round of the warps
constexpr float kBias = 6.f;                   // log2 of the largest weight right after m moved
constexpr float kSlack = 8.f;
constexpr float kNone = -1e30f;                // m of a row that has seen nothing
constexpr float kLn2 = 0.693147180559945f;

template <int D>
__device__ __forceinline__ int sigma(int n) {
  if (D == 128) return n ^ ((n & 1) << 2);
  const int m = n >> 1;
  return ((m & 1) | ((m >> 1) << 2)) ^ ((n & 1) * 3);
}
// Byte offset of 16-byte chunk c of row r of a 16-token box (the TMA's 128- or 64-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// RT: 16-row tiles; 0: one half tile (rows 8 .. 15 of the products stay empty).
template <int D, int RT>
struct FewShape {
  static constexpr int TILES = RT == 0 ? 1 : RT;
  static constexpr int E = RT == 0 ? 1 : 2;  // rows per lane and tile
  static constexpr int ROWS = TILES * 8 * E;
  static constexpr uint32_t BOX = 16 * D;
  static constexpr uint32_t STAGE = 4 * BOX;  // K of two groups, V of two groups
  static constexpr int STAGES = D == 128 && RT < 2 ? 2 : 3;
  static constexpr int CTAS = RT == 2 ? 2 : 3;  // per SM, by registers and shared memory
  static constexpr uint32_t RING = kFewWarps * STAGES * STAGE;
  static constexpr int STATE = TILES * E * (8 * D + 16);  // floats of a warp's state
  static constexpr uint32_t BODY = RING > 2 * STATE * 4 ? RING : 2 * STATE * 4;
  static constexpr uint32_t Q_OFF = BODY;  // RT == 2: query fragments
  static constexpr uint32_t BARS = Q_OFF + (RT == 2 ? TILES * (D / 16) * 512 : 0);
  static constexpr uint32_t SMEM = BARS + kFewWarps * STAGES * 8 + 16 + 1024;
};

// d (rows 0 .. 7 of the tile) += a . b with rows 8 .. 15 of a zero.
__device__ __forceinline__ void mma_top(float& d0, float& d1, uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  [[maybe_unused]] float x, y;
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};\n"
      : "+f"(d0), "+f"(d1), "=f"(x), "=f"(y)
      : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}

// A warp that gives up at step i of `steps`: none of its copies may land in memory that the join is about to
// use.  (Inlined, it costs the loop registers: 1 % of the full batch's time.)
template <int S>
__device__ __noinline__ void drain_copies(uint32_t bars, int i, int steps) {
  const unsigned long long t0 = globaltimer();
  ring_drain<S>(i, steps, [&](int stage, uint32_t parity) {
    while (!mbar_try_wait(bars + 8 * stage, parity) && globaltimer() - t0 < kWaitLimitNs) {
    }
  });
}

// KEEP: the scores are kept for the tokens' weights.
template <int FMT, int D, int RT, bool KEEP>
__global__ void __launch_bounds__(32 * kFewWarps, FewShape<D, RT>::CTAS)
    attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams P) {
  using SH = FewShape<D, RT>;
  constexpr int TILES = SH::TILES, E = SH::E, S = SH::STAGES;
  constexpr int NV = D / 8;   // n-tiles of the output
  constexpr int KS = D / 16;  // k-steps of the scores
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  const View& V = P.V;
  const int b = blockIdx.z, chunk = blockIdx.x;
  const int h = blockIdx.y % V.Hkv, rg = blockIdx.y / V.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const Span s = span(V, b);
  const int rows = s.n * P.G;
  const int row_base = rg * SH::ROWS;
  if (row_base >= rows) return;
  // Tokens [j0, j1) that some row of the group sees; all rows see those up to `all`.
  const int last_i = (min(row_base + SH::ROWS, rows) - 1) / P.G;
  const int j0 = chunk * P.chunk;
  const int j1 = min(min(s.len, j0 + P.chunk), s.old + last_i + 1);
  const int all = min(s.old + row_base / P.G, j1 - 1);
  if (j0 >= j1 && chunk > 0) return;  // slice 0 still writes what an empty row gives
  const int steps = j1 > j0 ? (j1 - j0 + kStep - 1) / kStep : 0;
  const int mine = steps > warp ? (steps - warp + kFewWarps - 1) / kFewWarps : 0;

  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::BARS + kFewWarps * S * 8);
  if (tid == 0) {
    for (int i = 0; i < kFewWarps * S; ++i) mbar_init(base + SH::BARS + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  launch_dependents();

  // ---- pages and scales, 16 steps at a time and one batch ahead: lane 2 k + g has group g of the batch's step k
  struct Meta {
    int cell, slot;
    float ks, lv;
  };
  auto load_meta = [&](int batch) {
    const int j = j0 + ((batch * 16 + (lane >> 1)) * kFewWarps + warp) * kStep + 16 * (lane & 1);
    const int page = j < j1 ? page_of(V, V.table, b, V.table_stride, j >> V.t_shift) : -1;
    Meta m;
    m.cell = page >= 0 ? page * V.Hkv + h : -1;
    m.slot = j & ((1 << V.t_shift) - 1);
    m.ks = page >= 0 ? V.ks[m.cell] : 1.f;
    // 2^lv stands for vs; its own inverse takes it out of l again, so that lv's rounding stays in the output: 2 ulp
    // of lv, 2^-18.5 of vs at the smallest scales (|lv| of 16 or more), 2^-19.5 at scales above 2^-16.
    m.lv = page >= 0 ? __log2f(fmaxf(V.vs[m.cell], kScaleFloor)) : 0.f;
    return m;
  };
  Meta cur = load_meta(0), nxt = load_meta(1);
  const uint32_t ring = base + warp * S * SH::STAGE, bars = base + SH::BARS + warp * S * 8;
  auto issue = [&](int i, int batch) {  // batch: of `cur`
    if (i >= mine) return;
    const bool ahead = (i >> 4) != batch;
    const int from = (2 * i & 31) + (lane & 1);
    const int cell = __shfl_sync(0xffffffffu, ahead ? nxt.cell : cur.cell, from);
    const int slot = __shfl_sync(0xffffffffu, ahead ? nxt.slot : cur.slot, from);
    const uint32_t there = __popc(__ballot_sync(0xffffffffu, cell >= 0 && lane < 2));
    const uint32_t bar = bars + 8 * ring_stage<S>(i);
    if (lane == 0) mbar_expect_tx(bar, there * 2 * SH::BOX);
    __syncwarp();
    if (lane < 4 && cell >= 0)
      tma_load_3d(ring + ring_stage<S>(i) * SH::STAGE + lane * SH::BOX, lane < 2 ? &tmK : &tmV, 0, slot, cell, bar);
  };
#pragma unroll
  for (int i = 0; i < S; ++i) issue(i, 0);

  // ---- the queries, once, in the k order of the codes; bf16 rows are scaled by a
  // power of two into fp16's range: exact for elements of 2^-31 of the row's maximum or more, off by at most
  // 2^-39 of it for smaller ones
  uint32_t qa[RT == 2 ? 1 : KS][RT == 0 ? 2 : 4];
  float mul[TILES][E];
  int last[TILES][E];  // last visible token (-1: no row)
  size_t hr[TILES][E];
#pragma unroll
  for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int row = row_base + rt * 16 + gr + 8 * e;
      const bool ok = row < rows;
      const int i = ok ? row / P.G : 0;
      const int hq = h * P.G + (ok ? row - i * P.G : 0);
      last[rt][e] = ok ? min(s.old + i, s.len - 1) : -1;
      hr[rt][e] = (size_t)(s.row0 + i) * P.Hq + hq;
      const uint16_t* q = P.Q + (s.row0 + i) * P.q_stride + (long long)hq * D;
      uint32_t raw[KS][2];
#pragma unroll
      for (int j = 0; j < KS / 4; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 x = ok ? *reinterpret_cast<const uint4*>(q + 16 * (t + 4 * j) + 8 * k) : make_uint4(0, 0, 0, 0);
          raw[4 * j + 2 * k][0] = x.x;
          raw[4 * j + 2 * k][1] = x.y;
          raw[4 * j + 2 * k + 1][0] = x.z;
          raw[4 * j + 2 * k + 1][1] = x.w;
        }
      float qs = 1.f;
      if (P.bf16) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = unpack(raw[k][x], true);
            m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e2 = max((int)(__float_as_uint(m) >> 23) - 127, -100);  // m < 2^(e2 + 1)
        const float up = __uint_as_float((uint32_t)(127 + min(14 - e2, 126)) << 23);
        qs = __uint_as_float((uint32_t)(127 - min(14 - e2, 126)) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = unpack(raw[k][x], true);
            raw[k][x] = pack_half2(f.x * up, f.y * up);
          }
      }
      mul[rt][e] = qs * P.scale_log2;
      if constexpr (RT == 2) {
        if ((warp & 1) == rt) {  // two warps write the same values for each tile: no exchange needed
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t at = base + SH::Q_OFF + ((rt * KS + k) * 32 + lane) * 16 + 4 * e;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(raw[k][0]) : "memory");
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 8), "r"(raw[k][1]) : "memory");
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qa[k][e] = raw[k][0];
          qa[k][E + e] = raw[k][1];
        }
      }
    }
  if constexpr (RT == 2) __syncthreads();

  float o[TILES][NV][2 * E];
  float m[TILES][E], l[TILES][E];
#pragma unroll
  for (int rt = 0; rt < TILES; ++rt) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int x = 0; x < 2 * E; ++x) o[rt][i][x] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      m[rt][e] = kNone;
      l[rt][e] = 0.f;
    }
  }
  const int sg[2] = {sigma<D>(2 * t), sigma<D>(2 * t + 1)};
  const int kr = sigma<D>(gr);
  float* srow = P.scores + ((size_t)h * V.rows * P.G + (size_t)s.row0 * P.G + row_base + gr) * P.score_stride;

  for (int i = 0; i < mine; ++i) {
    const int batch = i >> 4;
    if (i > 0 && (i & 15) == 0) {
      cur = nxt;
      nxt = load_meta(batch + 1);
    }
    const bool alive = mbar_wait(bars + 8 * ring_stage<S>(i), ring_parity<S>(i), abort_flag, &s_err_kvbd);
    if (!__all_sync(0xffffffffu, alive)) {
      drain_copies<S>(bars, i, mine);
      break;
    }
    // plain shared loads, so that the compiler may bring them forward
    const uint8_t* kt = smem + (ring - base) + ring_stage<S>(i) * SH::STAGE;
    const uint8_t* vt = kt + 2 * SH::BOX;
    const int tok0 = j0 + (i * kFewWarps + warp) * kStep;
    float ks[2], lv[2];
    bool there[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int from = (2 * i & 31) + g;
      ks[g] = __shfl_sync(0xffffffffu, cur.ks, from);
      lv[g] = __shfl_sync(0xffffffffu, cur.lv, from);
      there[g] = __shfl_sync(0xffffffffu, cur.cell, from) >= 0;
    }
    // Whether some row does not see some token (warp-uniform).
    const bool part = tok0 + kStep - 1 > all || !there[0] || !there[1];
    // ---- scores: rows x 32 tokens
    float sc[TILES][4][2 * E];
#pragma unroll
    for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int x = 0; x < 2 * E; ++x) sc[rt][a][x] = 0.f;
    if constexpr (RT < 2) {
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int j = 0; j < KS / 4; ++j) {
          const uint4 x =
              *reinterpret_cast<const uint4*>(kt + (a >> 1) * SH::BOX + swz<D>(8 * (a & 1) + kr, t + 4 * j));
          const uint32_t kw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b0, b1;
            codes_half<FMT>(kw[k], b0, b1);
            if constexpr (RT == 0)
              mma_top(sc[0][a][0], sc[0][a][1], qa[4 * j + k][0], qa[4 * j + k][1], b0, b1);
            else
              mma_16816(sc[0][a], qa[4 * j + k], b0, b1);
          }
        }
    } else {
      // the queries' fragments come from shared memory: once for the four 8-token groups
#pragma unroll
      for (int j = 0; j < KS / 4; ++j) {
        uint32_t kw[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const uint4 x =
              *reinterpret_cast<const uint4*>(kt + (a >> 1) * SH::BOX + swz<D>(8 * (a & 1) + kr, t + 4 * j));
          kw[a][0] = x.x;
          kw[a][1] = x.y;
          kw[a][2] = x.z;
          kw[a][3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t fa[TILES][4];
#pragma unroll
          for (int rt = 0; rt < TILES; ++rt) {
            const uint4 f =
                *reinterpret_cast<const uint4*>(smem + SH::Q_OFF + ((rt * KS + 4 * j + k) * 32 + lane) * 16);
            fa[rt][0] = f.x;
            fa[rt][1] = f.y;
            fa[rt][2] = f.z;
            fa[rt][3] = f.w;
          }
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            uint32_t b0, b1;
            codes_half<FMT>(kw[a][k], b0, b1);
#pragma unroll
            for (int rt = 0; rt < TILES; ++rt) mma_16816(sc[rt][a], fa[rt], b0, b1);
          }
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int x = 0; x < 2; ++x) sc[rt][a][2 * e + x] *= ks[a >> 1] * mul[rt][e];
    if (part)
#pragma unroll
      for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!there[a >> 1] || tok0 + 8 * a + sg[x] > last[rt][e]) sc[rt][a][2 * e + x] = -INFINITY;
    // The scores for the weights.  With more than 8 rows a swap makes a lane's two tokens neighbours, so that four
    // lanes write a whole sector (16 x 5 drafts: 65 us, without 68 then); with 8 its registers cost more (32 x 4096
    // tokens: 66, without 64).
    if constexpr (KEEP && RT == 0) {
      if (last[0][0] >= 0) {
        float* row = srow + tok0;
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int x = 0; x < 2; ++x) row[8 * a + sg[x]] = sc[0][a][x];
      }
    } else if constexpr (KEEP) {
#pragma unroll
      for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* row = srow + (size_t)(rt * 16 + 8 * e) * P.score_stride + tok0 + 2 * t;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            float x = sc[rt][a][2 * e], y = sc[rt][a][2 * e + 1];
            if constexpr (D == 128) {
              y = __shfl_xor_sync(0xffffffffu, y, 2);
            } else {
              const float z = __shfl_xor_sync(0xffffffffu, t & 1 ? x : y, 1);
              x = t & 1 ? y : x;
              y = z;
            }
            if (last[rt][e] >= 0) *reinterpret_cast<float2*>(row + 8 * a) = make_float2(x, y);
          }
        }
    }
    // ---- softmax
    uint32_t pa[TILES][2][2 * E];  // per 16-token group: A fragment
    const float inv[2] = {ex2(-lv[0]), ex2(-lv[1])};
#pragma unroll
    for (int rt = 0; rt < TILES; ++rt) {
      float tm[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        auto v = [&](int a, int x) { return sc[rt][a][2 * e + x]; };
        tm[e] = fmaxf(fmaxf(fmaxf(v(0, 0), v(0, 1)), fmaxf(v(1, 0), v(1, 1))) + lv[0],
                      fmaxf(fmaxf(v(2, 0), v(2, 1)), fmaxf(v(3, 0), v(3, 1))) + lv[1]);
        tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xffffffffu, tm[e], 1));
        tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xffffffffu, tm[e], 2));
      }
      if (__any_sync(0xffffffffu, tm[0] > m[rt][0] + kSlack || tm[E - 1] > m[rt][E - 1] + kSlack)) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float mn = fmaxf(m[rt][e], tm[e]);
          const float f = ex2(m[rt][e] - mn);
          m[rt][e] = mn;
          l[rt][e] *= f;
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            o[rt][k][2 * e] *= f;
            o[rt][k][2 * e + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float off = lv[g] + kBias - m[rt][e];
          float sum = 0.f;
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const float p0 = ex2(sc[rt][2 * g + a][2 * e] + off), p1 = ex2(sc[rt][2 * g + a][2 * e + 1] + off);
            sum += p0 + p1;
            pa[rt][g][E * a + e] = pack_half2(p0, p1);  // the codes' type in the product; l keeps all bits
          }
          l[rt][e] = fmaf(sum, inv[g], l[rt][e]);
        }
    }
    // ---- values: rows x 32 tokens x D
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      constexpr int W = D / 32;  // words of codes per lane and token
      uint32_t wv[4][W];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 8 * (q >> 1) + sg[q & 1];
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vt + g * SH::BOX + swz<D>(r, gr));
          wv[q][0] = x.x;
          wv[q][1] = x.y;
          wv[q][2] = x.z;
          wv[q][3] = x.w;
        } else {
          const uint2 x =
              *reinterpret_cast<const uint2*>(vt + g * SH::BOX + swz<D>(r, gr >> 1) + 8 * (gr & 1));
          wv[q][0] = x.x;
          wv[q][1] = x.y;
        }
        // Slots past the end and the boxes of holes hold anything, NaN codes too.
        if (part && (!there[g] || tok0 + 16 * g + r >= j1))
#pragma unroll
          for (int k = 0; k < W; ++k) wv[q][k] = 0u;
      }
#pragma unroll
      for (int k = 0; k < W; ++k) {
        uint32_t b0[4], b1[4];
        codes_half_pairs<FMT>(wv[0][k], wv[1][k], b0);
        codes_half_pairs<FMT>(wv[2][k], wv[3][k], b1);
#pragma unroll
        for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if constexpr (RT == 0)
              mma_top(o[0][4 * k + c][0], o[0][4 * k + c][1], pa[0][g][0], pa[0][g][1], b0[c], b1[c]);
            else
              mma_16816(o[rt][4 * k + c], pa[rt][g], b0[c], b1[c]);
          }
      }
    }
    __syncwarp();  // the stage is read: it may be filled again
    issue(i + S, batch);
  }
  __syncthreads();

  // ---- join the four warps: 2, 3 into 0, 1, then 1 into 0
  float* st = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      l[rt][e] += __shfl_xor_sync(0xffffffffu, l[rt][e], 1);
      l[rt][e] += __shfl_xor_sync(0xffffffffu, l[rt][e], 2);
    }
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (warp >= step && warp < 2 * step) {
      float* dst = st + (size_t)(warp - step) * SH::STATE;
#pragma unroll
      for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* part = dst + (rt * E + e) * (8 * D + 16);
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            part[(2 * k) * 32 + lane] = o[rt][k][2 * e];
            part[(2 * k + 1) * 32 + lane] = o[rt][k][2 * e + 1];
          }
          if (t == 0) {
            part[8 * D + gr] = m[rt][e];
            part[8 * D + 8 + gr] = l[rt][e];
          }
        }
    }
    __syncthreads();
    if (warp < step) {
      const float* src = st + (size_t)warp * SH::STATE;
#pragma unroll
      for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float* part = src + (rt * E + e) * (8 * D + 16);
          const float m2 = part[8 * D + gr], l2 = part[8 * D + 8 + gr];
          const float mn = fmaxf(m[rt][e], m2), f1 = ex2(m[rt][e] - mn), f2 = ex2(m2 - mn);
          m[rt][e] = mn;
          l[rt][e] = l[rt][e] * f1 + l2 * f2;
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            o[rt][k][2 * e] = o[rt][k][2 * e] * f1 + part[(2 * k) * 32 + lane] * f2;
            o[rt][k][2 * e + 1] = o[rt][k][2 * e + 1] * f1 + part[(2 * k + 1) * 32 + lane] * f2;
          }
        }
    }
    __syncthreads();
  }
  if (warp != 0) return;
  // ---- one slice: the output; several: the state, for the second launch
  constexpr int SPAN = D / 8;  // dimensions of one column: column n of n-tile i is dimension SPAN n + i
#pragma unroll
  for (int rt = 0; rt < TILES; ++rt)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (row_base + rt * 16 + gr + 8 * e >= rows) continue;
      const size_t at = hr[rt][e];
      const float lsum = l[rt][e];
      if (P.chunks == 1) {
        const float r = lsum > 0.f || lsum != lsum ? __fdividef(1.f, lsum) : 0.f;
        uint16_t* out = P.out + at * D + 2 * t * SPAN;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < NV; i += 8) {
            uint32_t wd[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f0 = o[rt][i + 2 * k][2 * e + x] * r, f1 = o[rt][i + 2 * k + 1][2 * e + x] * r;
              wd[k] = P.bf16 ? pack_bf162(f0, f1) : pack_half2(f0, f1);
            }
            *reinterpret_cast<uint4*>(out + x * SPAN + i) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
          }
        if (t == 0 && P.lse) P.lse[at] = lsum == 0.f ? -INFINITY : (log2f(lsum) + m[rt][e] - kBias) * kLn2;
      } else {
        float* dst = P.part + (at * P.chunks + chunk) * D + 2 * t * SPAN;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < NV; i += 4)
            *reinterpret_cast<float4*>(dst + x * SPAN + i) = make_float4(o[rt][i][2 * e + x], o[rt][i + 1][2 * e + x],
                                                                         o[rt][i + 2][2 * e + x], o[rt][i + 3][2 * e + x]);
      }
      if (t == 0 && P.part_ml) P.part_ml[at * P.chunks + chunk] = make_float2(m[rt][e] - kBias, lsum);
    }
}

// Slices that the CTAs of row (query i, head g of the group) wrote: up to the
// last token that the rows they share see, and slice 0.
__device__ __forceinline__ int slices_of(const AttnParams& P, const Span& s, int i, int g) {
  const int per = P.rows_per_cta;
  const int last_i = (min(((i * P.G + g) / per + 1) * per, s.n * P.G) - 1) / P.G;
  const int end = min(s.len, s.old + last_i + 1);
  return end > 0 ? (end + P.chunk - 1) / P.chunk : 1;
}

// ---- second launch: blocks below `joins` join the slices of their rows
// (P.wpr warps per row), the others sum the weights that tokens drew, one thread per four
// tokens of a (sequence, KV head), rows in order.
constexpr int kFinishThreads = 256;
constexpr int kWeightTokens = 4 * kFinishThreads;

template <int D>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const AttnParams P, int joins) {
  constexpr int E = D / 32;
  __shared__ float acc_s[8][D], l_s[8];
  __shared__ float lse_s[kFewRows];
  __shared__ int see_s[kFewRows];  // the last token that a row sees
  const View& V = P.V;
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Span s = span(V, b);  // written before the first launch began
  grid_dependency_wait();
  if ((int)blockIdx.x < joins) {
    const int wpr = P.wpr, sub = warp % wpr;
    const int at = blockIdx.x * (8 / wpr) + warp / wpr;
    const int i = at / P.Hq;
    const bool ok = i < s.n;
    const size_t hr = (size_t)(s.row0 + (ok ? i : 0)) * P.Hq + (at - i * P.Hq);
    const int n = ok ? slices_of(P, s, i, (at - i * P.Hq) % P.G) : 0;
    const float2* ml = P.part_ml + hr * P.chunks;
    float m = kNone;
    for (int c = lane; c < n; c += 32) m = fmaxf(m, ml[c].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, acc[E] = {};
#pragma unroll 4
    for (int c = sub; c < n; c += wpr) {
      const float2 v = ml[c];
      const float f = ex2(v.x - m);
      l = fmaf(v.y, f, l);
      const float* src = P.part + (hr * P.chunks + c) * D + lane * E;
#pragma unroll
      for (int k = 0; k < E; ++k) acc[k] = fmaf(src[k], f, acc[k]);
    }
    if (wpr > 1) {  // the row's warps, in order
#pragma unroll
      for (int k = 0; k < E; ++k) acc_s[warp][lane * E + k] = acc[k];
      if (lane == 0) l_s[warp] = l;
      __syncthreads();
      if (sub) return;
      for (int x = 1; x < wpr; ++x) {
        l += l_s[warp + x];
#pragma unroll
        for (int k = 0; k < E; ++k) acc[k] += acc_s[warp + x][lane * E + k];
      }
    }
    if (!ok) return;
    const float r = l > 0.f || l != l ? __fdividef(1.f, l) : 0.f;
    uint32_t* out = reinterpret_cast<uint32_t*>(P.out + hr * D + lane * E);
#pragma unroll
    for (int k = 0; k < E; k += 2)
      out[k / 2] = P.bf16 ? pack_bf162(acc[k] * r, acc[k + 1] * r) : pack_half2(acc[k] * r, acc[k + 1] * r);
    if (lane == 0 && P.lse) P.lse[hr] = l == 0.f ? -INFINITY : (log2f(l) + m) * kLn2;
    return;
  }
  // ---- weights
  const int blocks = (int)((P.w_stride + kWeightTokens - 1) / kWeightTokens);
  const int h = ((int)blockIdx.x - joins) / blocks, part = ((int)blockIdx.x - joins) - h * blocks;
  const int rows = s.n * P.G;  // at most kFewRows
  if (part * kWeightTokens < s.len) {
    // lse of every row at once: eight threads per row, 32 rows at a time
    for (int row = tid >> 3; row < (rows + 31) / 32 * 32; row += 32) {
      float m = kNone, l = 0.f;
      if (row < rows) {
        const int i = row / P.G, g = row - i * P.G;
        const int n = slices_of(P, s, i, g);
        const float2* ml = P.part_ml + ((size_t)(s.row0 + i) * P.Hq + h * P.G + g) * P.chunks;
        for (int c = tid & 7; c < n; c += 8) {
          const float2 v = ml[c];
          const float mn = fmaxf(m, v.x);
          l = l * ex2(m - mn) + v.y * ex2(v.x - mn);
          m = mn;
        }
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        const float mn = fmaxf(m, m2);
        l = l * ex2(m - mn) + l2 * ex2(m2 - mn);
        m = mn;
      }
      if ((tid & 7) == 0 && row < rows) {
        lse_s[row] = l == 0.f ? INFINITY : log2f(l) + m;  // nothing seen: no weight
        see_s[row] = min(s.old + row / P.G, s.len - 1);
      }
    }
  }
  __syncthreads();
  // Four tokens per thread.  The rows' CTAs wrote every score up to the row's last visible token;
  // what the row does not see before that (holes) is -inf.
  const size_t head = ((size_t)b * V.Hkv + h) * P.w_stride;
  const int j = part * kWeightTokens + 4 * tid;
  if (j >= P.w_stride) return;
  float sum[4] = {};
  if (j < s.len) {
    const int r0 = max(j - s.old, 0) * P.G;  // rows from here on see the first of them,
    const int r4 = j + 3 < s.len ? min(max(j + 3 - s.old, 0) * P.G, rows) : rows;  // and from here on all four
    const float* sc = P.scores + ((size_t)h * V.rows + s.row0) * P.G * P.score_stride + j;
#pragma unroll 8
    for (int row = r0; row < r4; ++row) {
      const float4 x = *reinterpret_cast<const float4*>(sc + row * P.score_stride);
      const float y = lse_s[row];
      const int see = see_s[row] - j;
      sum[0] += see >= 0 ? ex2(x.x - y) : 0.f;
      sum[1] += see >= 1 ? ex2(x.y - y) : 0.f;
      sum[2] += see >= 2 ? ex2(x.z - y) : 0.f;
      sum[3] += see >= 3 ? ex2(x.w - y) : 0.f;
    }
#pragma unroll 8
    for (int row = r4; row < rows; ++row) {
      const float4 x = *reinterpret_cast<const float4*>(sc + row * P.score_stride);
      const float y = lse_s[row];
      sum[0] += ex2(x.x - y);
      sum[1] += ex2(x.y - y);
      sum[2] += ex2(x.z - y);
      sum[3] += ex2(x.w - y);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (j + k < P.w_stride) P.w_out[head + j + k] = (P.w_in ? P.w_in[head + j + k] : 0.f) + sum[k];
}

template <int FMT, int D, int RT, bool KEEP>
tm_status launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& P, int groups, cudaStream_t s) {
  using SH = FewShape<D, RT>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(attn_kernel<FMT, D, RT, KEEP>), SH::SMEM)) return TM_ERR_CUDA;
  const dim3 grid((unsigned)P.chunks, (unsigned)(P.V.Hkv * groups), (unsigned)P.V.B);
  attn_kernel<FMT, D, RT, KEEP><<<grid, 32 * kFewWarps, SH::SMEM, s>>>(tmK, tmV, P);
  return cudaGetLastError() == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

template <int FMT, int D, bool KEEP>
tm_status launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& P, int rt, int groups,
                      cudaStream_t s) {
  if (rt == 0) return launch_attn<FMT, D, 0, KEEP>(tmK, tmV, P, groups, s);
  if (rt == 1) return launch_attn<FMT, D, 1, KEEP>(tmK, tmV, P, groups, s);
  return launch_attn<FMT, D, 2, KEEP>(tmK, tmV, P, groups, s);
}

// A 16-token box of a pool [cells][T][D]; inner rows of D bytes, swizzled over their width.
static bool pool_map(CUtensorMap* map, void* pool, const View& V, int D) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t cells = (cuuint64_t)(V.pages > 0 ? V.pages : 1) * V.Hkv, T = 1ull << V.t_shift;
  const cuuint64_t dims[3] = {(cuuint64_t)D, T, cells};
  const cuuint64_t strides[2] = {(cuuint64_t)D, T * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, 16, 1}, ones[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch settings and the workspace's layout, from the host fields alone.
struct Plan {
  int rt;            // the kernel for few rows: its row tiles (0, 1, 2; see FewShape); -1: the tcgen05 kernel
  int rows_per_cta;  // rows that share a CTA
  int groups;        // CTAs along the rows
  int chunk, chunks;
  bool scores;  // token weights from kept scores (few rows), else from a second pass
  size_t part, part_ml, lse, score, bytes;  // offsets, total
};

static Plan make_plan(const View& V, int D, int Hq, bool weights) {
  Plan p = {};
  const int G = Hq / V.Hkv;
  const long long rows = (long long)V.max_q * G;
  const long long sms = num_sms(current_device());
  // 64 rows (16 sequences x 2000 tokens, 8 heads a group): this kernel 51.5 us, with weights 99.6; the tcgen05
  // kernel 47.6, with its second pass for the weights 124.  At 32 rows this one takes 39.
  p.rt = rows <= 8 ? 0 : rows <= 16 ? 1 : rows <= (weights ? kFewRows : kFewRows / 2) ? 2 : -1;
  p.rows_per_cta = p.rt == 0 ? 8 : p.rt > 0 ? 16 * p.rt : 256;
  p.groups = (int)((rows + p.rows_per_cta - 1) / p.rows_per_cta);
  const long long ctas = (long long)V.B * V.Hkv * p.groups;
  long long chunk, least, unit;
  if (p.rt >= 0) {
    // Slices for two waves of CTAs, none shorter than two steps per warp (2 x 131072 tokens: two waves
    // 94 us, four 98, eight 101 at the time: starting a CTA costs about 3 us).
    const long long slots = sms * (p.rt < 2 ? 3 : 2);
    unit = kTile;
    least = 2 * kTile;
    chunk = ((long long)V.max_len * ctas + 2 * slots - 1) / (2 * slots);
  } else {
    // Slices only where the rows alone leave SMs idle (300 tokens over 30000: 182 us; unsliced 574).
    unit = 128;
    least = 512;
    chunk = ctas >= sms ? V.max_len : ((long long)V.max_len * ctas + 2 * sms - 1) / (2 * sms);
  }
  chunk = (chunk + unit - 1) / unit * unit;
  if (chunk < least) chunk = least;
  long long chunks = (V.max_len + chunk - 1) / chunk;
  if (chunks < 1) chunks = 1;
  p.chunk = (int)(chunk > 0x7fffff80ll ? 0x7fffff80ll : chunk);
  p.chunks = (int)chunks;
  auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
  const size_t hr = (size_t)V.rows * Hq;
  size_t at = 0;
  p.scores = weights && p.rt >= 0;
  if (chunks > 1) {
    p.part = at;
    at = al(at + hr * chunks * D * 4);
  }
  if (chunks > 1 || p.scores) {
    p.part_ml = at;
    at = al(at + hr * chunks * 8);
  }
  if (weights) {
    if (p.scores) {
      p.score = at;
      at = al(at + hr * (((size_t)V.max_len + kTile - 1) / kTile * kTile) * 4);
    } else {
      p.lse = at;
      at = al(at + hr * 4);
    }
  }
  p.bytes = at;
  return p;
}

// Whether the first launch fits its grid, a KV head per group of rows along y.  (The others do by the limits of
// check and check_heads.)
static bool plan_fits(const View& V, const Plan& p) { return p.rt < 0 || (long long)V.Hkv * p.groups <= 65535; }

}  // namespace kvb

cudaError_t kvb_attn_error_bits(uint32_t* bits, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, kvb::s_err_kvbd, sizeof(v));
  if (e != cudaSuccess) return e;
  if (clear && v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(kvb::s_err_kvbd, &zero, sizeof(zero));
  }
  *bits = v;
  return e;
}

}  // namespace w4

using namespace w4;
using namespace w4::kvb;

static tm_status check_heads(const View& V, const tm_kvb_batch* batch, int Hq) {
  if (Hq < 1 || Hq % V.Hkv != 0) return TM_ERR_INVALID_ARG;
  const bool one_each = batch->q_start == nullptr;
  if (one_each && (batch->rows != batch->B || (batch->B > 0 && batch->max_q < 1))) return TM_ERR_INVALID_ARG;
  const long long rows = (long long)V.max_q * (Hq / V.Hkv);
  if (rows > 4000000ll || (long long)V.B * V.Hkv > 0x1fffffffll) return TM_ERR_UNSUPPORTED;  // the grid's limits
  return TM_OK;
}

extern "C" tm_status tm_kvb_attention_workspace(const tm_kvb_cache* cache, const tm_kvb_batch* batch, int Hq,
                                                int weights, size_t* bytes) {
  View V;
  if (!bytes) return TM_ERR_INVALID_ARG;
  tm_status st = check(cache, batch, false, &V);
  if (st == TM_OK) st = check_heads(V, batch, Hq);
  if (st != TM_OK) return st;
  *bytes = 0;
  if (V.B == 0 || V.rows == 0 || V.max_q == 0) return TM_OK;
  const Plan p = make_plan(V, cache->D, Hq, weights != 0);
  if (!plan_fits(V, p)) return TM_ERR_UNSUPPORTED;
  *bytes = p.bytes;
  return TM_OK;
}

template <int FMT, int D>
static tm_status run(AttnParams P, const Plan& p, const tm_kvb_cache* cache, cudaStream_t s, int* launches) {
  const View& V = P.V;
  tm_status st;
  if (p.rt < 0) {
    st = launch_prefill_attn(P, FMT, D, p.groups, s);
  } else {
    CUtensorMap tmK, tmV;
    if (!pool_map(&tmK, cache->k, V, D) || !pool_map(&tmV, cache->v, V, D)) return TM_ERR_CUDA;
    st = p.scores ? launch_attn<FMT, D, true>(tmK, tmV, P, p.rt, p.groups, s)
                  : launch_attn<FMT, D, false>(tmK, tmV, P, p.rt, p.groups, s);
  }
  if (st != TM_OK) return st;
  *launches = 1;
  // The second launch: the joins of several slices, and the weights from kept scores.
  // Eight warps a row where few rows have many slices (128 rows of 57: 91 us in all, with one warp 114), one
  // otherwise (4096 rows of 8: 39 us, with eight 45).
  P.wpr = P.chunks >= 8 && (long long)V.rows * P.Hq <= 8 * num_sms(current_device()) ? 8 : 1;
  const long long per = 8 / P.wpr;
  const long long joins = P.chunks > 1 ? ((long long)V.max_q * P.Hq + per - 1) / per : 0;
  const long long sums = p.scores ? (P.w_stride + kWeightTokens - 1) / kWeightTokens * V.Hkv : 0;
  if (joins + sums > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(joins + sums), (unsigned)V.B, 1);
    cfg.blockDim = dim3(kFinishThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, finish_kernel<D>, P, (int)joins) != cudaSuccess) return TM_ERR_CUDA;
    ++*launches;
  }
  if (P.w_out && !p.scores) {
    st = launch_row_weights(P, FMT, D, s);
    if (st != TM_OK) return st;
    ++*launches;
  }
  return TM_OK;
}

extern "C" tm_status tm_kvb_attention(const tm_kvb_cache* cache, const tm_kvb_batch* batch, const void* Q,
                                      long long q_stride, int Hq, int dtype, float scale, void* out, float* lse,
                                      const float* w_in, float* w_out, long long w_stride, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  AttnParams P = {};
  tm_status st = check(cache, batch, true, &P.V);
  if (st == TM_OK) st = check_heads(P.V, batch, Hq);
  if (st != TM_OK) return st;
  const View& V = P.V;
  if (dtype != TM_KVB_F16 && dtype != TM_KVB_BF16) return TM_ERR_INVALID_ARG;
  if (w_in && !w_out) return TM_ERR_INVALID_ARG;
  if (!(fabsf(scale) <= FLT_MAX)) return TM_ERR_INVALID_ARG;  // NaN too
  if (V.B == 0) return TM_OK;
  if (w_out && w_stride < V.max_len) return TM_ERR_INVALID_ARG;
  if (w_out && w_stride > 65535ll * 128) return TM_ERR_UNSUPPORTED;  // the grid's limit
  if (!aligned(w_in, 4) || !aligned(w_out, 4)) return TM_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (V.rows == 0 || V.max_q == 0) {  // no row draws weight: w_out = w_in
    if (!w_out || w_out == w_in) return TM_OK;
    const size_t bytes = (size_t)V.B * V.Hkv * w_stride * 4;
    const cudaError_t e = w_in ? cudaMemcpyAsync(w_out, w_in, bytes, cudaMemcpyDeviceToDevice, s)
                               : cudaMemsetAsync(w_out, 0, bytes, s);
    return e == cudaSuccess ? TM_OK : TM_ERR_CUDA;
  }
  if (!Q || !out || q_stride < (long long)Hq * cache->D) return TM_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || q_stride % 8 || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return TM_ERR_ALIGNMENT;
  const Plan p = make_plan(V, cache->D, Hq, w_out != nullptr);
  if (!plan_fits(V, p)) return TM_ERR_UNSUPPORTED;
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return TM_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.Q = static_cast<const uint16_t*>(Q);
  P.q_stride = q_stride;
  P.Hq = Hq;
  P.G = Hq / V.Hkv;
  P.bf16 = dtype == TM_KVB_BF16;
  P.scale_log2 = (scale != 0.f ? scale : cache->D == 64 ? 0.125f : 0.08838834764831845f) * 1.4426950408889634f;
  P.out = static_cast<uint16_t*>(out);
  P.lse = lse ? lse : w_out && !p.scores ? reinterpret_cast<float*>(ws + p.lse) : nullptr;
  P.w_in = w_in;
  P.w_out = w_out;
  P.w_stride = w_stride;
  P.chunk = p.chunk;
  P.chunks = p.chunks;
  P.rows_per_cta = p.rows_per_cta;
  if (p.chunks > 1) P.part = reinterpret_cast<float*>(ws + p.part);
  if (p.chunks > 1 || p.scores) P.part_ml = reinterpret_cast<float2*>(ws + p.part_ml);
  if (p.scores) {
    P.scores = reinterpret_cast<float*>(ws + p.score);
    P.score_stride = ((long long)V.max_len + kTile - 1) / kTile * kTile;
  }
  int launches = 0;
  if (cache->format == TM_KVB_INT8)
    st = cache->D == 64 ? run<TM_KVB_INT8, 64>(P, p, cache, s, &launches)
                        : run<TM_KVB_INT8, 128>(P, p, cache, s, &launches);
  else
    st = cache->D == 64 ? run<TM_KVB_E4M3, 64>(P, p, cache, s, &launches)
                        : run<TM_KVB_E4M3, 128>(P, p, cache, s, &launches);
  if (st == TM_OK) set_launch_count(launches);
  return st;
}
