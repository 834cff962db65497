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
// A CTA takes one (sequence, KV head), RT x 16 rows (query token, query head of
// the group) and a slice of the tokens, in tiles of 64: 4 RT warps, each 16
// rows x 16 tokens of the tile, with a running softmax of its own; the tile
// comes by 16-byte asynchronous copies, several tiles ahead.  Rows
// of different tokens of a draft share the tile's codes.  The slices' partial
// states go through a workspace and a second launch joins them.
//
// Order of tokens and dimensions: the K fragment's column n holds token
// sigma(n) of an 8-token group, a lane's 16-byte chunk holds 16 dimensions that
// four k-steps take word by word (the queries are read in the same order), and
// the V fragment's column n holds dimension 16 n + i of n-tile i (D = 128; 8 n + i
// for 64).  sigma and the swizzle make all shared loads conflict-free.
#include "kvb_attn.h"

namespace w4 {
namespace kvb {

constexpr int kTile = 64;    // tokens per tile
constexpr int kWarpTok = 16;  // tokens of a tile per warp
constexpr float kBias = 6.f;  // log2 of the largest weight right after m moved
constexpr float kSlack = 8.f;
constexpr float kNone = -1e30f;  // m of a row that has seen nothing

template <int D>
__device__ __forceinline__ int sigma(int n) {
  if (D == 128) return n ^ ((n & 1) << 2);
  const int m = n >> 1;
  return ((m & 1) | ((m >> 1) << 2)) ^ ((n & 1) * 3);
}
// Byte offset of 16-byte chunk c of tile row r.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, int RT>
struct AttnShape {
  static constexpr int THREADS = 128 * RT;
  static constexpr uint32_t K_BYTES = kTile * D;
  static constexpr uint32_t META = 2 * K_BYTES;       // ks[4], vs[4], page[4]
  static constexpr uint32_t SLOT = 2 * K_BYTES + 64;  // multiple of 64
  static constexpr int STAGES = 4;
  static constexpr uint32_t JOIN = 2 * RT * (16 * D + 32) * 4;  // two warps' states per row tile
  static constexpr uint32_t SMEM = STAGES * SLOT > JOIN ? STAGES * SLOT : JOIN;
};

template <int FMT, int D, int RT>
__global__ void __launch_bounds__(128 * RT) attn_kernel(const AttnParams P) {
  using SH = AttnShape<D, RT>;
  constexpr int NV = D / 8;   // n-tiles of the output
  constexpr int KS = D / 16;  // k-steps of the scores
  constexpr int CPR = D / 16;  // 16-byte chunks per token
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const View& V = P.V;
  const int b = blockIdx.z, chunk = blockIdx.x;
  const int h = blockIdx.y % V.Hkv, rg = blockIdx.y / V.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int rt = warp >> 2, ts = warp & 3;
  const Span s = span(V, b);
  const int rows = s.n * P.G;
  const int row_base = rg * RT * 16;
  if (row_base >= rows) return;
  // Tokens [j0, j1) that some row of the group sees.
  const int last_i = (min(row_base + RT * 16, rows) - 1) / P.G;
  const int j0 = chunk * P.chunk;
  const int j1 = min(min(s.len, j0 + P.chunk), s.old + last_i + 1);
  if (j0 >= j1 && chunk > 0) return;  // chunk 0 still writes what an empty row gives
  const int tiles = j1 > j0 ? (j1 - j0 + kTile - 1) / kTile : 0;

  // ---- copies: thread -> chunk c of tokens 16 r + ..., the page of each 16-token group ahead of its use
  const int c16 = tid % CPR, r16 = (tid / CPR);
  constexpr int ROWS_PER_PASS = SH::THREADS / CPR;
  constexpr int PASSES = kTile / ROWS_PER_PASS > 0 ? kTile / ROWS_PER_PASS : 1;
  auto issue = [&](int it) {
    if (it < tiles) {
      const uint32_t slot = base + (it % SH::STAGES) * SH::SLOT;
      const int tok0 = j0 + it * kTile;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = r16 + p * ROWS_PER_PASS;
        if (r < kTile) {
          const int j = tok0 + r;
          const int page = j < j1 ? page_of(V, V.table, b, V.table_stride, j >> V.t_shift) : -1;
          const size_t off = ((((size_t)max(page, 0) * V.Hkv + h) << V.t_shift) + (j & ((1 << V.t_shift) - 1))) * D + c16 * 16;
          const uint32_t at = swz<D>(r, c16);
          cp16(slot + at, V.k + (page >= 0 ? off : 0), page >= 0);
          cp16(slot + SH::K_BYTES + at, V.v + (page >= 0 ? off : 0), page >= 0);
          if (c16 == 0 && (r & 15) == 0) {
            const size_t cell = (size_t)max(page, 0) * V.Hkv + h;
            cp4(slot + SH::META + (r >> 4) * 4, V.ks + (page >= 0 ? cell : 0), page >= 0);
            cp4(slot + SH::META + 16 + (r >> 4) * 4, V.vs + (page >= 0 ? cell : 0), page >= 0);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot + SH::META + 32 + (r >> 4) * 4), "r"(page) : "memory");
          }
        }
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < SH::STAGES - 1; ++i) issue(i);

  // ---- the queries, once, in the k order of the codes; bf16 rows are scaled by a
  // power of two into fp16's range (exact down to 2^-39 of the row's maximum)
  uint32_t qa[KS][4];
  float qscale[2];
  int lastv[2];  // last visible token of the lane's two rows (-1: none)
  size_t hr[2];  // row index of the outputs
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = row_base + rt * 16 + gr + 8 * e;
    const bool ok = row < rows;
    const int i = ok ? row / P.G : 0;
    const int hq = h * P.G + (ok ? row - i * P.G : 0);
    lastv[e] = ok ? min(s.old + i, s.len - 1) : -1;
    hr[e] = (size_t)(s.row0 + i) * P.Hq + hq;
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
    qscale[e] = 1.f;
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
      qscale[e] = __uint_as_float((uint32_t)(127 - min(14 - e2, 126)) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 f = unpack(raw[k][x], true);
          raw[k][x] = pack_half2(f.x * up, f.y * up);
        }
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qa[k][e] = raw[k][0];
      qa[k][2 + e] = raw[k][1];
    }
  }

  float o[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {kNone, kNone}, l[2] = {0.f, 0.f};
  const int sg[2] = {sigma<D>(2 * t), sigma<D>(2 * t + 1)};
  const int kr = sigma<D>(gr);

  for (int it = 0; it < tiles; ++it) {
    cp_wait<SH::STAGES - 2>();
    __syncthreads();
    issue(it + SH::STAGES - 1);
    const uint32_t slot = base + (it % SH::STAGES) * SH::SLOT;
    const int tok0 = j0 + it * kTile + ts * kWarpTok;
    if (tok0 >= j1) continue;  // the warp's tokens lie past the end (warp-uniform)
    const int page = (int)lds32(slot + SH::META + 32 + ts * 4);
    const float ks = __uint_as_float(lds32(slot + SH::META + ts * 4));
    const float vs = fmaxf(__uint_as_float(lds32(slot + SH::META + 16 + ts * 4)), kScaleFloor);
    // ---- scores: 16 rows x 16 tokens
    float sc[2][4] = {};
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int j = 0; j < KS / 4; ++j) {
        const uint4 kw = lds128(slot + swz<D>(ts * kWarpTok + 8 * a + kr, t + 4 * j));
        const uint32_t wd[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          codes_half<FMT>(wd[i], b0, b1);
          mma_16816(sc[a], qa[4 * j + i], b0, b1);
        }
      }
    // ---- softmax
    // 2^lv stands for vs (to 2^-21 of it); its own inverse takes it out of l again.
    const float lv = __log2f(vs), inv = ex2(-lv);
    uint32_t pa[4];
    float tm[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float c = ks * qscale[e] * P.scale_log2;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int j = tok0 + 8 * a + sg[x];
          float v = sc[a][2 * e + x] * c;
          v = (page >= 0 && j <= lastv[e]) ? v : -INFINITY;
          sc[a][2 * e + x] = v;
          tm[e] = fmaxf(tm[e], v);
        }
      if (P.scores && lastv[e] >= 0) {
        float* row = P.scores + hr[e] * P.score_stride + tok0;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int x = 0; x < 2; ++x) row[8 * a + sg[x]] = sc[a][2 * e + x];
      }
      tm[e] += lv;
      tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xffffffffu, tm[e], 1));
      tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xffffffffu, tm[e], 2));
    }
    if (__any_sync(0xffffffffu, tm[0] > m[0] + kSlack || tm[1] > m[1] + kSlack)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[e], tm[e]);
        const float f = ex2(m[e] - mn);
        m[e] = mn;
        l[e] *= f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          o[i][2 * e] *= f;
          o[i][2 * e + 1] *= f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float off = lv + kBias - m[e];
      float sum = 0.f;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const float p0 = ex2(sc[a][2 * e] + off), p1 = ex2(sc[a][2 * e + 1] + off);
        sum += p0 + p1;
        pa[2 * a + e] = pack_half2(p0, p1);
      }
      l[e] = fmaf(sum, inv, l[e]);
    }
    // ---- values: 16 rows x 16 tokens x D
    const uint32_t vb = slot + SH::K_BYTES;
    const int r0 = ts * kWarpTok;
    if constexpr (D == 128) {
      const uint4 v0 = lds128(vb + swz<D>(r0 + sg[0], gr)), v1 = lds128(vb + swz<D>(r0 + sg[1], gr));
      const uint4 v2 = lds128(vb + swz<D>(r0 + 8 + sg[0], gr)), v3 = lds128(vb + swz<D>(r0 + 8 + sg[1], gr));
      const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
      const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t b0[4], b1[4];
        codes_half_pairs<FMT>(w0[i], w1[i], b0);
        codes_half_pairs<FMT>(w2[i], w3[i], b1);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_16816(o[4 * i + k], pa, b0[k], b1[k]);
      }
    } else {
      uint32_t wv[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t at = vb + swz<D>(r0 + 8 * (q >> 1) + sg[q & 1], gr >> 1) + 8 * (gr & 1);
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wv[q][0]), "=r"(wv[q][1]) : "r"(at));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t b0[4], b1[4];
        codes_half_pairs<FMT>(wv[0][i], wv[1][i], b0);
        codes_half_pairs<FMT>(wv[2][i], wv[3][i], b1);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_16816(o[4 * i + k], pa, b0[k], b1[k]);
      }
    }
  }
  cp_wait<0>();
  __syncthreads();

  // ---- join the four warps of a row tile: 2, 3 into 0, 1, then 1 into 0
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
  }
  float* st = reinterpret_cast<float*>(smem);
  constexpr int STATE = 16 * D + 32;
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (ts >= step && ts < 2 * step) {
      float* dst = st + (size_t)(rt * 2 + ts - step) * STATE;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) dst[(i * 4 + x) * 32 + lane] = o[i][x];
      if (t == 0) {
        dst[16 * D + gr] = m[0];
        dst[16 * D + 8 + gr] = m[1];
        dst[16 * D + 16 + gr] = l[0];
        dst[16 * D + 24 + gr] = l[1];
      }
    }
    __syncthreads();
    if (ts < step) {
      const float* src = st + (size_t)(rt * 2 + ts) * STATE;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float m2 = src[16 * D + 8 * e + gr], l2 = src[16 * D + 16 + 8 * e + gr];
        const float mn = fmaxf(m[e], m2), f1 = ex2(m[e] - mn), f2 = ex2(m2 - mn);
        m[e] = mn;
        l[e] = l[e] * f1 + l2 * f2;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            o[i][2 * e + x] = o[i][2 * e + x] * f1 + src[(i * 4 + 2 * e + x) * 32 + lane] * f2;
      }
    }
    __syncthreads();
  }
  if (ts != 0) return;
  // ---- one slice: the output; several: the state, for the joining launch
  constexpr int SPAN = D / 8;  // dimensions of one column: column n of n-tile i is dimension SPAN n + i
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = row_base + rt * 16 + gr + 8 * e;
    if (row >= rows) continue;
    if (P.chunks == 1) {
      const float r = l[e] > 0.f || l[e] != l[e] ? __fdividef(1.f, l[e]) : 0.f;
      uint16_t* out = P.out + hr[e] * D + 2 * t * SPAN;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < NV; i += 8) {
          uint32_t wd[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f0 = o[i + 2 * k][2 * e + x] * r, f1 = o[i + 2 * k + 1][2 * e + x] * r;
            wd[k] = P.bf16 ? pack_bf162(f0, f1) : pack_half2(f0, f1);
          }
          *reinterpret_cast<uint4*>(out + x * SPAN + i) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
        }
      if (t == 0 && P.lse) P.lse[hr[e]] = l[e] == 0.f ? -INFINITY : (log2f(l[e]) + m[e] - kBias) * 0.693147180559945f;
    } else {
      float* dst = P.part + (hr[e] * P.chunks + chunk) * D + 2 * t * SPAN;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < NV; i += 4)
          *reinterpret_cast<float4*>(dst + x * SPAN + i) =
              make_float4(o[i][2 * e + x], o[i + 1][2 * e + x], o[i + 2][2 * e + x], o[i + 3][2 * e + x]);
      if (t == 0) P.part_ml[hr[e] * P.chunks + chunk] = make_float2(m[e] - kBias, l[e]);
    }
  }
}

// ---- the slices' states of one row into its output: one warp per (row, head)
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const AttnParams P) {
  const View& V = P.V;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const Span s = span(V, b);
  const int at = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int i = at / P.Hq;
  if (i >= s.n) return;
  const size_t hr = (size_t)(s.row0 + i) * P.Hq + (at - i * P.Hq);
  // Slices that the row's group of rows wrote: those before its last row's last token, and slice 0.
  const int g = P.rows_per_cta, head = (at - i * P.Hq) % P.G;
  const int row = i * P.G + head;
  const int last_i = (min((row / g + 1) * g, s.n * P.G) - 1) / P.G;
  const int end = min(s.len, s.old + last_i + 1);
  const int n = end > 0 ? (end + P.chunk - 1) / P.chunk : 1;
  const float2* ml = P.part_ml + hr * P.chunks;
  float m = kNone;
  for (int c = lane; c < n; c += 32) m = fmaxf(m, ml[c].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f;
  constexpr int E = D / 32;
  float acc[E] = {};
  for (int c = 0; c < n; ++c) {
    const float2 v = ml[c];
    const float f = ex2(v.x - m);
    l = fmaf(v.y, f, l);
    const float* src = P.part + (hr * P.chunks + c) * D + lane * E;
#pragma unroll
    for (int k = 0; k < E; ++k) acc[k] = fmaf(src[k], f, acc[k]);
  }
  const float r = l > 0.f || l != l ? __fdividef(1.f, l) : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(P.out + hr * D + lane * E);
#pragma unroll
  for (int k = 0; k < E; k += 2)
    out[k / 2] = P.bf16 ? pack_bf162(acc[k] * r, acc[k + 1] * r) : pack_half2(acc[k] * r, acc[k + 1] * r);
  if (lane == 0 && P.lse) P.lse[hr] = l == 0.f ? -INFINITY : (log2f(l) + m) * 0.693147180559945f;
}

// ---- the weight that each token drew, from the scores and the rows' lse:
// one thread per (token, KV head), rows in order
__global__ void __launch_bounds__(256) score_weights_kernel(const AttnParams P) {
  const View& V = P.V;
  const int b = blockIdx.z, h = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= P.w_stride) return;
  const Span s = span(V, b);
  const size_t at = ((size_t)b * V.Hkv + h) * P.w_stride + j;
  float sum = 0.f;
  for (int i = 0; i < s.n; ++i) {
    // The scores that the row's CTAs wrote end with its group's last visible tile;
    // what the row itself does not see is -inf there.
    if (j >= s.len || j > s.old + i) continue;
    for (int g = 0; g < P.G; ++g) {
      const size_t hr = (size_t)(s.row0 + i) * P.Hq + h * P.G + g;
      const float lse = P.lse[hr];
      sum += lse == -INFINITY ? 0.f : ex2(P.scores[hr * P.score_stride + j] - lse * 1.44269504088896f);
    }
  }
  P.w_out[at] = (P.w_in ? P.w_in[at] : 0.f) + sum;
}

template <int FMT, int D, int RT>
tm_status launch_attn(const AttnParams& P, int groups, cudaStream_t s) {
  using SH = AttnShape<D, RT>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(attn_kernel<FMT, D, RT>), SH::SMEM)) return TM_ERR_CUDA;
  const dim3 grid((unsigned)P.chunks, (unsigned)(P.V.Hkv * groups), (unsigned)P.V.B);
  attn_kernel<FMT, D, RT><<<grid, SH::THREADS, SH::SMEM, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

// Launch settings and the workspace's layout, from the host fields alone.
struct Plan {
  int rt;            // 16-row tiles per CTA of the kernel for few rows; 0: the tcgen05 kernel
  int rows_per_cta;  // rows that share a CTA
  int groups;        // CTAs along the rows
  int chunk, chunks;
  bool scores;  // token weights from kept scores (few rows), else from a second pass
  size_t part, part_ml, lse, score, bytes;  // offsets, total
};

constexpr int kFewRows = 64;  // most rows per (sequence, KV head) of the kernel for few rows

static Plan make_plan(const View& V, int D, int Hq, bool weights) {
  Plan p = {};
  const int G = Hq / V.Hkv;
  const long long rows = (long long)V.max_q * G;
  const long long sms = num_sms(current_device());
  p.rt = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= kFewRows ? 4 : 0;
  p.rows_per_cta = p.rt ? 16 * p.rt : 256;
  p.groups = (int)((rows + p.rows_per_cta - 1) / p.rows_per_cta);
  const long long ctas = (long long)V.B * V.Hkv * p.groups;
  long long chunk, least, unit;
  if (p.rt) {
    // Enough slices for two waves of CTAs, none shorter than four tiles.
    const long long slots = sms * (p.rt == 1 ? 3 : p.rt == 2 ? 2 : 1);
    unit = kTile;
    least = 4 * kTile;
    chunk = ((long long)V.max_len * ctas + 2 * slots - 1) / (2 * slots);
  } else {
    // Slices only where the rows alone leave SMs idle.
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
  if (chunks > 1) {
    p.part = at;
    at = al(at + hr * chunks * D * 4);
    p.part_ml = at;
    at = al(at + hr * chunks * 8);
  }
  if (weights) {
    p.lse = at;
    at = al(at + hr * 4);
    p.scores = p.rt != 0;
    if (p.scores) {
      p.score = at;
      at = al(at + hr * (((size_t)V.max_len + kTile - 1) / kTile * kTile) * 4);
    }
  }
  p.bytes = at;
  return p;
}

}  // namespace kvb
}  // namespace w4

using namespace w4;
using namespace w4::kvb;

static tm_status check_heads(const View& V, const tm_kvb_batch* batch, int Hq) {
  if (Hq < 1 || Hq % V.Hkv != 0) return TM_ERR_INVALID_ARG;
  const bool one_each = batch->q_start == nullptr;
  if (one_each && (batch->rows != batch->B || (batch->B > 0 && batch->max_q < 1))) return TM_ERR_INVALID_ARG;
  const long long rows = (long long)V.max_q * (Hq / V.Hkv);
  if (rows > 4000000ll || (long long)V.B * V.Hkv > 0x7fffffffll) return TM_ERR_UNSUPPORTED;  // the grid's limits
  return TM_OK;
}

extern "C" tm_status tm_kvb_attention_workspace(const tm_kvb_cache* cache, const tm_kvb_batch* batch, int Hq,
                                                int weights, size_t* bytes) {
  View V;
  if (!bytes) return TM_ERR_INVALID_ARG;
  tm_status st = check(cache, batch, false, &V);
  if (st == TM_OK) st = check_heads(V, batch, Hq);
  if (st != TM_OK) return st;
  *bytes = V.B == 0 || V.rows == 0 || V.max_q == 0 ? 0 : make_plan(V, cache->D, Hq, weights != 0).bytes;
  return TM_OK;
}

template <int FMT, int D>
static tm_status run(const AttnParams& P, const Plan& p, cudaStream_t s, int* launches) {
  tm_status st = p.rt == 0   ? launch_prefill_attn(P, FMT, D, p.groups, s)
                 : p.rt == 1 ? launch_attn<FMT, D, 1>(P, p.groups, s)
                 : p.rt == 2 ? launch_attn<FMT, D, 2>(P, p.groups, s)
                             : launch_attn<FMT, D, 4>(P, p.groups, s);
  if (st != TM_OK) return st;
  *launches = 1;
  const View& V = P.V;
  if (P.chunks > 1) {
    const long long warps = (long long)V.max_q * P.Hq;
    join_kernel<D><<<dim3((unsigned)((warps + 3) / 4), (unsigned)V.B), 128, 0, s>>>(P);
    ++*launches;
  }
  if (P.w_out) {
    if (p.scores) {
      const dim3 grid((unsigned)((P.w_stride + 255) / 256), (unsigned)V.Hkv, (unsigned)V.B);
      score_weights_kernel<<<grid, 256, 0, s>>>(P);
    } else {
      st = launch_row_weights(P, FMT, D, s);
      if (st != TM_OK) return st;
    }
    ++*launches;
  }
  return cudaGetLastError() == cudaSuccess ? TM_OK : TM_ERR_CUDA;
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
  if (V.B == 0 || V.rows == 0 || V.max_q == 0) return TM_OK;
  if (!Q || !out || q_stride < (long long)Hq * cache->D) return TM_ERR_INVALID_ARG;
  if (w_out && w_stride < V.max_len) return TM_ERR_INVALID_ARG;
  if (w_out && w_stride > 65535ll * 128) return TM_ERR_UNSUPPORTED;  // the grid's limit
  if (!aligned(Q, 16) || q_stride % 8 || !aligned(out, 16) || !aligned(lse, 4) || !aligned(w_in, 4) ||
      !aligned(w_out, 4) || !aligned(workspace, 16))
    return TM_ERR_ALIGNMENT;
  const Plan p = make_plan(V, cache->D, Hq, w_out != nullptr);
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return TM_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.Q = static_cast<const uint16_t*>(Q);
  P.q_stride = q_stride;
  P.Hq = Hq;
  P.G = Hq / V.Hkv;
  P.bf16 = dtype == TM_KVB_BF16;
  P.scale_log2 = (scale != 0.f ? scale : cache->D == 64 ? 0.125f : 0.08838834764831845f) * 1.4426950408889634f;
  P.out = static_cast<uint16_t*>(out);
  P.lse = lse ? lse : w_out ? reinterpret_cast<float*>(ws + p.lse) : nullptr;
  P.w_in = w_in;
  P.w_out = w_out;
  P.w_stride = w_stride;
  P.chunk = p.chunk;
  P.chunks = p.chunks;
  P.rows_per_cta = p.rows_per_cta;
  if (p.chunks > 1) {
    P.part = reinterpret_cast<float*>(ws + p.part);
    P.part_ml = reinterpret_cast<float2*>(ws + p.part_ml);
  }
  if (p.scores) {
    P.scores = reinterpret_cast<float*>(ws + p.score);
    P.score_stride = ((long long)V.max_len + kTile - 1) / kTile * kTile;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int launches = 0;
  if (cache->format == TM_KVB_INT8)
    st = cache->D == 64 ? run<TM_KVB_INT8, 64>(P, p, s, &launches) : run<TM_KVB_INT8, 128>(P, p, s, &launches);
  else
    st = cache->D == 64 ? run<TM_KVB_E4M3, 64>(P, p, s, &launches) : run<TM_KVB_E4M3, 128>(P, p, s, &launches);
  if (st == TM_OK) set_launch_count(launches);
  return st;
}
