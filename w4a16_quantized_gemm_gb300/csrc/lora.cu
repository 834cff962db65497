// Low-rank adapters of many requests beside a shared projection:
//   out = Y + scale_a (X A_a^T) B_a^T,  a the adapter of the row's sequence.
//
// One launch: a cluster of eight CTAs takes rows that use an adapter.
//   T = X A^T: each CTA a share of K, on mma.m16n8k16;
//   the eight partial T meet in distributed shared memory: CTA c sums rows c, c + 8, ... and hands them, scaled by a
//     power of two into fp16's range, to all eight.  T is rounded there, once, since the products take 16-bit operands: in
//     two halves (the rounding and what it leaves) it would double the second product and its registers.  Against 64
//     bits the result is then off by 0.00023 to 0.00025 of itself (root mean square), with T in 32 bits by 0.00021,
//     which is the result's own rounding to fp16;
//   out: each CTA a share of N.
// No partial result goes through memory.
//
// Measured: one row (4096 x 4096, rank 16) 5.4 us: a launch, finding the row's adapter 1.1, T 1.0, the cluster's two
// barriers and the exchange 1.6, the output 0.5.  32 rows with 28 adapters (14336 x 4096, rank 16) 8.1 us; 256 rows
// with 64 adapters (4096 x 4096, rank 32) 17 us (16 rows a tile, an adapter read once per tile: 41).  Prompts of 4031
// tokens (4096 x 28672, rank 64) 155 to 157 us: 530 MB, 3.4 TB/s; while they are busy the SMs move 4.8, but 63 clusters on
// the 36 to 38 places that the GPCs have leave 27 % of them idle.  By the threads' own copies in place of TMA 186,
// straight from global memory 183.
#include <cuda_fp16.h>

#include <atomic>

#include "../../include/tm_lora.h"
#include "tm_common.cuh"

namespace w4 {
namespace lora {

static __device__ uint32_t s_err_lora;

constexpr int kThreads = 256;
constexpr int kCluster = 8;
constexpr int kDevices = 32;  // whose limits are kept

struct Params {
  const __half* X;
  const __half* Y;
  __half* out;
  long long xs, ys, os;
  const __half* A;
  const __half* B;
  const float* scale;
  const int* ids;
  const int* q_start;
  int rows, seqs, n, K, N, R;
  int splits;  // clusters that share a tile's columns (each computes T)
};

// NT: groups of 8 ranks.
template <int NT>
struct Shape {
  static constexpr int KW = 8;             // warps that share K
  static constexpr int RP = 8 * NT;        // ranks, padded
  static constexpr int KS = (NT + 1) / 2;  // k-steps of the second product
  static constexpr uint32_t PART = 0;      // [KW][16][RP] fp32
  static constexpr uint32_t SUM = PART + KW * 16 * RP * 4;  // [16][RP] fp32, this CTA's share of K
  static constexpr uint32_t FRAG = SUM + 16 * RP * 4;       // [KS][32] x 16 bytes: T as A fragments
  static constexpr uint32_t MUL = FRAG + KS * 512;            // [16] fp32
  static constexpr uint32_t SMEM = MUL + 16 * 4;
};

// Into L2, which holds less than 2^30 bytes.
__device__ __forceinline__ void prefetch_l2(const void* p, long long bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"((uint32_t)min(bytes, 1ll << 30)) : "memory");
}
__device__ __forceinline__ uint4 ldg16(const __half* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_dsmem_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// What a tile's rows use.
template <int ROWS>
struct Rows {
  int seq[ROWS];   // the sequence, -1: none
  int id[ROWS];    // its adapter; -1: none, -2: no sequence
  int list[ROWS];  // the different adapters, in the order of their first rows
  int count;
};
template <int ROWS>
__device__ __forceinline__ void find_rows(const Params& P, int row0, Rows<ROWS>& s) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int r = tid; r < ROWS; r += kThreads) s.seq[r] = P.q_start || row0 + r >= P.rows ? -1 : row0 + r;
  __syncthreads();
  if (P.q_start)
    for (int b = tid; b < P.seqs; b += kThreads) {
      const int lo = max(min(max(P.q_start[b], 0), P.rows), row0);
      const int hi = min(min(max(P.q_start[b + 1], 0), P.rows), row0 + ROWS);
      for (int r = lo; r < hi; ++r) atomicMax(&s.seq[r - row0], b);
    }
  __syncthreads();
  if (tid < ROWS) {
    const int b = s.seq[tid];
    const int a = b >= 0 ? P.ids[b] : -2;
    s.id[tid] = b >= 0 && (unsigned)a >= (unsigned)P.n ? -1 : a;
  }
  __syncthreads();
  if (tid < 32) {
    int found = 0;
    for (int r0 = 0; r0 < ROWS; r0 += 32) {
      const int r = r0 + lane;
      bool first = r < ROWS && s.id[r < ROWS ? r : 0] >= 0;
      if (first)
        for (int x = 0; x < r; ++x) first = first && s.id[x] != s.id[r];
      const uint32_t who = __ballot_sync(0xffffffffu, first);
      if (first) s.list[found + __popc(who & ((1u << lane) - 1u))] = s.id[r];
      found += __popc(who);
    }
    if (lane == 0) s.count = found;
  }
  __syncthreads();
}

// A row without an adapter, by one warp: columns c0 .. c1 - 1 of Y as they are.
__device__ __forceinline__ void copy_row(const Params& P, long long row, int c0, int c1) {
  const __half* src = P.Y + row * P.ys;
  __half* dst = P.out + row * P.os;
  for (int c = c0 + 8 * (int)(threadIdx.x & 31); c < min(c1, P.N); c += 256)
    *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + c);
}

// The eight partial T [ROWS][RP] (fp32, at `sum` of each CTA) meet: CTA c takes rows c, c + 8, ..., adds the CTAs'
// parts in order, scales, and hands them to all eight as fp16 A fragments (at `frag`) with their factors (at `mul`).
// word_of(rank of a k-step) -> the lane's place in its group of four and the word of the fragment's upper rows.
template <int ROWS, int RP, int KS, typename WordOf>
__device__ __forceinline__ void exchange(const Params& P, int a, int rank, uint32_t sum, uint32_t frag, uint32_t mul,
                                         WordOf&& word_of) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster_sync_all();
  const float factor = P.scale ? P.scale[a] : 1.f;
  for (int r = rank + kCluster * warp; r < ROWS; r += kCluster * 8) {
    constexpr int PER = (RP + 31) / 32;
    float v[PER], big = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = lane + 32 * k;
      v[k] = 0.f;
      if (c < P.R) {  // ranks that fill RP up stay 0: their sums of products with 0 are NaN where X is infinite
        const uint32_t at = sum + (r * RP + c) * 4;
        float x[kCluster];
#pragma unroll
        for (int q = 0; q < kCluster; ++q) x[q] = ld_dsmem_f32(map_shared_rank(at, q));
#pragma unroll
        for (int q = 0; q < kCluster; ++q) v[k] += x[q];
        v[k] *= factor;
      }
      big = fmaxf(big, fabsf(v[k]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    // big < 2^(e + 1): times 2^(14 - e) the row fits fp16.  Infinities and NaN pass.
    const int e = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 127);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23), down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int c = lane + 32 * k;
      if (c >= 16 * KS) continue;
      const uint16_t bits = __half_as_ushort(__float2half_rn(v[k] * up));
      int x, word;
      word_of(c & 15, x, word);
      const uint32_t at = frag + (((r >> 4) * KS + (c >> 4)) * 32 + (r & 7) * 4 + x) * 16 + (word + ((r >> 3) & 1)) * 4 + (c & 1) * 2;
#pragma unroll
      for (int q = 0; q < kCluster; ++q) st_dsmem_u16(map_shared_rank(at, q), bits);
    }
    if (lane < kCluster) st_dsmem_f32(map_shared_rank(mul + r * 4, lane), down);
    __syncwarp();
  }
  cluster_sync_all();
}

__device__ __forceinline__ uint32_t add_half2(uint32_t y, float a, float b, float f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y));
  const __half2 h = __floats2half2_rn(fmaf(a, f, v.x), fmaf(b, f, v.y));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Decode batches: up to 256 rows a tile, whose rows come together by adapter, 16 at a time (an item of work: an adapter
// and 16 of its rows), so that an adapter is read once however its rows lie.
constexpr int kSpan = 256;
constexpr int kItems = kSpan;  // at most one per row
constexpr int kSlots = 512;    // of the table of adapters, at most half full
struct Items {
  int seq[kSpan];               // as in Rows
  int key[kSlots], start[kSlots];           // an adapter, its first item
  uint32_t rows[kThreads / 32][kSlots / 4];  // a byte each: how many rows of a warp use it
  int sums[kThreads / 32];
  int total;                    // items
  int adapter[kItems], size[kItems];
  uint8_t pick[kItems * 16];    // the rows of each
};
// Returns the adapter of the thread's row: -1: none, -2: no sequence.
__device__ __forceinline__ int find_items(const Params& P, int row0, Items& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int here = min(kSpan, P.rows - row0);
  s.seq[tid] = P.q_start || tid >= here ? -1 : row0 + tid;
  for (int i = tid; i < kSlots; i += kThreads) {
    s.key[i] = -1;
    for (int w = 0; w < kThreads / 32; w += 4) (&s.rows[0][0])[i * 2 + w / 4] = 0u;
  }
  __syncthreads();
  if (P.q_start) {
    for (int b = tid; b < P.seqs; b += kThreads) {
      const int lo = max(min(max(P.q_start[b], 0), P.rows), row0);
      const int hi = min(min(max(P.q_start[b + 1], 0), P.rows), row0 + here);
      for (int r = lo; r < hi; ++r) atomicMax(&s.seq[r - row0], b);
    }
    __syncthreads();
  }
  const int b = s.seq[tid];
  int a = b >= 0 ? P.ids[b] : -2;
  if (b >= 0 && (unsigned)a >= (unsigned)P.n) a = -1;
  // Where an adapter stands in the table goes by who comes first; a row's place among its adapter's rows by their order,
  // so that all CTAs of a cluster agree.
  const uint32_t same = __match_any_sync(0xffffffffu, a);
  auto counts = [&](int w) { return reinterpret_cast<uint8_t*>(s.rows[w]); };
  int slot = 0, place = 0, rows = 0;
  if (a >= 0) {
    for (slot = a % kSlots;; slot = (slot + 1) % kSlots) {
      const int was = atomicCAS(&s.key[slot], -1, a);
      if (was == -1 || was == a) break;
    }
    place = __popc(same & ((1u << lane) - 1u));
    if (place == 0) counts(warp)[slot] = (uint8_t)__popc(same);
  }
  __syncthreads();
  if (a >= 0)
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int n = counts(w)[slot];
      rows += n;
      if (w < warp) place += n;
    }
  const int mine = a >= 0 && place == 0 ? (rows + 15) / 16 : 0;
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) s.sums[warp] = sum;
  __syncthreads();
  int before = sum - mine;
  for (int w = 0; w < warp; ++w) before += s.sums[w];
  if (mine) s.start[slot] = before;
  for (int j = 0; j < mine; ++j) {
    s.adapter[before + j] = a;
    s.size[before + j] = min(16, rows - 16 * j);
  }
  if (tid == kThreads - 1) s.total = before + mine;
  __syncthreads();
  if (a >= 0) s.pick[16 * (s.start[slot] + place / 16) + place % 16] = (uint8_t)tid;
  __syncthreads();
  return a;
}

// Operands go from global memory to the products' registers.  The sum over k may go in any order, so that a lane's 16-byte
// chunk of a row holds the eight k of two products and both operands are read in whole sectors.
template <int NT>
__global__ void __launch_bounds__(kThreads, NT <= 8 ? 2 : 1) add_kernel(const Params P) {
  using SH = Shape<NT>;
  constexpr int RP = SH::RP, KS = SH::KS, KW = SH::KW;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Items items;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int rank = (int)cluster_ctarank();
  const int cl = blockIdx.x / kCluster;
  const int tile = cl / P.splits, split = cl - tile * P.splits;
  const int row0 = tile * kSpan;
  const uint32_t base = smem_u32(smem);
  const int own = find_items(P, row0, items);
  const int count = items.total;

  // This CTA's columns, in blocks of 32.
  const int blocks = (P.N + 31) / 32, parts = kCluster * P.splits, part = split * kCluster + rank;
  const int n0 = (int)((long long)blocks * part / parts), n1 = (int)((long long)blocks * (part + 1) / parts);
  if (P.out != P.Y)  // rows without an adapter, shared out over the tile's clusters
    for (uint32_t left = __ballot_sync(0xffffffffu, own == -1 && tid % gridDim.y == blockIdx.y); left; left &= left - 1)
      copy_row(P, row0 + 32 * warp + __ffs(left) - 1, 32 * n0, 32 * n1);

  for (int z = blockIdx.y; z < count; z += gridDim.y) {
    const int a = items.adapter[z], size = items.size[z];
    const bool lo_ok = gr < size, hi_ok = gr + 8 < size;
    const long long r_lo = row0 + (lo_ok ? items.pick[16 * z + gr] : 0), r_hi = row0 + (hi_ok ? items.pick[16 * z + gr + 8] : 0);
    // Its columns of B, one run of memory, on their way to L2 while T is computed; and the next item's A, a share
    // of it by each CTA.
    if (tid == 0 && n1 > n0)
      prefetch_l2(P.B + ((size_t)a * P.N + 32 * n0) * P.R, (min(32 * n1, P.N) - 32 * n0) * (2ll * P.R));
    if (tid == 32 && z + (int)gridDim.y < count) {
      const long long units = (long long)P.R * P.K / 8, u0 = units * rank / kCluster, u1 = units * (rank + 1) / kCluster;
      if (u1 > u0)
        prefetch_l2(P.A + (size_t)items.adapter[z + gridDim.y] * P.R * P.K + 8 * u0, (u1 - u0) * 16);
    }
    // ---- T: this warp's chunks of 32 k
    {
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
      const __half* xl = P.X + r_lo * P.xs + 8 * t;
      const __half* xh = P.X + r_hi * P.xs + 8 * t;
      const __half* pa = P.A + ((size_t)a * P.R + gr) * P.K + 8 * t;
      const int chunks = (P.K + 31) / 32, stride = kCluster * KW;
      constexpr int AHEAD = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;  // chunks whose loads are in flight
      uint4 x0[AHEAD], x1[AHEAD], w[AHEAD][NT];
      auto fetch = [&](int ch, int q) {
        const int k = 32 * ch;
        const bool in = k + 8 * t < P.K;  // past the last chunk, too
        x0[q] = ldg16(xl + k, in && lo_ok);
        x1[q] = ldg16(xh + k, in && hi_ok);
#pragma unroll
        for (int i = 0; i < NT; ++i) w[q][i] = ldg16(pa + (size_t)(8 * i) * P.K + k, in && 8 * i + gr < P.R);
      };
      int ch = rank * KW + warp;
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) fetch(ch + q * stride, q);
      for (; ch < chunks; ch += AHEAD * stride) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
          const uint32_t f0[4] = {x0[q].x, x1[q].x, x0[q].y, x1[q].y}, f1[4] = {x0[q].z, x1[q].z, x0[q].w, x1[q].w};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma_16816(acc[i], f0, w[q][i].x, w[q][i].y);
            mma_16816(acc[i], f1, w[q][i].z, w[q][i].w);
          }
          fetch(ch + (q + AHEAD) * stride, q);
        }
      }
      float* dst = reinterpret_cast<float*>(smem + SH::PART) + (warp * 16 + gr) * RP + 2 * t;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(acc[i][0], acc[i][1]);
        *reinterpret_cast<float2*>(dst + 8 * RP + 8 * i) = make_float2(acc[i][2], acc[i][3]);
      }
    }
    __syncthreads();
    {
      const float* src = reinterpret_cast<const float*>(smem + SH::PART);
      float* dst = reinterpret_cast<float*>(smem + SH::SUM);
      for (int i = tid; i < 16 * RP; i += kThreads) {
        float v = src[i];
#pragma unroll
        for (int k = 1; k < KW; ++k) v += src[k * 16 * RP + i];
        dst[i] = v;
      }
    }
    // a lane holds ranks 4 x .. 4 x + 3 of a k-step, as it reads B
    exchange<16, RP, KS>(P, a, rank, base + SH::SUM, base + SH::FRAG, base + SH::MUL, [](int c, int& x, int& word) {
      x = c >> 2;
      word = 2 * ((c >> 1) & 1);
    });
    // ---- out: blocks of 32 columns; a lane's products are eight consecutive ones
    const float* mul = reinterpret_cast<const float*>(smem + SH::MUL);
    for (int nb = n0 + warp; nb < n1; nb += 8) {
      uint2 w[4][KS];  // column 32 nb + 8 (gr / 2) + 2 i + gr % 2, ranks 16 s + 4 t ..
      const __half* pb = P.B + ((size_t)a * P.N + 32 * nb + 8 * (gr >> 1) + (gr & 1)) * P.R + 4 * t;
      const bool col_ok = 32 * nb + 8 * (gr >> 1) < P.N;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < KS; ++s)
          w[i][s] = col_ok && 16 * s + 4 * t < P.R ? __ldg(reinterpret_cast<const uint2*>(pb + 2 * i * P.R + 16 * s))
                                                    : make_uint2(0u, 0u);
      const int c0 = 32 * nb + 8 * t;
      const bool in = c0 < P.N;
      uint4 y[2] = {};
      if (lo_ok && in) y[0] = *reinterpret_cast<const uint4*>(P.Y + r_lo * P.ys + c0);
      if (hi_ok && in) y[1] = *reinterpret_cast<const uint4*>(P.Y + r_hi * P.ys + c0);
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint4 f = *reinterpret_cast<const uint4*>(smem + SH::FRAG + (s * 32 + lane) * 16);
        const uint32_t fa[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_16816(acc[i], fa, w[i][s].x, w[i][s].y);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float f = mul[gr + 8 * half];
        const uint32_t yw[4] = {y[half].x, y[half].y, y[half].z, y[half].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = add_half2(yw[i], acc[i][2 * half], acc[i][2 * half + 1], f);
        if ((half ? hi_ok : lo_ok) && in)
          *reinterpret_cast<uint4*>(P.out + (half ? r_hi : r_lo) * P.os + c0) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// Tiles of 64 rows: prompts.  X, A, Y and B come in by TMA through a ring of shared memory (by the threads' own copies
// the load-store pipe was the bottleneck), the results leave in whole lines.
template <int RP>
struct Wide {
  static constexpr int ROWS = 64;
  static constexpr int KS = RP / 16;
  static constexpr int STAGES = RP <= 64 ? 4 : 3;
  static constexpr uint32_t TILE = ROWS * 128;            // 64 k of X, or 64 columns of Y
  static constexpr uint32_t STAGE = TILE + RP * 128;      // and 64 k of A, or 64 columns of B
  static constexpr uint32_t SUM = STAGES * STAGE;         // [ROWS][RP] fp32, this CTA's share of K
  static constexpr uint32_t FRAG = SUM + ROWS * RP * 4;   // [ROWS / 16][KS][32] x 16 bytes: T as A fragments
  static constexpr uint32_t MUL = FRAG + ROWS / 16 * KS * 512;
  static constexpr uint32_t OUT = (MUL + ROWS * 4 + 127) / 128 * 128;  // two steps' results
  static constexpr uint32_t BARS = OUT + 2 * TILE;
  static constexpr uint32_t SMEM = BARS + 64 + 1024;
};
struct Maps {
  CUtensorMap x, a, y, b;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int RP>
__global__ void __launch_bounds__(kThreads, RP <= 32 ? 3 : RP == 64 ? 2 : 1)
    add_wide_kernel(const __grid_constant__ Maps M, const Params P) {
  using SH = Wide<RP>;
  constexpr int ROWS = SH::ROWS, KS = SH::KS, S = SH::STAGES, NT = RP / 8;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  __shared__ Rows<ROWS> rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int lm = lane >> 3, lr = lane & 7;  // matrix and row that the lane names in an ldmatrix
  const int rank = (int)cluster_ctarank();
  const int cl = blockIdx.x / kCluster;
  const int tile = cl / P.splits, split = cl - tile * P.splits;
  const int row0 = tile * ROWS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::BARS + 8 * S);
  if (tid == 0) {
    for (int i = 0; i < S; ++i) mbar_init(base + SH::BARS + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  find_rows(P, row0, rows);
  const int count = rows.count;

  // This CTA's columns, in blocks of 64 (its CTAs' blocks interleaved, so that a cluster works on one KB of a row at a
  // time: 196 us for the prompts of 157).
  const int blocks = (P.N + 63) / 64, parts = kCluster * P.splits, part = split * kCluster + rank;
  const int n0 = (int)((long long)blocks * part / parts), cols = (int)((long long)blocks * (part + 1) / parts) - n0;
  auto column = [&](int i) { return 64 * (n0 + i); };
  if (blockIdx.y == 0 && P.out != P.Y)
    for (int r = warp; r < ROWS; r += kThreads / 32)
      if (rows.id[r] == -1) copy_row(P, row0 + r, 64 * n0, 64 * (n0 + cols));

  // Lines of 128 bytes, 16-byte chunk c of line r at c ^ (r % 8), as the copies lay them: what a warp reads at once (eight
  // lines, one chunk) covers all banks.
  auto at = [](int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); };
  // B has a row of ranks a column: several a line (the copy's 32- or 64-byte swizzle), or 64 ranks of all columns, then
  // the other 64.
  auto at_b = [&](int col, int c) {
    if (RP >= 64) return at(64 * (c >> 3) + col, c & 7);
    if (RP == 32) return (uint32_t)(col * 64 + ((c ^ ((col >> 1) & 3)) << 4));
    return (uint32_t)(col * 32 + ((c ^ ((col >> 2) & 1)) << 4));
  };
  int issued = 0, taken = 0;  // steps of the ring, over all adapters

  for (int z = blockIdx.y; z < count; z += gridDim.y) {
    const int a = rows.list[z];
    // The steps of this adapter: its CTA's chunks of 64 k (rank, rank + 8, ...), then its blocks of 64 columns, so
    // that what the second product needs first is on its way while T is put together.
    const int chunks = ((P.K + 63) / 64 - rank + kCluster - 1) / kCluster;
    auto load = [&](int i) {
      if (i >= chunks + cols) return;
      if (tid == 0) {
        const uint32_t bar = base + SH::BARS + 8 * (issued % S), dst = base + (issued % S) * SH::STAGE;
        mbar_expect_tx(bar, SH::STAGE);
        if (i < chunks) {
          const int k = 64 * (rank + kCluster * i);
          tma_load_2d(dst, &M.x, k, row0, bar);
          tma_load_3d(dst + SH::TILE, &M.a, k, 0, a, bar);
        } else {
          const int c = column(i - chunks);
          tma_load_2d(dst, &M.y, c, row0, bar);
#pragma unroll
          for (int r = 0; r < RP; r += 64) tma_load_3d(dst + SH::TILE + 128 * r, &M.b, r, c, a, bar);
        }
      }
      ++issued;
    };
    // Step i's data; the step after those under way goes into the stage that all warps have left.
    auto next = [&](int i) {
      mbar_wait(base + SH::BARS + 8 * (taken % S), (uint32_t)(taken / S) & 1u, abort_flag, &s_err_lora);
      __syncthreads();
      load(i + S - 1);
      return (uint32_t)(taken++ % S) * SH::STAGE;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load(i);

    // ---- T: each warp half of a chunk's k for 16 rows
    {
      const int mt = warp & 3, half = warp >> 2;
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
      for (int i = 0; i < chunks; ++i) {
        const uint32_t src = base + next(i);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          uint32_t x[4];
          ldmatrix4(x, src + at(16 * mt + 8 * (lm & 1) + lr, 4 * half + 2 * ks + (lm >> 1)));
#pragma unroll
          for (int p = 0; p < NT / 2; ++p) {
            uint32_t w[4];
            ldmatrix4(w, src + SH::TILE + at(16 * p + 8 * (lm >> 1) + lr, 4 * half + 2 * ks + (lm & 1)));
            mma_16816(acc[2 * p], x, w[0], w[1]);
            mma_16816(acc[2 * p + 1], x, w[2], w[3]);
          }
        }
      }
      float* dst = reinterpret_cast<float*>(smem + SH::SUM) + (16 * mt + gr) * RP + 2 * t;
#pragma unroll
      for (int turn = 1; turn >= 0; --turn) {  // the second half of the warps, then the first adds its own
        if (half == turn)
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float2* lo = reinterpret_cast<float2*>(dst + 8 * i);
            float2* hi = reinterpret_cast<float2*>(dst + 8 * RP + 8 * i);
            const float2 u = turn ? make_float2(0.f, 0.f) : *lo, v = turn ? make_float2(0.f, 0.f) : *hi;
            *lo = make_float2(acc[i][0] + u.x, acc[i][1] + u.y);
            *hi = make_float2(acc[i][2] + v.x, acc[i][3] + v.y);
          }
        __syncthreads();
      }
    }
    exchange<ROWS, RP, KS>(P, a, rank, base + SH::SUM, base + SH::FRAG, base + SH::MUL, [](int c, int& x, int& word) {
      x = (c >> 1) & 3;
      word = 2 * (c >> 3);
    });
    // ---- out: 64 columns a step, each warp eight of them for all rows
    uint32_t tf[4][KS][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint4 f = *reinterpret_cast<const uint4*>(smem + SH::FRAG + ((mt * KS + s) * 32 + lane) * 16);
        tf[mt][s][0] = f.x;
        tf[mt][s][1] = f.y;
        tf[mt][s][2] = f.z;
        tf[mt][s][3] = f.w;
      }
    float mul[4][2];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) mul[mt][h] = reinterpret_cast<const float*>(smem + SH::MUL)[16 * mt + gr + 8 * h];
    // A step's results leave while the next one's are computed: one barrier a step (next's).
    auto leave = [&](int i) {
      const uint8_t* from = smem + SH::OUT + (i & 1) * SH::TILE;
      const int c = column(i) + 8 * (tid & 7);
#pragma unroll
      for (int j = 0; j < ROWS / 32; ++j) {
        const int r = (tid >> 3) + 32 * j;
        if (c < P.N && rows.id[r] == a)
          *reinterpret_cast<uint4*>(P.out + (row0 + r) * P.os + c) = *reinterpret_cast<const uint4*>(from + at(r, tid & 7));
      }
    };
    for (int i = 0; i < cols; ++i) {
      const uint32_t off = next(chunks + i), src = base + off + SH::TILE;
      if (i > 0) leave(i - 1);
      const uint8_t* y = smem + off;
      uint8_t* to = smem + SH::OUT + (i & 1) * SH::TILE;
      uint32_t w[KS][2];
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        uint32_t v[4];
        ldmatrix4(v, src + at_b(8 * warp + lr, 2 * s + (KS == 1 ? lm & 1 : lm)));
        w[s][0] = v[0];
        w[s][1] = v[1];
        if (s + 1 < KS) {
          w[s + 1][0] = v[2];
          w[s + 1][1] = v[3];
        }
      }
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) mma_16816(acc, tf[mt][s], w[s][0], w[s][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t place = at(16 * mt + gr + 8 * h, warp) + 4 * t;
          *reinterpret_cast<uint32_t*>(to + place) =
              add_half2(*reinterpret_cast<const uint32_t*>(y + place), acc[2 * h], acc[2 * h + 1], mul[mt][h]);
        }
      }
    }
    __syncthreads();
    if (cols > 0) leave(cols - 1);
  }
  if (tid == 0 && *abort_flag) {  // a wait gave up: no copy may land after the CTA has left
    const unsigned long long t0 = globaltimer();
    for (int k = max(0, issued - S); k < issued; ++k)
      while (!mbar_try_wait(base + SH::BARS + 8 * (k % S), (uint32_t)(k / S) & 1u) && globaltimer() - t0 < kWaitLimitNs) {
      }
  }
}

static void configure(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, int smem, cudaStream_t s) {
  *cfg = {};
  cfg->blockDim = dim3(kThreads, 1, 1);
  cfg->dynamicSmemBytes = (size_t)smem;
  cfg->stream = s;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = kCluster;
  at->val.clusterDim.y = 1;
  at->val.clusterDim.z = 1;
  cfg->attrs = at;
  cfg->numAttrs = 1;
}

// A launch of `tiles` x `splits` x `slots` clusters.  Slots: adapters of a tile (or adapters and 16 of their rows) side by
// side, as many as there may be but no more clusters than start at once, which the driver knows (GPCs are no
// multiple of a cluster): a second wave costs as much as the first.  Splits: clusters that share a tile's columns
// where it leaves SMs idle; each reads the rows and A again, so no more than make B's part the smaller.
template <typename Kernel, typename... Args>
static tm_status launch(Kernel kernel, int smem, long long tiles, long long slots, std::atomic<unsigned long long>& done,
                        std::atomic<int>* room_at, Params P, cudaStream_t s, const Args&... args) {
  if (!smem_attr_once(done, reinterpret_cast<const void*>(kernel), smem)) return TM_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute at;
  configure(&cfg, &at, smem, s);
  const int device = current_device();
  std::atomic<int>* cached = device >= 0 && device < kDevices ? room_at + device : nullptr;
  int room = cached ? cached->load(std::memory_order_relaxed) : 0;
  if (room <= 0) {
    cfg.gridDim = dim3(kCluster, 1, 1);
    if (cudaOccupancyMaxActiveClusters(&room, kernel, &cfg) != cudaSuccess || room < 1) return TM_ERR_CUDA;
    if (cached) cached->store(room, std::memory_order_relaxed);
  }
  if (slots * tiles > room) slots = room / tiles;
  if (slots < 1) slots = 1;
  long long splits = room / 2 / (tiles * slots);
  const long long blocks = (P.N + 32 * kCluster - 1) / (32 * kCluster);
  if (splits > blocks) splits = blocks;
  if (splits > 1 + P.N / P.K) splits = 1 + P.N / P.K;
  if (splits < 1) splits = 1;
  if (tiles * splits * kCluster > 0x7fffffffll) return TM_ERR_UNSUPPORTED;
  P.splits = (int)splits;
  cfg.gridDim = dim3((unsigned)(tiles * splits * kCluster), (unsigned)slots, 1);
  return cudaLaunchKernelEx(&cfg, kernel, args..., P) == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

template <int NT>
static tm_status launch_add(const Params& P, long long tiles, long long slots, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  static std::atomic<int> room[kDevices];
  return launch(add_kernel<NT>, Shape<NT>::SMEM, tiles, slots, done, room, P, s);
}

// fp16 [d2][d1][d0], rows `stride` elements apart; boxes of b1 rows x b0 elements (of at most 128 bytes, swizzled over them).
static bool tensor_map(CUtensorMap* map, const void* p, long long d0, long long d1, long long d2, long long stride, int b0,
                       int b1) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const int rank = d2 > 0 ? 3 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)stride * d1 * 2};
  const cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, 1}, ones[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void*>(p), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             b0 == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
             : b0 == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                        : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int RP>
static tm_status launch_wide(const Params& P, long long tiles, long long slots, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  static std::atomic<int> room[kDevices];
  Maps M;
  if (!tensor_map(&M.x, P.X, P.K, P.rows, 0, P.xs, 64, 64) || !tensor_map(&M.a, P.A, P.K, P.R, P.n, P.K, 64, RP) ||
      !tensor_map(&M.y, P.Y, P.N, P.rows, 0, P.ys, 64, 64) ||
      !tensor_map(&M.b, P.B, P.R, P.N, P.n, P.R, RP < 64 ? RP : 64, 64))
    return TM_ERR_CUDA;
  return launch(add_wide_kernel<RP>, Wide<RP>::SMEM, tiles, slots, done, room, P, s, M);
}

static tm_status launch(const Params& P, bool wide, long long tiles, long long slots, cudaStream_t s) {
  if (P.R <= 8 && !wide) return launch_add<1>(P, tiles, slots, s);
  if (P.R <= 16) return wide ? launch_wide<16>(P, tiles, slots, s) : launch_add<2>(P, tiles, slots, s);
  if (P.R <= 32) return wide ? launch_wide<32>(P, tiles, slots, s) : launch_add<4>(P, tiles, slots, s);
  if (P.R <= 64) return wide ? launch_wide<64>(P, tiles, slots, s) : launch_add<8>(P, tiles, slots, s);
  return wide ? launch_wide<128>(P, tiles, slots, s) : launch_add<16>(P, tiles, slots, s);
}

}  // namespace lora

cudaError_t lora_error_bits(uint32_t* bits, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, lora::s_err_lora, sizeof(v));
  if (e != cudaSuccess) return e;
  if (clear && v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(lora::s_err_lora, &zero, sizeof(zero));
  }
  *bits = v;
  return e;
}

}  // namespace w4

using namespace w4;

static bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

extern "C" tm_status tm_lora_add(const tm_lora_adapters* ad, const void* X, long long x_stride, const void* Y,
                                 long long y_stride, void* out, long long out_stride, long long rows, const int* ids,
                                 const int* q_start, int B, void* stream) {
  if (!ad || ad->n < 0 || ad->K < 8 || ad->K % 8 || ad->N < 8 || ad->N % 8 || ad->R < 8 || ad->R > 128 || ad->R % 8)
    return TM_ERR_INVALID_ARG;
  if (rows < 0 || B < 0 || (!q_start && rows != B)) return TM_ERR_INVALID_ARG;
  // Row and column indices are 32-bit in the kernels, and run ahead of the last one.
  if (rows > 0x7fffff00ll || ad->K > 1 << 30 || ad->N > 1 << 30) return TM_ERR_UNSUPPORTED;
  if (rows == 0 || B == 0) return TM_OK;
  if (!X || !Y || !out || !ids || (ad->n > 0 && (!ad->A || !ad->B))) return TM_ERR_INVALID_ARG;
  if (x_stride < ad->K || y_stride < ad->N || out_stride < ad->N) return TM_ERR_INVALID_ARG;
  if (out == Y && out_stride != y_stride) return TM_ERR_INVALID_ARG;
  if (!aligned_to(X, 16) || !aligned_to(Y, 16) || !aligned_to(out, 16) || !aligned_to(ad->A, 16) ||
      !aligned_to(ad->B, 16) || !aligned_to(ad->scale, 4) || !aligned_to(ids, 4) || !aligned_to(q_start, 4) ||
      x_stride % 8 || y_stride % 8 || out_stride % 8)
    return TM_ERR_ALIGNMENT;
  lora::Params P = {static_cast<const __half*>(X), static_cast<const __half*>(Y), static_cast<__half*>(out), x_stride,
                    y_stride, out_stride, static_cast<const __half*>(ad->A), static_cast<const __half*>(ad->B), ad->scale,
                    ids, q_start, (int)rows, B, ad->n, ad->K, ad->N, ad->R, 1};
  // Rows come in runs of one adapter where sequences are long.
  const bool wide = rows >= 16ll * B && ad->n > 0;
  const int tile = wide ? 64 : lora::kSpan;
  const long long in_tile = rows < tile ? rows : tile;
  long long slots = ad->n < in_tile ? ad->n : in_tile;
  if (slots > B) slots = B;
  if (!wide) slots += in_tile / 16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const tm_status st = lora::launch(P, wide, (rows + tile - 1) / tile, slots, s);
  if (st == TM_OK) set_launch_count(1);
  return st;
}
