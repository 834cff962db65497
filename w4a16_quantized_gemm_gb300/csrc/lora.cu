// Low-rank adapters of many requests beside a shared projection:
//   out = Y + scale_a (X A_a^T) B_a^T,  a the adapter of the row's sequence.
//
// One launch: a cluster of eight CTAs takes a tile of 16 or 64 rows and the adapters that appear in it.
//   T = X A^T: each CTA a slice of K, each warp 16 rows of a part of it, on mma.m16n8k16 with operands straight from
//     global memory.  The sum over k may go in any order, so that a lane's 16-byte chunk of a row holds the eight k
//     of two products and both operands are read in whole sectors;
//   the eight partial T meet in distributed shared memory: CTA c sums the tile's rows c, c + 8, ... and hands them,
//     scaled by a power of two into fp16's range, to all eight;
//   out: each CTA a slice of N.  A lane's products are arranged to be eight consecutive columns.
// No partial result goes through memory, rows that use another adapter are computed along and not stored, and an
// adapter is read once per tile that uses it.
#include <cuda_fp16.h>

#include <atomic>

#include "../../include/tm_lora.h"
#include "tm_common.cuh"

namespace w4 {
namespace lora {

constexpr int kThreads = 256;
constexpr int kCluster = 8;

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

// MT: 16-row groups of the tile; NT: groups of 8 ranks.
template <int MT, int NT>
struct Shape {
  static constexpr int ROWS = 16 * MT;
  static constexpr int KW = 8 / MT;        // warps that share a row group along K
  static constexpr int RP = 8 * NT;        // ranks, padded
  static constexpr int KS = (NT + 1) / 2;  // k-steps of the second product
  static constexpr uint32_t PART = 0;      // [KW][ROWS][RP] fp32
  static constexpr uint32_t SUM = PART + KW * ROWS * RP * 4;       // [ROWS][RP] fp32, this CTA's share of K
  static constexpr uint32_t FRAG = SUM + ROWS * RP * 4;            // [MT][KS][32] x 16 bytes: T as A fragments
  static constexpr uint32_t MUL = FRAG + MT * KS * 512;            // [ROWS] fp32
  static constexpr uint32_t SMEM = MUL + ROWS * 4;
};

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

template <int MT, int NT>
__global__ void __launch_bounds__(kThreads) add_kernel(const Params P) {
  using SH = Shape<MT, NT>;
  constexpr int ROWS = SH::ROWS, RP = SH::RP, KS = SH::KS, KW = SH::KW;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int seq_s[ROWS], id_s[ROWS], list_s[ROWS];
  __shared__ int count_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int rank = (int)cluster_ctarank();
  const int cl = blockIdx.x / kCluster;
  const int tile = cl / P.splits, split = cl - tile * P.splits;
  const int row0 = tile * ROWS;
  const uint32_t base = smem_u32(smem);

  // ---- whose rows these are
  for (int r = tid; r < ROWS; r += kThreads) seq_s[r] = P.q_start || row0 + r >= P.rows ? -1 : row0 + r;
  __syncthreads();
  if (P.q_start)
    for (int b = tid; b < P.seqs; b += kThreads) {
      const int lo = max(min(max(P.q_start[b], 0), P.rows), row0);
      const int hi = min(min(max(P.q_start[b + 1], 0), P.rows), row0 + ROWS);
      for (int r = lo; r < hi; ++r) atomicMax(&seq_s[r - row0], b);
    }
  __syncthreads();
  if (tid < ROWS) {
    const int b = seq_s[tid];
    const int a = b >= 0 ? P.ids[b] : -2;
    id_s[tid] = b >= 0 && (unsigned)a >= (unsigned)P.n ? -1 : a;  // -1: no adapter, -2: no sequence
  }
  __syncthreads();
  if (warp == 0) {  // the different adapters, in the order of their first rows
    int found = 0;
    for (int r0 = 0; r0 < ROWS; r0 += 32) {
      const int r = r0 + lane;
      bool first = r < ROWS && id_s[r < ROWS ? r : 0] >= 0;
      if (first)
        for (int x = 0; x < r; ++x) first = first && id_s[x] != id_s[r];
      const uint32_t who = __ballot_sync(0xffffffffu, first);
      if (first) list_s[found + __popc(who & ((1u << lane) - 1u))] = id_s[r];
      found += __popc(who);
    }
    if (lane == 0) count_s = found;
  }
  __syncthreads();
  const int count = count_s;

  // This CTA's columns, in blocks of 32.
  const int blocks = (P.N + 31) / 32, parts = kCluster * P.splits, part = split * kCluster + rank;
  const int n0 = (int)((long long)blocks * part / parts), n1 = (int)((long long)blocks * (part + 1) / parts);
  if (blockIdx.y == 0 && P.out != P.Y) {  // rows without an adapter
    for (int r = warp; r < ROWS; r += 8) {
      if (id_s[r] != -1) continue;
      const __half* src = P.Y + (row0 + r) * P.ys;
      __half* dst = P.out + (row0 + r) * P.os;
      for (int c = 32 * n0 + 8 * lane; c < min(32 * n1, P.N); c += 256)
        *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + c);
    }
  }

  for (int z = blockIdx.y; z < count; z += gridDim.y) {
    const int a = list_s[z];
    // ---- T: this CTA's chunks of 32 k
    {
      const int mt = warp % MT, kw = warp / MT;
      const int r_lo = mt * 16 + gr, r_hi = r_lo + 8;
      const bool any = __any_sync(0xffffffffu, id_s[r_lo] == a || id_s[r_hi] == a);
      const bool lo_ok = id_s[r_lo] == a, hi_ok = id_s[r_hi] == a;
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
      if (any) {
        const __half* xl = P.X + (row0 + r_lo) * P.xs + 8 * t;
        const __half* xh = P.X + (row0 + r_hi) * P.xs + 8 * t;
        const __half* pa = P.A + ((size_t)a * P.R + gr) * P.K + 8 * t;
        const int chunks = (P.K + 31) / 32, stride = kCluster * KW;
#pragma unroll(NT <= 2 ? 4 : NT <= 4 ? 2 : 1)
        for (int ch = rank * KW + kw; ch < chunks; ch += stride) {
          const int k = 32 * ch;
          const bool in = k + 8 * t < P.K;
          const uint4 x0 = ldg16(xl + k, in && lo_ok), x1 = ldg16(xh + k, in && hi_ok);
          uint4 w[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i) w[i] = ldg16(pa + (size_t)(8 * i) * P.K + k, in && 8 * i + gr < P.R);
          const uint32_t f0[4] = {x0.x, x1.x, x0.y, x1.y}, f1[4] = {x0.z, x1.z, x0.w, x1.w};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma_16816(acc[i], f0, w[i].x, w[i].y);
            mma_16816(acc[i], f1, w[i].z, w[i].w);
          }
        }
      }
      float* dst = reinterpret_cast<float*>(smem + SH::PART) + ((size_t)kw * ROWS + r_lo) * RP + 2 * t;
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
      for (int i = tid; i < ROWS * RP; i += kThreads) {
        float v = src[i];
#pragma unroll
        for (int k = 1; k < KW; ++k) v += src[k * ROWS * RP + i];
        dst[i] = v;
      }
    }
    cluster_sync_all();
    // ---- rows rank, rank + 8, ...: the sum over the CTAs, to fp16, to all of them
    for (int r = rank + kCluster * warp; r < ROWS; r += kCluster * 8) {
      constexpr int PER = (RP + 31) / 32;
      float v[PER], big = 0.f;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = lane + 32 * k;
        v[k] = 0.f;
        if (c < RP) {
          const uint32_t at = base + SH::SUM + (r * RP + c) * 4;
          float x[kCluster];
#pragma unroll
          for (int q = 0; q < kCluster; ++q) x[q] = ld_dsmem_f32(map_shared_rank(at, q));
#pragma unroll
          for (int q = 0; q < kCluster; ++q) v[k] += x[q];
        }
        v[k] *= P.scale ? P.scale[a] : 1.f;
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
        const uint16_t bits = c < RP ? __half_as_ushort(__float2half_rn(v[k] * up)) : (uint16_t)0;
        // A fragment of k-step c / 16: lane (row % 8, x) holds ranks 4 x .. 4 x + 3 of it, rows r and r + 8
        const int x = (c >> 2) & 3, word = 2 * ((c >> 1) & 1) + ((r >> 3) & 1);
        const uint32_t at = base + SH::FRAG + (((r >> 4) * KS + (c >> 4)) * 32 + (r & 7) * 4 + x) * 16 + word * 4 + (c & 1) * 2;
#pragma unroll
        for (int q = 0; q < kCluster; ++q) st_dsmem_u16(map_shared_rank(at, q), bits);
      }
      if (lane < kCluster) st_dsmem_f32(map_shared_rank(base + SH::MUL + r * 4, lane), down);
    }
    cluster_sync_all();
    // ---- out: blocks of 32 columns
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
#pragma unroll 1
      for (int mt = 0; mt < MT; ++mt) {
        const int r_lo = mt * 16 + gr;
        const bool lo_ok = id_s[r_lo] == a && c0 < P.N, hi_ok = id_s[r_lo + 8] == a && c0 < P.N;
        if (!__any_sync(0xffffffffu, lo_ok || hi_ok)) continue;
        uint4 y[2] = {};
        if (lo_ok) y[0] = *reinterpret_cast<const uint4*>(P.Y + (row0 + r_lo) * P.ys + c0);
        if (hi_ok) y[1] = *reinterpret_cast<const uint4*>(P.Y + (row0 + r_lo + 8) * P.ys + c0);
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint4 f = *reinterpret_cast<const uint4*>(smem + SH::FRAG + ((mt * KS + s) * 32 + lane) * 16);
          const uint32_t fa[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_16816(acc[i], fa, w[i][s].x, w[i][s].y);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float f = mul[r_lo + 8 * half];
          const uint32_t yw[4] = {y[half].x, y[half].y, y[half].z, y[half].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&yw[i]));
            const __half2 h = __floats2half2_rn(fmaf(acc[i][2 * half], f, v.x), fmaf(acc[i][2 * half + 1], f, v.y));
            o[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (half ? hi_ok : lo_ok)
            *reinterpret_cast<uint4*>(P.out + (row0 + r_lo + 8 * half) * P.os + c0) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
}

template <int MT, int NT>
tm_status launch(const Params& P, dim3 grid, cudaStream_t s) {
  using SH = Shape<MT, NT>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(add_kernel<MT, NT>), SH::SMEM)) return TM_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = SH::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_kernel<MT, NT>, P) == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

template <int MT>
tm_status launch(const Params& P, dim3 grid, cudaStream_t s) {
  if (P.R <= 8) return launch<MT, 1>(P, grid, s);
  if (P.R <= 16) return launch<MT, 2>(P, grid, s);
  if (P.R <= 32) return launch<MT, 4>(P, grid, s);
  if (P.R <= 64) return launch<MT, 8>(P, grid, s);
  return launch<MT, 16>(P, grid, s);
}

}  // namespace lora
}  // namespace w4

using namespace w4;

static bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

extern "C" tm_status tm_lora_add(const tm_lora_adapters* ad, const void* X, long long x_stride, const void* Y,
                                 long long y_stride, void* out, long long out_stride, long long rows, const int* ids,
                                 const int* q_start, int B, void* stream) {
  if (!ad || ad->n < 0 || ad->K < 8 || ad->K % 8 || ad->N < 8 || ad->N % 8 || ad->R < 8 || ad->R > 128 || ad->R % 8)
    return TM_ERR_INVALID_ARG;
  if (rows < 0 || B < 0 || (!q_start && rows != B)) return TM_ERR_INVALID_ARG;
  if (rows > 0x7fffff00ll) return TM_ERR_UNSUPPORTED;  // row indices are 32-bit in the kernel
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
  // Rows come in runs of one adapter where sequences are long: tiles of 64 then read an adapter a quarter as often.
  const bool wide = rows >= 16ll * B;
  const int tile = wide ? 64 : 16;
  const long long tiles = (rows + tile - 1) / tile;
  const long long room = 2ll * num_sms(current_device()) / lora::kCluster;  // clusters that start at once
  long long slots = ad->n < tile ? ad->n : tile;                            // adapters of a tile side by side
  if (slots > rows) slots = rows;
  if (slots > B) slots = B;
  if (slots * tiles > room) slots = room / tiles;
  if (slots < 1) slots = 1;
  // Clusters that share a tile's columns: each reads the rows and A again, so no more than make B's part the smaller.
  long long splits = room / 2 / (tiles * slots);
  const long long blocks = (ad->N + 32 * lora::kCluster - 1) / (32 * lora::kCluster);
  if (splits > blocks) splits = blocks;
  if (splits > 1 + ad->N / ad->K) splits = 1 + ad->N / ad->K;
  if (splits < 1) splits = 1;
  P.splits = (int)splits;
  if (tiles * splits * lora::kCluster > 0x7fffffffll) return TM_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(tiles * splits * lora::kCluster), (unsigned)slots, 1);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const tm_status st = wide ? lora::launch<4>(P, grid, s) : lora::launch<1>(P, grid, s);
  if (st == TM_OK) set_launch_count(1);
  return st;
}
