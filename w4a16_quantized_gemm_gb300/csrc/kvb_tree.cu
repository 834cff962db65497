// Attention of trees of drafts over the paged 8-bit KV cache, up to 128 rows (nodes x query heads of a KV head): on
// tcgen05 like the kernel for prompts (kvb_prefill.cu, whose mathematics this is), but bound by what brings the codes
// in.
//
// A CTA takes one (sequence, KV head) and a slice of the tokens in tiles of 128, which its two halves take in turn,
// each with a running softmax and an output of its own; they are joined at the end.  With one row tile every tile of
// codes is converted for 128 rows alone, so that the conversion has eight warps, in two groups:
//   warps 0-3, 4-7: softmax of the even and of the odd tiles, one row per thread;
//   warps 8-11: K, 12-15: V codes -> fp16 numbers (exact) in shared memory, rings of three tiles each;
//   warp 16: S_i = Q K_n^T and O_i += P_i V_n, i = n % 2;
//   warp 17: pages and scales of the tiles to come, whose codes it requests into L2.
// All waits are bounded.
//
// What has fewer than 32 bits, since one product takes one 16-bit type and fp16 is the one that holds both formats'
// codes exactly: the weights, rounded once (the sum that divides takes them unrounded), so that fp16 results are off by
// 0.00025 to 0.00028 of themselves against 64 bits, with weights in 32 bits by 0.00021, the results' own rounding (bf16
// results: 0.0017 either way); and bf16 queries, which a power of two a row carries into fp16: exact down to 2^-31 of the
// row's largest element.  Scores, maxima, sums and outputs are fp32.
//
// Measured: 16 trees of up to 26 nodes over up to 4096 tokens, int8, 32 query and 8 KV heads (104 rows): 47 us for
// 108 MB of codes.  A tile takes 2.2 k cycles, which is what converting K takes four warps, and V four others (eight
// each: 56 us in all, by the registers that the softmax then lacks); the softmax of a row takes 2.3 k, one half's, and
// the hand-overs to the tensor cores and back 2 k more.  Tensor pipe 22 %, a third of it while the SMs are busy; 128
// CTAs of unequal length leave 37 % of the SMs' time idle, and cutting them evenly costs more than it saves.  What
// mattered, in us for that case: pages and scales of four tiles looked up at a time 71 -> 60, codes requested a page at
// a time 56; rows of no node out of the mask's way 49; scores kept and fetched ahead 47.5.
#include "kvb_attn.h"

namespace w4 {
namespace kvb {

static __device__ uint32_t s_err_kvbt;

constexpr int kTreeThreads = 640;  // the last two warps lend their registers
constexpr int kTreeTile = 128;  // tokens per tile, rows
constexpr int kTreeSlots = 3;   // K tiles in flight, V tiles
constexpr int kTreeMeta = 4;    // tiles whose scales are in flight
constexpr float kTreeBias = 6.f;
constexpr float kTreeSlack = 8.f;
constexpr float kTreeNone = -1e30f;

template <int D>
struct TreeShape {
  static constexpr int PANELS = D / 64;              // 64 fp16 = one 128-byte swizzled row
  static constexpr uint32_t PANEL = kTreeTile * 128;  // 16 KB
  static constexpr uint32_t TILE = PANELS * PANEL;
  static constexpr uint32_t K_OFF = TILE;            // behind the queries
  static constexpr uint32_t V_OFF = K_OFF + kTreeSlots * TILE;
  static constexpr uint32_t META = V_OFF + kTreeSlots * TILE;   // [kTreeMeta][8] x {ks, lv, 1 / vs, group}
  static constexpr uint32_t HOLES = META + kTreeMeta * 8 * 16;  // [kTreeMeta] bits of the 16-token groups
  static constexpr uint32_t BARS = HOLES + 16;
  static constexpr uint32_t DOWN = BARS + 256;       // [128]: what the rows' queries were scaled by, inverted
  static constexpr uint32_t SMEM = DOWN + 512 + 1024;
};

template <int FMT, int D>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const AttnParams P) {
  using SH = TreeShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  const View& V = P.V;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int b = blockIdx.x / V.Hkv, h = blockIdx.x - b * V.Hkv, chunk = blockIdx.y;
  const Span s = span(V, b);
  const int rows = s.n * P.G;
  const int j0 = chunk * P.chunk, j1 = min(s.len, j0 + P.chunk);
  if (rows == 0 || (j0 >= j1 && chunk > 0)) return;  // slice 0 still writes what an empty row gives
  const int N = j1 > j0 ? (j1 - j0 + kTreeTile - 1) / kTreeTile : 0;

  const uint32_t bars = base + SH::BARS;
  const uint32_t q_full = bars, o_full = bars + 8;
  auto s_full = [&](int i) { return bars + 16 + 8 * i; };
  auto p_full = [&](int i, int half) { return bars + 32 + 16 * i + 8 * half; };
  auto full = [&](int kv, int i) { return bars + 64 + 24 * kv + 8 * i; };
  auto empty = [&](int kv, int i) { return bars + 112 + 24 * kv + 8 * i; };
  auto meta_full = [&](int i) { return bars + 160 + 8 * i; };
  auto meta_empty = [&](int i) { return bars + 192 + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SH::BARS + 224);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::BARS + 228);
  if (tid == 0) {
    mbar_init(q_full, 8);
    mbar_init(o_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i, 0), 4);
      mbar_init(p_full(i, 1), 4);
      for (int k = 0; k < kTreeSlots; ++k) {
        mbar_init(full(i, k), 4);
        mbar_init(empty(i, k), 1);
      }
    }
    for (int i = 0; i < kTreeMeta; ++i) {
      mbar_init(meta_full(i), 1);
      mbar_init(meta_empty(i), 8 + 4);  // the converting warps, and the half that takes the tile
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S_0, S_1 (P_i over S_i), then O_0, O_1

  if (warp < 8) {
    // ---------------- softmax: one row per thread ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int i = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const bool ok = r < rows;
    const int qi = ok ? r / P.G : 0;
    const size_t hr = (size_t)(s.row0 + qi) * P.Hq + h * P.G + (ok ? r - qi * P.G : 0);
    const bool busy = __any_sync(0xffffffffu, ok);  // else the warp's rows are no one's: it keeps the tiles going
    const uint32_t* mask = P.tree + (s.row0 + qi) * P.tree_stride;
    float mul = fabsf(P.scale_log2);
    {
      // Queries into shared memory, 16 bytes a thread, a row by neighbouring lanes: as fp16, bf16 rows times a power of
      // two.  A negative scale is taken into their sign.
      constexpr int LANES = D / 8, STEP = 256 / LANES, PASSES = kTreeTile / STEP;
      const uint32_t flip = P.scale_log2 < 0.f ? 0x80008000u : 0u;
      const int c = tid % LANES, r0 = tid / LANES;
      uint4 x[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int row = r0 + p * STEP;
        const bool have = row < rows;
        const int q = have ? row / P.G : 0;
        const int head = h * P.G + (have ? row - q * P.G : 0);
        x[p] = ldg_or_zero(P.Q + (s.row0 + q) * P.q_stride + (long long)head * D + 8 * c, have);
      }
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int row = r0 + p * STEP;
        uint32_t wd[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
        if (P.bf16) {
          float2 f[4];
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] = unpack(wd[k], true);
            top = max3(top, fabsf(f[k].x), fabsf(f[k].y));
          }
#pragma unroll
          for (int k = 1; k < LANES; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
          const int e2 = max((int)(__float_as_uint(top) >> 23) - 127, -100);
          const float up = __uint_as_float((uint32_t)(127 + min(14 - e2, 126)) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) wd[k] = pack_half2(f[k].x * up, f[k].y * up);
          if (c == 0)
            reinterpret_cast<float*>(smem + SH::DOWN)[row] = __uint_as_float((uint32_t)(127 - min(14 - e2, 126)) << 23);
        }
        sts128(base + (c >> 3) * SH::PANEL + row * 128 + (((c & 7) ^ (row & 7)) << 4), wd[0] ^ flip, wd[1] ^ flip,
               wd[2] ^ flip, wd[3] ^ flip);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      if (P.bf16) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        mul *= reinterpret_cast<const float*>(smem + SH::DOWN)[r];
      }
    }

    float m = kTreeNone, l = 0.f;
    const uint32_t ts = tmem + lanes + 128 * i, to = tmem + lanes + 256 + D * i;
    bool alive = true;
#pragma unroll 1
    for (int n = i; n < N; n += 2) {
      const int turn = n >> 1, slot = n % kTreeMeta;
      alive = wait_bar(meta_full(slot), (uint32_t)(n / kTreeMeta) & 1u, abort_flag, &s_err_kvbt) &&
              wait_bar(s_full(i), (uint32_t)turn & 1u, abort_flag, &s_err_kvbt);
      if (!__all_sync(0xffffffffu, alive)) {
        alive = false;
        break;
      }
      if (!busy) {
        if (lane == 0) {
          mbar_arrive(p_full(i, 0));
          mbar_arrive(p_full(i, 1));
          mbar_arrive(meta_empty(slot));
        }
        continue;
      }
      tc_fence_after();
      const uint32_t meta = base + SH::META + slot * 128;
      const int rel = s.len - 1 - (j0 + n * kTreeTile);  // columns 0 .. rel are there
      const int fresh = j0 + n * kTreeTile - s.old;    // the tile's first token, counted in new ones
      const uint32_t holes = lds32(base + SH::HOLES + 4 * slot);
      const bool part = fresh + kTreeTile > 0 || rel < kTreeTile - 1 || holes;
      uint32_t v[2][32];
      // What the row does not see, in tensor memory, in a loop of its own: the tiles without any of this stay in the
      // instruction cache.
      if (part) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tc_ld_32x32b_x32(ts + 32 * c, v[0]);
          const uint32_t see = tree_columns(P, mask, fresh, rel, holes, c);
          tc_wait_ld_of(v[0]);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((see >> k) & 1u)) v[0][k] = 0xff800000u;
          tc_st_32x32b_x32(ts + 32 * c, v[0]);
        }
        tc_wait_st();
      }
      // A quarter of the tile's scores is on its way while the one before is used: 0 .. 3 for the maximum, then 2 and
      // 3, which are still there, and 0 and 1 again for the weights (all of them would take the registers of two warps).
      float tm = -INFINITY;
      tc_ld_32x32b_x32(ts, v[0]);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g == 0) {
            tc_wait_ld_of(v[0]);
            tc_ld_32x32b_x32(ts + 64 * half + 32, v[1]);
          } else if (g == 2) {
            tc_wait_ld_of(v[1]);
            if (half == 0) tc_ld_32x32b_x32(ts + 64, v[0]);
          }
          const float4 mt = lds_f4(meta + 64 * half + 16 * g);
          auto val = [&](int c) { return __uint_as_float(v[g >> 1][16 * (g & 1) + c]); };
          float a = max3(val(0), val(1), val(2)), a2 = max3(val(3), val(4), val(5));
#pragma unroll
          for (int c = 6; c < 14; c += 4) {
            a = max3(a, val(c), val(c + 1));
            a2 = max3(a2, val(c + 2), val(c + 3));
          }
          a = max3(a, a2, fmaxf(val(14), val(15)));
          tm = fmaxf(tm, fmaf(a, fmaxf(mt.x * mul, 1e-35f), mt.y));
        }
      }
      if (__any_sync(0xffffffffu, ok && tm > m + kTreeSlack)) {
        const float mn = fmaxf(m, tm), f = ex2(m - mn);
        m = mn;
        l *= f;
        if (turn > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tc_ld_32x32b_x32(to + c, o);
            tc_wait_ld_of(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tc_st_32x32b_x32(to + c, o);
          }
        }
      }
#pragma unroll
      for (int half = 1; half >= 0; --half) {
        uint32_t p[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g == 0 && half == 0) {
            tc_wait_ld_of(v[0]);
            tc_ld_32x32b_x32(ts + 32, v[1]);
          } else if (g == 2) {
            if (half == 1) {
              tc_ld_32x32b_x32(ts, v[0]);
            } else {
              tc_wait_ld_of(v[1]);
            }
          }
          const float4 mt = lds_f4(meta + 64 * half + 16 * g);
          const float cg = fmaxf(mt.x * mul, 1e-35f), off = mt.y + kTreeBias - m;
          const uint64_t cg2 = f32x2(cg, cg), off2 = f32x2(off, off);
          uint64_t sum = 0ull;
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const uint32_t* x = &v[g >> 1][16 * (g & 1) + c];
            const float2 e = f32x2_get(fma_f32x2(f32x2(__uint_as_float(x[0]), __uint_as_float(x[1])), cg2, off2));
            const float p0 = ex2(e.x), p1 = ex2(e.y);
            sum = add_f32x2(sum, f32x2(p0, p1));
            p[8 * (g & 1) + c / 2] = pack_half2(p0, p1);  // the codes' type in the product; l keeps all bits
          }
          const float2 part_sum = f32x2_get(sum);
          l = fmaf(part_sum.x + part_sum.y, mt.z, l);
          if (g & 1) tc_st_32x32b_x16(ts + 64 * half + 8 * (g - 1), p);  // over this half's scores
        }
        // One half goes to the tensor cores while the other is computed.
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(i, half));
      }
      if (lane == 0) mbar_arrive(meta_empty(slot));
    }
    if (N > 0 && alive) {
      alive = wait_bar(o_full, 0, abort_flag, &s_err_kvbt);
      alive = __all_sync(0xffffffffu, alive);
      tc_fence_after();
    }
    // ---- the halves are joined through the tiles' memory (free: all products are done), each for half the columns
    constexpr int COLS = D / 2;
    float* state = reinterpret_cast<float*>(smem + SH::K_OFF) + r;            // [m, l of the first, of the second][128]
    auto given = [&](int to_half) { return state + (4 + to_half * COLS) * kTreeTile; };  // [COLS][128]
    auto output = [&](int c, uint32_t (&o)[32]) {
      if (i < N) {
        tc_ld_32x32b_x32(to + c, o);
        tc_wait_ld_of(o);
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
      }
    };
    if (alive) {
      state[2 * i * kTreeTile] = m;
      state[(2 * i + 1) * kTreeTile] = l;
#pragma unroll 1
      for (int c = 0; c < COLS; c += 32) {
        uint32_t o[32];
        output((1 - i) * COLS + c, o);
#pragma unroll
        for (int k = 0; k < 32; ++k) given(1 - i)[(c + k) * kTreeTile] = __uint_as_float(o[k]);
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    // ---- the row's output, or its state for the joining launch
    if (alive) {
      const float m0 = state[0], m1 = state[2 * kTreeTile], top = fmaxf(m0, m1), f0 = ex2(m0 - top), f1 = ex2(m1 - top);
      const float sum = state[kTreeTile] * f0 + state[3 * kTreeTile] * f1;
      const float inv = sum > 0.f || sum != sum ? __fdividef(1.f, sum) : 0.f;
      const float mine = i ? f1 : f0, others = i ? f0 : f1;
#pragma unroll 1
      for (int c = 0; c < COLS; c += 32) {
        uint32_t o[32];
        output(i * COLS + c, o);
        if (ok) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(__uint_as_float(o[k]) * mine + given(i)[(c + k) * kTreeTile] * others);
          if (P.chunks == 1) {
            uint16_t* out = P.out + hr * D + i * COLS + c;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t wd[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = __uint_as_float(o[k + 2 * e]) * inv, a2 = __uint_as_float(o[k + 2 * e + 1]) * inv;
                wd[e] = P.bf16 ? pack_bf162(a, a2) : pack_half2(a, a2);
              }
              *reinterpret_cast<uint4*>(out + k) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
            }
          } else {
            float* dst = P.part + (hr * P.chunks + chunk) * D + i * COLS + c;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<uint4*>(dst + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        __syncwarp();  // whole again for the next load
      }
      if (ok && i == 0) {
        if (P.chunks > 1)
          P.part_ml[hr * P.chunks + chunk] = make_float2(top - kTreeBias, sum);
        else if (P.lse)
          P.lse[hr] = sum == 0.f ? -INFINITY : (log2f(sum) + top - kTreeBias) * 0.693147180559945f;
      }
    }
    tc_fence_before();
  } else if (warp < 16) {
    // ---------------- codes -> fp16 tiles: warps 8-11 the keys', 12-15 the values' ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int kv = (warp - 8) >> 2;
    // A warp's pass takes 4 (D = 64: 8) rows, the next one those 16 (32) rows further on: the same row of another
    // 16-token group, so that of all addresses only the group changes.  Eight lanes write two rows of one
    // 64-dimension panel: no bank conflicts.
    constexpr int PASSES = D == 128 ? 8 : 4;
    constexpr int STEP = kTreeTile / PASSES;
    const int c4 = lane & 3;
    const int panel = D == 128 ? (lane >> 3) & 1 : 0;
    const int r0 = (warp & 3) * (STEP / 4) + ((lane >> 2) & 1) + 2 * (D == 128 ? lane >> 4 : lane >> 3);
    const uint8_t* pool = (kv ? V.v : V.k) + (r0 & 15) * D + panel * 64 + c4 * 16;
    const uint32_t groups = base + SH::META + (r0 >> 4) * 16 + 12;
    const uint32_t tiles = base + (kv ? SH::V_OFF : SH::K_OFF) + panel * SH::PANEL + r0 * 128;
    const uint32_t at0 = tiles + (((2 * c4) ^ (r0 & 7)) << 4), at1 = tiles + (((2 * c4 + 1) ^ (r0 & 7)) << 4);
    uint4 x[PASSES];
    int group[PASSES];
    auto look_up = [&](int n) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) group[p] = (int)lds32(groups + (n % kTreeMeta) * 128 + p * STEP);
    };
    // The codes of tile n.  Rows past the end read as zeros: stale codes may be NaN.
    auto fetch = [&](int n, int p) {
      x[p] = ldg_or_zero(pool + (size_t)(unsigned)max(group[p], 0) * (16 * D),
                         group[p] >= 0 && j0 + n * kTreeTile + r0 + p * STEP < j1);
    };
    bool alive = N == 0 || wait_bar(meta_full(0), 0, abort_flag, &s_err_kvbt);
    alive = __all_sync(0xffffffffu, alive);
    if (N > 0 && alive) {
      look_up(0);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) fetch(0, p);
    }
#pragma unroll 1
    for (int n = 0; n < N && alive; ++n) {
      const int slot = n % kTreeSlots;
      const bool more = n + 1 < N;
      alive = wait_bar(empty(kv, slot), ((uint32_t)(n / kTreeSlots) & 1u) ^ 1u, abort_flag, &s_err_kvbt);
      if (more)
        alive = alive && wait_bar(meta_full((n + 1) % kTreeMeta), (uint32_t)((n + 1) / kTreeMeta) & 1u, abort_flag,
                                  &s_err_kvbt);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      if (more) look_up(n + 1);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        uint32_t o[8];
        codes_half<FMT>(x[p].x, o[0], o[1]);
        codes_half<FMT>(x[p].y, o[2], o[3]);
        codes_half<FMT>(x[p].z, o[4], o[5]);
        codes_half<FMT>(x[p].w, o[6], o[7]);
        if (more) fetch(n + 1, p);
        sts128(at0 + slot * SH::TILE + p * (STEP * 128), o[0], o[1], o[2], o[3]);
        sts128(at1 + slot * SH::TILE + p * (STEP * 128), o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full(kv, slot));
        mbar_arrive(meta_empty(n % kTreeMeta));  // tile n's groups were read when it was fetched
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 16) {
      // ---------------- products ----------------
      // The whole warp walks the loop, so that descriptors and addresses stay uniform; one lane issues.
      if (N > 0) {
        constexpr uint32_t id_s = idesc_f16_f32(128, 128);
        constexpr uint32_t id_o = idesc_f16_f32(128, D) | (1u << 16);  // B is MN-major
        constexpr uint64_t kTileDesc = SH::TILE >> 4, kPanelDesc = SH::PANEL >> 4;
        const uint64_t dq = smem_desc_sw128(base), dk = smem_desc_sw128(base + SH::K_OFF);
        const uint64_t dv = smem_desc_mn(base + SH::V_OFF, SH::PANEL);
        const uint32_t lead = elect_one();
        const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);  // known to be uniform
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
          return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, &s_err_kvbt)) != 0;
        };
        auto keys = [&](int n) { return wait_all(full(0, n % kTreeSlots), (uint32_t)(n / kTreeSlots) & 1u); };
        // Scores of tile n into those of half n % 2, whose weights of tile n - 2 have been used.
        auto scores = [&](int n) {
          const int i = n & 1, slot = n % kTreeSlots;
          tc_fence_after();
          const uint64_t db = dk + (uint64_t)slot * kTileDesc;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (k >> 2) * kPanelDesc + (k & 3) * 2;
            mma_ss_if(lead, tm0 + 128 * i, dq + off, db + off, id_s, k > 0);
          }
          commit_if(lead, s_full(i));
          commit_if(lead, empty(0, slot));
        };
        bool alive = wait_all(q_full, 0);
        // scores 0, 1, [output n, scores n + 2] ...
#pragma unroll 1
        for (int n = -2; n < N && alive; ++n) {
          if (n >= 0) {
            const int i = n & 1, turn = n >> 1, slot = n % kTreeSlots;
            alive = wait_all(full(1, slot), (uint32_t)(n / kTreeSlots) & 1u);
            const uint64_t db = dv + (uint64_t)slot * kTileDesc;
#pragma unroll
            for (int half = 1; half >= 0; --half) {
              alive = alive && wait_all(p_full(i, half), (uint32_t)turn & 1u);
              // The next keys are looked for here, not between the weights and the scores that wait for their place.
              if (half == 1 && n + 2 < N) alive = alive && keys(n + 2);
              if (!alive) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts_if(lead, tm0 + 256 + D * i, tm0 + 128 * i + 64 * half + 8 * k,
                          db + (uint64_t)(((4 * half + k) * 16 * 128) >> 4), id_o, turn > 0 || half == 0 || k > 0);
            }
            if (!alive) break;
            commit_if(lead, empty(1, slot));
          } else if (n + 2 < N) {
            alive = keys(n + 2);
          }
          if (n + 2 < N && alive) scores(n + 2);
        }
        commit_if(lead, o_full);
        if (lead) {
          // Nothing is left in flight when tensor memory is freed, on an abort either.
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(o_full, 0)) {
            if (globaltimer() - t0 > kWaitLimitNs) {
              atomicOr(&s_err_kvbt, kErrTimeout);
              break;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == 17) {
      // ---------------- pages and scales ----------------
      publish_pages<D, kTreeMeta>(V, b, h, j0, j1, N, base + SH::META, base + SH::HOLES, meta_full(0), meta_empty(0),
                                  abort_flag, &s_err_kvbt);
    }
  }
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int D>
static tm_status launch(const AttnParams& P, cudaStream_t stream) {
  using SH = TreeShape<D>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(tree_kernel<FMT, D>), SH::SMEM)) return TM_ERR_CUDA;
  tree_kernel<FMT, D><<<dim3((unsigned)(P.V.B * P.V.Hkv), (unsigned)P.chunks), kTreeThreads, SH::SMEM, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

tm_status launch_tree_attn(const AttnParams& P, int format, int D, cudaStream_t stream) {
  if (format == TM_KVB_INT8) return D == 64 ? launch<TM_KVB_INT8, 64>(P, stream) : launch<TM_KVB_INT8, 128>(P, stream);
  return D == 64 ? launch<TM_KVB_E4M3, 64>(P, stream) : launch<TM_KVB_E4M3, 128>(P, stream);
}

}  // namespace kvb

cudaError_t kvb_tree_error_bits(uint32_t* bits, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, kvb::s_err_kvbt, sizeof(v));
  if (e != cudaSuccess) return e;
  if (clear && v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(kvb::s_err_kvbt, &zero, sizeof(zero));
  }
  *bits = v;
  return e;
}

}  // namespace w4
