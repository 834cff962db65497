// Attention over the paged 8-bit KV cache for many rows (prompts and their
// chunks): bound by the tensor cores, on tcgen05 with the scores, the weights and
// the output in tensor memory.
//
// A CTA takes one (sequence, KV head), 2 x 128 rows (query token, query head of
// the group: heads that share keys share the tile) and, where there are few
// rows, a slice of the tokens; tiles of 128 tokens.
//   warps 0-3, 4-7: softmax of the first and the second 128 rows, one row per
//     thread: scores from tensor memory, the running maximum (which moves only
//     when it has grown by more than 8, so that the output is rarely rescaled), weights
//     as fp16 back into the columns of the scores;
//   warps 8-11, 14, 15: codes -> fp16 numbers (exact) in shared memory, K and V tiles in
//     turn through a ring of four; the next tile's codes are requested while
//     this one's are converted;
//   warp 12: S_i = Q_i K^T (A, B in shared memory) and O_i += P_i V (A in tensor
//     memory, V as it lies, MN-major), the two row tiles in turn, so that one
//     computes while the other's softmax runs;
//   warp 13: pages and scales of the tiles to come.
// The scales stay out of the products as in the kernel for few rows: ks
// multiplies the scores, log2 vs joins the exponent and leaves l again.
// All waits are bounded.
//
// Measured: 2048 tokens over 8192, 32 query and 8 KV heads: 214 us, 1.12 PFLOP/s, tensor pipe 47 %.  Between two
// products of a row tile lie the softmax (about 1.7 k cycles a row: 250 to fetch the scores, 500 for the
// maximum, 900 for the weights) and the hand-overs; the conversion of a K and a V tile takes six warps about
// 3 k.  What mattered, in us for that case: operands in uniform registers 376 -> 250 (the issuing warp was
// the bottleneck), packed pairs and weights in halves 239, six converting warps 227, registers 192 / 64 / 64
// 214 (184 / 80 / 64: 227; 200 / 64 / 48: 225).  Fresh prompts of 1499 tokens: 113 us, where starting a CTA for
// each 256 rows costs as much as its six token tiles.
#include <type_traits>

#include "kvb_attn.h"

namespace w4 {
namespace kvb {

static __device__ uint32_t s_err_kvb;

constexpr int kPreThreads = 512;
constexpr int kPreTile = 128;   // tokens per tile, rows per row tile
constexpr int kPreConv = 6;     // converting warps
constexpr int kPreSlots = 4;    // K and V tiles in flight
constexpr int kPreMeta = 4;     // tiles whose scales are in flight
constexpr float kPreBias = 6.f;
constexpr float kPreSlack = 8.f;
constexpr float kPreNone = -1e30f;

template <int D>
struct PreShape {
  static constexpr int PANELS = D / 64;                 // 64 fp16 = one 128-byte swizzled row
  static constexpr uint32_t PANEL = kPreTile * 128;     // 16 KB
  static constexpr uint32_t TILE = PANELS * PANEL;
  static constexpr uint32_t Q_OFF = 0;
  static constexpr uint32_t KV_OFF = 2 * TILE;
  static constexpr uint32_t META = KV_OFF + kPreSlots * TILE;  // [kPreMeta][8] x {ks, lv, 1 / vs, group}
  static constexpr uint32_t HOLES = META + kPreMeta * 8 * 16;  // [kPreMeta] bits of the 16-token groups
  static constexpr uint32_t BARS = HOLES + 16;
  static constexpr uint32_t SMEM = BARS + 256 + 1024;
};

// MN-major operand: rows of K (tokens) of 128 bytes, 128-byte swizzle, 8-row
// atoms 1024 bytes apart along K, 64-element panels `panel` bytes apart along N.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// 16 bytes, or zeros.
__device__ __forceinline__ uint4 ldg_or_zero(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)ok));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kPreThreads, 1) prefill_kernel(const AttnParams P) {
  using SH = PreShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  const View& V = P.V;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int b = blockIdx.x / V.Hkv, h = blockIdx.x - b * V.Hkv;
  const int chunk = blockIdx.y % P.chunks;
  const int pair = (int)(gridDim.y / P.chunks) - 1 - blockIdx.y / P.chunks;  // the longest rows first
  const Span s = span(V, b);
  const int rows = s.n * P.G;
  const int row_base = pair * 2 * kPreTile;
  if (row_base >= rows) return;
  const int last_i = (min(row_base + 2 * kPreTile, rows) - 1) / P.G;
  const int j0 = chunk * P.chunk;
  const int j1 = min(min(s.len, j0 + P.chunk), s.old + last_i + 1);
  if (j0 >= j1 && chunk > 0) return;  // slice 0 still writes what an empty row gives
  const int N = j1 > j0 ? (j1 - j0 + kPreTile - 1) / kPreTile : 0;
  const int M = rows - row_base > kPreTile ? 2 : 1;  // row tiles

  const uint32_t bars = base + SH::BARS;
  const uint32_t q_full = bars;
  auto s_full = [&](int i) { return bars + 8 + 8 * i; };
  auto p_full = [&](int i, int half) { return bars + 24 + 16 * i + 8 * half; };
  const uint32_t o_full = bars + 56;
  auto kv_full = [&](int i) { return bars + 64 + 8 * i; };
  auto kv_empty = [&](int i) { return bars + 96 + 8 * i; };
  auto meta_full = [&](int i) { return bars + 128 + 8 * i; };
  auto meta_empty = [&](int i) { return bars + 160 + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SH::BARS + 192);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::BARS + 196);
  if (tid == 0) {
    mbar_init(q_full, 4 * M);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i, 0), 4);
      mbar_init(p_full(i, 1), 4);
    }
    mbar_init(o_full, 1);
    for (int i = 0; i < kPreSlots; ++i) {
      mbar_init(kv_full(i), kPreConv);
      mbar_init(kv_empty(i), 1);
    }
    for (int i = 0; i < kPreMeta; ++i) {
      mbar_init(meta_full(i), 1);
      mbar_init(meta_empty(i), kPreConv + 4 * M);
    }
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
  const uint32_t tmem = *tmem_slot;  // S_0, S_1 (P_i over S_i), then O_0, O_1

  // ---------------- codes -> fp16 tiles ----------------
  // A converting warp's passes of 4 (D = 64: 8) rows: rows `first`, `first` + `stride`, ...  Warps 8-11 take
  // three quarters of a tile's rows, warps 14 and 15 the rest.
  constexpr int kWarpRows = 512 / D;
  auto convert = [&](auto passes, int first, int stride) {
    constexpr int PASSES = decltype(passes)::value;
    // Eight lanes write two rows of one 64-dimension panel: no bank conflicts.
    const int c4 = lane & 3;
    const int panel = D == 128 ? (lane >> 3) & 1 : 0;
    const int r0 = first + ((lane >> 2) & 1) + 2 * (D == 128 ? lane >> 4 : lane >> 3);
    const int code_off = panel * 64 + c4 * 16;
    const int items = 2 * N;  // K_0, V_0, K_1, V_1, ...
    uint4 x[PASSES];
    int grp[PASSES];  // 16-token groups of the pool that the thread's rows of the tile lie in
    auto groups = [&](int n) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        grp[p] = (int)lds32(base + SH::META + (n % kPreMeta) * 128 + ((r0 + p * stride) >> 4) * 16 + 12);
    };
    auto fetch = [&](int item, int p) {
      // Rows past the end read as zeros: stale codes may be NaN.
      const int r = r0 + p * stride;
      const uint8_t* src = (item & 1 ? V.v : V.k) + (size_t)(unsigned)max(grp[p], 0) * (16 * D) + (r & 15) * D + code_off;
      x[p] = ldg_or_zero(src, grp[p] >= 0 && j0 + (item >> 1) * kPreTile + r < j1);
    };
    bool alive = true;
    if (items) {
      alive = wait_bar(meta_full(0), 0, abort_flag, &s_err_kvb);
      if (__all_sync(0xffffffffu, alive)) {
        groups(0);
#pragma unroll
        for (int p = 0; p < PASSES; ++p) fetch(0, p);
      } else {
        alive = false;
      }
    }
    for (int item = 0; item < items && alive; ++item) {
      const int slot = item % kPreSlots;
      alive = wait_bar(kv_empty(slot), ((uint32_t)(item / kPreSlots) & 1u) ^ 1u, abort_flag, &s_err_kvb);
      const bool more = item + 1 < items;
      if (more && !((item + 1) & 1))
        alive = alive && wait_bar(meta_full(((item + 1) >> 1) % kPreMeta), (uint32_t)(((item + 1) >> 1) / kPreMeta) & 1u,
                                   abort_flag, &s_err_kvb);
      if (!__all_sync(0xffffffffu, alive)) {
        alive = false;
        break;
      }
      if (more && (item & 1)) groups((item + 1) >> 1);
      const uint32_t dst = base + SH::KV_OFF + slot * SH::TILE + panel * SH::PANEL;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = r0 + p * stride;
        uint32_t o[8];
        codes_half<FMT>(x[p].x, o[0], o[1]);
        codes_half<FMT>(x[p].y, o[2], o[3]);
        codes_half<FMT>(x[p].z, o[4], o[5]);
        codes_half<FMT>(x[p].w, o[6], o[7]);
        if (more) fetch(item + 1, p);
        const uint32_t at = dst + r * 128;
        sts128(at + (((2 * c4) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
        sts128(at + (((2 * c4 + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(kv_full(slot));
        // Tile n's groups were read into registers before K_n was fetched.
        if (!(item & 1)) mbar_arrive(meta_empty((item >> 1) % kPreMeta));
      }
    }
  };

  if (warp < 8) {
    // ---------------- softmax: one row per thread ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int i = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int row = row_base + i * kPreTile + r;
    const bool ok = row < rows;
    const int qi = ok ? row / P.G : 0;
    const size_t hr = (size_t)(s.row0 + qi) * P.Hq + h * P.G + (ok ? row - qi * P.G : 0);
    const int last = ok ? min(s.old + qi, s.len - 1) : -1;  // last visible token
    float mul = fabsf(P.scale_log2);
    if (i < M) {
      // The row's queries into shared memory, as fp16; bf16 rows times a power of two.  A negative
      // scale is taken into their sign.
      const uint32_t flip = P.scale_log2 < 0.f ? 0x80008000u : 0u;
      const uint16_t* q = P.Q + (s.row0 + qi) * P.q_stride + (long long)(h * P.G + (ok ? row - qi * P.G : 0)) * D;
      uint4 x[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        x[c] = ok ? *reinterpret_cast<const uint4*>(q + 8 * c) : make_uint4(0, 0, 0, 0);
      float up = 1.f;
      if (P.bf16) {
        float m = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t wd[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack(wd[k], true);
            m = max3(m, fabsf(f.x), fabsf(f.y));
          }
        }
        const int e2 = max((int)(__float_as_uint(m) >> 23) - 127, -100);
        up = __uint_as_float((uint32_t)(127 + min(14 - e2, 126)) << 23);
        mul *= __uint_as_float((uint32_t)(127 - min(14 - e2, 126)) << 23);
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint32_t wd[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        if (P.bf16)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack(wd[k], true);
            wd[k] = pack_half2(f.x * up, f.y * up);
          }
        sts128(base + SH::Q_OFF + i * SH::TILE + (c >> 3) * SH::PANEL + r * 128 + (((c & 7) ^ (r & 7)) << 4),
               wd[0] ^ flip, wd[1] ^ flip, wd[2] ^ flip, wd[3] ^ flip);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      float m = kPreNone, l = 0.f;
      const uint32_t ts = tmem + lanes + 128 * i, to = tmem + lanes + 256 + D * i;
      bool alive = true;
      for (int n = 0; n < N; ++n) {
        const int slot = n % kPreMeta;
        const uint32_t ph = (uint32_t)(n / kPreMeta) & 1u;
        alive = wait_bar(meta_full(slot), ph, abort_flag, &s_err_kvb) &&
                wait_bar(s_full(i), (uint32_t)n & 1u, abort_flag, &s_err_kvb);
        if (!__all_sync(0xffffffffu, alive)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t meta = base + SH::META + slot * 128;
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld_32x32b_x32(ts + 32 * c, v[c]);
        tc_wait_ld();
        const int rel = last - (j0 + n * kPreTile);  // columns 0 .. rel are visible
        const uint32_t holes = lds32(base + SH::HOLES + 4 * slot);
        if (!__all_sync(0xffffffffu, rel >= kPreTile - 1) || holes) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > rel || ((holes >> (c >> 4)) & 1u)) v[c >> 5][c & 31] = 0xff800000u;
        }
        float tm = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 mt = lds_f4(meta + 16 * g);
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
        if (__any_sync(0xffffffffu, tm > m + kPreSlack)) {
          const float mn = fmaxf(m, tm), f = ex2(m - mn);
          m = mn;
          l *= f;
          if (n > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc_ld_32x32b_x32(to + c, o);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tc_st_32x32b_x32(to + c, o);
            }
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int g = 4 * half + k;
            const float4 mt = lds_f4(meta + 16 * g);
            const float cg = fmaxf(mt.x * mul, 1e-35f), off = mt.y + kPreBias - m;
            const uint64_t cg2 = f32x2(cg, cg), off2 = f32x2(off, off);
            uint64_t sum = 0ull;
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const float2 e = f32x2_get(fma_f32x2(f32x2(__uint_as_float(v[g >> 1][16 * (g & 1) + c]),
                                                         __uint_as_float(v[g >> 1][16 * (g & 1) + c + 1])),
                                                   cg2, off2));
              const float p0 = ex2(e.x), p1 = ex2(e.y);
              sum = add_f32x2(sum, f32x2(p0, p1));
              p[8 * k + c / 2] = pack_half2(p0, p1);  // the codes' type in the product; l keeps all bits
            }
            const float2 part = f32x2_get(sum);
            l = fmaf(part.x + part.y, mt.z, l);
          }
          // The first half of the weights goes to the tensor cores while the second is computed.
          tc_st_32x32b_x32(ts + 32 * half, p);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(i, half));
        }
        if (lane == 0) mbar_arrive(meta_empty(slot));
      }
      // ---- the row's output, or its state for the joining launch
      if (N > 0 && alive) {
        alive = wait_bar(o_full, 0, abort_flag, &s_err_kvb);
        alive = __all_sync(0xffffffffu, alive);
        tc_fence_after();
      }
      if (alive) {
        const float inv = l > 0.f || l != l ? __fdividef(1.f, l) : 0.f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (N > 0) {
            tc_ld_32x32b_x32(to + c, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (!ok) continue;
          if (P.chunks == 1) {
            uint16_t* out = P.out + hr * D + c;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t wd[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float f0 = __uint_as_float(o[k + 2 * e]) * inv, f1 = __uint_as_float(o[k + 2 * e + 1]) * inv;
                wd[e] = P.bf16 ? pack_bf162(f0, f1) : pack_half2(f0, f1);
              }
              *reinterpret_cast<uint4*>(out + k) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
            }
          } else {
            float* dst = P.part + (hr * P.chunks + chunk) * D + c;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<uint4*>(dst + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        if (ok) {
          if (P.chunks > 1)
            P.part_ml[hr * P.chunks + chunk] = make_float2(m - kPreBias, l);
          else if (P.lse)
            P.lse[hr] = l == 0.f ? -INFINITY : (log2f(l) + m - kPreBias) * 0.693147180559945f;
        }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    convert(std::integral_constant<int, D == 128 ? 6 : 3>{}, (warp - 8) * kWarpRows, 4 * kWarpRows);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12) {
      // ---------------- MMA issuer ----------------
      // The whole warp walks the loop, so that descriptors and addresses stay uniform; one lane issues.
      if (N > 0) {
        constexpr uint32_t id_s = idesc_f16_f32(128, 128);
        constexpr uint32_t id_o = idesc_f16_f32(128, D) | (1u << 16);  // B is MN-major
        constexpr uint64_t kTileDesc = SH::TILE >> 4, kPanelDesc = SH::PANEL >> 4;
        const uint64_t dq = smem_desc_sw128(base + SH::Q_OFF), dk = smem_desc_sw128(base + SH::KV_OFF);
        const uint64_t dv = smem_desc_mn(base + SH::KV_OFF, SH::PANEL);
        const uint32_t lead = elect_one();
        const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);  // known to be uniform
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
          return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, &s_err_kvb)) != 0;
        };
        auto wait_kv = [&](int item) {
          return wait_all(kv_full(item % kPreSlots), (uint32_t)(item / kPreSlots) & 1u);
        };
        auto scores = [&](int i, int n) {
          const uint64_t da = dq + i * kTileDesc, db = dk + (uint64_t)((2 * n) % kPreSlots) * kTileDesc;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (k >> 2) * kPanelDesc + (k & 3) * 2;
            mma_ss_if(lead, tm0 + 128 * i, da + off, db + off, id_s, k > 0);
          }
          commit_if(lead, s_full(i));
        };
        bool alive = wait_all(q_full, 0) && wait_kv(0);
        if (alive) {
          tc_fence_after();
          for (int i = 0; i < M; ++i) scores(i, 0);
          commit_if(lead, kv_empty(0));
        }
        for (int n = 0; n < N && alive; ++n) {
          alive = wait_kv(2 * n + 1);
          const uint64_t db = dv + (uint64_t)((2 * n + 1) % kPreSlots) * kTileDesc;
          for (int i = 0; i < M && alive; ++i) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              alive = alive && wait_all(p_full(i, half), (uint32_t)n & 1u);
              if (!alive) break;
              tc_fence_after();
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                mma_ts_if(lead, tm0 + 256 + D * i, tm0 + 128 * i + 8 * k, db + (uint64_t)((k * 16 * 128) >> 4), id_o,
                          n > 0 || k > 0);
            }
            if (!alive) break;
            if (n + 1 < N) {
              if (i == 0) alive = wait_kv(2 * n + 2);
              if (!alive) break;
              tc_fence_after();
              scores(i, n + 1);
            }
          }
          if (!alive) break;
          commit_if(lead, kv_empty((2 * n + 1) % kPreSlots));
          if (n + 1 < N) commit_if(lead, kv_empty((2 * n + 2) % kPreSlots));
        }
        commit_if(lead, o_full);
        if (lead) {
          // Nothing is left in flight when tensor memory is freed, on an abort either.
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(o_full, 0)) {
            if (globaltimer() - t0 > kWaitLimitNs) {
              atomicOr(&s_err_kvb, kErrTimeout);
              break;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp >= 14) {
      convert(std::integral_constant<int, D == 128 ? 4 : 2>{}, 96 + (warp - 14) * kWarpRows, 2 * kWarpRows);
    } else if (warp == 13) {
      // ---------------- pages and scales ----------------
      for (int n = 0; n < N; ++n) {
        const int slot = n % kPreMeta;
        const bool alive =
            wait_bar(meta_empty(slot), ((uint32_t)(n / kPreMeta) & 1u) ^ 1u, abort_flag, &s_err_kvb);
        if (!__all_sync(0xffffffffu, alive)) break;
        const int j = j0 + n * kPreTile + 16 * lane;
        bool hole = false;
        if (lane < 8) {
          const int page = j < j1 ? page_of(V, V.table, b, V.table_stride, j >> V.t_shift) : -1;
          hole = j < j1 && page < 0;
          float ks = 1.f, vs = 1.f;
          uint32_t group = 0xffffffffu;
          if (page >= 0) {
            const size_t cell = (size_t)page * V.Hkv + h;
            group = (uint32_t)(((cell << V.t_shift) + (j & ((1 << V.t_shift) - 1))) >> 4);
            ks = V.ks[cell];
            vs = fmaxf(V.vs[cell], kScaleFloor);
          }
          const float lv = __log2f(vs);
          sts128(base + SH::META + slot * 128 + lane * 16, __float_as_uint(ks), __float_as_uint(lv),
                 __float_as_uint(ex2(-lv)), group);
        }
        const uint32_t holes = __ballot_sync(0xffffffffu, hole);
        if (lane == 0)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + SH::HOLES + 4 * slot), "r"(holes) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(meta_full(slot));
        __syncwarp();
      }
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int D>
static tm_status launch(const AttnParams& P, int pairs, cudaStream_t stream) {
  using SH = PreShape<D>;
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(done, reinterpret_cast<const void*>(prefill_kernel<FMT, D>), SH::SMEM)) return TM_ERR_CUDA;
  const dim3 grid((unsigned)(P.V.B * P.V.Hkv), (unsigned)(pairs * P.chunks));
  prefill_kernel<FMT, D><<<grid, kPreThreads, SH::SMEM, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? TM_OK : TM_ERR_CUDA;
}

tm_status launch_prefill_attn(const AttnParams& P, int format, int D, int pairs, cudaStream_t stream) {
  if (format == TM_KVB_INT8)
    return D == 64 ? launch<TM_KVB_INT8, 64>(P, pairs, stream) : launch<TM_KVB_INT8, 128>(P, pairs, stream);
  return D == 64 ? launch<TM_KVB_E4M3, 64>(P, pairs, stream) : launch<TM_KVB_E4M3, 128>(P, pairs, stream);
}

}  // namespace kvb

cudaError_t kvb_error_bits(uint32_t* bits, bool clear) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, kvb::s_err_kvb, sizeof(v));
  if (e != cudaSuccess) return e;
  if (clear && v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(kvb::s_err_kvb, &zero, sizeof(zero));
  }
  *bits = v;
  return e;
}

}  // namespace w4
