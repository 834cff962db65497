/*
 * tm_lora.h -- C ABI of low-rank adapters beside a shared projection (GB300, sm_103a).
 *
 * Many requests share one quantised projection (tm_w4a16_gemm, tm_w8a8_gemm)
 * and each adds the product of its own adapter, two thin fp16 matrices:
 *   out[m] = Y[m] + scale[a] (X[m] . A[a]^T) . B[a]^T,   a = the adapter of row m
 *
 * Conventions are those of tm_w4a16.h: device pointers of the current device,
 * nothing throws, no call allocates or synchronises, every call is
 * asynchronous on `stream` (a cudaStream_t; NULL = the legacy default stream)
 * and can be captured into a CUDA graph.  No index makes a kernel leave the
 * buffers that the call names.
 */
#ifndef TM_LORA_H
#define TM_LORA_H

#include "tm_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The adapters of one projection, all of one rank (pad lower ranks with zeros). */
typedef struct {
  const void* A;      /* device fp16 [n][R][K], contiguous, 16-byte aligned */
  const void* B;      /* device fp16 [n][N][R], contiguous, 16-byte aligned */
  const float* scale; /* device fp32 [n]; NULL: 1 */
  int n;              /* adapters, >= 0 */
  int K, N;           /* of the projection, multiples of 8, at most 2^30 */
  int R;              /* a multiple of 8, 8 .. 128 */
} tm_lora_adapters;

/*
 * X     : device fp16 [rows][K], row stride x_stride in elements
 * Y     : device fp16 [rows][N], the projection's output, row stride y_stride
 * out   : device fp16 [rows][N], row stride out_stride; may be Y (with its stride),
 *         else it overlaps neither X nor Y
 *         (all strides multiples of 8, all pointers 16-byte aligned: slices of a fused projection are fine)
 * ids   : device int32 [B]: the adapter of each sequence; outside 0 .. n-1: none, out = Y
 * q_start: device int32 [B + 1]: sequence b's rows are q_start[b] .. q_start[b+1]-1
 *         (clamped to 0 .. rows), as in tm_kvb_batch; NULL: one row each (B == rows).
 *         Rows of no sequence are left as they are in out; of a row that
 *         several claim the last one's adapter counts.
 * The products accumulate in fp32.  X . A^T is rounded once to fp16 relative to
 * its row's largest element (11 bits; elements below 2^-29 of it lose bits), the
 * result once to fp16 from the fp32 sum.  The same inputs give the same bits.
 * K or N past 2^30, 2^31 - 256 rows and more: TM_ERR_UNSUPPORTED.
 * One launch, no workspace.  B, rows == 0 is a no-op.
 */
tm_status tm_lora_add(const tm_lora_adapters* adapters, const void* X, long long x_stride, const void* Y,
                      long long y_stride, void* out, long long out_stride, long long rows, const int* ids,
                      const int* q_start, int B, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TM_LORA_H */
