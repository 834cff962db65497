"""Small caches for the tests of the paged 8-bit KV cache: host copies for the
oracle, device copies for the kernels, and the error bounds."""
import numpy as np
import torch

import oracle.kvb as ref
from w4a16_quantized_gemm_gb300 import synth

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
TOP = {"fp16": 65504.0, "bf16": 3.3895313892515355e38}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def normal(tag, *shape):
    return synth.normal64(tag, 1, int(np.prod(shape))).reshape(shape)


def rounded(x, dtype):
    """binary64 x to the dtype, as a CPU tensor and as exact float32."""
    t = torch.from_numpy(np.asarray(x)).to(DT[dtype])
    return t, t.float().numpy()


def device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Cache:
    """Pages full of random tokens (stale slots included), scales of their own."""

    def __init__(self, tag, lens, Hkv, D, T, fmt, spare=2, spread=1.0):
        self.fmt, self.T = fmt, T
        held = [-(-max(n, 0) // T) for n in lens]
        pages = sum(held) + spare
        self.pools = []
        for name in "kv":
            x = normal(f"{tag}/{name}", pages, Hkv, T, D).astype(np.float32)
            x *= np.exp(spread * normal(f"{tag}/{name}s", pages, Hkv, 1, 1)).astype(np.float32)
            s = np.maximum(np.abs(x).max((2, 3)) / ref.QMAX[fmt], ref.FLOOR).astype(np.float32)
            self.pools.append((ref.encode(x / s[:, :, None, None], fmt), s))
        order = np.argsort(normal(f"{tag}/order", pages)).astype(np.int32)
        self.table = np.full((len(lens), max(held + [1])), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.kv_len = np.array(lens, dtype=np.int32)

    def to_device(self, binding):
        (k, ks), (v, vs) = self.pools
        code = lambda c: device(c.view(np.uint8)).view(CODE[self.fmt])  # noqa: E731
        return binding.KVBlocks(code(k), code(v), device(ks), device(vs))

    def same(self, blocks):
        """Whether the device pages equal the host's, to the bit."""
        (k, ks), (v, vs) = self.pools
        bits = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
        return (np.array_equal(bits(blocks.k), k.view(np.uint8)) and np.array_equal(bits(blocks.v), v.view(np.uint8))
                and np.array_equal(blocks.ks.cpu().numpy().view(np.uint32), ks.view(np.uint32))
                and np.array_equal(blocks.vs.cpu().numpy().view(np.uint32), vs.view(np.uint32)))


def bounds(out, lse, w, size, reach, D, dtype):
    """Largest errors of attention's results, from the number formats alone.

    Scores: D products summed in fp32, each addition off by at most 2^-23 of the sum of
    magnitudes (truncating adders), the scaling by a few 2^-24: es = (D + 4) 2^-23 reach,
    and a weight is off by 2 es of itself, its exponential by 2^-21 and the normalisation
    by the same.  Values: each weight once to fp16 (2^-11), or to its subnormals, which are
    2^-25 / 2^6 of the largest weight.  The result once to its type."""
    es = ((D + 4) * 2.0 ** -23 * reach)[..., None]
    half = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    fine = 2 * es + 2.0 ** -19
    b_out = (2.0 ** -11 + 2 * fine) * size + 2.0 ** -20 * size.max(initial=0.0) + half * np.abs(out) + 2.0 ** -25
    b_lse = es[..., 0] + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
    b_w = (2 * fine.max(initial=0.0) + 2.0 ** -21) * np.abs(w) + 2.0 ** -30
    return b_out, b_lse, b_w
