"""Tree attention whose sequences pass the host's bounds: more new tokens than max_q, more tokens than max_len.  Rows
past max_q are not computed, new tokens past the mask's ceil(max_q / 32) words are not seen, lengths end at max_len, in
every kernel alike; against binary64 within bounds counted from the number formats."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import DT, Cache, bounds, device, normal, rounded
from tests.test_gpu_tree import starts
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def run(c, new, Hq, dtype, tag, max_q, max_len=0, weights=True):
    Hkv, D = c.pools[0][0].shape[1], c.pools[0][0].shape[3]
    q_start = starts(new)
    rows, words = int(q_start[-1]), -(-max_q // 32)
    # half of all bits, and every bit for a third of the rows: a word taken for another one shows
    mask = (normal(f"{tag}/mask", rows, words) * 2.0 ** 30).astype(np.int64).astype(np.int32)
    mask[::3] = -1
    held = device(np.concatenate([mask, np.full((rows, 1), -1, np.int32)], 1))  # a word behind them that does not count
    Q = rounded(normal(f"{tag}/q", rows, Hq, D) * 1.5, dtype)[0].cuda()
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=max_q, max_len=max_len)
    room = c.table.shape[1] * c.T
    w_in = np.abs(normal(f"{tag}/w", len(new), Hkv, room)).astype(np.float32)
    wi = device(w_in)
    wo = torch.full_like(wi, 7.0) if weights else None
    lse = torch.full((rows, Hq), 5.0, device="cuda")
    out = torch.full((rows, Hq, D), 5.0, dtype=DT[dtype], device="cuda")
    binding.kvb_attention_tree(blocks, batch, Q, held, out=out, lse=lse, w_in=wi if weights else None, w_out=wo)
    torch.cuda.synchronize()
    assert binding.device_error(clear=True) == 0 and c.same(blocks)
    (k, ks), (v, vs) = c.pools
    o, l, w, size, reach = ref.attention(Q.double().cpu().numpy(), k, v, ks, vs, c.table, c.kv_len, q_start, c.fmt, tree=mask,
                                         max_q=max_q, max_len=max_len or room)
    bo, bl, bw = bounds(o, l, w, size, reach, D, dtype)
    live = np.zeros(rows, dtype=bool)
    for b, n in enumerate(new):
        live[q_start[b]:q_start[b] + min(n, max_q)] = True
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (got[~live] == 5.0).all() and (gl[~live] == 5.0).all()
    assert np.all(np.abs(got - o)[live] <= bo[live])
    assert np.array_equal(np.isneginf(gl[live]), np.isneginf(l[live]))
    seen = live[:, None] & np.isfinite(l)
    assert np.all(np.abs(gl[seen] - l[seen]) <= bl[seen])
    if weights:
        want, tol = w_in.astype(np.float64), np.zeros(w_in.shape)
        m = min(room, w.shape[2])
        want[:, :, :m] += w[:, :, :m]
        tol[:, :, :m] = bw[:, :, :m]
        err = np.abs(wo.double().cpu().numpy() - want)
        assert np.all(err <= tol + 2.0 ** -23 * want), np.argwhere(err > tol + 2.0 ** -23 * want)[:4]


# Hq, Hkv, max_q, new, and the rows of a KV head: the kernel for few rows (8, 16, 32 a CTA), the tcgen05 kernels of one
# row tile and of pairs, weights by kept scores, by the pass of up to 512 rows and by that of more
ROWS = [(4, 2, 4, [40, 5, 70]), (4, 1, 4, [37, 33, 4]), (8, 2, 7, [40, 9, 33]), (4, 1, 10, [40, 75, 8]), (2, 2, 40, [80, 41, 100]),
        (8, 1, 40, [100, 65, 30]), (16, 1, 40, [100, 65, 30])]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("fmt,dtype,D,T", [("int8", "fp16", 128, 64), ("e4m3", "bf16", 64, 16)])
@pytest.mark.parametrize("Hq,Hkv,max_q,new", ROWS)
def test_more_new_tokens_than_max_q(Hq, Hkv, max_q, new, fmt, dtype, D, T, weights):
    tag = f"bounds/q/{fmt}/{Hq}/{Hkv}/{max_q}"
    run(Cache(tag, [new[0] + 230, new[1], new[2] + 51], Hkv, D, T, fmt), new, Hq, dtype, tag, max_q, weights=weights)


@pytest.mark.parametrize("fmt,dtype,D,T", [("int8", "bf16", 64, 32), ("e4m3", "fp16", 128, 128)])
@pytest.mark.parametrize("Hq,Hkv,max_q,new", ROWS)
def test_more_tokens_than_max_len(Hq, Hkv, max_q, new, fmt, dtype, D, T):
    """A bound among the new tokens of one sequence, before all those of another."""
    tag = f"bounds/len/{fmt}/{Hq}/{Hkv}/{max_q}"
    c = Cache(tag, [new[0] + 290, new[1] + 320, new[2] + 51], Hkv, D, T, fmt)
    run(c, new, Hq, dtype, tag, max_q, max_len=new[0] + 290 - max(new[0] - 20, 3))
    run(c, new, Hq, dtype, tag, max(new), max_len=290)
