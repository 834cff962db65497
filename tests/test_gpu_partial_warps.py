"""Attention on tensor memory where warps have rows of their own and rows of no one: 33 to 160 rows a KV head that end at
every place of a warp, alone and in several slices, causal and as trees (chains: the same mask, so the same results)."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import Cache, bounds, device, normal, rounded
from tests.test_gpu_tree import starts
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [33, 39, 47, 63, 64, 65, 95, 97, 127, 129, 159])
def test_rows_that_end_inside_a_warp(new, D):
    lens = [new + 3, 1400]
    c = Cache(f"partial/{new}", lens, 1, D, 64, "int8")
    n = [new, 1 + new % 32]  # a full and a nearly empty sequence
    q_start = starts(n)
    rows = int(q_start[-1])
    Q = rounded(normal(f"partial/q/{new}", rows, 1, D) * 1.5, "bf16")[0].cuda()
    chains = binding.tree_masks([list(range(-1, k - 1)) for k in n]).cuda()
    blocks = c.to_device(binding)
    (k, ks), (v, vs) = c.pools
    o, l, w, size, reach = ref.attention(Q.double().cpu().numpy(), k, v, ks, vs, c.table, c.kv_len, q_start, "int8")
    bo, bl, bw = bounds(o, l, w, size, reach, D, "bf16")
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=new)
    for call, more in ((binding.kvb_attention, ()), (binding.kvb_attention_tree, (chains,))):
        out, lse = torch.full((rows + 1, 1, D), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows + 1, 1), 5.0, device="cuda")
        wo = torch.empty(2, 1, c.table.shape[1] * 64, device="cuda")
        call(blocks, batch, Q, *more, out=out[:rows], lse=lse[:rows], w_out=wo)
        torch.cuda.synchronize()
        assert binding.device_error(clear=True) == 0 and (out[rows] == 5.0).all() and (lse[rows] == 5.0).all()
        assert np.all(np.abs(out[:rows].double().cpu().numpy() - o) <= bo)
        assert np.all(np.abs(lse[:rows].double().cpu().numpy() - l) <= bl)
        got = wo.double().cpu().numpy()
        assert np.all(np.abs(got[:, :, :w.shape[2]] - w) <= bw) and not got[:, :, w.shape[2]:].any()
