"""Tree attention in workspaces of other sizes than its own: fewer slices, the same results within the bounds."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import Cache, bounds, device, normal, rounded
from tests.test_gpu_tree import random_trees, starts
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("B,Hq,new", [(1, 8, 3), (1, 8, 5), (1, 8, 20), (20, 16, 10), (20, 16, 33), (3, 8, 150)])
def test_smaller_workspaces(B, Hq, new, weights):
    """The tree's own workspace, the causal call's, and what holds two slices."""
    Hkv, D = 8 if B == 20 else 2, 64
    lens = [4000 if B == 20 else 2300] + [new + 40 + 7 * b for b in range(B - 1)]
    c = Cache(f"work/{B}/{new}", lens, Hkv, D, 64, "int8")
    q_start = starts([new] * B)
    rows = int(q_start[-1])
    mask = binding.tree_masks(random_trees(f"work/{new}", [new] * B))
    Q = rounded(normal(f"work/q/{new}", rows, Hq, D), "fp16")[0].cuda()
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=new)
    own = binding.kvb_attention_tree_workspace(blocks, batch, Hq, rows, weights)
    causal = binding.kvb_attention_workspace(blocks, batch, Hq, rows, weights)
    if (B, new, weights) == (20, 33, False):  # 160 CTAs of 66 rows
        assert causal == 0 < own
    (k, ks), (v, vs) = c.pools
    o, l, w, size, reach = ref.attention(Q.double().cpu().numpy(), k, v, ks, vs, c.table, c.kv_len, q_start, "int8",
                                         tree=mask.numpy())
    bo, bl, bw = bounds(o, l, w, size, reach, D, "fp16")
    for n in sorted({own, min(own, causal), causal + 2 * rows * Hq * (D + 2) * 4 + 1024}):
        guard = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
        wo = torch.zeros(B, Hkv, c.table.shape[1] * 64, device="cuda") if weights else None
        lse = torch.empty(rows, Hq, device="cuda")
        out = binding.kvb_attention_tree(blocks, batch, Q, mask.cuda(), lse=lse, w_out=wo, workspace=guard[:n])
        torch.cuda.synchronize()
        assert binding.device_error(clear=True) == 0 and (guard[n:] == 77).all()
        assert np.all(np.abs(out.double().cpu().numpy() - o) <= bo)
        assert np.all(np.abs(lse.double().cpu().numpy() - l) <= bl)
        if weights:
            got = wo.double().cpu().numpy()
            assert np.all(np.abs(got[:, :, :w.shape[2]] - w) <= bw) and not got[:, :, w.shape[2]:].any()
    if weights:  # no room for the weights' parts
        with pytest.raises(binding.TMError):
            binding.kvb_attention_tree(blocks, batch, Q, mask.cuda(), w_out=wo, workspace=guard[:64])
