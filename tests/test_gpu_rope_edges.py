"""Append with rotation: lengths at the end of 32 bits."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import Cache, device, normal, rounded
from tests.test_gpu_tree import angles, starts
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("T", [16, 128])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_slots_up_to_the_last_one(n, T):
    """The last slots that 32 bits count have no page, but their queries turn, by the table's end and by positions; a
    sequence beside them is as ever."""
    Hq, Hkv, D = 4, 2, 64
    c = Cache(f"rope/last/{T}", [n + 3, n + 50], Hkv, D, T, "int8")
    lens = np.array([2 ** 31 - 1, n + 50], np.int32)
    rows = 2 * n
    x, exact = rounded(normal(f"rope/last/x/{n}", rows, Hq + 2 * Hkv, D), "fp16")
    fused, table = x.cuda(), angles(100, D)
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(lens), device(starts([n, n])), max_q=n)
    slots = np.concatenate([np.full(n, 99), np.arange(50, n + 50)])  # the first sequence's: past the table, its end
    given = np.arange(rows)[::-1].astype(np.int32)
    for pos in (slots, given):
        q = binding.kvb_append_rope(blocks, batch, fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:], binding.Rope(device(table)),
                                    Q=fused[:, :Hq], pos=device(given) if pos is given else None)
        torch.cuda.synchronize()
        want = torch.from_numpy(ref.rotate(exact[:, :Hq], table, pos)).half()
        assert torch.equal(q.cpu(), want)
        turned = ref.rotate(exact[:, Hq:Hq + Hkv], table, pos)
        ref.append(*c.pools[0], c.table, lens, starts([n, n]), turned, "int8")
        ref.append(*c.pools[1], c.table, lens, starts([n, n]), exact[:, Hq + Hkv:], "int8")
        assert c.same(blocks)
