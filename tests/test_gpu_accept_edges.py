"""Accepted drafts: paths without an entry."""
import numpy as np
import pytest
import torch

from tests.kvb_util import Cache, device, normal
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def test_no_path_at_all():
    """A path [B][0]: nothing is kept, whatever the counts are; the weights of the new tokens are cleared."""
    c = Cache("accept/none", [60, 33, 7], 2, 64, 16, "int8")
    blocks, w = c.to_device(binding), np.abs(normal("accept/none/w", 3, 2, 64)).astype(np.float32)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(np.array([0, 20, 20, 27], np.int32)), max_q=20)
    wd = device(w)
    got = binding.kvb_accept(blocks, batch, torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                             device(np.array([4, 0, -1], np.int32)), w=wd)
    torch.cuda.synchronize()
    w[0, :, 40:60] = 0.0
    w[2, :, 0:7] = 0.0
    assert got.tolist() == [40, 33, 0] and c.same(blocks) and np.array_equal(wd.cpu().numpy(), w)
