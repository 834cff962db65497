"""Accepted drafts: paths without an entry, lengths at the end of 32 bits."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
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


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 256, 2 ** 31 - 257])
def test_as_many_new_tokens_as_32_bits_count(n):
    """A length and a row start that no cache holds: tokens past the table's room have no page, those past the weights'
    stride no weight, and nothing outside is touched."""
    c = Cache("accept/long", [64, 40], 2, 64, 16, "e4m3", spread=1.0)
    blocks, w = c.to_device(binding), np.abs(normal("accept/long/w", 2, 2, 64)).astype(np.float32)
    batch = binding.KVBatch(device(c.table), device(np.array([n, 40], np.int32)), device(np.array([0, n, n], np.int32)), max_q=20)
    path = np.array([[2, 5, 17, 33, 63, n - 1], [0, 1, 2, 3, 4, 5]])
    wide = torch.full((3, 2, 2, 64), 7.0, device="cuda")
    wide[1] = device(w)
    got = binding.kvb_accept(blocks, batch, device(path.astype(np.int32)), device(np.array([5, 3], np.int32)), w=wide[1])
    torch.cuda.synchronize()
    # as if the first sequence had all of its room as new tokens, and the second none
    want = ref.accept(c.pools, c.table, c.kv_len, np.array([0, 64, 64]), path, np.array([5, 3]), w, "e4m3")
    assert got.tolist() == want.tolist() == [5, 40]
    assert c.same(blocks) and np.array_equal(wide[1].cpu().numpy(), w)
    assert (wide[0] == 7.0).all() and (wide[2] == 7.0).all()
