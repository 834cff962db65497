"""Paged 8-bit KV cache on the GPU: steps without rows, streams, guards around every
buffer, long slices, shared selections (tests/test_gpu_kvb.py has the operators themselves)."""
import numpy as np
import pytest
import torch

from tests.kvb_util import Cache, device, normal
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("given", ["apart", "in place", "none"])
def test_weights_of_a_step_without_rows(given):
    """No row draws weight: w_out = w_in, over the whole stride."""
    c = Cache("kvb/norows", [70, 0, 33], 2, 64, 32, "int8")
    batch = binding.KVBatch(device(c.table), device(c.kv_len), torch.zeros(4, dtype=torch.int32, device="cuda"), max_q=4)
    Q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    w_in = device(np.abs(normal("kvb/norows/w", 3, 2, c.table.shape[1] * 32 + 5)).astype(np.float32))
    want = torch.zeros_like(w_in) if given == "none" else w_in.clone()
    w_out = w_in if given == "in place" else torch.full_like(w_in, float("nan"))
    out = binding.kvb_attention(c.to_device(binding), batch, Q, w_in=None if given == "none" else w_in, w_out=w_out)
    torch.cuda.synchronize()
    assert out.shape == Q.shape and torch.equal(w_out, want)
    assert binding.device_error() == 0
