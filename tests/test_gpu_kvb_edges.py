"""Paged 8-bit KV cache on the GPU: steps without rows, streams, guards around every
buffer, long slices, shared selections (tests/test_gpu_kvb.py has the operators themselves)."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import Cache, device, normal, rounded
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


def _owner(t):
    """Handle of the stream whose memory t lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"])


def test_memory_of_calls_on_another_stream(monkeypatch):
    """What a call on a given stream allocates is that stream's: blocks that the current stream gave back are
    still written there by pending work."""
    c = Cache("kvb/side", [900, 411], 2, 128, 64, "int8")
    blocks, batch = c.to_device(binding), binding.KVBatch(device(c.table), device(c.kv_len))
    Q = rounded(normal("kvb/side/q", 2, 8, 128), "fp16")[0].cuda()
    w = device(np.abs(normal("kvb/side/w", 2, 2, c.table.shape[1] * 64)).astype(np.float32))
    w_want, w_got, w_evict = torch.empty_like(w), torch.empty_like(w), torch.empty(2, 2, 100, device="cuda")
    want = binding.kvb_attention(blocks, batch, Q, w_in=w, w_out=w_want)
    fresh, kept_want = c.to_device(binding), ref.evict(c.pools, c.table, c.table, c.kv_len, w.cpu().numpy(), 100, 4, 9,
                                                       "int8")[0]
    side, made, plain = torch.cuda.Stream(), [], torch.empty
    size = binding.kvb_attention_workspace(blocks, batch, 8, 2, True)
    a = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    given_back = [torch.empty_like(want), torch.empty(size, dtype=torch.uint8, device="cuda"),
                  torch.empty(2, 2, 100, dtype=torch.int32, device="cuda"),
                  torch.empty(2, dtype=torch.int32, device="cuda")]
    for _ in range(20):
        a = a @ a * 0.01
    for t in given_back:
        t.fill_(1)  # pending behind the products
    given_back.clear()
    del t
    monkeypatch.setattr(torch, "empty", lambda *x, **k: made.append(plain(*x, **k)) or made[-1])
    out = binding.kvb_attention(blocks, batch, Q, w_in=w, w_out=w_got, stream=side)
    kept, new_len = binding.kvb_evict(fresh, batch, w, 100, first=4, recent=9, dst_table=batch.table, w_out=w_evict,
                                      stream=side)
    monkeypatch.undo()
    assert len(made) == 4 and [_owner(t) for t in made] == [side.cuda_stream] * 4
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(w_got, w_want)
    assert np.array_equal(kept.cpu().numpy(), kept_want) and new_len.tolist() == [100, 100]
    assert c.same(fresh)
