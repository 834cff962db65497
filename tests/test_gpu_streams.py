"""Calls on a stream that is not the current one: what the binding allocates for them is that stream's
memory (a block that the current stream gave back may still be written by work pending there), and the
results are those of the current stream."""
import pytest
import torch

from tests.gpu_util import activations, packed
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

M, K, N, G = 5, 512, 256, 128


def _owner(t):
    """Handle of the stream whose memory t lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"])


def _calls():
    gen = torch.Generator("cuda").manual_seed(3)
    w = packed(K, N, G)
    X = torch.from_numpy(activations(M, K, N, G)).cuda()
    wide = torch.cat([X, X], 1)[:, :K]  # rows with a stride: copied first
    W = torch.randn(K, N, generator=gen, device="cuda").half()
    wide_W = torch.cat([W, W], 1)[:, :N]
    heads = torch.randn(1, 2, 256, 128, generator=gen, device="cuda").half()
    codes, ks, kz = binding.kv_quantize(heads, 8)
    tiles = binding.kv_pack_v(codes, 8)
    Q = torch.randn(1, 8, 128, generator=gen, device="cuda").half()
    length = torch.tensor([200], dtype=torch.int32, device="cuda")
    xq, sx = binding.w8a8_quantize_act(X)
    xq16, sx16 = binding.w8a8_quantize_act_f16(X)
    w8 = binding.pack_w8(*binding.w8_quantize_weight(W))
    return [
        ("gemm", 1, lambda st: binding.gemm(X, w, stream=st)),
        ("gemm_copy", 1, lambda st: binding.gemm(wide, w, stream=st)),
        ("gemm_silu_mul", 1, lambda st: binding.gemm_silu_mul(wide, w, stream=st)),
        ("gemm_grouped", 2, lambda st: binding.gemm_grouped([(X, w, None, False), (wide, w, None, True)], stream=st)),
        ("gemm_host", 3, lambda st: binding.gemm_host(X.cpu(), w, stream=st)),  # out, on the host, and two buffers
        ("quantize_rtn", 3, lambda st: binding.quantize_rtn(wide_W, G, stream=st)),
        ("kv_quantize", 3, lambda st: binding.kv_quantize(heads, 8, stream=st)),
        ("kv_pack_v", 1, lambda st: binding.kv_pack_v(codes, 8, stream=st)),
        ("kv_decode_attention", 1, lambda st: binding.kv_decode_attention(Q, (codes, ks, kz), (tiles, ks, kz), length,
                                                                         8, stream=st)),
        ("w8a8_quantize_act", 2, lambda st: binding.w8a8_quantize_act(X, stream=st)),
        ("w8a8_quantize_act_f16", 2, lambda st: binding.w8a8_quantize_act_f16(X, stream=st)),
        ("w8_quantize_weight", 2, lambda st: binding.w8_quantize_weight(W, stream=st)),
        ("w8a8_gemm", 1, lambda st: binding.w8a8_gemm(xq, sx, w8, stream=st)),
        ("w8a8_gemm_f16", 1, lambda st: binding.w8a8_gemm_f16(xq16, sx16, w8, stream=st)),
    ]


def test_memory_and_results_on_another_stream(monkeypatch):
    side, plain = torch.cuda.Stream(), torch.empty
    flat = lambda r: [r] if isinstance(r, torch.Tensor) else list(r)  # noqa: E731
    for name, n, call in _calls():
        want = flat(call(None))
        torch.cuda.synchronize()
        made = []
        with monkeypatch.context() as patch:
            patch.setattr(torch, "empty", lambda *a, **k: made.append(plain(*a, **k)) or made[-1])
            side.wait_stream(torch.cuda.current_stream())
            got = flat(call(side))
        torch.cuda.synchronize()
        assert len(made) == n, name
        assert all(_owner(t) == side.cuda_stream for t in made if t.is_cuda), name
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want), name
    assert binding.device_error(clear=True) == 0
