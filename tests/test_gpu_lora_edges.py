"""Adapters: what the formula gives for infinities, at every rank and in both kernels."""
import pytest
import torch

from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("rows", [1, 5, 40])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 48, 64, 72, 104, 128])
def test_an_infinity_is_an_infinity(R, rows):
    """Every product and sum of the formula is +inf where X has one and A and B are positive: no rank that the kernels
    fill up with has a say (0 inf is NaN).  Rows of one sequence each, and of one sequence."""
    K, N = 128, 72
    g = torch.Generator().manual_seed(R)
    A = (torch.rand(2, R, K, generator=g) + 0.5).half().cuda()
    B = (torch.rand(2, N, R, generator=g) + 0.5).half().cuda()
    X, Y = torch.ones(rows, K).half().cuda(), torch.ones(rows, N).half().cuda()
    X[rows // 2, 77] = float("inf")
    ad = binding.Adapters(A, B)
    for ids, q_start in ((torch.ones(rows), None), (torch.ones(1), torch.tensor([0, rows], dtype=torch.int32).cuda())):
        got = binding.lora_add(Y, X, ad, ids.int().cuda(), q_start=q_start, out=torch.empty_like(Y))
        clean = torch.arange(rows, device="cuda") != rows // 2
        assert (got[rows // 2] == float("inf")).all()
        assert torch.isfinite(got[clean]).all()
