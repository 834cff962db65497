"""The paged cache as a program uses it: prompt chunks, decode and eviction together
(examples/kv_budget_decode.py), against the same stack in plain binary32."""
import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _module():
    spec = importlib.util.spec_from_file_location("kv_budget_decode",
                                                  os.path.join(ROOT, "examples", "kv_budget_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(stack, tokens):
    """All tokens [B][n][hidden] through the stack at once, binary32, nothing quantised but the weights."""
    x = tokens.float()
    for layer in stack.layers:
        B, n, _ = x.shape
        h = (x * torch.rsqrt(x.square().mean(2, keepdim=True) + 1e-6)) @ layer.qkv_plain
        h = h.view(B, n, -1, layer.D).transpose(1, 2)
        G = layer.Hq // layer.Hkv
        q = h[:, :layer.Hq]
        k = h[:, layer.Hq:layer.Hq + layer.Hkv].repeat_interleave(G, 1)
        v = h[:, layer.Hq + layer.Hkv:].repeat_interleave(G, 1)
        s = (q @ k.transpose(2, 3)) / layer.D ** 0.5
        s = s.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool, device="cuda"), 1), -float("inf"))
        x = x + (s.softmax(3) @ v).transpose(1, 2).reshape(B, n, -1) @ layer.o_plain
    return x


@pytest.mark.parametrize("fmt,tol", [(torch.int8, 0.02), (torch.float8_e4m3fn, 0.06)])
def test_prompt_and_decode_without_eviction(fmt, tol):
    """Keys and values are off by half a code: int8 1/254 of a page's maximum (about
    4 sigma: 1.6 % of sigma at most, a uniform error of 0.9 % rms), e4m3 2^-4 at most, 2.6 % rms;
    the attention's branch is part of the sum with the residual, and errors of independent tokens average
    out.  Twice the rms bounds the relative distance of the outputs."""
    m = _module()
    stack = m.Stack(budget=160, slack=96, fmt=fmt)
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(stack.B, 203, 1024, generator=gen, device="cuda").half()
    got = [stack.prompt(x[:, :150])]
    for t in range(150, 203):
        got.append(stack.step(x[:, t].contiguous(), 1)[:, None])
    assert stack.evictions == 0
    got, want = torch.cat(got, 1).float(), _plain(stack, x)
    assert ((got - want).norm() / want.norm()).item() < tol
    # every row of a softmax adds up to one: the weights drawn are the rows that were computed
    for layer in stack.layers:
        rows = 203 * layer.Hq // layer.Hkv
        assert torch.allclose(layer.weights.sum(2), torch.full_like(layer.weights[:, :, 0], rows), rtol=1e-4)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_a_bounded_cache_goes_on(fmt):
    """Far more tokens than the cache holds: lengths stay bounded, nothing but the pages' own place is used,
    and the result stays near the unbounded one (the recent tokens and the heavy ones are kept)."""
    m = _module()
    stack = m.Stack(budget=96, slack=32, fmt=fmt)
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(stack.B, 300, 1024, generator=gen, device="cuda").half()
    out = [stack.prompt(x[:, :200])]
    for t in range(200, 300):
        out.append(stack.decode(x[:, t]).clone()[:, None])  # a replayed graph
        assert stack.held[0] <= stack.capacity and stack.kv_len.max().item() == stack.held[0]
    got, want = torch.cat(out, 1).float(), _plain(stack, x)
    assert stack.evictions > 2 and torch.isfinite(got).all()
    cos = torch.nn.functional.cosine_similarity(got.flatten(1), want.flatten(1))
    assert cos.min().item() > 0.9
