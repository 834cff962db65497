"""Adapters, rotated append, tree attention and accepted paths as a program uses them together
(examples/tree_decode.py), against the same stack in plain binary32."""
import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _module():
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(stack, b, tokens):
    """One sequence's tokens through the stack at once, binary32, nothing quantised but the weights."""
    x = stack.embed[tokens].float()
    n = x.shape[0]
    cs = stack.rope.table[:n, None]
    for layer in stack.layers:
        def project(y, plain, lora):
            a = int(stack.ids[b])
            out = y @ plain
            return out + (y @ lora.A[a].float().T) @ lora.B[a].float().T if a >= 0 else out

        def turn(v):
            half = layer.D // 2
            c, s = cs[..., :half], cs[..., half:]
            return torch.cat([v[..., :half] * c - v[..., half:] * s, v[..., half:] * c + v[..., :half] * s], 2)

        h = project(x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6), layer.qkv_plain, layer.qkv_lora).view(n, -1, layer.D)
        G = layer.Hq // layer.Hkv
        q = turn(h[:, :layer.Hq]).transpose(0, 1)
        k = turn(h[:, layer.Hq:layer.Hq + layer.Hkv]).repeat_interleave(G, 1).transpose(0, 1)
        v = h[:, layer.Hq + layer.Hkv:].repeat_interleave(G, 1).transpose(0, 1)
        s = (q @ k.transpose(1, 2)) / layer.D ** 0.5
        s = s.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool, device="cuda"), 1), -float("inf"))
        x = x + project((s.softmax(2) @ v).transpose(0, 1).reshape(n, -1), layer.o_plain, layer.o_lora)
    return x


@pytest.mark.parametrize("fmt,tol", [(torch.int8, 0.02), (torch.float8_e4m3fn, 0.06)])
def test_accepted_paths_are_the_sequences_own(fmt, tol):
    """What the kept nodes gave equals what their sequence gives read from front to back.  Keys and values are off by
    half a code: int8 1/254 of a page's maximum (about 4 sigma: 0.9 % of sigma rms), e4m3 2.6 % rms; the attention's branch
    is part of the sum with the residual.  Twice the rms bounds the relative distance."""
    m = _module()
    stack = m.Stack(room=400, fmt=fmt, vocab=12)  # few tokens: guesses come true
    gen = torch.Generator("cuda").manual_seed(3)
    prompt = torch.randint(0, stack.vocab, (stack.B, 150), generator=gen, device="cuda")
    first = stack.prompt(prompt)
    tokens = [list(prompt[b]) for b in range(stack.B)]
    hidden = [list(first[b]) for b in range(stack.B)]
    most = 0
    for _ in range(20):
        t, kept, x = stack.step()
        for b in range(stack.B):
            at = kept[b].nonzero().flatten().tolist()
            assert at[0] == 0 and all(m.PARENTS[i] in at for i in at[1:])
            most = max(most, len(at))
            tokens[b] += list(t[b, at])
            hidden[b] += list(x[b, at].clone())
    assert stack.kv_len.tolist() == [len(v) for v in tokens] and most > 1
    for b in range(stack.B):
        want = _plain(stack, b, torch.stack(tokens[b]))
        got = torch.stack(hidden[b]).float()
        assert ((got - want).norm() / want.norm()).item() < tol


def test_main_runs(capsys, monkeypatch):
    m = _module()
    monkeypatch.setattr("sys.argv", ["tree_decode.py", "--prompt", "70", "--steps", "5", "--batch", "3"])
    m.main()
    assert "tokens per step" in capsys.readouterr().out
