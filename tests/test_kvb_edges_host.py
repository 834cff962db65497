"""Paged 8-bit KV cache: the edges of its calls that need no GPU (made-up device
addresses: nothing is read through them)."""
import contextlib
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from tests.conftest import ROOT
from tests.test_kvb_host import A, ALIGN, INVALID, OK, UNSUP, batch, cache


@pytest.fixture(scope="module")
def lib():
    from w4a16_quantized_gemm_gb300 import binding, build
    build.build()
    return binding.load()


def attention(lib, c, b, Q=A, qs=1024, Hq=8, out=A, wi=None, wo=None, ws=0, work=None, size=0, scale=0.0):
    return lib.tm_kvb_attention(c, b, Q, qs, Hq, 0, scale, out, None, wi, wo, ws, work, size, None)


@pytest.mark.parametrize("none", [dict(q_start=A, rows=0), dict(q_start=A, max_q=0)])
def test_weights_of_a_step_without_rows_are_checked(lib, none):
    """w_out is written in such a step too, so its size and alignment count."""
    b = batch(**none)
    assert attention(lib, cache(), b, Q=None, out=None, wo=A, ws=255) == INVALID  # 256 tokens may be there
    assert attention(lib, cache(), b, Q=None, out=None, wo=A + 2, ws=256) == ALIGN
    assert attention(lib, cache(), b, Q=None, out=None, wi=A + 2, wo=A, ws=256) == ALIGN
    assert attention(lib, cache(), b, Q=None, out=None, wo=A, ws=65536 * 128) == UNSUP
    assert attention(lib, cache(), b, Q=None, out=None, wi=A, wo=A, ws=256) == OK  # in place: nothing to do
    assert attention(lib, cache(), b, Q=None, out=None) == OK


def test_memory_made_for_a_call_is_its_streams(monkeypatch):
    """binding._empty allocates with the given stream current, and records the caller's own."""
    from w4a16_quantized_gemm_gb300 import binding
    log = []

    @contextlib.contextmanager
    def stream(s):
        log.append(("enter", s))
        yield
        log.append(("leave", s))

    class Made:
        device = "dev"

        def record_stream(self, s):
            log.append(("record", s))

    def empty(*a, **k):
        log.append("empty")
        return Made()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: ("current", d))
    monkeypatch.setattr(torch, "empty", empty)
    assert isinstance(binding._empty(3, torch.uint8, "dev", "side"), Made)
    assert log == [("enter", "side"), "empty", ("leave", "side"), ("record", ("current", "dev"))]
    log.clear()
    binding._empty(3, torch.uint8, "dev", None)
    assert log == ["empty"]


def test_a_warp_that_gives_up_waits_for_its_copies(tmp_path):
    """The few-row kernel's ring: a warp that leaves its loop drains each copy in flight on that copy's own phase."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "ring")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "w4a16_quantized_gemm_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "kvb_ring_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert [int(n) for n in r.stdout.split()] == [sum(k + 1 for k in range(5 * S + 2)) for S in (2, 3, 4)]


def test_calls_with_other_rows_share_no_struct():
    """One batch in two threads, a workspace query beside a launch: each call sees its own number of rows."""
    from w4a16_quantized_gemm_gb300 import binding
    b = binding.KVBatch.__new__(binding.KVBatch)  # without device tensors
    b.q_start, b.B, b._c = object(), 3, batch(q_start=A)
    b._ref = ctypes.byref(b._c)
    refs = {n: b._rows(n) for n in (7, 3, 12, 7)}
    assert {n: r._obj.rows for n, r in refs.items()} == {7: 7, 3: 3, 12: 12}
    assert all(r._obj.q_start == A and r._obj.table_stride == 4 for r in refs.values())
    b.q_start = None
    assert b._rows(3)._obj.rows == 3
    with pytest.raises(ValueError):
        b._rows(4)


def test_grids_that_no_launch_takes_are_refused(lib):
    """33 to 64 rows a head with weights: two groups of 32 rows, 80000 along the grid's y for 40000 heads."""
    n, size = ctypes.c_size_t(7), lambda c, b, Hq, w: lib.tm_kvb_attention_workspace(c, b, Hq, w, ctypes.byref(n))
    c, b, Hq = cache(Hkv=40000), batch(q_start=A, max_q=40, rows=120), 40000
    assert size(c, b, Hq, 1) == UNSUP and size(c, b, Hq, 0) == OK
    big = dict(qs=Hq * 128, Hq=Hq, wo=A, ws=256, work=A, size=1 << 62)
    assert attention(lib, c, b, **big) == UNSUP


def test_scales_of_the_scores(lib):
    """NaN and infinities are refused, and so is what would quietly become 0, the default."""
    from w4a16_quantized_gemm_gb300 import binding
    none = batch(q_start=A, rows=0)
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert attention(lib, cache(), none, scale=bad) == INVALID
    assert attention(lib, cache(), none, scale=-0.5) == OK and attention(lib, cache(), none) == OK
    for tiny in (1e-60, -1e-60):
        with pytest.raises(ValueError, match="scale"):
            binding.kvb_attention(None, None, None, scale=tiny)
