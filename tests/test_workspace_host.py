"""Workspace of the paged cache's attention, from the host fields alone: what each of the two calls asks for."""
import ctypes

import pytest

from tests.test_kvb_host import batch, cache

OK = 0
A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from w4a16_quantized_gemm_gb300 import binding, build
    build.build()
    return binding.load()


def query(lib, tree, Hq, Hkv, D, B, max_q, room, weights=0, rows=None, max_len=0):
    n = ctypes.c_size_t(7)
    b = batch(B=B, q_start=A, rows=B * max_q if rows is None else rows, max_q=max_q, max_len=max_len, table=None, kv_len=None,
              table_stride=room // 64)
    call = lib.tm_kvb_attention_tree_workspace if tree else lib.tm_kvb_attention_workspace
    assert call(cache(T=64, Hkv=Hkv, D=D, k=None, v=None, ks=None, vs=None), b, Hq, weights, ctypes.byref(n)) == OK
    return n.value


@pytest.mark.parametrize("B,max_q,room", [(1, 2048, 32768), (1, 2048, 131072), (4, 512, 32768), (2, 2048, 32768),
                                          (1, 1280, 131072), (1, 4096, 131072), (32, 77, 4096)])
def test_prompts_that_fill_the_gpu_ask_for_nothing(lib, B, max_q, room):
    """160 and more CTAs of 256 rows (32 query and 8 KV heads): the causal call has no slices, and no partial results."""
    assert query(lib, False, 32, 8, 128, B, max_q, room) == 0
    rows = B * max_q * 32
    assert query(lib, False, 32, 8, 128, B, max_q, room, weights=1) == -(-4 * rows // 256) * 256  # the rows' lse


def test_slices_of_a_chunk(lib):
    """512 new tokens over 131072, 64 CTAs: five slices of the causal call, fp32 partial results and two numbers a row."""
    rows = 512 * 32
    assert query(lib, False, 32, 8, 128, 1, 512, 131072) == 5 * rows * (128 + 2) * 4


@pytest.mark.parametrize("weights", [0, 1])
@pytest.mark.parametrize("Hkv,G,D", [(1, 1, 64), (8, 4, 128), (2, 7, 128), (12, 1, 64)])
def test_a_causal_workspace_holds_one_slice_of_a_tree(lib, Hkv, G, D, weights):
    """A room of 512 tokens or fewer is one slice whatever the rows are: never more for the tree than for the causal call."""
    for max_q in (1, 2, 5, 8, 9, 16, 17, 32, 33, 40, 64, 65, 128, 129, 600):
        for room in (64, 128, 512):
            for B in (1, 40):
                one = query(lib, True, Hkv * G, Hkv, D, B, max_q, room, weights)
                if max_q * G > 16:  # fewer rows take the same kernel, with shorter slices
                    assert one <= query(lib, False, Hkv * G, Hkv, D, B, max_q, room, weights)
                else:
                    assert one == query(lib, False, Hkv * G, Hkv, D, B, max_q, room, weights)


def test_slices_of_large_trees_fit_their_grid(lib):
    """A tree's CTAs stand side by side along one axis of the grid, groups of 256 rows times slices: at most 65535."""
    G, D, room = 8, 64, 1 << 24
    most = 0
    for groups in list(range(200, 15600, 97)) + [1023, 1024, 4095, 4096, 7000, 13107, 15625]:
        max_q = groups * 256 // G
        n = query(lib, True, G, 1, D, 1, max_q, room, rows=1)  # one row: the partial results of a slice are G (D + 2) numbers
        slices = max(n // (G * (D + 2) * 4), 1)
        most = max(most, groups * slices)
    assert most <= 65535
