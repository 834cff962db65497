"""Adapters whose sizes pass what the kernels count in 32 bits: refused before any launch (made-up device addresses)."""
import pytest

from tests.test_tree_host import A, UNSUP, adapters


@pytest.fixture(scope="module")
def lib():
    from w4a16_quantized_gemm_gb300 import binding, build
    build.build()
    return binding.load()


@pytest.mark.parametrize("change", [dict(K=2 ** 30 + 8), dict(N=2 ** 30 + 8), dict(K=2 ** 31 - 8), dict(N=2 ** 31 - 8)])
def test_sizes_past_the_kernels_indices(lib, change):
    ad = adapters(**change)
    for rows, starts in ((3, None), (64, A)):
        assert lib.tm_lora_add(ad, A, ad.K, A, ad.N, 2 * A, ad.N, rows, A, starts, 3, None) == UNSUP
