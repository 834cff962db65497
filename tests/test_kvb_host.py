"""Host side of the paged 8-bit KV cache: refusals before any launch (made-up
device addresses: nothing is read through them), workspace sizes, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.kvb as ref

INVALID, ALIGN, UNSUP, OK = 1, 2, 3, 0
A = 1 << 20  # an aligned address


@pytest.fixture(scope="module")
def lib():
    from w4a16_quantized_gemm_gb300 import binding, build
    build.build()
    return binding.load()


def cache(**change):
    from w4a16_quantized_gemm_gb300.binding import KVBCacheStruct
    f = dict(k=A, v=A, ks=A, vs=A, pages=8, Hkv=2, T=64, D=128, format=0)
    f.update(change)
    return KVBCacheStruct(**f)


def batch(**change):
    from w4a16_quantized_gemm_gb300.binding import KVBBatchStruct
    f = dict(table=A, kv_len=A, q_start=None, B=3, table_stride=4, max_q=1, max_len=0, rows=3)
    f.update(change)
    return KVBBatchStruct(**f)


BAD_CACHES = [(dict(pages=-1), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=70000), INVALID), (dict(T=48), INVALID),
              (dict(T=256), INVALID), (dict(D=96), INVALID), (dict(format=2), INVALID), (dict(k=None), INVALID),
              (dict(vs=None), INVALID), (dict(k=A + 8), ALIGN), (dict(ks=A + 2), ALIGN)]
BAD_BATCHES = [(dict(B=-1), INVALID), (dict(B=70000), INVALID), (dict(table_stride=-1), INVALID),
               (dict(max_q=-1), INVALID), (dict(max_len=-1), INVALID), (dict(rows=-1), INVALID),
               (dict(table=None), INVALID), (dict(kv_len=None), INVALID), (dict(table=A + 2), ALIGN),
               (dict(table_stride=1 << 30), UNSUP), (dict(rows=1 << 40, q_start=A), UNSUP)]


def calls(lib):
    def append(c, b, K=A, ks=256, V=A, vs=256, dtype=0, w=None, ws=0):
        return lib.tm_kvb_append(c, b, K, ks, V, vs, dtype, w, ws, None)

    def attention(c, b, Q=A, qs=1024, Hq=8, dtype=0, out=A, lse=None, wi=None, wo=None, ws=0, work=None, size=0):
        return lib.tm_kvb_attention(c, b, Q, qs, Hq, dtype, 0.0, out, lse, wi, wo, ws, work, size, None)

    def evict(c, b, dst=A, ds=4, w=A, ws=256, wo=A, wos=256, budget=100, first=4, recent=8, kept=A, new=2 * A):
        return lib.tm_kvb_evict(c, b, dst, ds, w, ws, wo, wos, budget, first, recent, kept, new, None)

    return append, attention, evict


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(lib, change, status):
    for call in calls(lib):
        assert call(cache(**change), batch()) == status


@pytest.mark.parametrize("change,status", BAD_BATCHES)
def test_bad_batches(lib, change, status):
    for call in calls(lib):
        assert call(cache(), batch(**change)) == status


def test_bad_arguments(lib):
    append, attention, evict = calls(lib)
    c, b = cache(), batch()
    assert lib.tm_kvb_append(None, b, A, 256, A, 256, 0, None, 0, None) == INVALID
    assert append(c, b, dtype=2) == INVALID
    assert append(c, b, K=None) == INVALID and append(c, b, V=None) == INVALID
    assert append(c, b, ks=248) == INVALID and append(c, b, vs=260) == ALIGN and append(c, b, K=A + 8) == ALIGN
    assert append(c, batch(rows=2)) == INVALID  # one row per sequence without q_start
    assert attention(c, b, Hq=0) == INVALID and attention(c, b, Hq=3) == INVALID
    assert attention(c, b, dtype=5) == INVALID
    assert attention(c, b, Q=None) == INVALID and attention(c, b, out=None) == INVALID
    assert attention(c, b, qs=1016) == INVALID and attention(c, b, qs=1028) == ALIGN
    assert attention(c, b, Q=A + 2) == ALIGN and attention(c, b, out=A + 8) == ALIGN and attention(c, b, lse=A + 1) == ALIGN
    assert attention(c, b, wi=A) == INVALID                          # w_in without w_out
    assert attention(c, b, wo=A, ws=255) == INVALID                  # fewer weights than tokens
    assert attention(c, b, wo=A, ws=256) == INVALID                  # no workspace
    assert attention(c, b, wo=A, ws=256, work=A, size=64) == INVALID  # too small a one
    assert attention(c, batch(max_q=0)) == INVALID
    assert evict(c, b, budget=0) == INVALID and evict(c, b, first=-1) == INVALID and evict(c, b, recent=97) == INVALID
    assert evict(c, b, dst=None) == INVALID and evict(c, b, ds=1) == INVALID and evict(c, b, w=None) == INVALID
    assert evict(c, b, ws=255) == INVALID and evict(c, b, wos=99) == INVALID
    assert evict(c, b, wos=128) == INVALID                           # in place with another stride
    assert evict(c, b, new=A) == INVALID                             # new_len over kv_len
    assert evict(c, b, kept=A + 2) == ALIGN
    # a length that no 32-bit product holds
    assert evict(c, b, budget=1 << 30, first=1 << 30, recent=1 << 30) == INVALID


def test_nothing_to_do(lib):
    append, attention, evict = calls(lib)
    c = cache()
    for b in (batch(B=0, rows=0), batch(q_start=A, rows=0), batch(q_start=A, max_q=0)):
        assert append(c, b) == OK and attention(c, b) == OK
    assert evict(c, batch(B=0)) == OK


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(7)
    size = lambda c, b, Hq, w: (lib.tm_kvb_attention_workspace(c, b, Hq, w, ctypes.byref(n)), n.value)  # noqa: E731
    none = dict(table=None, kv_len=None)
    assert size(cache(k=None, v=None, ks=None, vs=None), batch(**none), 8, 0) == (OK, 0)  # 256 tokens: one slice
    st, long = size(cache(), batch(table_stride=2048, **none), 8, 0)
    assert st == OK and long > 0
    st, weights = size(cache(), batch(table_stride=2048, **none), 8, 1)
    assert st == OK and weights > long
    assert size(cache(), batch(table_stride=2048, max_len=100, **none), 8, 0) == (OK, 0)
    assert size(cache(), batch(B=0, rows=0), 8, 1) == (OK, 0)
    assert size(cache(), batch(), 3, 0)[0] == INVALID
    assert lib.tm_kvb_attention_workspace(cache(), batch(), 8, 0, None) == INVALID


def test_binding_refuses_host_tensors():
    from w4a16_quantized_gemm_gb300 import binding
    k = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        binding.KVBlocks(k, k, torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        binding.KVBlocks(k[0], k[0], torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(ValueError):
        binding.KVBatch(torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.KVBatch(torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# ---- the oracle ----

def test_oracle_e4m3_equals_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.decode(codes, "e4m3"), want, equal_nan=True)
    v = ref.decode(codes[:127], "e4m3")
    y = np.concatenate([v, (v[1:] + v[:-1]) / 2, v * 1.03, -v, np.linspace(-448, 448, 9999)]).astype(np.float32)
    y = np.clip(y, -448, 448)
    assert np.array_equal(ref.encode(y, "e4m3"), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert np.array_equal(ref.encode(np.float32([449, 1e9, -1e9]), "e4m3"), [0x7E, 0x7E, 0xFE])


def test_oracle_append_by_hand():
    """A page of 16 with three tokens of scale 1; a token with maximum 254 doubles it."""
    codes, s = np.zeros((1, 1, 16, 64), np.int8), np.ones((1, 1), np.float32)
    codes[0, 0, :3, 0] = [127, 3, 5]  # 3 / 2 and 5 / 2 are ties: to the even 2
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :2] = [254.0, -7.0]
    ref.append(codes, s, np.array([[0]]), np.array([4]), np.array([0, 1]), x, "int8")
    assert s[0, 0] == 2.0
    assert list(codes[0, 0, :4, 0]) == [64, 2, 2, 127] and codes[0, 0, 3, 1] == -4
    ref.append(codes, s, np.array([[0]]), np.array([5]), np.array([0, 1]), x / 254, "int8")
    assert s[0, 0] == 2.0 and list(codes[0, 0, :5, 0]) == [64, 2, 2, 127, 0]  # 1/2: a tie


def test_oracle_attention_equals_torch():
    r = np.random.default_rng(3)
    codes = [r.integers(-127, 128, (5, 2, 16, 64)).astype(np.int8) for _ in range(2)]
    s = [r.uniform(0.005, 0.02, (5, 2)).astype(np.float32) for _ in range(2)]
    table, Q = np.array([[3, 0, 4]]), r.standard_normal((6, 4, 64))
    out, lse, w, _, _ = ref.attention(Q, codes[0], codes[1], s[0], s[1], table, np.array([41]), np.array([0, 6]), "int8")
    k, v = [(c.astype(float) * x[:, :, None, None])[table[0]].transpose(1, 0, 2, 3).reshape(2, 48, 64)[:, :41]
            for c, x in zip(codes, s)]
    sc = torch.from_numpy(np.einsum("ihd,hjd->hij", Q, np.repeat(k, 2, 0)) / 8.0)
    sc.masked_fill_(torch.arange(41) > torch.arange(35, 41)[:, None], -np.inf)
    p = sc.softmax(2)
    assert np.allclose(out, np.einsum("hij,hjd->ihd", p.numpy(), np.repeat(v, 2, 0)), atol=1e-12)
    assert np.allclose(lse, sc.logsumexp(2).numpy().T, atol=1e-12)
    assert np.allclose(w[0], p.sum(1).reshape(2, 2, 41).sum(1).numpy(), atol=1e-12)


def test_oracle_evict_by_hand():
    """Six tokens to four: the first, the last and the two heaviest; equal ones by index."""
    codes, s = np.zeros((3, 1, 16, 64), np.int8), np.ones((3, 1), np.float32)
    codes[0, 0, :6, 0] = [10, 127, 30, 40, 50, 60]
    w = np.zeros((1, 1, 16), np.float32)
    w[0, 0, :6] = [0.0, 2.0, 3.0, 1.0, 2.0, 0.0]
    pools = [(codes, s), (codes.copy(), s.copy())]
    kept, n, wo = ref.evict(pools, np.array([[0]]), np.array([[2]]), np.array([6]), w, 4, 1, 1, "int8")
    assert list(kept[0, 0]) == [0, 1, 2, 5] and n[0] == 4 and list(wo[0, 0]) == [0.0, 2.0, 3.0, 0.0]
    assert list(codes[2, 0, :5, 0]) == [10, 127, 30, 60, 0] and s[2, 0] == 1.0
    kept, n, _ = ref.evict(pools, np.array([[0]]), np.array([[1]]), np.array([6]), w, 8, 1, 1, "int8")
    assert n[0] == 6 and list(kept[0, 0]) == [0, 1, 2, 3, 4, 5, -1, -1]
    assert np.array_equal(codes[1], np.pad(codes[0][:, :6], ((0, 0), (0, 10), (0, 0))))
