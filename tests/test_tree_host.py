"""Host side of rotated appends, tree attention, accepted drafts and adapters: refusals before any launch (made-up
device addresses: nothing is read through them), the masks of trees, and the oracles' own pins."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
import oracle.lora as lora_ref
from tests.test_kvb_host import BAD_BATCHES, BAD_CACHES, batch, cache

INVALID, ALIGN, UNSUP, OK = 1, 2, 3, 0
A = 1 << 20  # an aligned address


@pytest.fixture(scope="module")
def lib():
    from w4a16_quantized_gemm_gb300 import binding, build
    build.build()
    return binding.load()


def rope(**change):
    from w4a16_quantized_gemm_gb300.binding import KVBRopeStruct
    f = dict(table=A, positions=100, dims=128, interleaved=0, pos=None)
    f.update(change)
    return KVBRopeStruct(**f)


def adapters(**change):
    from w4a16_quantized_gemm_gb300.binding import LoraAdaptersStruct
    f = dict(A=A, B=A, scale=A, n=4, K=256, N=128, R=16)
    f.update(change)
    return LoraAdaptersStruct(**f)


def calls(lib):
    def append(c, b, r=None, K=A, ks=256, V=A, vs=256, Q=A, qs=1024, Hq=8, qo=2 * A, qos=1024, dtype=0, w=None, ws=0):
        return lib.tm_kvb_append_rope(c, b, K, ks, V, vs, Q, qs, Hq, qo, qos, r or rope(), dtype, w, ws, None)

    def tree(c, b, mask=A, ms=1, Q=A, qs=1024, Hq=8, dtype=0, scale=0.0, out=A, lse=None, wi=None, wo=None, ws=0, work=None,
             size=0):
        return lib.tm_kvb_attention_tree(c, b, Q, qs, Hq, dtype, scale, mask, ms, out, lse, wi, wo, ws, work, size, None)

    def accept(c, b, path=A, ps=4, count=A, w=None, ws=0, new=2 * A):
        return lib.tm_kvb_accept(c, b, path, ps, count, w, ws, new, None)

    return append, tree, accept


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(lib, change, status):
    for call in calls(lib):
        assert call(cache(**change), batch()) == status


@pytest.mark.parametrize("change,status", BAD_BATCHES)
def test_bad_batches(lib, change, status):
    for call in calls(lib):
        assert call(cache(), batch(**change)) == status


def test_bad_arguments(lib):
    append, tree, accept = calls(lib)
    c, b = cache(), batch()
    for change in (dict(positions=0), dict(dims=8), dict(dims=24), dict(dims=144), dict(table=None)):
        assert append(c, b, rope(**change)) == INVALID
    assert append(cache(D=64), b, rope(dims=128)) == INVALID
    assert append(c, b, rope(table=A + 8)) == ALIGN and append(c, b, rope(pos=A + 2)) == ALIGN
    assert append(c, b, K=None) == INVALID and append(c, b, V=None) == INVALID and append(c, b, dtype=2) == INVALID
    assert append(c, b, ks=248) == INVALID and append(c, b, vs=260) == ALIGN and append(c, b, K=A + 8) == ALIGN
    assert append(c, b, Hq=3) == INVALID and append(c, b, Hq=0) == INVALID and append(c, b, qo=None) == INVALID
    assert append(c, b, qs=1016) == INVALID and append(c, b, qos=1016) == INVALID and append(c, b, qs=1028) == ALIGN
    assert append(c, b, Q=A + 2) == ALIGN and append(c, b, qo=A + 8) == ALIGN
    assert append(c, b, qo=A, qos=2048) == INVALID                   # in place with another stride
    assert append(c, batch(rows=2)) == INVALID
    assert lib.tm_kvb_append_rope(c, b, A, 256, A, 256, None, 0, 0, None, 0, None, 0, None, 0, None) == INVALID
    assert tree(c, b, mask=None) == INVALID and tree(c, b, ms=0) == INVALID and tree(c, b, mask=A + 2) == ALIGN
    assert tree(c, batch(max_q=33, q_start=A), ms=1) == INVALID      # two words a row
    assert tree(c, b, Hq=3) == INVALID and tree(c, b, scale=float("nan")) == INVALID
    assert tree(c, b, wi=A) == INVALID and tree(c, b, wo=A, ws=255) == INVALID
    assert tree(c, b, wo=A, ws=256, work=A, size=64) == INVALID
    assert accept(c, b, path=None) == INVALID and accept(c, b, count=None) == INVALID and accept(c, b, new=None) == INVALID
    assert accept(c, b, ps=-1) == INVALID and accept(c, b, ws=-1) == INVALID
    assert accept(c, b, new=A) == INVALID                            # new_len over kv_len
    assert accept(c, b, path=A + 2) == ALIGN and accept(c, b, count=A + 1) == ALIGN and accept(c, b, w=A + 2) == ALIGN
    assert accept(c, batch(rows=2)) == INVALID


def test_nothing_to_do(lib):
    append, tree, accept = calls(lib)
    for b in (batch(B=0, rows=0), batch(q_start=A, rows=0), batch(q_start=A, max_q=0)):
        assert append(cache(), b) == OK and tree(cache(), b) == OK
    assert accept(cache(), batch(B=0, rows=0)) == OK


def test_bad_adapters(lib):
    def add(ad, X=A, xs=256, Y=A, ys=128, out=A, os_=128, rows=3, ids=A, q_start=None, B=3):
        return lib.tm_lora_add(ad, X, xs, Y, ys, out, os_, rows, ids, q_start, B, None)

    for change in (dict(n=-1), dict(K=0), dict(K=100), dict(N=4), dict(N=132), dict(R=0), dict(R=12), dict(R=136),
                   dict(A=None), dict(B=None)):
        assert add(adapters(**change)) == INVALID
    ad = adapters()
    assert lib.tm_lora_add(None, A, 256, A, 128, A, 128, 3, A, None, 3, None) == INVALID
    assert add(adapters(A=A + 8)) == ALIGN and add(adapters(scale=A + 2)) == ALIGN
    assert add(ad, rows=-1) == INVALID and add(ad, B=-1) == INVALID and add(ad, rows=4) == INVALID
    assert add(ad, X=None) == INVALID and add(ad, Y=None) == INVALID and add(ad, out=None) == INVALID
    assert add(ad, ids=None) == INVALID and add(ad, xs=248) == INVALID and add(ad, ys=120) == INVALID
    assert add(ad, os_=136) == INVALID                               # in place with another stride
    assert add(ad, xs=260) == ALIGN and add(ad, X=A + 8) == ALIGN and add(ad, ids=A + 2) == ALIGN
    assert add(ad, q_start=A + 2, rows=9) == ALIGN
    assert add(ad, rows=1 << 40, q_start=A) == UNSUP
    assert add(ad, rows=0, B=0) == OK and add(ad, rows=0, q_start=A) == OK and add(ad, rows=5, q_start=A, B=0) == OK


def test_binding_refuses():
    from w4a16_quantized_gemm_gb300 import binding
    with pytest.raises(ValueError):
        binding.Rope(torch.zeros(4, 24))
    with pytest.raises(ValueError):
        binding.Rope(torch.zeros(4, 32))  # on the host
    with pytest.raises(ValueError):
        binding.Adapters(torch.zeros(2, 16, 64).half(), torch.zeros(2, 32, 8).half())
    with pytest.raises(ValueError):
        binding.Adapters(torch.zeros(2, 12, 64).half(), torch.zeros(2, 32, 12).half())
    with pytest.raises(ValueError):
        binding.Adapters(torch.zeros(2, 16, 64).half(), torch.zeros(2, 32, 16).half())  # on the host


def test_tree_masks():
    from w4a16_quantized_gemm_gb300 import binding
    m = binding.tree_masks([[-1, 0, 0, 1], [], [-1, -1]])
    assert m.dtype == torch.int32 and m.flatten().tolist() == [1, 3, 5, 11, 1, 2]
    chain = binding.tree_masks([list(range(-1, 39))])
    assert chain.shape == (40, 2) and chain[31].tolist() == [-1, 0] and chain[39].tolist() == [-1, 255]
    with pytest.raises(ValueError):
        binding.tree_masks([[-1, 1]])


# ---- the oracles ----

@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_a_complex_product(interleaved):
    r = np.random.default_rng(1)
    x, ang = r.standard_normal((5, 3, 64)).astype(np.float32), r.uniform(-3, 3, (9, 16))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = np.array([0, 3, 8, 20, -4])
    y = ref.rotate(x, table, pos, interleaved)
    z = np.exp(1j * ang[np.clip(pos, 0, 8)])[:, None]
    a, b = (x[..., 0:32:2], x[..., 1:32:2]) if interleaved else (x[..., :16], x[..., 16:32])
    t = (a + 1j * b) * z
    c, d = (y[..., 0:32:2], y[..., 1:32:2]) if interleaved else (y[..., :16], y[..., 16:32])
    assert np.abs(c - t.real).max() < 1e-6 and np.abs(d - t.imag).max() < 1e-6 and np.array_equal(y[..., 32:], x[..., 32:])


def test_oracle_tree_of_a_chain_is_causal():
    r = np.random.default_rng(2)
    codes = [r.integers(-127, 128, (4, 1, 16, 64)).astype(np.int8) for _ in range(2)]
    s = [r.uniform(0.005, 0.02, (4, 1)).astype(np.float32) for _ in range(2)]
    table, Q, n = np.array([[3, 0, 2]]), r.standard_normal((35, 2, 64)), np.array([0, 35])
    chain = np.array([[(1 << min(i + 1, 32)) - 1, (1 << max(i - 31, 0)) - 1] for i in range(35)])
    for a, b in zip(ref.attention(Q, codes[0], codes[1], s[0], s[1], table, np.array([41]), n, "int8"),
                    ref.attention(Q, codes[0], codes[1], s[0], s[1], table, np.array([41]), n, "int8", tree=chain)):
        assert np.array_equal(a, b)


def test_oracle_accept_by_hand():
    """Pages of 16: 15 tokens held, new ones in slots 15 .. 19; nodes 0, 2 and 4 are kept.  Node 2 crosses into the
    first page, whose scale doubles; node 4 stays in the second, whose scale stays."""
    codes, s = np.zeros((2, 1, 16, 64), np.int8), np.array([[1.0], [2.0]], np.float32)
    codes[0, 0, :16, 0] = range(1, 17)
    codes[1, 0, :4, 0] = [50, 127, 70, 80]
    w = np.arange(32, dtype=np.float32).reshape(1, 1, 32)
    pools = [(codes, s), (codes.copy(), s.copy())]
    n = ref.accept(pools, np.array([[0, 1]]), np.array([20]), np.array([0, 5]), np.array([[0, 2, 4, 1]]), np.array([4]), w,
                   "int8")
    assert n[0] == 18 and list(w[0, 0, 14:21]) == [14.0, 15.0, 17.0, 19.0, 0.0, 0.0, 20.0]
    assert s[0, 0] == 1.0 and s[1, 0] == np.float32(254 * np.float32(1) / np.float32(127)) == 2.0
    assert list(codes[0, 0, :16, 0]) == list(range(1, 17))  # node 0 is where it was, node 2 goes to slot 16
    assert list(codes[1, 0, :4, 0]) == [127, 80, 70, 80]
    # 14 held: nodes 3 and 4 (second page, the largest 127 * 2) land in the first
    codes[0, 0, :16, 0] = range(1, 17)
    codes[1, 0, :4, 0] = [50, 127, 70, 80]
    n = ref.accept(pools, np.array([[0, 1]]), np.array([19]), np.array([0, 5]), np.array([[3, 4]]), np.array([2]), None, "int8")
    assert n[0] == 16 and s[0, 0] == 2.0 and list(codes[0, 0, 13:16, 0]) == [7, 127, 70] and codes[0, 0, 0, 0] == 0
    assert s[1, 0] == 2.0 and list(codes[1, 0, :4, 0]) == [50, 127, 70, 80]


def test_oracle_adapters_by_hand():
    X, Y = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]), np.ones((3, 1))
    A, B = np.array([[[1.0, 0.0]], [[0.0, 2.0]]]), np.array([[[10.0]], [[100.0]]])
    out, bound = lora_ref.add(Y, X, A, B, np.array([1.0, 0.5]), [1, -1], np.array([0, 1, 2]), np.full((3, 1), 7.0))
    assert out[:, 0].tolist() == [1.0 + 0.5 * 4.0 * 100.0, 1.0, 7.0] and bound[1:, 0].tolist() == [0.0, 0.0]
