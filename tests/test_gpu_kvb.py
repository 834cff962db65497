"""GPU parity of the paged 8-bit KV cache: append and eviction to the bit against
the binary32 oracle; attention against binary64 within bounds counted from the
number formats (tests/kvb_util.py)."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import CODE, DT, TOP, Cache, bounds, device, normal, rounded
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def run_attention(c, new, Hq, dtype, tag, weights=True, scale=None, in_place=False, stride=0, max_len=0, one_each=False,
                  q_mult=1.0, workspace=None, stream=None):
    Hkv, D = c.pools[0][0].shape[1], c.pools[0][0].shape[3]
    q_start = starts(new)
    rows = int(q_start[-1])
    wide, _ = rounded(normal(f"{tag}/q", rows, Hq + stride, D) * 1.5 * q_mult, dtype)
    Q = wide.cuda()[:, :Hq]
    exact = Q.double().cpu().numpy()
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), None if one_each else device(q_start),
                            max_q=max(list(new) + [1]), max_len=max_len)
    room = c.table.shape[1] * c.T
    w_in = np.abs(normal(f"{tag}/w", len(new), Hkv, room)).astype(np.float32)
    wi = device(w_in)
    wo = (wi if in_place else torch.full_like(wi, 7.0)) if weights else None
    lse = torch.zeros(rows, Hq, device="cuda")
    out = binding.kvb_attention(blocks, batch, Q, lse=lse, w_in=wi if weights else None, w_out=wo, scale=scale,
                                workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    assert c.same(blocks)  # read only
    (k, ks), (v, vs) = c.pools
    o, l, w, size, reach = ref.attention(exact, k, v, ks, vs, c.table, c.kv_len, q_start, c.fmt, scale)
    bo, bl, bw = bounds(o, l, w, size, reach, D, dtype)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - o) <= bo), np.max(np.abs(got - o) / bo)
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(l))
    seen = np.isfinite(l)
    assert np.all(np.abs(gl - l)[seen] <= bl[seen])
    if weights:
        want = w_in.astype(np.float64)
        want[:, :, :w.shape[2]] += w[:, :, :room]
        tol = np.zeros_like(want)
        tol[:, :, :w.shape[2]] = bw[:, :, :room]
        err = np.abs(wo.double().cpu().numpy() - want)
        assert np.all(err <= tol + 2.0 ** -23 * want), np.max(err)
    return out


SHAPES = [  # fmt, dtype, D, T, Hq, Hkv
    ("int8", "fp16", 128, 64, 32, 8), ("e4m3", "bf16", 128, 128, 16, 2), ("e4m3", "fp16", 128, 16, 6, 2),
    ("int8", "bf16", 128, 32, 5, 1), ("int8", "fp16", 64, 16, 4, 4), ("e4m3", "bf16", 64, 32, 14, 2),
    ("e4m3", "fp16", 64, 64, 8, 4), ("int8", "bf16", 64, 128, 12, 1),
]


@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv", SHAPES)
def test_decode_ragged(fmt, dtype, D, T, Hq, Hkv):
    """One token each: lengths of zero and one, pages that end inside a tile, several slices."""
    lens = [1, 0, T, T + 1, 63, 64, 65, 333, 1030]
    c = Cache(f"kvb/dec/{fmt}/{dtype}/{D}/{T}", lens, Hkv, D, T, fmt)
    run_attention(c, [1] * len(lens), Hq, dtype, "dec", one_each=True)


@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv", SHAPES)
def test_drafts_and_chunks(fmt, dtype, D, T, Hq, Hkv):
    """Several tokens each, none for one sequence, a fresh prompt, strided rows, weights in place."""
    c = Cache(f"kvb/draft/{fmt}/{dtype}/{D}/{T}", [70, 9, 5, 259], Hkv, D, T, fmt)
    run_attention(c, [3, 0, 5, 4], Hq, dtype, "draft", stride=3, in_place=True)
    c = Cache(f"kvb/chunk/{fmt}/{dtype}/{D}/{T}", [90, 41, 200], Hkv, D, T, fmt)
    run_attention(c, [90, 17, 33], Hq, dtype, "chunk", stride=2)


@pytest.mark.parametrize("new", [1, 4, 40])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_holes_and_rows_that_see_nothing(new, fmt):
    """Table entries that name no page, a sequence of holes alone, more rows than tokens."""
    c = Cache(f"kvb/holes/{fmt}", [200, 150, 64, 45, 0], 2, 128, 32, fmt)
    c.table[0, 1], c.table[0, 3], c.table[0, 6] = -1, 10 ** 6, c.pools[0][0].shape[0]
    c.table[1, :] = -7
    c.kv_len[2] = 2  # more rows than tokens: the first ones see nothing
    run_attention(c, [new] * 5, 8, "fp16", f"holes/{new}")


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_stale_slots_say_nothing(new, fmt):
    """Slots past each length hold the largest codes and NaN codes, pages of no sequence NaN scales."""
    lens = [70, 130]
    c = Cache(f"kvb/stale/{fmt}", lens, 2, 64, 64, fmt)
    for codes, s in c.pools:
        for b, n in enumerate(lens):
            codes.view(np.uint8)[c.table[b, n // 64], :, n % 64:] = 127
        s[c.free] = np.nan
    run_attention(c, [new] * 2, 4, "fp16", f"stale/{new}")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_scales_far_apart(dtype):
    """Value scales over ten decades, keys that make the softmax nearly one-hot, large and tiny queries."""
    c = Cache(f"kvb/far/{dtype}", [300, 300], 2, 128, 16, "int8", spread=0.3)
    for b in range(2):
        for i in range(19):
            c.pools[1][1][c.table[b, i]] *= np.float32(10.0 ** (3 - 10 * ((i * 7) % 19) / 18))
    run_attention(c, [1, 1], 8, dtype, "far1")
    run_attention(c, [20, 20], 8, dtype, "far2", q_mult=6.0)
    run_attention(c, [2, 1], 8, dtype, "far3", q_mult=1e-3 if dtype == "fp16" else 1e-30)


def test_scale_argument_and_host_bounds():
    c = Cache("kvb/args", [100, 20], 2, 128, 64, "int8")
    a = run_attention(c, [1, 1], 4, "fp16", "args", scale=0.03)
    b = run_attention(c, [1, 1], 4, "fp16", "args", scale=0.03, max_len=100)
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of the pool."""
    T, D, Hkv = 128, 128, 8
    pages = 2 ** 32 // (T * D * Hkv) + 5
    small = Cache("kvb/big", [300, 128], Hkv, D, T, "int8", spare=0)
    blocks = binding.KVBlocks.empty(pages, Hkv, T, D)
    n = small.pools[0][0].shape[0]
    at = pages - n
    (k, ks), (v, vs) = small.pools
    blocks.k[at:], blocks.v[at:] = device(k), device(v)
    blocks.ks[at:], blocks.vs[at:] = device(ks), device(vs)
    table = np.where(small.table >= 0, small.table + at, -1).astype(np.int32)
    for new in ([1, 1], [70, 70]):
        q_start = starts(new)
        Q, _ = rounded(normal("kvb/big/q", int(q_start[-1]), 16, D), "fp16")
        batch = binding.KVBatch(device(table), device(small.kv_len), device(q_start), max_q=max(new))
        out = binding.kvb_attention(blocks, batch, Q.cuda())
        plain = small.to_device(binding)
        batch = binding.KVBatch(device(small.table), device(small.kv_len), device(q_start), max_q=max(new))
        assert torch.equal(out, binding.kvb_attention(plain, batch, Q.cuda()))
    x, xf = rounded(normal("kvb/big/x", 2, Hkv, D), "fp16")
    batch = binding.KVBatch(device(table), device(small.kv_len))
    binding.kvb_append(blocks, batch, x.cuda(), x.cuda())
    for codes, s in small.pools:
        ref.append(codes, s, small.table, small.kv_len, starts([1, 1]), xf, "int8")
    (k, ks), (v, vs) = small.pools
    assert np.array_equal(blocks.k[at:].cpu().numpy(), k) and np.array_equal(blocks.vs[at:].cpu().numpy(), vs)
    w = device(np.abs(normal("kvb/big/w", 2, Hkv, 384)).astype(np.float32))
    kept, _ = binding.kvb_evict(blocks, batch, w.clone(), 100, first=2, recent=9)
    want, _, _ = ref.evict(small.pools, small.table, small.table, small.kv_len, w.cpu().numpy(), 100, 2, 9, "int8")
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(blocks.k[at:].cpu().numpy(), small.pools[0][0])


# ---- append ----

def run_append(c, new, dtype, tag, weights=True, stride=0, mult=1.0, change=None):
    Hkv, D = c.pools[0][0].shape[1], c.pools[0][0].shape[3]
    q_start = starts(new)
    rows = int(q_start[-1])
    x = normal(f"{tag}/x", rows, 2 * Hkv + stride, D) * mult
    if change is not None:
        change(x)
    wide, _ = rounded(x, dtype)
    dev = wide.cuda()
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=max(list(new) + [1]))
    room = c.table.shape[1] * c.T
    w = np.abs(normal(f"{tag}/w", len(new), Hkv, room)).astype(np.float32)
    wd = device(w)
    binding.kvb_append(blocks, batch, dev[:, :Hkv], dev[:, Hkv:2 * Hkv], w=wd if weights else None)
    torch.cuda.synchronize()
    f = wide.float().numpy()
    for (codes, s), part in zip(c.pools, (f[:, :Hkv], f[:, Hkv:2 * Hkv])):
        ref.append(codes, s, c.table, c.kv_len, q_start, part, c.fmt, TOP[dtype])
    assert c.same(blocks)
    if weights:
        for b, n in enumerate(new):
            w[b, :, max(c.kv_len[b] - n, 0):max(c.kv_len[b], 0)] = 0
    assert np.array_equal(wd.cpu().numpy(), w)


@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv", SHAPES)
def test_append_bit_exact(fmt, dtype, D, T, Hq, Hkv):
    """Single tokens (most pages keep their scale), larger ones (it grows), prompts over many pages."""
    tag = f"kvb/app/{fmt}/{dtype}/{D}/{T}"
    lens = [1, T, T + 1, 100, 333, 0]
    run_append(Cache(tag, lens, Hkv, D, T, fmt), [1] * 5 + [0], dtype, tag, stride=1)
    run_append(Cache(tag, lens, Hkv, D, T, fmt), [1] * 5 + [0], dtype, tag + "/large", mult=40.0)
    run_append(Cache(tag, [300, 40, 129], Hkv, D, T, fmt), [300, 23, 128], dtype, tag + "/prompt", stride=2)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_special_values(fmt, dtype):
    """NaN, infinities, zeros, values below the scale's floor, exact ties, a page of zeros."""
    def change(x):
        x[0, 0, :4] = [np.nan, 1.0, -2.0, 0.25]
        x[1, 0, :2] = [np.inf, -np.inf]
        x[2:40, 1] = 0.0
        x[40:70, 0] = 1e-12 if dtype == "bf16" else 6e-8
        x[70, 1] = 127.0
        x[71:75, 1] = np.arange(4 * 64).reshape(4, 64) / 2.0 - 63.5
    tag = f"kvb/special/{fmt}/{dtype}"
    run_append(Cache(tag, [80], 2, 64, 16, fmt), [80], dtype, tag, change=change)


def test_append_leaves_holes_and_other_slots():
    c = Cache("kvb/apphole", [100, 50, 3], 2, 128, 32, "int8")
    c.table[0, 2], c.table[1, 1] = -1, 10 ** 7
    c.kv_len[2] = 1  # three new rows, one token: the last row alone has a place
    run_append(c, [60, 20, 3], "fp16", "kvb/apphole")


def test_append_token_by_token_keeps_one_scale_per_page():
    """A page filled one token at a time equals the oracle's after each step."""
    c = Cache("kvb/steps", [40], 2, 64, 32, "int8", spread=0.0)
    for n in range(1, 41):
        c.kv_len[0] = n
        run_append(c, [1], "fp16", f"kvb/steps/{n}", mult=1.0 + 0.1 * n)


# ---- eviction ----

def run_evict(c, budget, first, recent, tag, in_place=False, w=None):
    B, Hkv = len(c.kv_len), c.pools[0][0].shape[1]
    room = c.table.shape[1] * c.T
    if w is None:  # a few equal weights: ties go to the lowest index
        w = (np.floor(np.exp(2 * normal(f"{tag}/w", B, Hkv, room)) * 16) / 16).astype(np.float32)
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len))
    wd = device(w)
    if in_place:
        dst, wo = c.table, wd
    else:
        nb = -(-budget // c.T)
        dst = c.free[:B * nb].reshape(B, nb).astype(np.int32)
        wo = torch.full((B, Hkv, budget + 3), 5.0, device="cuda")
    kept, new_len = binding.kvb_evict(blocks, batch, wd, budget, first=first, recent=recent,
                                      dst_table=None if in_place else device(dst), w_out=wo)
    torch.cuda.synchronize()
    k0, n0, w0 = ref.evict(c.pools, c.table, dst, c.kv_len, w, budget, first, recent, c.fmt)
    assert np.array_equal(new_len.cpu().numpy(), n0)
    assert np.array_equal(kept.cpu().numpy(), k0)
    assert np.array_equal(wo.cpu().numpy()[:, :, :budget], w0, equal_nan=True)
    if not in_place:
        assert np.all(wo.cpu().numpy()[:, :, budget:] == 5.0)
    assert c.same(blocks)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv", SHAPES)
def test_evict_bit_exact(fmt, dtype, D, T, Hq, Hkv, in_place):
    lens = [500, 37, 0, 1, 129, 260]
    for budget, first, recent in [(128, 4, 32), (37, 0, 0), (100, 50, 50)]:
        spare = len(lens) * -(-budget // T)
        c = Cache(f"kvb/ev/{fmt}/{D}/{T}/{budget}", lens, Hkv, D, T, fmt, spare=spare)
        run_evict(c, budget, first, recent, f"ev/{budget}", in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_special_weights(in_place):
    """Equal weights, NaN, infinities, negative zeros and a hole."""
    c = Cache("kvb/evspecial", [300, 300], 2, 64, 32, "e4m3", spare=8)
    c.table[1, 2] = -1
    w = np.abs(normal("kvb/evspecial/w", 2, 2, c.table.shape[1] * 32)).astype(np.float32)
    w[0, 0] = 1.0
    w[0, 1, 5:200] = np.nan
    w[1, 0, 7:250:3], w[1, 0, 8:250:3] = 0.0, -0.0
    w[1, 1, 3], w[1, 1, 100], w[1, 1, 120:140] = np.inf, -np.inf, -1.0
    run_evict(c, 120, 3, 10, "evspecial", in_place, w)


def test_evict_long():
    """More tokens than a CTA holds keys of, and several waves of pages."""
    c = Cache("kvb/evlong", [140001], 1, 64, 16, "int8", spare=0)
    run_evict(c, 9000, 16, 100, "evlong", in_place=True)


# ---- streams, graphs, repeats ----

def test_another_stream_and_graph_and_repeat():
    c = Cache("kvb/graph", [900, 411], 2, 128, 64, "int8")
    new = [1, 1]
    want = run_attention(c, new, 8, "fp16", "graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(run_attention(c, new, 8, "fp16", "graph", stream=side), want)
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len))
    Q = rounded(normal("graph/q", 2, 8, 128) * 1.5, "fp16")[0].cuda()
    w = torch.zeros(2, 2, c.table.shape[1] * 64, device="cuda")
    ws = torch.empty(binding.kvb_attention_workspace(blocks, batch, 8, 2, True), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(Q)
    step = lambda: binding.kvb_attention(blocks, batch, Q, out=out, w_in=w, w_out=w, workspace=ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    once = w.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    w.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(w, once + once)  # a fixed order of sums: the same bits each time


def test_refusals_of_the_binding():
    blocks = binding.KVBlocks.empty(4, 2, 64, 128)
    batch = binding.KVBatch(torch.zeros(1, 2, dtype=torch.int32, device="cuda"),
                            torch.ones(1, dtype=torch.int32, device="cuda"))
    Q = torch.zeros(1, 4, 128, dtype=torch.float16, device="cuda")
    for bad in (Q.float(), Q[:, :, :64], Q.cpu(), Q.transpose(0, 1)):
        with pytest.raises((ValueError, binding.TMError)):
            binding.kvb_attention(blocks, batch, bad)
    with pytest.raises(binding.TMError):
        binding.kvb_attention(blocks, batch, Q[:, :3])  # 2 KV heads do not divide 3
    with pytest.raises(binding.TMError):  # a workspace that is too small
        w = torch.zeros(1, 2, 128, device="cuda")
        binding.kvb_attention(blocks, batch, Q, w_out=w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.TMError):  # weights for fewer tokens than a sequence may have
        binding.kvb_attention(blocks, batch, Q, w_out=torch.zeros(1, 2, 100, device="cuda"))
    with pytest.raises(ValueError):
        binding.kvb_append(blocks, batch, Q[:, :2], Q[:, :2].bfloat16())
    with pytest.raises(binding.TMError):
        binding.kvb_evict(blocks, batch, torch.zeros(1, 2, 128, device="cuda"), 100, first=60, recent=60)
    with pytest.raises(ValueError):
        binding.KVBlocks(blocks.k, blocks.v, blocks.ks[:2], blocks.vs)
    with pytest.raises(ValueError):
        binding.KVBlocks(blocks.k.view(torch.uint8), blocks.v, blocks.ks, blocks.vs)


@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv", SHAPES)
def test_prompts(fmt, dtype, D, T, Hq, Hkv):
    """Many rows: one and two row tiles, several pairs of them, tiles cut by the length, slices."""
    tag = f"kvb/prompt/{fmt}/{dtype}/{D}/{T}"
    c = Cache(tag, [200, 131, 64, 300, 0, 1], Hkv, D, T, fmt)
    run_attention(c, [200, 128, 40, 3, 0, 1], Hq, dtype, tag, stride=1)
    c = Cache(tag, [1500], Hkv, D, T, fmt)
    run_attention(c, [70], Hq, dtype, tag)
    assert binding.device_error() == 0


def test_prompt_with_holes_and_negative_scale():
    c = Cache("kvb/prompt/holes", [400, 256], 2, 128, 16, "e4m3")
    c.table[0, 3], c.table[0, 8:16], c.table[1, :] = -1, -1, 2 ** 30
    run_attention(c, [150, 90], 8, "fp16", "prompt/holes", scale=-0.1)
    run_attention(c, [2, 2], 8, "fp16", "draft/holes", scale=-0.1)
    assert binding.device_error() == 0


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,Hkv,new", [(40, 1, 1), (64, 1, 1), (100, 1, 1), (13, 1, 4), (24, 2, 2), (22, 2, 3), (6, 6, 33)])
def test_rows_per_head(Hq, Hkv, new, weights):
    """From 33 to over 64 rows of one KV head: each kernel, with and without the tokens' weights."""
    c = Cache(f"kvb/rows/{Hq}/{new}", [300, 90], Hkv, 64, 32, "int8")
    run_attention(c, [new, new], Hq, "bf16", f"rows/{Hq}", weights=weights)
    assert binding.device_error() == 0


@pytest.mark.parametrize("new", [2, 70])
def test_bounds_of_the_host_hold(new):
    """A sequence longer than max_len is read up to it; rows past max_q are not computed; lengths and row
    starts out of range stay inside the buffers."""
    c = Cache("kvb/bounds", [400, 200], 2, 128, 16, "e4m3")
    blocks, q_start = c.to_device(binding), starts([new, new])
    Q = rounded(normal("kvb/bounds/q", 2 * new, 4, 128), "fp16")[0].cuda()
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=new, max_len=144)
    out = binding.kvb_attention(blocks, batch, Q)
    (k, ks), (v, vs) = c.pools
    exact = Q.double().cpu().numpy()
    # rows past token 144 all see the first 144 tokens
    for b in range(2):
        if c.kv_len[b] - new < 144:
            continue
        for i in range(new):
            r = q_start[b] + i
            one = ref.attention(exact[r:r + 1], k, v, ks, vs, c.table[b:b + 1], np.array([144]), np.array([0, 1]), "e4m3")
            bo, _, _ = bounds(*one, 128, "fp16")
            assert np.all(np.abs(out[r].double().cpu().numpy() - one[0][0]) <= bo[0])
    # wrong numbers on the device: clamped, never followed
    bad_len = torch.tensor([10 ** 9, -5], dtype=torch.int32, device="cuda")
    bad_start = torch.tensor([5, 10 ** 9, -3], dtype=torch.int32, device="cuda")
    batch = binding.KVBatch(device(c.table), bad_len, bad_start, max_q=new)
    room = c.table.shape[1] * 16
    w = torch.zeros(2, 2, room, device="cuda")
    binding.kvb_attention(blocks, batch, Q, w_in=w, w_out=w)
    binding.kvb_append(blocks, batch, Q[:, :2], Q[:, 2:], w=w)
    binding.kvb_evict(blocks, batch, w, 40)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
