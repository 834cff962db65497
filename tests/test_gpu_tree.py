"""GPU parity of rotated appends, tree attention and accepted drafts of the paged 8-bit KV cache: pages to the bit
against the binary32 oracle, attention against binary64 within bounds counted from the number formats."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import DT, TOP, Cache, bounds, device, normal, rounded
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

FLT_MAX = float(np.finfo(np.float32).max)


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def angles(positions, dims, base=10000.0):
    half = dims // 2
    a = np.arange(positions)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


# ---- append with rotation ----

def run_rope(c, new, Hq, dtype, tag, dims, interleaved=False, pos=None, queries=True, in_place=False, values=None,
             positions=None, one_each=False, max_q=0, tail=0):
    """`tail`: rows behind the last sequence."""
    Hkv, D = c.pools[0][0].shape[1], c.pools[0][0].shape[3]
    q_start = starts(new)
    rows = int(q_start[-1]) + tail
    # q, k, v of one fused projection, a stray head between them
    x = normal(f"{tag}/x", rows, Hq + 2 * Hkv + 1, D) * 2.0
    if values is not None:
        x = values(x)
    t, exact = rounded(x, dtype)
    fused = t.cuda()
    lens = np.maximum(c.kv_len, 0)
    table = angles(positions or int(lens.max()) + 3, dims)
    slots = np.concatenate([np.arange(lens[b] - n, lens[b]) for b, n in enumerate(new)] + [np.zeros(tail)]).astype(np.int64)
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), None if one_each else device(q_start),
                            max_q=max_q or max(list(new) + [1]))
    room = c.table.shape[1] * c.T
    w = torch.full((len(new), Hkv, room), 3.0, device="cuda")
    Q = fused[:, :Hq]
    q_out = Q if in_place else torch.full((rows, Hq, D), 9.0, dtype=DT[dtype], device="cuda")
    got = binding.kvb_append_rope(blocks, batch, fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv + 1:],
                                  binding.Rope(device(table), interleaved), Q=Q if queries else None,
                                  q_out=q_out if queries else None, pos=None if pos is None else device(pos), w=w)
    torch.cuda.synchronize()
    at = slots if pos is None else pos.astype(np.int64)
    turned = ref.rotate(ref.finite(exact[:, Hq:Hq + Hkv], TOP[dtype]), table, at, interleaved)
    want_w = np.full(w.shape, 3.0, np.float32)
    live = np.zeros(rows, dtype=bool)
    for b, n in enumerate(new):
        old = int(lens[b]) - n
        n_here = min(n, batch.max_q)
        live[q_start[b]:q_start[b] + n_here] = True
        want_w[b, :, max(old, 0):max(old + n_here, 0)] = 0.0
    ref.append(*c.pools[0], c.table, c.kv_len, q_start, turned, c.fmt, top=FLT_MAX)
    ref.append(*c.pools[1], c.table, c.kv_len, q_start, exact[:, Hq + Hkv + 1:], c.fmt, top=TOP[dtype])
    assert c.same(blocks)
    assert np.array_equal(w.cpu().numpy(), want_w)
    if not queries:
        assert got is None
        return
    want = torch.from_numpy(ref.rotate(exact[:, :Hq], table, at, interleaved)).to(DT[dtype])
    kept = t[:, :Hq] if in_place else torch.full_like(want, 9.0)
    want = torch.where(torch.from_numpy(live)[:, None, None], want, kept)
    assert torch.equal(got.cpu().view(torch.int16), want.contiguous().view(torch.int16)) or (
        torch.equal(got.cpu().isnan(), want.isnan()) and torch.equal(got.cpu().nan_to_num(0.5), want.nan_to_num(0.5)))


ROPES = [  # fmt, dtype, D, T, Hq, Hkv, dims, interleaved
    ("int8", "fp16", 128, 64, 32, 8, 128, False), ("e4m3", "bf16", 128, 128, 14, 2, 64, True),
    ("e4m3", "fp16", 64, 16, 5, 5, 48, False), ("int8", "bf16", 64, 32, 9, 1, 64, True),
    ("int8", "bf16", 128, 16, 6, 2, 96, False), ("e4m3", "fp16", 128, 32, 8, 4, 16, True),
    ("e4m3", "bf16", 64, 128, 4, 4, 32, False), ("int8", "fp16", 64, 64, 3, 1, 16, False),
]


@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv,dims,inter", ROPES)
def test_rope_append(fmt, dtype, D, T, Hq, Hkv, dims, inter):
    """Single tokens; fresh and continued pages, ragged, one sequence without new tokens; positions given."""
    lens = [1, T, T + 1, 63, 333]
    c = Cache(f"rope/one/{fmt}/{dtype}/{D}/{T}", lens, Hkv, D, T, fmt)
    run_rope(c, [1] * 5, Hq, dtype, "rope1", dims, inter, one_each=True)
    c = Cache(f"rope/many/{fmt}/{dtype}/{D}/{T}", [T + 5, 40, 2 * T, 150], Hkv, D, T, fmt, spread=0.2)
    new = [7, 0, 2 * T, 150]
    run_rope(c, new, Hq, dtype, "rope2", dims, inter, in_place=True, tail=3)
    c = Cache(f"rope/pos/{fmt}/{dtype}/{D}/{T}", [T + 9, 70], Hkv, D, T, fmt)
    pos = np.array([3, 5, 5, 6, 0, 900, 899, 12, 901, 902, -1, 5], np.int32)  # beyond the table: its ends
    run_rope(c, [9, 3], Hq, dtype, "rope3", dims, inter, pos=pos, positions=901)


@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv,dims,inter", ROPES)
def test_rope_append_of_many_pages(fmt, dtype, D, T, Hq, Hkv, dims, inter):
    """More CTAs than start at once, of single tokens, of whole pages, and of a few tokens."""
    B = 520 // Hkv + 1
    c = Cache(f"rope/wide/one/{fmt}/{D}/{T}", [1 + 7 * b % (T + 3) for b in range(B)], Hkv, D, T, fmt)
    run_rope(c, [1] * B, Hq, dtype, "rope4", dims, inter, one_each=True)
    new = [(2 * T, 5, 1, T + 3, 0)[b % 5] for b in range(B // 2)]
    c = Cache(f"rope/wide/many/{fmt}/{D}/{T}", [n + 3 * b % T for b, n in enumerate(new)], Hkv, D, T, fmt, spread=0.2)
    run_rope(c, new, Hq, dtype, "rope5", dims, inter)
    new = [1 + b % 5 for b in range(B)]
    c = Cache(f"rope/wide/few/{fmt}/{D}/{T}", [n + 5 * b % (T + 9) for b, n in enumerate(new)], Hkv, D, T, fmt, spread=0.2)
    run_rope(c, new, Hq, dtype, "rope6", dims, inter, in_place=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rope_append_of_infinities_and_nan(fmt, dtype):
    def values(x):
        x[3, :, 5], x[4, 7, 64 + 5], x[10, 6:, 100], x[11, 9, 0] = np.inf, np.nan, -np.inf, np.nan
        x[20:, :, :] *= 1e4 if dtype == "fp16" else 2e37  # two large halves pass the type's range
        return x
    for dims, inter in ((128, False), (64, True)):
        c = Cache(f"rope/inf/{fmt}/{dtype}", [70, 33], 2, 128, 32, fmt)
        run_rope(c, [30, 2], 6, dtype, "ropeinf", dims, inter, values=values)


def test_rope_append_holes_and_odd_sequences():
    """Holes, tokens past the table's room, more rows than tokens, rows past max_q, no queries."""
    c = Cache("rope/holes", [200, 90, 4, 64], 2, 64, 32, "int8")
    c.table[0, 5], c.table[1, :] = -1, 10 ** 6
    c.kv_len[2] = 3
    run_rope(c, [60, 9, 5, 1], 4, "fp16", "ropeholes", 64)
    c = Cache("rope/queryless", [50, 20], 3, 64, 16, "e4m3")
    run_rope(c, [20, 20], 6, "bf16", "queryless", 32, queries=False)
    c = Cache("rope/past", [64, 64], 1, 64, 32, "int8")
    c.kv_len[0] = 70  # six tokens have no page
    run_rope(c, [20, 3], 2, "fp16", "ropepast", 64)


def test_rope_rows_past_max_q():
    """Rows past the host's bound keep what they hold, queries included."""
    c = Cache("rope/maxq", [64, 30], 1, 64, 32, "int8")
    Hq, D = 2, 64
    t, exact = rounded(normal("maxq/x", 24, Hq + 2, D), "fp16")
    x, table = t.cuda(), angles(70, 64)
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(starts([20, 4])), max_q=8)
    q = torch.full((24, Hq, D), 9.0, dtype=torch.float16, device="cuda")
    binding.kvb_append_rope(blocks, batch, x[:, Hq:Hq + 1], x[:, Hq + 1:], binding.Rope(device(table)), Q=x[:, :Hq], q_out=q)
    torch.cuda.synchronize()
    q = q.cpu()
    assert (q[8:20] == 9.0).all() and not (q[:8] == 9.0).any() and not (q[20:] == 9.0).any()
    # the eight that count are those of slots 44 .. 51
    part = np.concatenate([exact[:8], exact[20:]])
    turned = ref.rotate(part[:, Hq:Hq + 1], table, np.r_[44:52, 26:30])
    for pool, y in zip(c.pools, (turned, part[:, Hq + 1:])):
        ref.append(*pool, c.table, np.array([52, 30]), starts([8, 4]), y, c.fmt)
    assert c.same(blocks)


# ---- tree attention ----

def random_trees(tag, new):
    """Parents of random trees: as bushy as chains."""
    r = normal(f"{tag}/parents", sum(new) + 1, 2)[:, 0]
    out, at = [], 0
    for n in new:
        out.append([int(np.floor((0.5 + 0.5 * np.tanh(r[at + i])) * (i + 1))) - 1 for i in range(n)])
        at += n
    return out


def run_tree(c, new, Hq, dtype, tag, mask=None, weights=True, scale=None, wide=0, max_len=0, q_mult=1.0, one_each=False,
             tail=0):
    Hkv, D = c.pools[0][0].shape[1], c.pools[0][0].shape[3]
    q_start = starts(new)
    rows = int(q_start[-1]) + tail
    words = -(-max(list(new) + [1]) // 32)
    if mask is None:
        mask = binding.tree_masks(random_trees(tag, new)).numpy()
    mask = np.pad(mask, ((0, rows - mask.shape[0]), (0, words - mask.shape[1])))
    # words past those that count, and bits past the tokens, hold anything
    held = torch.from_numpy(np.concatenate([mask, np.full((rows, wide), -1, np.int32)], 1).astype(np.int32)).cuda()
    x, _ = rounded(normal(f"{tag}/q", rows, Hq + 1, D) * 1.5 * q_mult, dtype)
    Q = x.cuda()[:, :Hq]
    blocks = c.to_device(binding)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), None if one_each else device(q_start),
                            max_q=max(list(new) + [1]), max_len=max_len)
    room = c.table.shape[1] * c.T
    w_in = np.abs(normal(f"{tag}/w", len(new), Hkv, room)).astype(np.float32)
    wi = device(w_in)
    wo = torch.full_like(wi, 7.0) if weights else None
    lse = torch.full((rows, Hq), 5.0, device="cuda")
    out = torch.full((rows, Hq, D), 5.0, dtype=DT[dtype], device="cuda")
    binding.kvb_attention_tree(blocks, batch, Q, held, out=out, lse=lse, w_in=wi if weights else None, w_out=wo, scale=scale)
    torch.cuda.synchronize()
    assert binding.device_error(clear=True) == 0 and c.same(blocks)
    n = int(q_start[-1])
    (k, ks), (v, vs) = c.pools
    o, l, w, size, reach = ref.attention(Q[:n].double().cpu().numpy(), k, v, ks, vs, c.table, c.kv_len, q_start, c.fmt, scale,
                                         tree=mask)
    bo, bl, bw = bounds(o, l, w, size, reach, D, dtype)
    assert (out[n:] == 5.0).all() and (lse[n:] == 5.0).all()
    got, gl = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    assert np.all(np.abs(got - o) <= bo), np.max(np.abs(got - o) / bo)
    assert np.array_equal(np.isneginf(gl), np.isneginf(l))
    seen = np.isfinite(l)
    assert np.all(np.abs(gl[seen] - l[seen]) <= bl[seen])
    if weights:
        want, tol = w_in.astype(np.float64), np.zeros(w_in.shape)
        m = min(room, w.shape[2])
        want[:, :, :m] += w[:, :, :m]
        tol[:, :, :m] = bw[:, :, :m]
        err = np.abs(wo.double().cpu().numpy() - want)
        assert np.all(err <= tol + 2.0 ** -23 * want), np.max(err)
    return out


TREES = [  # fmt, dtype, D, T, Hq, Hkv
    ("int8", "fp16", 128, 64, 32, 8), ("e4m3", "bf16", 128, 128, 16, 2), ("e4m3", "fp16", 128, 16, 6, 2),
    ("int8", "bf16", 128, 32, 5, 1), ("int8", "fp16", 64, 16, 4, 4), ("e4m3", "bf16", 64, 32, 14, 2),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("fmt,dtype,D,T,Hq,Hkv", TREES)
def test_trees(fmt, dtype, D, T, Hq, Hkv, weights):
    """Few rows a head (mma.sync), many (tcgen05), several slices; trees over a page's or a tile's end; a sequence
    without rows, one that is its tree alone."""
    tag = f"tree/{fmt}/{dtype}/{D}/{T}"
    run_tree(Cache(tag + "/a", [70, 9, 2, 259], Hkv, D, T, fmt), [2, 0, 2, 1], Hq, dtype, tag + "a", weights=weights, tail=2)
    run_tree(Cache(tag + "/b", [70, 129, 5, 1259], Hkv, D, T, fmt), [3, 5, 5, 4], Hq, dtype, tag + "b", weights=weights, wide=2)
    run_tree(Cache(tag + "/c", [131, 41, 300], Hkv, D, T, fmt), [33, 41, 64], Hq, dtype, tag + "c", weights=weights)


@pytest.mark.parametrize("fmt,dtype,D", [("int8", "bf16", 128), ("e4m3", "fp16", 128), ("e4m3", "bf16", 64)])
def test_weights_of_one_row_tile(fmt, dtype, D):
    """33 to 128 rows a head: several slices of the tokens, trees over a tile's and a slice's end, a sequence shorter than
    a tile, one without rows, weights past the longest sequence."""
    c = Cache(f"tree/second/{fmt}/{D}", [1300, 650, 21, 1036, 300], 2, D, 64, fmt)
    run_tree(c, [21, 17, 21, 20, 0], 8, dtype, f"second/{fmt}/{D}", wide=1)
    run_tree(c, [21, 17, 21, 20, 0], 12, dtype, f"second/{fmt}/{D}/six", max_len=1300, scale=-0.1)


@pytest.mark.parametrize("fmt,dtype,D", [("int8", "fp16", 128), ("e4m3", "bf16", 64)])
@pytest.mark.parametrize("Hq,new", [(5, [30, 52, 3]), (8, [64, 17, 40]), (8, [65, 70, 1]), (2, [140, 256, 201])])
def test_weights_of_more_row_tiles(fmt, dtype, D, Hq, new):
    """Two to four row tiles, not all of them used by every sequence, and more; masks of up to eight words."""
    c = Cache(f"tree/rows/{fmt}/{Hq}/{new[0]}", [new[0] + 700, new[1], new[2] + 130], 1, D, 32, fmt)
    run_tree(c, new, Hq, dtype, f"rows/{fmt}/{Hq}/{new[0]}", wide=1)


@pytest.mark.parametrize("nodes", [1, 2, 3, 8, 16, 17, 31, 32, 33, 64, 65, 129])
def test_tree_sizes(nodes):
    """Every kernel and row tile, masks of one to five words, tokens before the tree in every phase of a tile."""
    lens = [nodes, nodes + 1, nodes + 127, nodes + 161, 640]
    run_tree(Cache(f"tree/n{nodes}", lens, 1, 64, 32, "int8"), [nodes] * 5, 3, "fp16", f"sizes{nodes}", weights=nodes % 2 == 0)


@pytest.mark.parametrize("new", [2, 9, 40])
def test_masks_that_leave_rows_empty(new):
    """No bit at all, all of them, later nodes alone; nothing before the tree; holes."""
    c = Cache(f"tree/empty{new}", [new, new + 200, new, new + 3], 2, 128, 32, "e4m3")
    words = -(-new // 32)
    mask = np.zeros((4 * new, words), np.int32)
    mask[new:2 * new] = -1
    mask[3 * new:, 0] = 2
    c.table[1, 2] = -1
    c.table[3, :] = -1
    run_tree(c, [new] * 4, 8, "fp16", f"empty{new}", mask=mask)


def test_tree_that_is_a_chain_equals_causal_attention():
    for new, Hq in ((4, 8), (40, 8)):
        c = Cache("tree/chain", [90, 300], 2, 128, 64, "int8")
        rows = 2 * new
        chain = binding.tree_masks([list(range(-1, new - 1))] * 2).cuda()
        Q = rounded(normal("chain/q", rows, Hq, 128), "fp16")[0].cuda()
        blocks, batch = c.to_device(binding), binding.KVBatch(device(c.table), device(c.kv_len), device(starts([new] * 2)), max_q=new)
        a, b = binding.kvb_attention(blocks, batch, Q), binding.kvb_attention_tree(blocks, batch, Q, chain)
        assert torch.equal(a, b)


@pytest.mark.parametrize("new", [3, 40])
def test_tree_stale_slots_and_garbage_in_masked_places(new):
    """NaN codes past the lengths; a hidden token's values are the type's largest."""
    c = Cache(f"tree/stale{new}", [70, 130], 2, 64, 64, "e4m3")
    for codes, s in c.pools:
        for b, n in enumerate([70, 130]):
            codes.view(np.uint8)[c.table[b, n // 64], :, n % 64:] = 127
    c.pools[0][0][c.table[0, 1], :, (70 - 1) % 64] = 0x7E  # the last node: no other row sees it
    run_tree(c, [new, new], 4, "fp16", f"treestale{new}", scale=-0.05)


def test_tree_arguments():
    c = Cache("tree/args", [100, 20], 2, 128, 64, "int8")
    a = run_tree(c, [1, 1], 4, "fp16", "treeargs", scale=0.03, one_each=True, mask=np.ones((2, 1), np.int32))
    b = run_tree(c, [1, 1], 4, "fp16", "treeargs", scale=0.03, max_len=100, mask=np.ones((2, 1), np.int32))
    assert torch.equal(a, b)


# ---- accepted drafts ----

def run_accept(c, new, path, count, weights=True, in_place_len=False):
    Hkv = c.pools[0][0].shape[1]
    blocks = c.to_device(binding)
    q_start = starts(new)
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=max(list(new) + [1]))
    room = c.table.shape[1] * c.T
    w = np.abs(normal("accept/w", len(new), Hkv, room)).astype(np.float32) if weights else None
    wd = device(w) if weights else None
    got = binding.kvb_accept(blocks, batch, device(path.astype(np.int32)), device(np.asarray(count, np.int32)), w=wd)
    torch.cuda.synchronize()
    want = ref.accept(c.pools, c.table, c.kv_len, q_start, path, np.asarray(count), w, c.fmt)
    assert np.array_equal(got.cpu().numpy(), want)
    assert c.same(blocks)
    if weights:
        assert np.array_equal(wd.cpu().numpy(), w)


@pytest.mark.parametrize("fmt,D,T", [("int8", 128, 64), ("e4m3", 128, 16), ("int8", 64, 16), ("e4m3", 64, 128), ("int8", 128, 32)])
def test_accept(fmt, D, T):
    """Paths of every length, within a page, over its end, over several pages and passes; page scales far apart."""
    new = [1, 5, 26, 40, 63, 0, 150, 300]
    lens = [n + x for n, x in zip(new, [0, T - 2, 37, 3 * T, 61, 9, 130, 2 * T - 1])]
    for spread in (0.1, 2.0):
        c = Cache(f"accept/{fmt}/{D}/{T}/{spread}", lens, 2, D, T, fmt, spread=spread)
        path = np.full((8, 200), 10 ** 6)
        count = []
        for b, n in enumerate(new):
            on = np.nonzero(normal(f"accept/path/{b}", n + 1, 1)[:n, 0] > (0.8 if b < 5 else -0.4))[0][:200]
            path[b, :len(on)] = on
            count.append(len(on))
        run_accept(c, new, path, count, weights=spread < 1)


def test_accept_refuses_bad_paths_by_ending_them():
    """Out of range, repeated, descending, negative counts and ones past the path's room; holes; more rows than tokens."""
    c = Cache("accept/bad", [60, 60, 60, 60, 60, 60, 5, 40], 1, 64, 16, "int8", spread=1.0)
    path = np.array([[0, 3, 3, 5], [2, 1, 4, 5], [-1, 2, 3, 4], [4, 9, 20, 21], [1, 2, 4, 6], [1, 3, 4, 19], [0, 1, 2, 3],
                     [5, 7, 11, 19]])
    c.table[5, 2], c.table[7, 1] = -1, 10 ** 6
    run_accept(c, [20] * 8, path, [4, 4, 4, 4, 9, 4, 4, 4])
    run_accept(c, [20] * 8, path, [-3, 0, 1, 2, 3, 4, 4, 2 ** 31 - 1], weights=False)


def test_accept_past_the_tables_room():
    c = Cache("accept/room", [64, 64], 1, 64, 32, "int8")
    c.kv_len[:] = [80, 66]
    run_accept(c, [40, 10], np.array([[3, 20, 22, 30, 39], [1, 8, 9, 9, 9]]), [5, 3])


# ---- offsets, streams, graphs ----

def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of the pool, in all three calls."""
    T, D, Hkv, Hq = 128, 128, 8, 16
    pages = 2 ** 32 // (T * D * Hkv) + 5
    c = Cache("tree/big", [150, 128], Hkv, D, T, "int8", spare=0)
    (k, ks), (v, vs) = c.pools
    n = k.shape[0]
    at = pages - n
    blocks = binding.KVBlocks.empty(pages, Hkv, T, D)
    blocks.k[at:], blocks.v[at:], blocks.ks[at:], blocks.vs[at:] = device(k), device(v), device(ks), device(vs)
    table = np.where(c.table >= 0, c.table + at, -1).astype(np.int32)
    new = [40, 12]
    rows, q_start, rope = sum(new), starts(new), angles(160, 128)
    x, exact = rounded(normal("tree/bigx", rows, Hq + 2 * Hkv, D), "fp16")
    x = x.cuda()
    batch = binding.KVBatch(device(table), device(c.kv_len), device(q_start), max_q=40)
    q = binding.kvb_append_rope(blocks, batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], binding.Rope(device(rope)), Q=x[:, :Hq])
    slots = np.r_[110:150, 116:128]
    ref.append(k, ks, c.table, c.kv_len, q_start, ref.rotate(exact[:, Hq:Hq + Hkv], rope, slots), "int8")
    ref.append(v, vs, c.table, c.kv_len, q_start, exact[:, Hq + Hkv:], "int8")
    mask = binding.tree_masks(random_trees("big", new))
    out = binding.kvb_attention_tree(blocks, batch, q, mask.cuda())
    o, l, w, size, reach = ref.attention(q.double().cpu().numpy(), k, v, ks, vs, c.table, c.kv_len, q_start, "int8",
                                         tree=mask.numpy())
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= bounds(o, l, w, size, reach, D, "fp16")[0])
    path, count = np.array([[0, 4, 20, 31, 39], [2, 3, 5, 7, 11]], np.int32), np.array([5, 4], np.int32)
    binding.kvb_accept(blocks, batch, device(path), device(count))
    ref.accept(c.pools, c.table, c.kv_len, q_start, path, count, None, "int8")
    assert np.array_equal(blocks.k[at:].cpu().numpy(), k) and np.array_equal(blocks.vs[at:].cpu().numpy(), vs)
    assert not blocks.k[:at].any() and not blocks.v[:at].any()


def test_streams_and_graphs():
    """The three calls on a stream of their own, then captured and replayed: the same bits."""
    def state():
        c = Cache("tree/graph", [200, 77], 2, 64, 16, "e4m3")
        x = rounded(normal("tree/graphx", 30, 8 + 4, 64), "bf16")[0].cuda()
        batch = binding.KVBatch(device(c.table), device(c.kv_len), device(starts([20, 10])), max_q=20)
        mask = binding.tree_masks(random_trees("graph", [20, 10])).cuda()
        return (c.to_device(binding), batch, x, mask, binding.Rope(device(angles(210, 64))),
                device(np.array([[1, 4, 7, 19], [0, 2, 5, 9]], np.int32)), device(np.array([4, 3], np.int32)),
                torch.zeros(2, 2, 208, device="cuda"))

    def calls(s, stream=None):
        blocks, batch, x, mask, rope, path, count, w = s
        q = binding.kvb_append_rope(blocks, batch, x[:, 8:10], x[:, 10:], rope, Q=x[:, :8], w=w, stream=stream)
        out = binding.kvb_attention_tree(blocks, batch, q, mask, w_in=w, w_out=w, stream=stream)
        n = binding.kvb_accept(blocks, batch, path, count, w=w, stream=stream)
        return out, n, blocks.k.view(torch.uint8), blocks.vs, w

    want = [t.clone() for t in calls(state())]
    own, s = torch.cuda.Stream(), state()
    torch.cuda.synchronize()
    got = calls(s, own)
    own.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s, graph = state(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = calls(s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    """Attention calls that overlap, each with its workspace: sliced on tensor cores, few rows, many rows."""
    runs = []
    for new, lens in (([26, 9], [1300, 2900]), ([3, 2], [1500, 700]), ([70, 66], [900, 1700])):
        c = Cache(f"tree/two{new[0]}", lens, 2, 128, 64, "int8")
        rows = sum(new)
        Q = rounded(normal(f"two{new[0]}/q", rows, 8, 128), "fp16")[0].cuda()
        mask = binding.tree_masks(random_trees(f"two{new[0]}", new)).cuda()
        blocks = c.to_device(binding)
        batch = binding.KVBatch(device(c.table), device(c.kv_len), device(starts(new)), max_q=max(new))
        size = binding.kvb_attention_workspace(blocks, batch, 8, rows)
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        alone = binding.kvb_attention_tree(blocks, batch, Q, mask)
        runs.append((blocks, batch, Q, mask, ws, alone, torch.cuda.Stream(), [torch.zeros_like(alone) for _ in range(12)]))
    torch.cuda.synchronize()
    for i in range(12):
        for blocks, batch, Q, mask, ws, _, stream, outs in runs:
            binding.kvb_attention_tree(blocks, batch, Q, mask, out=outs[i], workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert binding.device_error(clear=True) == 0
    for *_, alone, _, outs in runs:
        assert all(torch.equal(o, alone) for o in outs)
