"""Paged 8-bit KV cache on the GPU: steps without rows, streams, guards around every
buffer, long slices, shared selections (tests/test_gpu_kvb.py has the operators themselves)."""
import numpy as np
import pytest
import torch

import oracle.kvb as ref
from tests.kvb_util import DT, Cache, device, normal, rounded
from tests.test_gpu_kvb import run_attention, run_evict, starts
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.mark.parametrize("given", ["apart", "in place", "none"])
def test_weights_of_a_step_without_rows(given):
    """No row draws weight: w_out = w_in, over the whole stride."""
    c = Cache("kvb/norows", [70, 0, 33], 2, 64, 32, "int8")
    batch = binding.KVBatch(device(c.table), device(c.kv_len), torch.zeros(4, dtype=torch.int32, device="cuda"), max_q=4)
    Q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    w_in = device(np.abs(normal("kvb/norows/w", 3, 2, c.table.shape[1] * 32 + 5)).astype(np.float32))
    want = torch.zeros_like(w_in) if given == "none" else w_in.clone()
    w_out = w_in if given == "in place" else torch.full_like(w_in, float("nan"))
    out = binding.kvb_attention(c.to_device(binding), batch, Q, w_in=None if given == "none" else w_in, w_out=w_out)
    torch.cuda.synchronize()
    assert out.shape == Q.shape and torch.equal(w_out, want)
    assert binding.device_error() == 0


def _owner(t):
    """Handle of the stream whose memory t lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"])


def test_memory_of_calls_on_another_stream(monkeypatch):
    """What a call on a given stream allocates is that stream's: blocks that the current stream gave back are
    still written there by pending work."""
    c = Cache("kvb/side", [900, 411], 2, 128, 64, "int8")
    blocks, batch = c.to_device(binding), binding.KVBatch(device(c.table), device(c.kv_len))
    Q = rounded(normal("kvb/side/q", 2, 8, 128), "fp16")[0].cuda()
    w = device(np.abs(normal("kvb/side/w", 2, 2, c.table.shape[1] * 64)).astype(np.float32))
    w_want, w_got, w_evict = torch.empty_like(w), torch.empty_like(w), torch.empty(2, 2, 100, device="cuda")
    want = binding.kvb_attention(blocks, batch, Q, w_in=w, w_out=w_want)
    fresh, kept_want = c.to_device(binding), ref.evict(c.pools, c.table, c.table, c.kv_len, w.cpu().numpy(), 100, 4, 9,
                                                       "int8")[0]
    side, made, plain = torch.cuda.Stream(), [], torch.empty
    size = binding.kvb_attention_workspace(blocks, batch, 8, 2, True)
    a = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    given_back = [torch.empty_like(want), torch.empty(size, dtype=torch.uint8, device="cuda"),
                  torch.empty(2, 2, 100, dtype=torch.int32, device="cuda"),
                  torch.empty(2, dtype=torch.int32, device="cuda")]
    for _ in range(20):
        a = a @ a * 0.01
    for t in given_back:
        t.fill_(1)  # pending behind the products
    given_back.clear()
    del t
    monkeypatch.setattr(torch, "empty", lambda *x, **k: made.append(plain(*x, **k)) or made[-1])
    out = binding.kvb_attention(blocks, batch, Q, w_in=w, w_out=w_got, stream=side)
    kept, new_len = binding.kvb_evict(fresh, batch, w, 100, first=4, recent=9, dst_table=batch.table, w_out=w_evict,
                                      stream=side)
    monkeypatch.undo()
    assert len(made) == 4 and [_owner(t) for t in made] == [side.cuda_stream] * 4
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(w_got, w_want)
    assert np.array_equal(kept.cpu().numpy(), kept_want) and new_len.tolist() == [100, 100]
    assert c.same(fresh)


# ---- long slices, shared selections ----

@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,new", [(8, 1), (32, 3), (32, 8)])
def test_slices_of_more_than_2048_tokens(Hq, new, weights):
    """8, 16 and 32 rows a CTA under a bound of 131072 tokens: slices of 4608 or more (on 152 SMs), in which a
    warp takes more than the 16 steps whose pages it reads at once."""
    c = Cache(f"kvb/slice/{Hq}/{new}", [3000, 4600, 2049, 100], 8, 64, 128, "int8")
    c.table = np.pad(c.table, ((0, 0), (0, 1024 - c.table.shape[1])), constant_values=-1)
    c.table[0, 17] = -1  # a hole behind the first 2048
    run_attention(c, [new] * 4, Hq, "fp16", f"slice/{Hq}/{new}", weights=weights)
    assert binding.device_error() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fmt,D,T", [("e4m3", 128, 32), ("int8", 128, 64), ("e4m3", 64, 16)])
def test_evict_in_clusters(fmt, D, T, in_place):
    """Several heads of more tokens than a CTA selects from alone, beside short ones, with waves of pages."""
    lens, budget = [9000, 4097, 20000, 4096, 300], 3000
    c = Cache(f"kvb/evcluster/{fmt}/{D}", lens, 2, D, T, fmt, spare=len(lens) * -(-budget // T))
    run_evict(c, budget, 5, 200, f"evcluster/{T}", in_place)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_repeats_are_equal_to_the_bit(fmt):
    """Each kernel's sums have a fixed order."""
    c = Cache(f"kvb/again/{fmt}", [700, 333], 2, 128, 32, fmt)
    blocks = c.to_device(binding)
    for new in (1, 3, 7, 70):
        Q = rounded(normal(f"kvb/again/q{new}", 2 * new, 8, 128), "bf16")[0].cuda()
        batch = binding.KVBatch(device(c.table), device(c.kv_len), device(starts([new] * 2)), max_q=new)
        got = []
        for _ in range(3):
            w, lse = torch.full((2, 2, 704), 0.5, device="cuda"), torch.empty(2 * new, 8, device="cuda")
            got.append((binding.kvb_attention(blocks, batch, Q, lse=lse, w_in=w, w_out=w), lse, w))
        for other in got[1:]:
            assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# ---- value scales far apart: each row against its own size ----

def row_bounds(c, Q, q_start, dtype, scale=None):
    """The oracle's out, and how far a kernel's may be from it, row by row.

    Relative to sum p |v|: a weight to fp16 2^-11; its score (D products in fp32, (D + 4) 2^-23 of the sum of
    magnitudes, twice: numerator and sum); the exponent's own roundings and log2 of a scale, 2^-17 in all; the
    sums, at most 2^-23 a token.  Weights below 2^-14 are fp16 subnormals, off by 2^-25 where the largest
    p vs of their slice stands for 2^6 or more: 2^-31 of the largest p vs times the code, taken twice.  Then the type."""
    (k, ks), (v, vs) = c.pools
    o, _, _, size, reach = ref.attention(Q, k, v, ks, vs, c.table, c.kv_len, q_start, c.fmt, scale)
    Hkv, T, D = v.shape[1:]
    G = Q.shape[1] // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    sub = np.zeros_like(o)
    for b, length in enumerate(c.kv_len):
        pages = c.table[b, np.arange(length) // T]
        slots = np.arange(length) % T
        for h in range(Hkv):
            kh = ref.decode(k[pages, h, slots], c.fmt) * ks[pages, h].astype(np.float64)[:, None]
            code = np.abs(ref.decode(v[pages, h, slots], c.fmt))
            for r in range(q_start[b], q_start[b + 1]):
                seen = length - (q_start[b + 1] - r) + 1
                for g in range(h * G, h * G + G):
                    x = scale * (kh[:seen] @ Q[r, g])
                    p = np.exp(x - x.max())
                    top = (p / p.sum() * vs[pages[:seen], h]).max()
                    sub[r, g] = 2.0 ** -30 * top * code[:seen].sum(0)
    score = ((D + 4) * 2.0 ** -23 * reach)[..., None]
    rel = 2.0 ** -11 + 4 * score + 2.0 ** -17 + 2.0 ** -23 * max(c.kv_len)
    return o, rel * size + sub + torch.finfo(DT[dtype]).eps / 2 * np.abs(o)


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_value_scales_decades_apart_in_one_call(fmt, new):
    """Sequences and heads whose values differ by up to twelve decades, and pages of one sequence by six: every
    row is near its own result, not near the largest one of the call."""
    c = Cache(f"kvb/decades/{fmt}", [300, 290, 310], 2, 128, 16, fmt, spread=0.3)
    vs = c.pools[1][1]
    for b in range(3):
        for i, page in enumerate(p for p in c.table[b] if p >= 0):
            vs[page] *= np.float32(10.0 ** (2 - 3 * b - 6 * ((i * 7) % 19) / 18))
    vs[:, 1] *= np.float32(1e-1)
    np.maximum(vs, ref.FLOOR, out=vs)
    q_start = starts([new] * 3)
    Q = rounded(normal(f"kvb/decades/q/{new}", 3 * new, 8, 128) * 1.5, "bf16")[0].cuda()
    batch = binding.KVBatch(device(c.table), device(c.kv_len), device(q_start), max_q=new)
    out = binding.kvb_attention(c.to_device(binding), batch, Q).double().cpu().numpy()
    want, tol = row_bounds(c, Q.double().cpu().numpy(), q_start, "bf16")
    assert np.all(np.abs(out - want) <= tol), np.max(np.abs(out - want) / tol)
    small = np.abs(want[-1]).max()  # the smallest sequence is looked at for itself
    assert 0 < small < 1e-2 * np.abs(want[0]).max() and tol[-1].max() < 0.1 * small


# ---- pages that sequences share, pages that nothing was written to ----

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_shared_pages_are_read_and_moved_into_fresh_ones(fmt):
    """Three sequences with one prefix: attention over it, and an eviction that leaves it as it was."""
    T, budget = 32, 100
    c = Cache(f"kvb/shared/{fmt}", [300, 170, 129], 2, 128, T, fmt, spare=3 * 4)
    c.table[1:, :4] = c.table[0, :4]
    for new in (1, 40):
        run_attention(c, [new] * 3, 8, "fp16", f"shared/{new}")
    before = [(codes[c.table[0]].copy(), s[c.table[0]].copy()) for codes, s in c.pools]
    run_evict(c, budget, 40, 10, "shared")
    assert all(np.array_equal(codes[c.table[0]], b) and np.array_equal(s[c.table[0]], d)
               for (codes, s), (b, d) in zip(c.pools, before))


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("new", [1, 3, 50])
def test_pages_that_nothing_was_written_to(fmt, new):
    """Zero codes under scale 0: values of 0, equal scores."""
    blocks = binding.KVBlocks.empty(6, 2, 32, 64, fmt)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6)
    batch = binding.KVBatch(table, device(np.array([180], np.int32)), device(starts([new])), max_q=new)
    Q = torch.randn(new, 4, 64, device="cuda").half()
    lse = torch.empty(new, 4, device="cuda")
    out = binding.kvb_attention(blocks, batch, Q, lse=lse)
    seen = torch.arange(180 - new + 1, 181, device="cuda").double().log()[:, None].expand(new, 4)
    assert torch.equal(out, torch.zeros_like(out))
    assert ((lse.double() - seen).abs() <= 2.0 ** -20 * (1 + seen)).all()  # a log2 and a product in fp32


# ---- nothing outside the buffers, whatever the numbers on the device say ----

class Guards:
    """Tensors inside larger buffers of a known byte."""

    def __init__(self, pad=8192, byte=0xA5):
        self.pad, self.byte, self.whole = pad, byte, []

    def __call__(self, t):
        n = t.numel() * t.element_size()
        raw = torch.full((n + 2 * self.pad,), self.byte, dtype=torch.uint8, device="cuda")
        inner = raw[self.pad:self.pad + n].view(t.dtype).view(t.shape)
        inner.view(torch.uint8).copy_(t.contiguous().view(torch.uint8)) if n else None
        self.whole.append((raw, n))
        return inner

    def intact(self):
        return all(bool((raw[:self.pad] == self.byte).all()) and bool((raw[self.pad + n:] == self.byte).all())
                   for raw, n in self.whole)


BIG = 2 ** 31 - 1
NUMBERS = [  # lengths, row starts (rows are 2 new)
    ([10 ** 9, -5], [5, 10 ** 9, -3]),
    ([BIG, BIG], [-BIG, 2, BIG]),
    ([400, 200], [3, 1, 0]),       # falling starts: no rows
    ([-BIG - 1, 7], [0, BIG, BIG]),
    ([3, 0], [0, 2, 4]),
]


@pytest.mark.parametrize("lens,begins", NUMBERS)
@pytest.mark.parametrize("new", [2, 70])
def test_numbers_out_of_range_stay_inside_every_buffer(new, lens, begins):
    """Wrong lengths, row starts and table entries: guards around each buffer, pages that no table names and the
    inputs stay as they were."""
    T, D, Hkv, Hq, B = 16, 128, 2, 4, 2
    c = Cache("kvb/guard", [400, 200], Hkv, D, T, "e4m3", spare=9)
    c.table[0, 2], c.table[0, 3], c.table[1, 1] = -BIG - 1, BIG, c.pools[0][0].shape[0]
    room = c.table.shape[1] * T
    rows = 2 * new
    guard = Guards()
    plain = c.to_device(binding)
    blocks = binding.KVBlocks(*(guard(t) for t in (plain.k, plain.v, plain.ks, plain.vs)))
    table, kv_len = guard(device(c.table)), guard(device(np.array(lens, np.int32)))
    q_start = guard(device(np.array(begins, np.int32)))
    Q = guard(rounded(normal("kvb/guard/q", rows, Hq, D), "fp16")[0].cuda())
    w = guard(torch.rand(B, Hkv, room, device="cuda"))
    out, lse = guard(torch.zeros_like(Q)), guard(torch.zeros(rows, Hq, device="cuda"))
    w_out = guard(torch.zeros_like(w))
    inputs = [(t, t.clone()) for t in (table, kv_len, q_start, Q)]
    batch = binding.KVBatch(table, kv_len, q_start, max_q=new)
    size = binding.kvb_attention_workspace(blocks, batch, Hq, rows, True)
    work = guard(torch.zeros(size, dtype=torch.uint8, device="cuda"))
    pools = [t.view(torch.uint8).clone() for t in (blocks.k, blocks.v)]
    binding.kvb_attention(blocks, batch, Q, out=out, lse=lse, w_in=w, w_out=w_out, workspace=work)
    binding.kvb_attention(blocks, batch, Q, out=out)
    torch.cuda.synchronize()
    assert guard.intact() and all(torch.equal(t.view(torch.uint8), p)
                                  for t, p in zip((blocks.k, blocks.v), pools))  # attention reads
    binding.kvb_append(blocks, batch, Q[:, :Hkv], Q[:, Hkv:], w=w)
    torch.cuda.synchronize()
    assert guard.intact()
    dst = guard(device(c.free[:6].reshape(2, 3).astype(np.int32)))
    kept = guard(torch.zeros(B, Hkv, 40, dtype=torch.int32, device="cuda"))
    new_len, evicted = guard(torch.zeros(B, dtype=torch.int32, device="cuda")), guard(torch.zeros(B, Hkv, 41, device="cuda"))
    binding.kvb_evict(blocks, batch, w, 40, first=1, recent=3, dst_table=dst, w_out=evicted, kept=kept, new_len=new_len)
    binding.kvb_evict(blocks, batch, w, 40, kept=kept, new_len=new_len)
    torch.cuda.synchronize()
    assert guard.intact() and binding.device_error() == 0
    named = set(c.table.ravel()) | set(c.free[:6])
    others = [p for p in range(blocks.pages) if p not in named]
    assert others and all(torch.equal(t.view(torch.uint8)[others], p[others])
                          for t, p in zip((blocks.k, blocks.v), pools))
    assert all(torch.equal(t, before) for t, before in inputs)
    assert new_len.tolist() == [min(max(n, 0), room, 40) for n in lens]


@pytest.mark.parametrize("budget", [1, 2, 6])
def test_example_with_a_small_budget(budget):
    """The example's kept ends fit every budget."""
    from tests.test_gpu_kvb_example import _module
    m = _module()
    stack = m.Stack(layers=1, B=2, budget=budget, slack=3)
    gen = torch.Generator("cuda").manual_seed(7)
    x = stack.prompt(torch.randn(2, 20, 1024, generator=gen, device="cuda").half())
    for _ in range(5):
        y = stack.decode(stack.norm(x[:, -1]))
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and stack.evictions > 2 and stack.kv_len.tolist() == stack.held
    with pytest.raises(ValueError):
        m.Stack(slack=0)
