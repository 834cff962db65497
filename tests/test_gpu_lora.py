"""GPU parity of low-rank adapters beside a shared projection: binary64, within bounds counted from the number formats."""
import numpy as np
import pytest
import torch

import oracle.lora as ref
from tests.kvb_util import device, normal
from w4a16_quantized_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def halves(tag, *shape, mult=1.0):
    return torch.from_numpy(normal(tag, *shape) * mult).half()


class Problem:
    def __init__(self, tag, new, K, N, R, n, ids, tail=0, x_mult=1.0, scale=True):
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.q_start[-1]) + tail
        self.K, self.N, self.ids = K, N, np.asarray(ids, np.int32)
        self.X, self.Y = halves(f"{tag}/x", self.rows, K + 8, mult=x_mult), halves(f"{tag}/y", self.rows, N + 16)
        self.A, self.B = halves(f"{tag}/a", n, R, K, mult=K ** -0.5), halves(f"{tag}/b", n, N, R, mult=R ** -0.5)
        self.scale = np.abs(normal(f"{tag}/s", n)).astype(np.float32) if scale else None

    def check(self, one_each=False, in_place=False, stream=None):
        ad = binding.Adapters(self.A.cuda(), self.B.cuda(), None if self.scale is None else device(self.scale))
        X, Y = self.X.cuda()[:, 8:], self.Y.cuda()[:, 8:8 + self.N]  # strided rows
        wide = torch.full((self.rows, self.N + 24), 7.0, dtype=torch.float16, device="cuda")
        out = Y if in_place else wide[:, 8:8 + self.N]
        torch.cuda.synchronize()
        got = binding.lora_add(Y, X, ad, device(self.ids), q_start=None if one_each else device(self.q_start),
                               out=None if in_place else out, stream=stream)
        torch.cuda.synchronize()
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        held = f(self.Y[:, 8:8 + self.N]) if in_place else np.full((self.rows, self.N), 7.0)
        scale = np.ones(self.A.shape[0]) if self.scale is None else self.scale.astype(np.float64)
        want, bound = ref.add(f(self.Y[:, 8:8 + self.N]), f(self.X[:, 8:]), f(self.A), f(self.B), scale, self.ids, self.q_start,
                              held)
        err = np.abs(f(got) - want)
        assert np.all(err <= bound), (np.max(err - bound), np.argwhere(err > bound)[:4])
        if not in_place:
            assert (wide[:, :8] == 7.0).all() and (wide[:, 8 + self.N:] == 7.0).all()
        return got


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 104, 128])
@pytest.mark.parametrize("K,N", [(256, 320), (72, 40), (8, 8), (1000, 2056)])
def test_ranks_and_sizes(R, K, N):
    """Decode rows (one each) and runs of rows, K and N that end inside a block, rows without an adapter."""
    Problem(f"lora/d/{R}/{K}", [1] * 7, K, N, R, 4, [3, 0, 0, -1, 2, 3, 9]).check(one_each=True)
    Problem(f"lora/p/{R}/{K}", [33, 1, 0, 70, 5], K, N, R, 3, [1, 2, 0, 0, -5], tail=2).check(in_place=R % 16 == 0)


def test_one_row_one_adapter():
    Problem("lora/one", [1], 4096, 4096, 16, 1, [0]).check(one_each=True, in_place=True)
    Problem("lora/wide", [1], 512, 8192, 64, 2, [1], scale=False).check(one_each=True)


def test_many_adapters_in_a_batch():
    """More adapters than a launch takes side by side, the same ones again and again, in tiles of both sizes."""
    ids = [(7 * b) % 61 - 1 for b in range(150)]
    Problem("lora/many", [1] * 150, 256, 512, 16, 60, ids).check(one_each=True)
    Problem("lora/short", [3, 2, 1, 17, 0, 2] * 12, 256, 256, 32, 30, [(5 * b) % 31 - 1 for b in range(72)], tail=5).check()
    Problem("lora/runs", [40, 16, 3, 130, 1, 64], 512, 264, 64, 3, [0, 1, 0, 2, 1, 2]).check()


@pytest.mark.parametrize("x_mult", [2.0 ** -20, 300.0])
def test_magnitudes(x_mult):
    """Products far below and above fp16's comfortable range on their way."""
    p = Problem("lora/mag", [5, 20], 1024, 64, 16, 2, [0, 1], x_mult=x_mult)
    if x_mult > 1:  # T beyond fp16's largest, brought back by small B
        p.A = (p.A.float() * 500).half()
        p.B = (p.B.float() * 2.0 ** -14).half()
    p.check()


def test_infinities_stay_in_their_rows():
    p = Problem("lora/inf", [1] * 20, 256, 64, 16, 2, [b % 3 - 1 for b in range(20)])
    ad, ids = binding.Adapters(p.A.cuda(), p.B.cuda(), device(p.scale)), device(p.ids)
    X, Y = p.X[:, 8:].cuda(), p.Y[:, :64].contiguous().cuda()
    clean = binding.lora_add(Y, X, ad, ids, out=torch.empty_like(Y))
    X[4, 3], X[8, 100], X[6, 5] = float("inf"), float("nan"), float("nan")  # row 6 has no adapter
    got = binding.lora_add(Y, X, ad, ids, out=torch.empty_like(Y))
    bad = ~torch.isfinite(got).all(1)
    assert bad.nonzero().flatten().tolist() == [4, 8]
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("rows", [40, 400])
def test_claims_that_overlap_and_run_out_of_range(rows):
    """Row starts that are no partition (few rows a sequence, and many): nothing outside is touched, a row that several
    claim takes the last one's."""
    p = Problem(f"lora/claims/{rows}", [1] * rows, 64, 64, 16, 3, [0] * rows)
    ad = binding.Adapters(p.A.cuda(), p.B.cuda())
    X, Y = p.X[:, 8:].cuda(), p.Y[:, :64].contiguous().cuda()
    u = rows // 4
    out = binding.lora_add(Y, X, ad, device(np.array([0, 1, 2, 1], np.int32)),
                           q_start=device(np.array([-5, 2 * u, u, 3 * u, 10 ** 9], np.int32)),
                           out=torch.full_like(Y, 7.0))
    whole = [binding.lora_add(Y, X, ad, torch.full((4,), a, dtype=torch.int32, device="cuda"),
                              q_start=device(np.arange(0, rows + 1, u).astype(np.int32)), out=torch.empty_like(Y))
             for a in range(3)]
    # sequence 0: rows 0 .. 2 u - 1; 1: none; 2: u .. 3 u - 1; 3: 3 u ..
    assert torch.equal(out[:u], whole[0][:u]) and torch.equal(out[u:3 * u], whole[2][u:3 * u])
    assert torch.equal(out[3 * u:], whole[1][3 * u:])


def test_no_adapters_at_all():
    p = Problem("lora/none", [2, 3], 64, 64, 16, 1, [0, 0])
    empty = binding.Adapters(torch.empty(0, 16, 64, dtype=torch.float16, device="cuda"),
                             torch.empty(0, 64, 16, dtype=torch.float16, device="cuda"))
    Y = p.Y[:, :64].contiguous().cuda()
    out = binding.lora_add(Y, p.X[:, 8:].cuda(), empty, device(p.ids), q_start=device(p.q_start), out=torch.zeros_like(Y))
    assert torch.equal(out, Y)


def test_stream_graph_and_repeats():
    p = Problem("lora/graph", [1] * 9, 512, 512, 32, 5, [b % 5 for b in range(9)])
    want = p.check(one_each=True)
    assert torch.equal(p.check(one_each=True, stream=torch.cuda.Stream()), want)
    ad, ids = binding.Adapters(p.A.cuda(), p.B.cuda(), device(p.scale)), device(p.ids)
    X, Y = p.X.cuda()[:, 8:], p.Y.cuda()[:, 8:8 + p.N]
    out, graph = torch.zeros_like(want), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.lora_add(Y, X, ad, ids, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_more_rows_and_adapters_than_one_tile_holds():
    """700 rows of 600 adapters: three tiles, every slot of the table of adapters taken by several."""
    Problem("lora/spans", [1] * 700, 64, 72, 8, 600, [(b * 512 + b // 7) % 601 for b in range(700)]).check(one_each=True)


def test_two_streams_at_once():
    """Calls that overlap, of both kernels: each as it is alone."""
    p = Problem("lora/two", [1] * 40, 1024, 512, 16, 6, [b % 6 for b in range(40)])
    q = Problem("lora/two/q", [300, 21], 1024, 512, 16, 6, [1, 4])
    runs = []
    for x, one_each in ((p, True), (q, False)):
        ad = binding.Adapters(x.A.cuda(), x.B.cuda(), device(x.scale))
        args = (x.Y.cuda()[:, 8:8 + x.N], x.X.cuda()[:, 8:], ad, device(x.ids))
        starts = None if one_each else device(x.q_start)
        alone = binding.lora_add(*args, q_start=starts, out=torch.zeros(x.rows, x.N, dtype=torch.float16, device="cuda"))
        runs.append((args, starts, alone, torch.cuda.Stream(), [torch.zeros_like(alone) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for args, starts, _, stream, outs in runs:
            binding.lora_add(*args, q_start=starts, out=outs[i], stream=stream)
    torch.cuda.synchronize()
    for _, _, alone, _, outs in runs:
        assert all(torch.equal(o, alone) for o in outs)


def test_offsets_past_32_bits():
    """Adapters beyond 4 GiB of A and B."""
    n, R, K, N = 2100, 128, 8192, 8192
    A = torch.zeros(n, R, K, dtype=torch.float16, device="cuda")
    B = torch.zeros(n, N, R, dtype=torch.float16, device="cuda")
    p = Problem("lora/far", [1, 1], K, N, R, 1, [n - 1, 0])
    A[n - 1], B[n - 1] = p.A[0].cuda(), p.B[0].cuda()
    X, Y = p.X.cuda()[:, 8:], p.Y.cuda()[:, 8:8 + N]
    out = binding.lora_add(Y, X, binding.Adapters(A, B), device(p.ids), out=torch.empty(2, N, dtype=torch.float16, device="cuda"))
    near = binding.lora_add(Y, X, binding.Adapters(p.A.cuda(), p.B.cuda()), device(np.array([0, -1], np.int32)),
                            out=torch.empty(2, N, dtype=torch.float16, device="cuda"))
    assert torch.equal(out[0], near[0]) and torch.equal(out[1], Y[1])
