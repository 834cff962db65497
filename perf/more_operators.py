"""Cases of a serving step with drafted trees and adapters: keys rotated by their
position on the way into the paged 8-bit cache, attention for a tree of drafted
tokens, the accepted path moved together, and low-rank adapters of many requests
beside a shared projection.

The cache is paged: a page holds T tokens of one sequence, codes [pages][Hkv][T][D]
(int8 or e4m3) and one fp32 scale per (page, KV head), for keys and for values; a
sequence's row of the table lists its pages.  The calls that write to it return the
whole pools as the numbers that they hold beside their scales, which both forms
compute to the bit: binary32 at each step, division, rounding to the nearest, ties
to even.

``own`` false: the operators in elementary torch operations; true: the calls of
``w4a16_quantized_gemm_gb300.binding``.
"""
import math

import torch

own = False

FLOOR = 2.0 ** -30  # the smallest scale
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
QMAX = {"int8": 127.0, "e4m3": 448.0}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def _rope(name, B, Hq, Hkv, D, T, fmt, dtype, tq, kv, dims, interleaved, tree):
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "fmt": fmt, "dtype": dtype,
            "tq": tq, "kv": kv, "dims": dims, "interleaved": interleaved, "tree": tree}


def _tree(name, B, Hq, Hkv, D, T, fmt, dtype, tq, kv, weights):
    return {"name": name, "op": "tree", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "fmt": fmt, "dtype": dtype,
            "tq": tq, "kv": kv, "weights": weights}


def _accept(name, B, Hkv, D, T, fmt, tq, kv, depth):
    return {"name": name, "op": "accept", "B": B, "Hkv": Hkv, "D": D, "T": T, "fmt": fmt, "tq": tq, "kv": kv,
            "depth": depth}


def _lora(name, B, tq, K, N, R, adapters):
    return {"name": name, "op": "lora", "B": B, "tq": tq, "K": K, "N": N, "R": R, "adapters": adapters}


def listed():
    return [
        # every decode step's token of a full batch
        _rope("rope_token", 32, 32, 8, 128, 64, "int8", "fp16", 1, 4096, 128, False, False),
        # a drafted tree of each of 16 users: positions by depth; neighbours rotate, half of the dimensions do
        _rope("rope_drafts", 16, 32, 4, 64, 32, "e4m3", "bf16", 26, 1777, 32, True, True),
        # four long prompts going into the cache
        _rope("rope_prompt", 4, 32, 8, 128, 64, "e4m3", "bf16", 8191, 8191, 128, False, False),
        # one user with a short context and a handful of drafts: latency alone counts
        _tree("tree_one", 1, 32, 8, 128, 64, "int8", "fp16", 7, 333, False),
        # a serving batch, a tree of 26 nodes for each
        _tree("tree_batch", 16, 32, 8, 128, 64, "int8", "fp16", 26, 4096, False),
        # two users with long contexts and large trees
        _tree("tree_long", 2, 64, 8, 128, 128, "e4m3", "bf16", 63, 65536, False),
        # small heads, none shared, the weights kept for an eviction
        _tree("tree_weights", 9, 12, 12, 64, 16, "e4m3", "bf16", 13, 1531, True),
        # paths of up to 6 nodes of those 26
        _accept("accept_batch", 32, 8, 128, 64, "int8", 26, 4096, 6),
        # long paths through small pages
        _accept("accept_pages", 64, 8, 128, 16, "e4m3", 63, 2047, 40),
        # one request with its adapter beside a square projection
        _lora("lora_token", 1, 1, 4096, 4096, 16, 8),
        # a decode batch with many adapters beside the down projection
        _lora("lora_batch", 32, 1, 14336, 4096, 16, 48),
        # prompts of a few users beside the gate and up projections
        _lora("lora_prompt", 5, 1023, 4096, 28672, 64, 6),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "accept", "lora", "lora"])
    if op == "lora":
        K, N = 64 * _log_uniform(rng, 8, 224), 16 * _log_uniform(rng, 16, 1792)
        tq = 1 if rng.random() < 0.5 else _log_uniform(rng, 2, 2048)
        B = _log_uniform(rng, 1, 64 if tq > 1 else 256)
        B = max(1, min(B, 2 ** 27 // (tq * (K + 2 * N)), 2 ** 13 // tq))  # at most the prompts' bytes
        R = rng.choice([8, 16, 16, 24, 32, 64, 64, 128])
        c = _lora("", B, tq, K, N, R, rng.randint(1, 2 * B if B < 24 else 48))
        del c["name"]
        return c
    D, T = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    fmt, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8])
    G = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8])
    B = _log_uniform(rng, 1, 64)
    if op == "rope":
        tq = _log_uniform(rng, 1, 8192)
        kv = max(tq, _log_uniform(rng, 1, 32768))
        B = max(1, min(B, 2 ** 19 // (Hkv * G * tq), 2 ** 21 // (Hkv * kv)))
        dims = rng.choice([d for d in (16, 32, 48, 64, 96, 128, D, D) if d <= D])
        c = _rope("", B, Hkv * G, Hkv, D, T, fmt, dtype, tq, kv, dims, rng.random() < 0.4, tq < 65 and rng.random() < 0.7)
    elif op == "tree":
        tq = _log_uniform(rng, 2, 64)
        kv = max(tq, _log_uniform(rng, 8, 65536))
        B = max(1, min(B, 2 ** 20 // (Hkv * kv), 2 ** 29 // (Hkv * G * tq * kv)))
        c = _tree("", B, Hkv * G, Hkv, D, T, fmt, dtype, tq, kv, rng.random() < 0.4)
    else:
        tq = _log_uniform(rng, 1, 128)
        kv = max(tq, _log_uniform(rng, 1, 16384))
        B = max(1, min(B, 2 ** 20 // (Hkv * kv)))
        c = _accept("", B, Hkv, D, T, fmt, tq, kv, rng.randint(1, tq))
    del c["name"]
    return c


def _lengths(case):
    """Tokens held and new tokens of each sequence: ragged, and the case's own for the first."""
    kv, tq = case.get("kv", 0), case["tq"]
    n = [max(1, tq - (3 * b % 4) * tq // 8) for b in range(case["B"])]
    total = [max(n[b], kv - (5 * b % 8) * kv // 16) if tq < kv else n[b] for b in range(case["B"])]
    return total, n


def _paths(case):
    """How many nodes of each tree are accepted."""
    _, n = _lengths(case)
    return [min(n[b], case["depth"] - b % (case["depth"] + 1)) for b in range(case["B"])]


def _adapter_of(case):
    """Each sequence's adapter; one in eight has none."""
    return [-1 if b % 8 == 5 else 5 * b % case["adapters"] for b in range(case["B"])]


def work(case):
    total, n = _lengths(case)
    rows = sum(n)
    if case["op"] == "lora":
        K, N, R = case["K"], case["N"], case["R"]
        ids = _adapter_of(case)
        with_one = sum(k for k, a in zip(n, ids) if a >= 0)
        used = len({a for a in ids if a >= 0})
        return {"bytes": used * R * (K + N) * 2 + with_one * K * 2 + rows * N * 4, "flops": 2 * with_one * R * (K + N)}
    Hkv, D, T = case["Hkv"], case["D"], case["T"]
    if case["op"] == "rope":
        size = rows * Hkv * 2 * (3 * D + 4 / T) + 4 * rows * Hkv + rows * case["Hq"] * D * 4
        return {"bytes": size, "flops": 6 * rows * (case["Hq"] + Hkv) * case["dims"] // 2}
    if case["op"] == "tree":
        Hq, pages = case["Hq"], sum(-(-t // T) for t in total)
        seen = sum(k * t for k, t in zip(n, total))
        size = sum(total) * Hkv * 2 * D + pages * Hkv * 8 + rows * (Hq * (2 * D * 2 + 4) + 4 * -(-case["tq"] // 32))
        if case["weights"]:
            size += sum(total) * Hkv * 8
        return {"bytes": size, "flops": 4 * D * Hq * seen}
    kept = sum(_paths(case))
    return {"bytes": kept * Hkv * (4 * D + 8) + 8 * kept + 4 * rows * Hkv, "flops": 0}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _code(y, fmt):
    if fmt == "int8":
        return y.round().clamp(-127, 127).to(torch.int8)
    return y.to(torch.float8_e4m3fn)


def _pool(gen, pages, Hkv, T, D, fmt, channels):
    """Random pages with the scales that they need."""
    x = torch.randn(pages, Hkv, T, D, generator=gen, device="cuda")
    x *= channels * (0.5 + torch.rand(pages, Hkv, 1, 1, generator=gen, device="cuda"))
    s = (x.abs().amax((2, 3)) / QMAX[fmt]).clamp_min(FLOOR)
    return _code(x / s[:, :, None, None], fmt), s


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _trees(gen, B, tq):
    """Random trees: each node's depth, and a mask whose word w, bit j says that node 32 w + j is on its path."""
    parent = torch.rand(B, tq, generator=gen, device="cuda")
    parent = (parent * (torch.arange(tq, device="cuda") + 1)).long() - 1  # -1: the root's child
    sees = torch.zeros(B, tq + 1, tq, dtype=torch.bool, device="cuda")  # the last row: nothing
    for i in range(tq):
        sees[:, i] = sees.gather(1, torch.where(parent[:, i] < 0, tq, parent[:, i])[:, None, None].expand(-1, 1, tq))[:, 0]
        sees[:, i, i] = True
    sees = sees[:, :tq]
    words = -(-tq // 32)
    bits = torch.nn.functional.pad(sees.long(), (0, 32 * words - tq)).reshape(B, tq, words, 32)
    mask = (bits << torch.arange(32, device="cuda")).sum(3)
    return sees.sum(2) - 1, torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    total, n = _lengths(case)
    rows = sum(n)
    st = {"case": case, "q_start": _int32([sum(n[:b]) for b in range(case["B"] + 1)]), "max_q": max(n)}
    if case["op"] == "lora":
        K, N, R, count = case["K"], case["N"], case["R"], case["adapters"]
        st["x"] = torch.randn(rows, K, generator=gen, device="cuda").half()
        st["y"] = torch.randn(rows, N, generator=gen, device="cuda").half()
        st["a"] = (torch.randn(count, R, K, generator=gen, device="cuda") * K ** -0.5).half()
        st["b"] = (torch.randn(count, N, R, generator=gen, device="cuda") * R ** -0.5).half()
        st["scale"] = 0.25 + torch.rand(count, generator=gen, device="cuda")
        st["ids"] = _int32(_adapter_of(case))
        st["out"] = torch.zeros_like(st["y"])
        return st
    B, Hkv, D, T, fmt = case["B"], case["Hkv"], case["D"], case["T"], case["fmt"]
    held = [-(-t // T) for t in total]
    pages = sum(held) + 3  # the last one stays out of every table
    # keys have a few strong channels, as the rotary embedding leaves them
    channels = torch.ones(Hkv, 1, D, device="cuda")
    channels[:, :, 3::29] = 4.0
    st["k"], st["ks"] = _pool(gen, pages, Hkv, T, D, fmt, channels)
    st["v"], st["vs"] = _pool(gen, pages, Hkv, T, D, fmt, torch.ones_like(channels))
    order = torch.randperm(pages - 1, generator=gen, device="cuda").to(torch.int32)
    wide = max(held)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([sum(held[:b]) for b in range(B)], device="cuda")[:, None] + torch.arange(wide, device="cuda")
    there = torch.arange(wide, device="cuda") < torch.tensor(held, device="cuda")[:, None]
    table[there] = order[at[there]]
    st["table"], st["kv_len"], st["max_len"] = table, _int32(total), max(total)
    if case["op"] in ("rope", "accept") or case["weights"]:
        st["w"] = torch.rand(B, Hkv, max(total), generator=gen, device="cuda")
    if case["op"] == "accept":
        # a path's nodes in their order: those with the smallest of random keys
        count = torch.tensor(_paths(case), device="cuda")
        key = torch.rand(B, case["tq"], generator=gen, device="cuda")
        key = torch.where(torch.arange(case["tq"], device="cuda") < torch.tensor(n, device="cuda")[:, None], key, 2.0)
        place = key.argsort(1).argsort(1)
        on = place < count[:, None]
        st["path"] = torch.where(on, torch.arange(case["tq"], device="cuda"), case["tq"]).sort(1).values
        st["path"] = st["path"][:, :case["depth"]].to(torch.int32).contiguous()
        st["count"] = count.to(torch.int32)
        st["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return st
    # the three parts of one fused projection
    Hq = case["Hq"]
    qkv = torch.randn(rows, Hq + 2 * Hkv, D, generator=gen, device="cuda")
    qkv[:, Hq:Hq + Hkv] *= channels[:, 0]
    qkv[:, Hq:] *= 0.5 + torch.rand(rows, 1, 1, generator=gen, device="cuda")
    st["qkv"] = qkv.to(DTYPES[case["dtype"]])
    st["out"] = torch.zeros(rows, Hq, D, dtype=DTYPES[case["dtype"]], device="cuda")
    seq = torch.arange(B, device="cuda").repeat_interleave(torch.tensor(n, device="cuda"))
    node = torch.arange(rows, device="cuda") - st["q_start"].long()[seq]
    if case["op"] == "tree":
        st["mask"] = _trees(gen, B, case["tq"])[1][seq, node].contiguous()
        st["lse"] = torch.zeros(rows, Hq, device="cuda")
        if case["weights"]:
            st["w_out"] = torch.zeros_like(st["w"])
        return st
    # cosines and sines of every position, computed in 64 bits
    half = case["dims"] // 2
    far = max(total) + 1
    turn = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * turn
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["tree"]:
        depth = _trees(gen, B, case["tq"])[0]
        st["pos"] = (st["kv_len"].long() - torch.tensor(n, device="cuda"))[seq].add(depth[seq, node]).to(torch.int32)
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "tree": _own_tree, "accept": _own_accept, "lora": _own_lora}[op](state)
    return {"rope": _plain_rope, "tree": _plain_tree, "accept": _plain_accept, "lora": _plain_lora}[op](state)


def _own_handles(state):
    """What a program makes once: the cache of a layer, and the batch of a step."""
    if "cache" not in state:
        from w4a16_quantized_gemm_gb300 import binding
        state["binding"] = binding
        state["cache"] = binding.KVBlocks(state["k"], state["v"], state["ks"], state["vs"])
        state["batch"] = binding.KVBatch(state["table"], state["kv_len"], q_start=state["q_start"],
                                         max_q=state["max_q"], max_len=state["max_len"])
    return state["binding"], state["cache"], state["batch"]


def _own_rope(state):
    binding, cache, batch = _own_handles(state)
    Hq, Hkv, qkv = state["case"]["Hq"], state["case"]["Hkv"], state["qkv"]
    if "rope" not in state:
        state["rope"] = binding.Rope(state["cos_sin"], interleaved=state["case"]["interleaved"])
    binding.kvb_append_rope(cache, batch, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], state["rope"], Q=qkv[:, :Hq],
                            q_out=state["out"], pos=state.get("pos"), w=state["w"])
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["out"], state["w"]]


def _own_tree(state):
    binding, cache, batch = _own_handles(state)
    Hq, weights = state["case"]["Hq"], state["case"]["weights"]
    if "workspace" not in state:
        # the call's own query (a library without one has a query for both calls)
        query = getattr(binding, "kvb_attention_tree_workspace", binding.kvb_attention_workspace)
        size = query(cache, batch, Hq, state["qkv"].shape[0], weights)
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    more = {"w_in": state["w"], "w_out": state["w_out"]} if weights else {}
    binding.kvb_attention_tree(cache, batch, state["qkv"][:, :Hq], state["mask"], out=state["out"], lse=state["lse"],
                               workspace=state["workspace"], **more)
    return [state["out"], state["lse"]] + ([state["w_out"]] if weights else [])


def _own_accept(state):
    binding, cache, batch = _own_handles(state)
    binding.kvb_accept(cache, batch, state["path"], state["count"], w=state["w"], new_len=state["new_len"])
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["w"], state["new_len"]]


def _own_lora(state):
    if "adapters" not in state:
        from w4a16_quantized_gemm_gb300 import binding
        state["binding"] = binding
        state["adapters"] = binding.Adapters(state["a"], state["b"], state["scale"])
    return state["binding"].lora_add(state["y"], state["x"], state["adapters"], state["ids"], q_start=state["q_start"],
                                     out=state["out"])


def _raw(codes, *at):
    """Codes at an index, as the numbers that they are in 32 bits."""
    return codes.view(torch.uint8)[at].view(codes.dtype).float()


def _turn(x, cs, interleaved):
    """x [rows][heads][D] in 32 bits, its first dimensions rotated in pairs by cs [rows][dims]: cosines, then sines."""
    half = cs.shape[1] // 2
    c, s = cs[:, None, :half], cs[:, None, half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * c - b * s, b * c + a * s], 3).flatten(2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * c - b * s, b * c + a * s], 2)
    return torch.cat([y, x[..., 2 * half:]], 2)


def _plain_rope(state):
    case = state["case"]
    Hq, Hkv, T, fmt = case["Hq"], case["Hkv"], case["T"], case["fmt"]
    start, length = state["q_start"].long(), state["kv_len"].long()
    old = length - (start[1:] - start[:-1])  # tokens held before
    r = torch.arange(state["qkv"].shape[0], device="cuda")
    b = (r[:, None] >= start[1:]).sum(1)
    pos = state["pos"].long() if "pos" in state else old[b] + r - start[b]
    cs = state["cos_sin"][pos]
    state["out"].copy_(_turn(state["qkv"][:, :Hq].float(), cs, case["interleaved"]))
    keys = _turn(state["qkv"][:, Hq:Hq + Hkv].float(), cs, case["interleaved"])
    span = -(-state["max_q"] // T) + 1  # pages that a sequence's new tokens can touch
    block = (old // T)[:, None] + torch.arange(span, device="cuda")
    page = state["table"].long().gather(1, block.clamp_max(state["table"].shape[1] - 1))
    page = torch.where(block * T < length[:, None], page, state["k"].shape[0] - 1)  # the spare page takes the rest
    at = block[:, :, None] * T + torch.arange(T, device="cuda")
    fresh = ((at >= old[:, None, None]) & (at < length[:, None, None]))[:, :, None, :, None]
    before = (at < old[:, None, None])[:, :, None, :, None]
    row = (start[:-1, None, None] + at - old[:, None, None]).clamp(0, r.shape[0] - 1)
    continued = (old[:, None] > block * T)[:, :, None]
    for codes, scales, x in ((state["k"], state["ks"], keys), (state["v"], state["vs"], state["qkv"][:, Hq + Hkv:].float())):
        _plain_write(codes, scales, page, x[row].permute(0, 1, 3, 2, 4), fresh, before, continued, fmt)
    t = torch.arange(state["w"].shape[2], device="cuda")
    state["w"].masked_fill_(((t >= old[:, None]) & (t < length[:, None]))[:, None], 0.0)
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["out"], state["w"]]


def _plain_write(codes, scales, page, x, fresh, before, keeps, fmt):
    """New values x where `fresh` into pages; codes `before` are rounded anew where a page's scale has to grow.
    A page that keeps nothing takes the scale that the new values need."""
    need = (torch.where(fresh, x.abs(), 0.0).amax((3, 4)) * (1.0 / QMAX[fmt])).clamp_min(FLOOR)
    was = scales[page]
    s = torch.where(keeps, torch.maximum(was, need), need)
    s = torch.where(fresh.any(3)[..., 0].expand_as(s), s, was)
    have = codes.view(torch.uint8)[page]
    again = _code(have.view(codes.dtype).float() * was[..., None, None] / s[..., None, None], fmt).view(torch.uint8)
    new = _code(x / s[..., None, None], fmt).view(torch.uint8)
    kept = torch.where(before & (s > was)[..., None, None], again, have)
    codes.view(torch.uint8)[page] = torch.where(fresh, new, kept)
    scales[page] = s


def _dense(codes, scales, table):
    """The values of every sequence's pages, [B][Hkv][tokens][D] in 32 bits."""
    page = table.long().clamp_min(0)
    x = _raw(codes, page).mul_(scales[page][..., None, None])
    B, nb, Hkv, T, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, nb * T, D)


def _plain_tree(state):
    case = state["case"]
    B, Hq, Hkv, D, tq = case["B"], case["Hq"], case["Hkv"], case["D"], state["max_q"]
    G = Hq // Hkv
    k, v = _dense(state["k"], state["ks"], state["table"]), _dense(state["v"], state["vs"], state["table"])
    L = k.shape[2]
    start, length = state["q_start"].long(), state["kv_len"].long()
    new = start[1:] - start[:-1]
    old = length - new
    i = torch.arange(tq, device="cuda")
    row = (start[:-1, None] + i).clamp_max(state["qkv"].shape[0] - 1)
    q = state["qkv"][:, :Hq][row].float().reshape(B, tq, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, tq * G, D)
    # query i of a sequence sees the tokens before the tree and those of the tree that its mask names
    j = torch.arange(L, device="cuda")
    node = (j - old[:, None]).clamp(0, 32 * state["mask"].shape[1] - 1)[:, None].expand(B, tq, L)
    bit = (state["mask"][row].long().gather(2, node // 32) >> (node % 32)) & 1
    seen = (j < old[:, None])[:, None] | ((bit == 1) & (j < length[:, None])[:, None])
    seen = (seen & (i < new[:, None])[:, :, None]).repeat_interleave(G, 1)[:, None]
    s = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).masked_fill_(~seen, -math.inf)
    m = s.amax(3, keepdim=True).clamp_min(-1e30)
    p = s.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    p = p.div_(total.clamp_min(1e-30))
    out = (p @ v).reshape(B, Hkv, tq, G, D).transpose(1, 2).reshape(B * tq, Hq, D)
    lse = (m + total.log()).reshape(B, Hkv, tq, G).transpose(1, 2).reshape(B * tq, Hq)
    # back to the packed rows: row r is query r - start[b] of its sequence b
    r = torch.arange(state["qkv"].shape[0], device="cuda")
    b = (r[:, None] >= start[1:]).sum(1)
    at = b * tq + r - start[b]
    got = [out[at].to(state["out"].dtype), lse[at]]
    if case["weights"]:
        got.append(state["w"] + p.sum(2)[:, :, :state["w"].shape[2]])
    return got


def _plain_accept(state):
    case = state["case"]
    B, T, fmt = case["B"], case["T"], case["fmt"]
    start, length, path = state["q_start"].long(), state["kv_len"].long(), state["path"].long()
    n = start[1:] - start[:-1]
    old, count = length - n, state["count"].long()
    last = state["table"].shape[1] - 1
    span = -(-path.shape[1] // T) + 1
    block = (old // T)[:, None] + torch.arange(span, device="cuda")
    at = block[:, :, None] * T + torch.arange(T, device="cuda")
    i = at - old[:, None, None]  # which token of the path lands here
    lands = (i >= 0) & (i < count[:, None, None])
    src = path.gather(1, i.clamp(0, path.shape[1] - 1).flatten(1)).reshape(i.shape)
    src = torch.where(lands, src + old[:, None, None], 0)
    page = state["table"].long().gather(1, block.clamp_max(last))
    page = torch.where(lands.any(2), page, state["k"].shape[0] - 1)  # the spare page takes the rest
    from_page = state["table"].long().gather(1, (src // T).clamp_max(last).flatten(1)).reshape(src.shape)
    other = lands & (src // T != block[:, :, None])
    same = lands & ~other
    keeps = ((old[:, None] > block * T) | same.any(2))[:, :, None]
    before = ((at < old[:, None, None]) | same)[:, :, None, :, None]
    for codes, scales in ((state["k"], state["ks"]), (state["v"], state["vs"])):
        moved = codes.view(torch.uint8)[from_page, :, src % T].permute(0, 1, 3, 2, 4)  # [B][span][Hkv][T][D]
        s = scales[from_page].permute(0, 1, 3, 2)[..., None]
        x = moved.contiguous().view(codes.dtype).float() * s
        # what stays in its page goes to its slot with its code
        have = codes.view(torch.uint8)[page]
        codes.view(torch.uint8)[page] = torch.where(same[:, :, None, :, None], moved, have)
        _plain_write(codes, scales, page, x, other[:, :, None, :, None], before, keeps, fmt)
    t = torch.arange(state["w"].shape[2], device="cuda")
    k = t - old[:, None]
    to = torch.where((k >= 0) & (k < count[:, None]), path.gather(1, k.clamp(0, path.shape[1] - 1)) + old[:, None], t)
    w = state["w"].gather(2, to.clamp_max(t.shape[0] - 1)[:, None].expand_as(state["w"]))
    w.masked_fill_(((k >= count[:, None]) & (t < length[:, None]))[:, None], 0.0)
    state["w"].copy_(w)
    state["new_len"].copy_(old + count)
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["w"], state["new_len"]]


def _plain_lora(state):
    start, ids = state["q_start"].long(), state["ids"].long()
    rows = state["x"].shape[0]
    i = torch.arange(state["max_q"], device="cuda")
    row = (start[:-1, None] + i).clamp_max(rows - 1)
    a, b = state["a"][ids.clamp_min(0)].float(), state["b"][ids.clamp_min(0)].float()
    t = (state["x"][row].float() @ a.transpose(1, 2)) * torch.where(ids >= 0, state["scale"][ids.clamp_min(0)], 0.0)[:, None, None]
    d = t @ b.transpose(1, 2)
    r = torch.arange(rows, device="cuda")
    seq = (r[:, None] >= start[1:]).sum(1)
    return (state["y"].float() + d[seq, r - start[seq]]).half()


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "accept": _exact_accept, "lora": _exact_lora}[case["op"]](case, st)


def _round64(y, fmt):
    """y (64 bits) to the nearest number of the format, as 64 bits; ties to the even one."""
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _as_codes(x, fmt):
    return x.to(torch.int8) if fmt == "int8" else x


def _exact_rope(case, st):
    total, n = _lengths(case)
    Hq, Hkv, T, D, fmt, half = case["Hq"], case["Hkv"], case["T"], case["D"], case["fmt"], case["dims"] // 2
    pos = [p for b in range(case["B"]) for p in range(total[b] - n[b], total[b])]
    cs = st["cos_sin"].double()[st["pos"].long() if case["tree"] else torch.tensor(pos, device="cuda")]
    # as a product of complex numbers
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    z = torch.complex(cs[:, :half], cs[:, half:])[:, None]
    x = st["qkv"].double()
    t = torch.complex(x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second]) * z
    x[:, :Hq + Hkv, first], x[:, :Hq + Hkv, second] = t.real, t.imag
    got = []
    for codes, scales, h0 in ((st["k"], st["ks"], Hq), (st["v"], st["vs"], Hq + Hkv)):
        c, s = codes.float().double(), scales.double()
        r = 0
        for b in range(case["B"]):
            old = total[b] - n[b]
            for j in range(old // T, -(-total[b] // T)):
                page = int(st["table"][b, j])
                lo, hi = max(old, j * T), min(total[b], (j + 1) * T)
                y = x[r + lo - old:r + hi - old, h0:h0 + Hkv].transpose(0, 1)
                need = (y.abs().amax((1, 2)) / QMAX[fmt]).clamp_min(FLOOR)
                if lo > j * T:
                    was = s[page].clone()
                    need = torch.maximum(need, was)
                    c[page, :, :lo - j * T] = _round64(c[page, :, :lo - j * T] * (was / need)[:, None, None], fmt)
                s[page] = need
                c[page, :, lo - j * T:hi - j * T] = _round64(y / need[:, None, None], fmt)
            r += n[b]
        got.append((_as_codes(c[:-1], fmt), s[:-1]))
    w = st["w"].double()
    for b in range(case["B"]):
        w[b, :, total[b] - n[b]:total[b]] = 0.0
    return [got[0][0], got[1][0], got[0][1], got[1][1], x[:, :Hq], w]


def _exact_tree(case, st):
    total, n = _lengths(case)
    Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], case["T"]
    G = Hq // Hkv
    rows = sum(n)
    out = torch.zeros(rows, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, Hq, dtype=torch.float64, device="cuda")
    w = st["w"].double() if case["weights"] else None
    masks = [[v & 0xffffffff for v in words] for words in st["mask"].tolist()]
    r = 0
    for b in range(case["B"]):
        pages = st["table"][b, :-(-total[b] // T)].long()
        hidden = torch.tensor([[not masks[r + i][j // 32] >> (j % 32) & 1 for j in range(n[b])] for i in range(n[b])], device="cuda")
        for h in range(Hkv):
            kh = st["k"].view(torch.uint8)[pages, h].view(st["k"].dtype).double() * st["ks"][pages, h].double()[:, None, None]
            vh = st["v"].view(torch.uint8)[pages, h].view(st["v"].dtype).double() * st["vs"][pages, h].double()[:, None, None]
            kh, vh = kh.reshape(-1, D)[:total[b]], vh.reshape(-1, D)[:total[b]]
            for g in range(G):
                s = st["qkv"][r:r + n[b], h * G + g].double() @ kh.T / math.sqrt(D)
                s[:, total[b] - n[b]:].masked_fill_(hidden, -math.inf)
                lse[r:r + n[b], h * G + g] = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                out[r:r + n[b], h * G + g] = p @ vh
                if w is not None:
                    w[b, h, :total[b]] += p.sum(0)
        r += n[b]
    return [out, lse] + ([w] if w is not None else [])


def _exact_accept(case, st):
    total, n = _lengths(case)
    counts, T, fmt = _paths(case), case["T"], case["fmt"]
    path = st["path"].tolist()
    table = st["table"].tolist()
    got = []
    for codes, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        c, s = codes.float().double(), scales.double()
        for b in range(case["B"]):
            old, row = total[b] - n[b], table[b]
            for j in range(old // T, -(-(old + counts[b]) // T) if counts[b] else 0):
                here = [i for i in range(counts[b]) if (old + i) // T == j]
                away = [i for i in here if (old + path[b][i]) // T != j]
                stay = [i for i in here if (old + path[b][i]) // T == j]
                page, begin = row[j], max(0, old - j * T)
                for i in stay:
                    c[page, :, (old + i) % T] = c[page, :, (old + path[b][i]) % T]
                if not away:
                    continue
                source = [(row[(old + path[b][i]) // T], (old + path[b][i]) % T) for i in away]
                x = torch.stack([c[p, :, t] * s[p][:, None] for p, t in source], 1)
                need = (x.abs().amax((1, 2)) / QMAX[fmt]).clamp_min(FLOOR)
                held = list(range(begin)) + [(old + i) % T for i in stay]
                if held:
                    need = torch.maximum(need, s[page])
                    c[page][:, held] = _round64(c[page][:, held] * (s[page] / need)[:, None, None], fmt)
                c[page][:, [(old + i) % T for i in away]] = _round64(x / need[:, None, None], fmt)
                s[page] = need
        got.append((_as_codes(c[:-1], fmt), s[:-1]))
    w = st["w"].double()
    for b in range(case["B"]):
        old = total[b] - n[b]
        moved = w[b][:, [old + i for i in path[b][:counts[b]]]].clone()
        w[b, :, old:total[b]] = 0.0
        w[b, :, old:old + counts[b]] = moved
    lens = torch.tensor([total[b] - n[b] + counts[b] for b in range(case["B"])], dtype=torch.int32)
    return [got[0][0], got[1][0], got[0][1], got[1][1], w, lens]


def _exact_lora(case, st):
    _, n = _lengths(case)
    y, r = st["y"].double(), 0
    for b, a in enumerate(_adapter_of(case)):
        if a >= 0:
            y[r:r + n[b]] += (st["x"][r:r + n[b]].double() @ st["a"][a].double().T) @ st["b"][a].double().T * st["scale"][a].double()
        r += n[b]
    return y
