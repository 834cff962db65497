"""Cases of the block-scaled 8-bit KV cache: appending tokens, attention over the
cache, and eviction by accumulated attention weight.

The cache is paged.  A page holds T tokens of one sequence: codes
[pages][Hkv][T][D] (int8 or e4m3) for keys and for values and one fp32 scale per
(page, KV head) for each; a sequence's row of the table lists its pages.

Appending and evicting return the whole pools as the numbers that they hold (a
plain int8 or e4m3 number each, none packed) beside their scales, which both
forms compute to the bit: binary32 division, rounding to the nearest, ties to even.

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

def _attention(name, B, Hq, Hkv, D, T, fmt, dtype, tq, kv, weights):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "fmt": fmt,
            "dtype": dtype, "tq": tq, "kv": kv, "weights": weights}


def _append(name, B, Hkv, D, T, fmt, dtype, tq, kv):
    return {"name": name, "op": "append", "B": B, "Hq": 4 * Hkv, "Hkv": Hkv, "D": D, "T": T, "fmt": fmt,
            "dtype": dtype, "tq": tq, "kv": kv}


def _evict(name, B, Hkv, D, T, fmt, kv, budget, first, recent):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "D": D, "T": T, "fmt": fmt, "kv": kv,
            "budget": budget, "first": first, "recent": recent}


def listed():
    return [
        # the second word of an answer to a short question: one user, latency alone counts
        _attention("decode_short", 1, 32, 8, 128, 64, "int8", "fp16", 1, 37, False),
        # a full serving batch, every head's weights kept for the eviction
        _attention("decode_batch", 32, 32, 8, 128, 64, "int8", "fp16", 1, 4096, True),
        # two users with whole books in the context
        _attention("decode_long", 2, 64, 8, 128, 128, "e4m3", "bf16", 1, 131072, False),
        # a small model without shared heads, small pages, ragged lengths
        _attention("decode_small_heads", 13, 12, 12, 64, 16, "e4m3", "bf16", 1, 1531, True),
        # five drafted tokens of each of 16 users checked at once
        _attention("verify", 16, 40, 8, 128, 32, "int8", "fp16", 5, 2777, True),
        # the last chunk of a long prompt over what is cached of it
        _attention("prefill_chunk", 1, 32, 8, 128, 64, "int8", "fp16", 2048, 8192, False),
        # three fresh prompts, their weights kept for the eviction that follows
        _attention("prompt_weights", 3, 64, 8, 128, 64, "e4m3", "bf16", 1499, 1499, True),
        # every decode step's keys and values of a full batch
        _append("append_token", 32, 8, 128, 64, "int8", "fp16", 1, 4096),
        # four long prompts going into the cache
        _append("append_prompt", 4, 8, 128, 64, "e4m3", "bf16", 8191, 8191),
        # one user falls back to the budget every 256 tokens
        _evict("evict_one", 1, 8, 128, 64, "int8", 2304, 2048, 4, 256),
        # a full batch of prompts cut to a quarter
        _evict("evict_batch", 32, 8, 128, 32, "e4m3", 4001, 1000, 4, 128),
        # two whole books cut to a few pages
        _evict("evict_long", 2, 8, 128, 64, "int8", 131072, 4096, 64, 512),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "verify", "prefill", "append", "evict"])
    D, T = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    fmt, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 8])
    G = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8])
    kv = _log_uniform(rng, 1, 65536)
    B = _log_uniform(rng, 1, 64)
    if op in ("decode", "verify"):
        tq = 1 if op == "decode" else rng.randint(2, 8)
        kv = max(kv, tq)
        B = max(1, min(B, 2 ** 21 // (Hkv * kv)))  # at most the long decode case's cache
        c = _attention("", B, Hkv * G, Hkv, D, T, fmt, dtype, tq, kv, rng.random() < 0.5)
    elif op == "prefill":
        tq = _log_uniform(rng, 9, 2048)
        kv = tq if rng.random() < 0.5 else max(tq, min(kv % 8192, 2 ** 29 // (Hkv * G * tq)))
        B = max(1, min(B, 2 ** 29 // (Hkv * G * tq * kv)))  # at most the prompt chunk's products
        c = _attention("", B, Hkv * G, Hkv, D, T, fmt, dtype, tq, kv, rng.random() < 0.5)
    elif op == "append":
        tq = _log_uniform(rng, 1, 8192)
        kv = max(tq, kv)
        B = max(1, min(B, 2 ** 18 // (Hkv * tq), 2 ** 21 // (Hkv * kv)))
        c = _append("", B, Hkv, D, T, fmt, dtype, tq, kv)
    else:
        kv = max(kv, 32)
        B = max(1, min(B, 2 ** 21 // (Hkv * kv)))
        budget = min(_log_uniform(rng, 8, 8192), kv)
        first = rng.randint(0, min(64, budget // 4))
        recent = rng.randint(0, min(512, budget // 2))
        c = _evict("", B, Hkv, D, T, fmt, kv, budget, first, recent)
    del c["name"]
    return c


def _lengths(case):
    """Tokens held and new tokens of each sequence: ragged, and the case's own for the first."""
    kv, tq = case["kv"], case.get("tq", 0)
    n = [max(min(tq, 1), tq - (3 * b % 4) * tq // 8) for b in range(case["B"])]
    total = [max(n[b], kv - (5 * b % 8) * kv // 16) if tq < kv else n[b] for b in range(case["B"])]
    return total, n


def work(case):
    total, n = _lengths(case)
    Hkv, D, T = case["Hkv"], case["D"], case["T"]
    pages = sum(-(-t // T) for t in total)
    if case["op"] == "attention":
        Hq, rows = case["Hq"], sum(n)
        seen = sum(k * t - k * (k - 1) // 2 for k, t in zip(n, total))  # visible (query, token) pairs
        size = sum(total) * Hkv * 2 * D + pages * Hkv * 8 + rows * Hq * (2 * D * 2 + 4)
        if case["weights"]:
            size += sum(total) * Hkv * 8
        return {"bytes": size, "flops": 4 * D * Hq * seen}
    if case["op"] == "append":
        rows = sum(n)
        return {"bytes": rows * Hkv * 2 * (3 * D + 4 / T) + 4 * rows * Hkv, "flops": 0}
    kept = sum(min(t, case["budget"]) for t in total)
    return {"bytes": sum(total) * Hkv * 4 + kept * Hkv * (2 * 2 * D + 2 * 8 / T + 8), "flops": 0}


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


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    B, Hkv, D, T, fmt = case["B"], case["Hkv"], case["D"], case["T"], case["fmt"]
    total, n = _lengths(case)
    if case["op"] == "evict":
        held = [-(-t // T) for t in total]
        kept = -(-case["budget"] // T)
    else:
        held, kept = [-(-t // T) for t in total], 0
    used = sum(held) + B * kept
    pages = used + 3  # the last one stays out of every table
    # keys have a few strong channels, as the rotary embedding leaves them
    channels = torch.ones(Hkv, 1, D, device="cuda")
    channels[:, :, 3::29] = 4.0
    k, ks = _pool(gen, pages, Hkv, T, D, fmt, channels)
    v, vs = _pool(gen, pages, Hkv, T, D, fmt, torch.ones_like(channels))
    order = torch.randperm(pages - 1, generator=gen, device="cuda").to(torch.int32)[:used]
    wide = max(held)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([sum(held[:b]) for b in range(B)], device="cuda")[:, None] + torch.arange(wide, device="cuda")
    there = torch.arange(wide, device="cuda") < torch.tensor(held, device="cuda")[:, None]
    table[there] = order[at[there]]
    vs[table[:, 0].long()] *= 0.1  # the first tokens draw much weight and say little
    st = {"case": case, "k": k, "v": v, "ks": ks, "vs": vs, "table": table,
          "kv_len": torch.tensor(total, dtype=torch.int32, device="cuda"), "max_len": max(total)}
    if case["op"] == "evict":
        # sums of softmax weights: a heavy tail, and enough equal ones to need the rule for ties
        w = torch.randn(B, Hkv, max(total), generator=gen, device="cuda").mul_(2.0).exp_()
        st["w"] = (w * 64).floor_() / 64
        st["dst_table"] = order[sum(held):].reshape(B, kept).contiguous()
        st["w_out"] = torch.zeros(B, Hkv, case["budget"], device="cuda")
        st["kept"] = torch.zeros(B, Hkv, case["budget"], dtype=torch.int32, device="cuda")
        st["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return st
    rows, dt = sum(n), DTYPES[case["dtype"]]
    st["q_start"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    st["max_q"] = max(n)
    # the three parts of one fused projection
    Hq = case["Hq"]
    qkv = torch.randn(rows, Hq + 2 * Hkv, D, generator=gen, device="cuda")
    qkv[:, Hq:Hq + Hkv] *= channels[:, 0]
    qkv[:, Hq:] *= 0.5 + torch.rand(rows, 1, 1, generator=gen, device="cuda")
    st["qkv"] = qkv.to(dt)
    if case["op"] == "append":
        st["w"] = torch.rand(B, Hkv, max(total), generator=gen, device="cuda")
        return st
    st["out"] = torch.zeros(rows, Hq, D, dtype=dt, device="cuda")
    st["lse"] = torch.zeros(rows, Hq, device="cuda")
    if case["weights"]:
        st["w"] = torch.rand(B, Hkv, max(total), generator=gen, device="cuda")
        st["w_out"] = torch.zeros_like(st["w"])
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "evict": _own_evict}[op](state)
    return {"attention": _plain_attention, "append": _plain_append, "evict": _plain_evict}[op](state)


def _own_handles(state):
    """What a program makes once: the cache of a layer, and the batch of a step."""
    if "cache" not in state:
        from w4a16_quantized_gemm_gb300 import binding
        state["binding"] = binding
        state["cache"] = binding.KVBlocks(state["k"], state["v"], state["ks"], state["vs"])
        state["batch"] = binding.KVBatch(state["table"], state["kv_len"], q_start=state.get("q_start"),
                                         max_q=state.get("max_q", 1), max_len=state["max_len"])
    return state["binding"], state["cache"], state["batch"]


def _own_attention(state):
    binding, cache, batch = _own_handles(state)
    Hq = state["case"]["Hq"]
    if "workspace" not in state:
        size = binding.kvb_attention_workspace(cache, batch, Hq, state["qkv"].shape[0], state["case"]["weights"])
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    weights = {"w_in": state["w"], "w_out": state["w_out"]} if state["case"]["weights"] else {}
    binding.kvb_attention(cache, batch, state["qkv"][:, :Hq], out=state["out"], lse=state["lse"],
                          workspace=state["workspace"], **weights)
    return [state["out"], state["lse"]] + ([state["w_out"]] if weights else [])


def _own_append(state):
    binding, cache, batch = _own_handles(state)
    Hq, Hkv = state["case"]["Hq"], state["case"]["Hkv"]
    qkv = state["qkv"]
    binding.kvb_append(cache, batch, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], w=state["w"])
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["w"]]


def _own_evict(state):
    binding, cache, batch = _own_handles(state)
    case = state["case"]
    binding.kvb_evict(cache, batch, state["w"], case["budget"], first=case["first"], recent=case["recent"],
                      dst_table=state["dst_table"], w_out=state["w_out"], kept=state["kept"],
                      new_len=state["new_len"])
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["kept"], state["new_len"],
            state["w_out"]]


def _dense(codes, scales, table):
    """The values of every sequence's pages, [B][Hkv][tokens][D] in 32 bits."""
    page = table.long().clamp_min(0)
    raw = codes.view(torch.uint8)[page].view(codes.dtype).float()
    x = raw.mul_(scales[page][..., None, None])
    B, nb, Hkv, T, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, nb * T, D)


def _plain_attention(state):
    case = state["case"]
    B, Hq, Hkv, D, tq = case["B"], case["Hq"], case["Hkv"], case["D"], state["max_q"]
    G = Hq // Hkv
    k = _dense(state["k"], state["ks"], state["table"])
    v = _dense(state["v"], state["vs"], state["table"])
    L = k.shape[2]
    start, length = state["q_start"].long(), state["kv_len"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(tq, device="cuda")
    row = (start[:-1, None] + i).clamp_max(state["qkv"].shape[0] - 1)
    q = state["qkv"][:, :Hq][row].float().reshape(B, tq, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, tq * G, D)
    # query i of a sequence sees the tokens up to its own
    last = torch.where(i < new[:, None], length[:, None] - new[:, None] + i, -1)
    seen = (torch.arange(L, device="cuda") <= last[:, :, None]).repeat_interleave(G, 1)[:, None]
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
        size = state["w"].shape[2]
        got.append(state["w"] + p.sum(2)[:, :, :size])
    return got


def _plain_append(state):
    case = state["case"]
    Hq, Hkv, T, D, fmt = case["Hq"], case["Hkv"], case["T"], case["D"], case["fmt"]
    start, length = state["q_start"].long(), state["kv_len"].long()
    old = length - (start[1:] - start[:-1])  # tokens held before
    span = -(-state["max_q"] // T) + 1       # pages that a sequence's new tokens can touch
    block = (old // T)[:, None] + torch.arange(span, device="cuda")
    touched = block * T < length[:, None]
    page = state["table"].long().gather(1, block.clamp_max(state["table"].shape[1] - 1))
    page = torch.where(touched, page, state["k"].shape[0] - 1)  # the spare page takes the rest
    pos = block[:, :, None] * T + torch.arange(T, device="cuda")
    fresh = ((pos >= old[:, None, None]) & (pos < length[:, None, None]))[:, :, None, :, None]
    before = (pos < old[:, None, None])[:, :, None, :, None]
    row = (start[:-1, None, None] + pos - old[:, None, None]).clamp(0, state["qkv"].shape[0] - 1)
    continued = (old[:, None] > block * T)[:, :, None]
    new = state["qkv"][:, Hq:][row].permute(0, 1, 3, 2, 4)
    _plain_write(state["k"], state["ks"], page, new[:, :, :Hkv], fresh, before, continued, fmt)
    _plain_write(state["v"], state["vs"], page, new[:, :, Hkv:], fresh, before, continued, fmt)
    t = torch.arange(state["w"].shape[2], device="cuda")
    state["w"].masked_fill_(((t >= old[:, None]) & (t < length[:, None]))[:, None], 0.0)
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["w"]]


def _plain_write(codes, scales, page, new, fresh, before, continued, fmt):
    """New tokens into their pages; a page whose scale has to grow has its earlier codes rounded anew."""
    x = torch.where(fresh, new.float(), 0.0)
    need = (x.abs().amax((3, 4)) / QMAX[fmt]).clamp_min(FLOOR)
    was = scales[page]
    s = torch.where(continued, torch.maximum(was, need), need)
    have = codes.view(torch.uint8)[page].view(codes.dtype)
    again = _code((have.float() * was[..., None, None]) / s[..., None, None], fmt)
    fresh_codes = _code(x / s[..., None, None], fmt)
    kept = torch.where(before & (s > was)[..., None, None], again.view(torch.uint8), have.view(torch.uint8))
    codes.view(torch.uint8)[page] = torch.where(fresh, fresh_codes.view(torch.uint8), kept)
    scales[page] = s


def _plain_evict(state):
    case = state["case"]
    B, Hkv, D, T, fmt = case["B"], case["Hkv"], case["D"], case["T"], case["fmt"]
    budget, w = case["budget"], state["w"]
    length = state["kv_len"].long()[:, None, None]
    t = torch.arange(w.shape[2], device="cuda")
    rank = torch.where((t < case["first"]) | (t >= length - case["recent"]), math.inf, w)
    rank = torch.where(t < length, rank, -math.inf)
    count = length.clamp_max(budget)
    best = rank.argsort(dim=2, descending=True, stable=True)
    place = torch.empty_like(best).scatter_(2, best, t.expand_as(best))
    chosen = (place < count) & (t < length)
    kept = (~chosen).to(torch.uint8).argsort(dim=2, stable=True)[:, :, :budget]  # the chosen, in their order
    slot = torch.arange(kept.shape[2], device="cuda")
    there = slot < count
    state["new_len"].copy_(count[:, 0, 0])
    state["kept"].fill_(-1)[:, :, :kept.shape[2]] = torch.where(there, kept, -1).to(torch.int32)
    state["w_out"].zero_()[:, :, :kept.shape[2]] = torch.where(there, w.gather(2, kept), 0.0)
    pad = state["dst_table"].shape[1] * T - kept.shape[2]
    src = torch.nn.functional.pad(kept, (0, pad))
    there = torch.nn.functional.pad(there.expand(B, Hkv, -1), (0, pad))
    _plain_move(state["k"], state["ks"], state, src, there, fmt)
    _plain_move(state["v"], state["vs"], state, src, there, fmt)
    return [state["k"][:-1], state["v"][:-1], state["ks"][:-1], state["vs"][:-1], state["kept"], state["new_len"],
            state["w_out"]]


def _plain_move(codes, scales, state, src, there, fmt):
    """The kept tokens into their new pages; a page that loses nothing keeps its codes and scale."""
    B, Hkv, n = src.shape
    T, D = codes.shape[2:]
    page = state["table"].long().clamp_min(0).gather(1, (src // T).reshape(B, -1)).reshape(B, Hkv, n)
    head = torch.arange(Hkv, device="cuda")[:, None]
    have = codes.view(torch.uint8)[page, head, src % T].view(codes.dtype)
    x = torch.where(there[..., None], have.float() * scales[page, head][..., None], 0.0)
    s = (x.reshape(B, Hkv, n // T, T * D).abs().amax(3) / QMAX[fmt]).clamp_min(FLOOR)
    same = ((src == torch.arange(n, device="cuda")) | ~there).reshape(B, Hkv, n // T, T).all(3)
    s = torch.where(same, scales[page, head].reshape(B, Hkv, n // T, T)[..., 0], s)
    new = _code(x / s.repeat_interleave(T, 2)[..., None], fmt).view(torch.uint8)
    new = torch.where(same.repeat_interleave(T, 2)[..., None] & there[..., None], have.view(torch.uint8), new)
    new = new.reshape(B, Hkv, n // T, T, D).transpose(1, 2)
    # pages past the kept tokens stay as they are: the spare page takes what falls there
    filled = there.reshape(B, Hkv, n // T, T)[:, 0, :, 0]
    to = torch.where(filled, state["dst_table"].long(), codes.shape[0] - 1)
    codes.view(torch.uint8)[to] = new
    scales[to] = s.transpose(1, 2)


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "evict": _exact_evict}[case["op"]](case, st)


def _exact_attention(case, st):
    total, n = _lengths(case)
    Hq, Hkv, D, T = case["Hq"], case["Hkv"], case["D"], case["T"]
    G = Hq // Hkv
    rows = sum(n)
    out = torch.zeros(rows, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, Hq, dtype=torch.float64, device="cuda")
    w = st["w"].double() if case["weights"] else None
    r = 0
    for b in range(case["B"]):
        pages = st["table"][b, :-(-total[b] // T)].long()
        for h in range(Hkv):
            kh = st["k"].view(torch.uint8)[pages, h].view(st["k"].dtype).double() * st["ks"][pages, h].double()[:, None, None]
            vh = st["v"].view(torch.uint8)[pages, h].view(st["v"].dtype).double() * st["vs"][pages, h].double()[:, None, None]
            kh, vh = kh.reshape(-1, D)[:total[b]], vh.reshape(-1, D)[:total[b]]
            for g in range(G):
                q = st["qkv"][r:r + n[b], h * G + g].double()
                s = q @ kh.T / math.sqrt(D)
                ahead = torch.arange(total[b], device="cuda") > torch.arange(n[b], device="cuda")[:, None] + total[b] - n[b]
                s[ahead] = -math.inf
                lse[r:r + n[b], h * G + g] = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                out[r:r + n[b], h * G + g] = p @ vh
                if w is not None:
                    w[b, h, :total[b]] += p.sum(0)
        r += n[b]
    return [out, lse] + ([w] if w is not None else [])


def _round64(y, fmt):
    """y (64 bits) to the nearest number of the format, as 64 bits; ties to the even one."""
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _as_codes(x, fmt):
    return x.to(torch.int8) if fmt == "int8" else x


def _exact_append(case, st):
    total, n = _lengths(case)
    Hq, Hkv, T, fmt = case["Hq"], case["Hkv"], case["T"], case["fmt"]
    got = []
    for codes, scales, h0 in ((st["k"], st["ks"], Hq), (st["v"], st["vs"], Hq + Hkv)):
        c, s = codes.float().double(), scales.double()
        r = 0
        for b in range(case["B"]):
            old = total[b] - n[b]
            for j in range(old // T, -(-total[b] // T)):
                page = int(st["table"][b, j])
                lo, hi = max(old, j * T), min(total[b], (j + 1) * T)
                x = st["qkv"][r + lo - old:r + hi - old, h0:h0 + Hkv].double().transpose(0, 1)
                need = (x.abs().amax((1, 2)) / QMAX[fmt]).clamp_min(FLOOR)
                if lo > j * T:
                    was = s[page].clone()
                    need = torch.maximum(need, was)
                    head = c[page, :, :lo - j * T] * (was / need)[:, None, None]
                    c[page, :, :lo - j * T] = _round64(head, fmt)
                s[page] = need
                c[page, :, lo - j * T:hi - j * T] = _round64(x / need[:, None, None], fmt)
            r += n[b]
        got.append((_as_codes(c[:-1], fmt), s[:-1]))
    w = st["w"].double()
    for b in range(case["B"]):
        w[b, :, total[b] - n[b]:total[b]] = 0.0
    return [got[0][0], got[1][0], got[0][1], got[1][1], w]


def _exact_evict(case, st):
    total, _ = _lengths(case)
    B, Hkv, T, fmt, budget = case["B"], case["Hkv"], case["T"], case["fmt"], case["budget"]
    if B * Hkv * max(total) > 2 ** 21 or B * Hkv * budget // T > 2 ** 16:
        return None
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    w_out = torch.zeros(B, Hkv, budget, dtype=torch.float64)
    pools = [[st["k"].float().double(), st["ks"].double()], [st["v"].float().double(), st["vs"].double()]]
    w = st["w"].double().cpu()
    for b in range(B):
        count = min(total[b], budget)
        for h in range(Hkv):
            row = w[b, h].tolist()
            forced = [t for t in range(total[b]) if t < case["first"] or t >= total[b] - case["recent"]]
            held = set(forced[:count])
            rest = sorted((t for t in range(total[b]) if t not in held), key=lambda t: (-row[t], t))
            keep = sorted(list(held) + rest[:count - len(held)])
            kept[b, h, :count] = torch.tensor(keep, dtype=torch.int32)
            at = torch.tensor(keep)
            w_out[b, h, :count] = w[b, h, at]
            at = at.cuda()
            page = st["table"][b].long()[at // T]
            for pool, first in zip(pools, ((st["k"], st["ks"]), (st["v"], st["vs"]))):
                raw = first[0].view(torch.uint8)[page, h, at % T].view(first[0].dtype).double()
                scale = first[1][page, h].double()
                for j in range(-(-count // T)):
                    to = int(st["dst_table"][b, j])
                    part = slice(j * T, min(count, (j + 1) * T))
                    x = raw[part] * scale[part, None]
                    size = x.shape[0]
                    if keep[part.stop - 1] == part.stop - 1:
                        new, s = raw[part], scale[part][0]
                    else:
                        s = (x.abs().max() / QMAX[fmt]).clamp_min(FLOOR)
                        new = _round64(x / s, fmt)
                    pool[0][to, h, :size], pool[0][to, h, size:], pool[1][to, h] = new, 0.0, s
    counts = torch.tensor([min(t, budget) for t in total], dtype=torch.int32)
    return [_as_codes(pools[0][0][:-1], fmt), _as_codes(pools[1][0][:-1], fmt), pools[0][1][:-1], pools[1][1][:-1],
            kept, counts, w_out]
