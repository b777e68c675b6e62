"""Timing cases of the serving operators around the paged KV cache: rotary positions, appending to
the cache, attention over a cache held in 8 bits with block scales, and attention over packed prompts.

Each operator has two forms here that take the same inputs.  With ``own`` false ``run`` computes it
from elementary torch operations in 32 bits (64 for the rotation angles), rounded once at the end;
with ``own`` true it makes the library calls a serving program makes.  ``exact`` gives the results
from the definitions in 64 bits."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3, I8, BF16 = "e4m3", "i8", "bf16"
QMAX = {E4M3: 448.0, I8: 127.0}
CODES = {E4M3: torch.float8_e4m3fn, I8: torch.int8}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a 64-request batch, far into a long context, frequencies stretched by 8
        dict(name="rope_step", op="rope", tokens=64, hq=64, hk=8, d=128, rope=128, layout="halves", theta=500000.0,
             factor=8.0, far=131072, fused=False),
        # a prompt batch of 16384 tokens
        dict(name="rope_prompt", op="rope", tokens=16384, hq=32, hk=8, d=128, rope=128, layout="interleaved",
             theta=10000.0, factor=1.0, far=16384, fused=False),
        # a quarter-ish of the head rotated, q and k read as slices of one fused projection, odd count
        dict(name="rope_partial", op="rope", tokens=2047, hq=8, hk=2, d=64, rope=32, layout="halves", theta=10000.0,
             factor=1.0, far=4096, fused=True),
        # one decode step: 64 requests append one token each to an 8-bit cache; q is rotated on the way
        dict(name="append_step_e4m3", op="append", requests=64, new_lo=1, new_hi=1, len_lo=1, len_hi=512, hq=64, hk=8,
             d=128, page=16, block=16, cache=E4M3, rope=128, layout="halves", theta=10000.0, lens=11),
        # ragged prompts written to an 8-bit cache with one scale per 64-token page and head
        dict(name="append_prompts_e4m3", op="append", requests=16, new_lo=100, new_hi=2000, len_lo=0, len_hi=100, hq=0,
             hk=8, d=128, page=64, block=64, cache=E4M3, rope=128, layout="interleaved", theta=10000.0, lens=12),
        # prompts and single tokens mixed, bf16 cache, small heads
        dict(name="append_mixed_bf16", op="append", requests=37, new_lo=1, new_hi=300, len_lo=0, len_hi=700, hq=8, hk=2,
             d=64, page=16, block=0, cache=BF16, rope=64, layout="halves", theta=10000.0, lens=13),
        # a few short requests: latency
        dict(name="decode_short_i8", op="decode", requests=4, len_lo=37, len_hi=256, q_len=1, causal=False, hq=8, hk=2,
             d=64, page=16, block=16, cache=I8, lens=21),
        # 64-request decode of the 64/8-head shape
        dict(name="decode_batch_e4m3", op="decode", requests=64, len_lo=1024, len_hi=8192, q_len=1, causal=False, hq=64,
             hk=8, d=128, page=16, block=16, cache=E4M3, lens=22),
        # drafted tokens verified together: 4 query tokens per request, causal among themselves
        dict(name="verify_long_i8", op="decode", requests=16, len_lo=1000, len_hi=16384, q_len=4, causal=True, hq=32,
             hk=8, d=128, page=64, block=64, cache=I8, lens=23),
        # a few short prompts: latency
        dict(name="prompt_short", op="prompt", requests=4, q_lo=37, q_hi=256, past=0, hq=8, hk=2, d=64, causal=True,
             lens=31),
        # ragged prompts packed back to back
        dict(name="prompt_ragged", op="prompt", requests=16, q_lo=64, q_hi=2048, past=0, hq=32, hk=8, d=128, causal=True,
             lens=32),
        # the last 4096 tokens of a 16384-token prompt taken in chunks
        dict(name="prompt_chunk", op="prompt", requests=1, q_lo=4096, q_hi=4096, past=12288, hq=32, hk=8, d=128,
             causal=True, lens=33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "prompt"])
    heads = rng.choice([(8, 2), (16, 2), (32, 8), (64, 8), (12, 4), (8, 8), (5, 1)])
    d, layout = rng.choice([64, 128]), rng.choice(["halves", "interleaved"])
    lens = rng.randrange(1 << 20)
    c = dict(op=op, hq=heads[0], hk=heads[1], d=d)
    if op == "rope":
        return dict(c, tokens=_log(rng, 1, 8192), rope=rng.choice([d, d // 2, 48]), layout=layout,
                    theta=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 8.0]),
                    far=_log(rng, 10, 1 << 20), fused=rng.random() < 0.5)
    if op == "append":
        page, cache = rng.choice([16, 32, 64]), rng.choice([E4M3, BF16])
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, 6000 // n)
        return dict(c, hq=rng.choice([0, heads[0]]), requests=n, new_lo=1, new_hi=hi, len_lo=0,
                    len_hi=_log(rng, 1, 600), page=page, block=0 if cache == BF16 else rng.choice([16, page]),
                    cache=cache, rope=rng.choice([0, d, d // 2]), layout=layout, theta=10000.0, lens=lens)
    if op == "decode":
        page = rng.choice([16, 32, 64])
        n, hi = _log(rng, 1, 64), _log(rng, 16, 8192)
        return dict(c, requests=n, len_lo=max(1, hi // 8), len_hi=hi, q_len=rng.choice([1, 1, 2, 4]), causal=True,
                    page=page, block=rng.choice([16, page]), cache=rng.choice([E4M3, I8]), lens=lens)
    hi, past = _log(rng, 1, 2048), rng.choice([0, 0, _log(rng, 1, 2048)])
    most = max(1, (1 << 31) // (hi * (hi + past) * heads[0]))
    return dict(c, requests=_log(rng, 1, min(16, most)), q_lo=max(1, hi // 16), q_hi=hi, past=past,
                causal=rng.random() < 0.8, lens=lens)


def _lengths(case, lo, hi, count, salt=0):
    r = random.Random(case["lens"] * 7 + salt)
    out = [r.randint(lo, hi) for _ in range(count)]
    if count > 1:
        out[0], out[1] = lo, hi
    return out


def _append_lens(case):
    old = _lengths(case, case["len_lo"], case["len_hi"], case["requests"], 1)
    new = _lengths(case, case["new_lo"], case["new_hi"], case["requests"], 2)
    return old[::-1], new


def _prompt_lens(case):
    q = _lengths(case, case["q_lo"], case["q_hi"], case["requests"])
    return q, [n + case["past"] for n in q]


def work(case):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": 4 * t * (hq + hk) * d + 4 * t, "flops": 3 * t * (hq + hk) * case["rope"]}
    if case["op"] == "append":
        old, new = _append_lens(case)
        t = sum(new)
        size = 2 if case["cache"] == BF16 else 1
        scales = 0 if not case["block"] else sum(-(-(o + n) // case["block"]) - o // case["block"]
                                                 for o, n in zip(old, new)) * hk * 8
        return {"bytes": t * (2 * hk * d * (2 + size) + hq * d * 4) + scales, "flops": 3 * t * (hq + hk) * case["rope"]}
    if case["op"] == "decode":
        lens = _lengths(case, case["len_lo"], case["len_hi"], case["requests"])
        rows = case["requests"] * case["q_len"] * hq
        blocks = sum(-(-n // case["block"]) for n in lens)
        return {"bytes": 2 * sum(lens) * hk * d + blocks * hk * 8 + rows * (4 * d + 4),
                "flops": 4 * d * hq * case["q_len"] * sum(lens)}
    q, kv = _prompt_lens(case)
    pairs = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(q, kv))
    return {"bytes": sum(q) * hq * (4 * d + 4) + 4 * sum(kv) * hk * d, "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------------------- inputs
def _i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device=DEV)


def _inv_freq(case):
    half = case["rope"] // 2
    return np.array([case["theta"] ** (-i / half) / case.get("factor", 1.0) for i in range(half)])


def _pages(lens, page, gen):
    """Host page-table shape of requests of these lengths, and their page ids in a seeded order."""
    n = [-(-x // page) for x in lens]
    indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    last = np.array([x - (k - 1) * page if k else 1 for x, k in zip(lens, n)], dtype=np.int32)
    total = int(indptr[-1]) + 3
    ids = torch.randperm(total, generator=gen, device=DEV)[:int(indptr[-1])].to(torch.int32)
    return indptr, last, ids, total


def _quantised(case, pages, gen):
    """An 8-bit cache as earlier appends left it: codes, and one scale for each block and head."""
    shape = (pages, case["page"] // case["block"], case["block"], case["hk"], case["d"])
    x = torch.randn(shape, generator=gen, device=DEV) * (
        0.5 + torch.rand(shape[0], shape[1], 1, shape[3], 1, generator=gen, device=DEV))
    scale = x.abs().amax(dim=(2, 4)) / QMAX[case["cache"]]
    y = x / scale[:, :, None, :, None]
    y = y.round().clamp(-127, 127) if case["cache"] == I8 else y.clamp(-448, 448)
    return y.to(CODES[case["cache"]]).reshape(pages, case["page"], case["hk"], case["d"]), scale.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    hq, hk, d = case["hq"], case["hk"], case["d"]
    s = {"case": case}
    if case["op"] == "rope":
        t = case["tokens"]
        if case["fused"]:
            qkv = rand(t, hq + 2 * hk, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            s["q"], s["k"] = rand(t, hq, d), rand(t, hk, d)
        s["positions"] = torch.randint(0, case["far"], (t,), generator=gen, device=DEV, dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case)
    elif case["op"] == "append":
        old, new = _append_lens(case)
        after = [a + b for a, b in zip(old, new)]
        s["kv_indptr_h"], s["last_h"], s["kv_indices"], pages = _pages(after, case["page"], gen)
        s["append_indptr_h"] = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["kv_indptr"], s["last"] = _i32(s["kv_indptr_h"]), _i32(s["last_h"])
        s["append_indptr"] = _i32(s["append_indptr_h"])
        t = sum(new)
        s["k"], s["v"] = rand(t, hk, d), rand(t, hk, d)
        s["q"] = rand(t, hq, d) if hq else None
        if case["cache"] == BF16:
            s["k_cache"], s["v_cache"] = (rand(pages, case["page"], hk, d) for _ in range(2))
            s["k_scale"] = s["v_scale"] = None
        else:
            s["k_cache"], s["k_scale"] = _quantised(case, pages, gen)
            s["v_cache"], s["v_scale"] = _quantised(case, pages, gen)
        s["inv_freq"] = _inv_freq(case) if case["rope"] else None
    elif case["op"] == "decode":
        lens = _lengths(case, case["len_lo"], case["len_hi"], case["requests"])
        s["kv_indptr_h"], s["last_h"], s["kv_indices"], pages = _pages(lens, case["page"], gen)
        s["kv_indptr"], s["last"] = _i32(s["kv_indptr_h"]), _i32(s["last_h"])
        s["qo_indptr_h"] = (np.arange(len(lens) + 1) * case["q_len"]).astype(np.int32)
        s["lens"] = _i32(lens)
        s["q"] = rand(len(lens) * case["q_len"], hq, d)
        s["k_cache"], s["k_scale"] = _quantised(case, pages, gen)
        s["v_cache"], s["v_scale"] = _quantised(case, pages, gen)
        if own:  # a step plans once for all its layers
            import split_kv_merge_b200 as skv
            s["plan"] = skv.plan_paged_scaled(s["qo_indptr_h"], s["kv_indptr_h"], s["last_h"], case["page"], hq, hk, d,
                                              causal=case["causal"]).to(DEV)
    else:
        q, kv = _prompt_lens(case)
        s["qo_indptr_h"] = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        s["kv_indptr_h"] = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)
        s["qo_indptr"], s["kv_indptr"] = _i32(s["qo_indptr_h"]), _i32(s["kv_indptr_h"])
        s["q"], s["k"], s["v"] = rand(sum(q), hq, d), rand(sum(kv), hk, d), rand(sum(kv), hk, d)
        if own:
            import split_kv_merge_b200 as skv
            s["plan"] = skv.plan_prompt(s["qo_indptr_h"], s["kv_indptr_h"], hq, hk, d, causal=case["causal"]).to(DEV)
    return s


# ---------------------------------------------------------------------------------- plain forms
def _rotate(x, positions, inv_freq, layout):
    """x [T, H, D] in 32 bits, its first 2 * len(inv_freq) values turned by position * inv_freq."""
    r = 2 * len(inv_freq)
    angle = positions.double()[:, None] * torch.tensor(inv_freq, device=DEV)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    if layout == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., r:]], dim=-1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2), x[..., r:]], dim=-1)


def _rope_plain(s):
    c = s["case"]
    return tuple(_rotate(s[n], s["positions"], s["inv_freq"], c["layout"]).to(torch.bfloat16) for n in ("q", "k"))


def _quantise_blocks(x, cache, scale, at_page, at_slot, old, case):
    """New rows x [T, H, D] into their blocks: the block's scale grows to hold them, the codes that
    were there are written again where it grew."""
    bt, page = case["block"], case["page"]
    nb = page // bt
    key = at_page * nb + at_slot // bt                                       # block of each new token
    amax = torch.zeros(cache.shape[0] * nb, cache.shape[2], device=DEV)
    amax.scatter_reduce_(0, key[:, None].expand(-1, cache.shape[2]), x.abs().amax(-1), "amax")
    touched = torch.unique(key)
    flat = scale.view(-1, cache.shape[2])
    kept = torch.zeros(flat.shape[0], dtype=torch.bool, device=DEV)          # holds tokens of before
    kept[key[old]] = True
    before = torch.where(kept[:, None], flat, 0.0)[touched]
    after = torch.maximum(before, amax[touched] / QMAX[case["cache"]])
    codes = cache.view(-1, bt, *cache.shape[2:])
    was = codes[touched].float() * before[:, None, :, None]
    again = _encode(was, after[:, None, :, None], case["cache"])
    grew = (kept[touched][:, None] & (after > before))[:, None, :, None]
    raw = codes.view(torch.uint8)
    raw[touched] = torch.where(grew, again.view(torch.uint8), raw[touched])
    flat[touched] = after
    raw_rows = cache.view(torch.uint8)
    raw_rows[at_page, at_slot] = _encode(x, flat[key][..., None], case["cache"]).view(torch.uint8)


def _encode(x, scale, cache):
    y = torch.where(scale > 0, x / scale, 0.0)
    y = y.round().clamp(-127, 127) if cache == I8 else y.clamp(-448, 448)
    return y.to(CODES[cache])


def _append_places(s):
    """Position, page and slot of every new token, and whether its block holds tokens of before."""
    c = s["case"]
    ip = s["append_indptr"].long()
    t = s["k"].shape[0]
    row = torch.arange(t, device=DEV)
    req = torch.searchsorted(ip, row, right=True) - 1
    n_pages = (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).long()
    length = (n_pages - 1) * c["page"] + s["last"].long()
    first = length - (ip[1:] - ip[:-1])
    pos = first[req] + row - ip[req]
    page = s["kv_indices"][s["kv_indptr"].long()[req] + pos // c["page"]].long()
    # a block holds earlier tokens where its first position is before the request's first new one
    block = c["block"] or 1
    kept = (first[req] // block == pos // block) & (first[req] % block > 0)
    return pos, page, pos % c["page"], kept


def _append_plain(s):
    c = s["case"]
    pos, page, slot, kept = _append_places(s)
    turn = lambda x: _rotate(x, pos, s["inv_freq"], c["layout"]) if c["rope"] else x.float()  # noqa: E731
    k, v = turn(s["k"]), s["v"].float()
    if c["cache"] == BF16:
        s["k_cache"][page, slot] = k.to(torch.bfloat16)
        s["v_cache"][page, slot] = v.to(torch.bfloat16)
    else:
        _quantise_blocks(k, s["k_cache"], s["k_scale"], page, slot, kept, c)
        _quantise_blocks(v, s["v_cache"], s["v_scale"], page, slot, kept, c)
    return [turn(s["q"]).to(torch.bfloat16) if s["q"] is not None else None, s["k_cache"], s["v_cache"], s["k_scale"],
            s["v_scale"]]


def _softmax_attend(scores, seen, values):
    """scores [..., q, k] in 32 bits (overwritten), seen the keys each row has, values [..., k, d]."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = scores.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, values) / torch.where(total > 0, total, 1.0)
    return o, (top + total.log()).squeeze(-1)


def _decode_plain(s):
    c = s["case"]
    hq, hk, d, bt, n, ql = c["hq"], c["hk"], c["d"], c["block"], c["requests"], c["q_len"]
    lens = s["lens"].long()
    t = torch.arange(c["len_hi"], device=DEV)
    at = s["kv_indptr"].long()[:-1, None] + torch.minimum(t[None], (lens - 1)[:, None]) // c["page"]
    page, slot = s["kv_indices"].long()[at], (t % c["page"])[None].expand(n, -1)

    def rows(codes, scale):  # [n, Hk, L, D]
        x = codes.view(torch.uint8)[page, slot].view(codes.dtype).float() * scale[page, slot // bt][..., None]
        return torch.where((t[None] < lens[:, None])[..., None, None], x, 0.0).transpose(1, 2)

    q = s["q"].float().view(n, ql, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    scores = torch.matmul(q, rows(s["k_cache"], s["k_scale"]).transpose(-1, -2)) * d ** -0.5
    limit = lens[:, None] - (torch.arange(ql - 1, -1, -1, device=DEV) if c["causal"] else torch.zeros(ql, device=DEV, dtype=torch.long))
    seen = (t < limit[..., None]).repeat(1, hq // hk, 1)[:, None]             # rows are (group head, query token)
    o, lse = _softmax_attend(scores, seen, rows(s["v_cache"], s["v_scale"]))
    o = o.view(n, hk, hq // hk, ql, d).permute(0, 3, 1, 2, 4).reshape(n * ql, hq, d)
    lse = lse.view(n, hk, hq // hk, ql).permute(0, 3, 1, 2).reshape(n * ql, hq)
    return o.to(torch.bfloat16), lse


def _prompt_plain(s):
    c = s["case"]
    hq, hk, d, n = c["hq"], c["hk"], c["d"], c["requests"]
    qi, ki = s["qo_indptr"].long(), s["kv_indptr"].long()
    ql, kl = (qi[1:] - qi[:-1])[:, None], (ki[1:] - ki[:-1])[:, None]
    i, t = torch.arange(c["q_hi"], device=DEV), torch.arange(c["q_hi"] + c["past"], device=DEV)
    pad = lambda x, ip, length, at: torch.where(  # noqa: E731  packed [T, H, D] -> [n, H, len, D]
        (at < length)[..., None, None], x[torch.minimum(ip[:-1, None] + at, ip[-1] - 1)].float(), 0.0).transpose(1, 2)
    q = pad(s["q"], qi, ql, i).reshape(n, hk, -1, d)                          # rows (group head, query token)
    k, v = pad(s["k"], ki, kl, t), pad(s["v"], ki, kl, t)
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).view(n, hk, hq // hk, c["q_hi"], -1)
    limit = (kl - ql + i + 1) if c["causal"] else kl.expand(-1, c["q_hi"])
    seen = (t < torch.minimum(limit, kl)[..., None])[:, None, None]
    o, lse = _softmax_attend(scores, seen, v[:, :, None])
    row = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(qi, row, right=True) - 1
    o = o.reshape(n, hq, c["q_hi"], d)[r, :, row - qi[r]]
    return o.to(torch.bfloat16), lse.reshape(n, hq, c["q_hi"])[r, :, row - qi[r]]


# ------------------------------------------------------------------------------- library calls
def _rope_own(s):
    import split_kv_merge_b200 as skv
    c = s["case"]
    return skv.rope_apply(s["q"], s["k"], s["positions"], rope_dim=c["rope"], rope_layout=c["layout"],
                          inv_freq=s["inv_freq"])


def _append_own(s):
    import split_kv_merge_b200 as skv
    c = s["case"]
    q = skv.paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["append_indptr"], s["kv_indptr"],
                            s["kv_indices"], s["last"], k_scale=s["k_scale"], v_scale=s["v_scale"], q=s["q"],
                            rope_dim=c["rope"], rope_layout=c["layout"], inv_freq=s["inv_freq"])
    return [q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _decode_own(s):
    import split_kv_merge_b200 as skv
    o, lse, _ = skv.paged_attention_scaled(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                           s["qo_indptr_h"], s["kv_indptr_h"], s["kv_indices"], s["last_h"],
                                           causal=s["case"]["causal"], kv_indptr=s["kv_indptr"],
                                           kv_last_page_len=s["last"], plan=s["plan"], o_dtype=torch.bfloat16)
    return o, lse


def _prompt_own(s):
    import split_kv_merge_b200 as skv
    o, lse, _ = skv.prompt_attention(s["q"], s["k"], s["v"], s["qo_indptr_h"], s["kv_indptr_h"],
                                     causal=s["case"]["causal"], plan=s["plan"], o_dtype=torch.bfloat16)
    return o, lse


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _rope_own, "append": _append_own, "decode": _decode_own, "prompt": _prompt_own}[op](state)
    return {"rope": _rope_plain, "append": _append_plain, "decode": _decode_plain, "prompt": _prompt_plain}[op](state)


# ------------------------------------------------------------------------------ 64-bit results
def _turned(x, positions, inv_freq, layout):
    """Pair p of a row as a complex number, times e^(i position inv_freq[p])."""
    out = x.double().clone()
    half = len(inv_freq)
    first = [p if layout == "halves" else 2 * p for p in range(half)]
    second = [p + half if layout == "halves" else 2 * p + 1 for p in range(half)]
    turn = torch.polar(torch.ones(len(positions), half, dtype=torch.double, device=DEV),
                       positions.double()[:, None] * torch.tensor(inv_freq, device=DEV))[:, None]
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _attend(q, k, v, limits, scale):
    """One head's rows [q, d] over keys [k, d]; row i has the first limits[i] of them."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.double, device=DEV)
    x = (q @ k.T) * scale
    x = torch.where(torch.arange(k.shape[0], device=DEV)[None] < limits[:, None], x, -math.inf)
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "rope":
        return tuple(_turned(s[n], s["positions"], s["inv_freq"], case["layout"]) for n in ("q", "k"))
    if case["op"] == "append":
        ip, ki = s["append_indptr_h"], s["kv_indptr_h"]
        pos = np.concatenate([np.arange(n) for n in np.diff(ip)] or [[]])
        olds = []
        for r in range(case["requests"]):
            total = (ki[r + 1] - ki[r] - 1) * case["page"] + s["last_h"][r]
            olds.append(int(total - (ip[r + 1] - ip[r])))
            pos[ip[r]:ip[r + 1]] += olds[r]
        at = torch.tensor(pos.astype(np.int64), device=DEV)
        turn = lambda x: _turned(x, at, s["inv_freq"], case["layout"]) if case["rope"] else x.double()  # noqa: E731
        new = {"k": turn(s["k"]), "v": s["v"].double()}
        out = [turn(s["q"]) if s["q"] is not None else None]
        ids = s["kv_indices"].cpu().numpy()
        scales = [None, None]
        for n, (name, x) in enumerate(new.items()):
            cache, scale = s[name + "_cache"].double(), s[name + "_scale"]
            if scale is not None:
                scale = scales[n] = scale.double()
            for r in range(case["requests"]):
                step = case["block"] or case["page"]
                t = olds[r]
                while t < olds[r] + ip[r + 1] - ip[r]:
                    start = t // step * step
                    end = min(start + step, olds[r] + int(ip[r + 1] - ip[r]))
                    page, slot = ids[ki[r] + t // case["page"]], start % case["page"]
                    rows = x[ip[r] + t - olds[r]:ip[r] + end - olds[r]]
                    if scale is None:
                        cache[page, slot + t - start:slot + end - start] = rows
                    else:
                        b = slot // step
                        want = rows.abs().amax(dim=(0, 2)) / QMAX[case["cache"]]
                        if t > start:
                            want = torch.maximum(want, scale[page, b])
                            cache[page, slot:slot + t - start] *= (scale[page, b] / want)[:, None]
                        scale[page, b] = want
                        cache[page, slot + t - start:slot + end - start] = rows / want[:, None]
                    t = end
            out.append(cache)
        return out + scales
    if case["op"] == "decode":
        ki, ids = s["kv_indptr_h"], s["kv_indices"].long()
        ql = case["q_len"]
        o = torch.empty(s["q"].shape[0], hq, d, dtype=torch.double, device=DEV)
        lse = torch.empty(s["q"].shape[0], hq, dtype=torch.double, device=DEV)
        for r, length in enumerate(s["lens"].tolist()):
            pages = ids[int(ki[r]):int(ki[r + 1])]
            k, v = ((s[n + "_cache"].view(torch.uint8)[pages].view(s[n + "_cache"].dtype).double() * s[n + "_scale"][pages]
                     .double().repeat_interleave(case["block"], dim=1)[..., None]).flatten(0, 1)[:length] for n in "kv")
            limits = torch.arange(length - ql + 1, length + 1, device=DEV) if case["causal"] else torch.full((ql,), length, device=DEV)
            for h in range(hq):
                rows = slice(r * ql, (r + 1) * ql)
                kh = h // (hq // hk)
                o[rows, h], lse[rows, h] = _attend(s["q"][rows, h].double(), k[:, kh], v[:, kh], limits, d ** -0.5)
        return o, lse
    qi, ki = s["qo_indptr_h"], s["kv_indptr_h"]
    o = torch.empty(s["q"].shape[0], hq, d, dtype=torch.double, device=DEV)
    lse = torch.empty(s["q"].shape[0], hq, dtype=torch.double, device=DEV)
    for r in range(case["requests"]):
        rows, keys = slice(int(qi[r]), int(qi[r + 1])), slice(int(ki[r]), int(ki[r + 1]))
        n, m = rows.stop - rows.start, keys.stop - keys.start
        limits = torch.arange(m - n + 1, m + 1, device=DEV) if case["causal"] else torch.full((n,), m, device=DEV)
        for h in range(hq):
            kh = h // (hq // hk)
            o[rows, h], lse[rows, h] = _attend(s["q"][rows, h].double(), s["k"][keys, kh].double(),
                                               s["v"][keys, kh].double(), limits, d ** -0.5)
    return o, lse
