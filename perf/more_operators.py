"""Cases, plain forms and 64-bit values of what a serving loop does around the paged caches.

Three operators.  Attention in a sliding window with a few first tokens that stay visible
(``packed_window_attention`` over prompts, ``paged_window_attention`` over the caches);
attention of a batch whose sequences share a prefix (``paged_prefix_attention``); and the
paging itself (``kv_cache_extend``, ``kv_cache_slots``, ``kv_cache_truncate``): pages taken
from a free list and given back, block tables and slot maps from the requests' lengths.

``own`` chooses what ``run`` does: the plain torch form (false) or the calls of this
repository's library (true).
"""
import math
import random

import torch

own = False

WORKSPACE_BYTES = 64 << 20       # what the window attention calls are content with
SCORES = 1 << 30                 # score elements that the plain form holds at a time
EXACT_FLOPS = 3e12               # beyond this the 64-bit value takes too long

HALF = {"bf16": torch.bfloat16, "fp16": torch.float16}
STORED = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, **HALF}
SIZE = {"bf16": 2, "fp16": 2, "int8": 1, "e4m3": 1, "e5m2": 1}


# ---------------------------------------------------------------- cases
def _packed(name, B, q, nq, nkv, d, window, sinks, ragged, dtype="bf16", layout="BSD"):
    """B prompts of q tokens in all."""
    return {"op": "packed", "name": name, "B": B, "q": q, "nq": nq, "nkv": nkv, "d": d, "window": window,
            "sinks": sinks, "ragged": ragged, "dtype": dtype, "layout": layout}


def _paged(name, variant, B, N, heads, Dkv, Dv, R, mode, bs, ctx, new, window, sinks, kt, vt, dtype="bf16", ragged=True):
    """B sequences of up to ctx cached tokens, the last up to `new` of them attending."""
    return {"op": "paged", "name": name, "variant": variant, "B": B, "N": N, "heads": heads, "Dkv": Dkv, "Dv": Dv,
            "R": R, "mode": mode, "bs": bs, "ctx": ctx, "new": new, "window": window, "sinks": sinks, "kt": kt, "vt": vt,
            "dtype": dtype, "ragged": ragged}


def _prefix(name, variant, B, N, heads, Dkv, Dv, R, mode, bs, prefix, ctx, new, kt, vt, dtype="bf16", ragged=True):
    """B sequences behind `prefix` shared tokens, each with up to ctx tokens of its own, the
    last up to `new` of them attending."""
    return {"op": "prefix", "name": name, "variant": variant, "B": B, "N": N, "heads": heads, "Dkv": Dkv, "Dv": Dv,
            "R": R, "mode": mode, "bs": bs, "prefix": prefix, "ctx": ctx, "new": new, "kt": kt, "vt": vt, "dtype": dtype,
            "ragged": ragged}


def _paging(name, op, B, bs, ctx, new, short=False):
    """B requests of up to ctx cached tokens: extended by up to `new`, their slots of all ctx
    listed, or cut back by up to `new`.  short: the free list does not last for all."""
    return {"op": op, "name": name, "B": B, "bs": bs, "ctx": ctx, "new": new, "short": short}


def listed():
    return [
        # two heads of 64, 128 tokens: latency of one call
        _packed("window_prompt_tiny", 1, 128, 2, 2, 64, 32, 4, False),
        # packed prompts of different lengths, grouped heads: a language model's prefill
        _packed("window_prompt_packed", 7, 9001, 32, 8, 128, 1024, 4, True),
        # one long document
        _packed("window_prompt_long", 1, 16411, 32, 8, 128, 4096, 4, False),
        # one token for each of 8 long sequences, V2 int8 cache: a decode step
        _paged("window_decode_v2_int8", 2, 8, 8, 64, 192, 128, 64, "PA_BNSD", 128, 32768, 1, 4096, 64, "int8", "int8"),
        # chunked prefill over long contexts, 16-bit cache
        _paged("window_chunk_v2", 2, 4, 8, 32, 192, 128, 64, "PA_BNSD", 128, 16384, 512, 2048, 16, "bf16", "bf16"),
        # a decode step of 32 sequences behind one long system prompt, V2 int8 cache
        _prefix("prefix_decode_v2_int8", 2, 32, 8, 64, 192, 128, 64, "PA_BNSD", 128, 8192, 512, 1, "int8", "int8"),
        # the same over the MLA latent, 16 query heads (a shard of 128)
        _prefix("prefix_decode_mla", 1, 32, 1, 16, 576, 512, 64, "PA_BNSD", 128, 16384, 256, 1, "bf16", "bf16"),
        # two short chats, a few tokens each: latency
        _prefix("prefix_short", 2, 2, 2, 8, 192, 128, 64, "PA", 16, 501, 40, 4, "bf16", "bf16"),
        # a decode step's bookkeeping: a token more for each of 256 requests
        _paging("extend_decode", "extend", 256, 16, 4096, 1),
        # prompts arriving: some 33,000 tokens for 16 requests
        _paging("extend_prompts", "extend", 16, 128, 2000, 4099),
        # the slots of whole contexts, for reading a cache back
        _paging("slots_contexts", "slots", 32, 128, 4096, 0),
        # requests rolled back or ended, their pages returned
        _paging("truncate", "truncate", 300, 32, 5000, 5000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["packed", "packed", "paged", "paged", "paged", "prefix", "prefix", "prefix", "extend", "slots", "truncate"])
    while True:
        sinks = rng.choice([0, 1, 4, 4, 16, 64, 100, 130, 500])
        if kind == "packed":
            B = rng.choice([1, 1, 2, 3, 5, 8, 17])
            nkv = rng.choice([1, 2, 4, 5, 8])
            case = _packed("", B, B * _log_int(rng, 1, 12000 // B), nkv * rng.choice([1, 1, 2, 4, 7, 8]), nkv,
                           rng.choice([64, 128, 128, 80, 96, 16, 112]), _log_int(rng, 1, 6000), sinks, rng.random() < 0.6,
                           rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["BSD", "BSD", "NBSD"]))
        elif kind in ("paged", "prefix"):
            variant = rng.choice([1, 2, 2])
            kt, vt = rng.choice(["int8", "bf16", "e4m3", "e5m2"]), rng.choice(["int8", "bf16", "e4m3"])
            kt, vt = (kt, kt) if rng.random() < 0.7 else (kt, vt)
            N = 1 if variant == 1 else rng.choice([1, 2, 4, 8])
            Dkv, Dv, R = (576, 512, 64) if variant == 1 else rng.choice([(192, 128, 64), (128, 128, 64), (64, 64, 32), (96, 80, 32)])
            heads = N * (rng.choice([16, 32, 64, 128, 5]) if variant == 1 else rng.choice([1, 2, 4, 8, 16, 3]))
            B, bs = rng.choice([1, 1, 2, 4, 7, 16, 32, 61]), rng.choice([32, 64, 96, 128, 256])
            new = 1 if rng.random() < 0.5 else _log_int(rng, 1, 700)
            if kind == "paged":
                mode = rng.choice(["PA", "PA_BNSD", "PA_BNSD"] + (["Norm"] if variant == 2 else []))
                case = _paged("", variant, B, N, heads, Dkv, Dv, R, mode, bs, _log_int(rng, 1, 40000), new,
                              _log_int(rng, 1, 9000), sinks, kt, vt, ragged=rng.random() < 0.7)
            else:
                case = _prefix("", variant, B, N, heads, Dkv, Dv, R, rng.choice(["PA", "PA_BNSD"]), bs,
                               _log_int(rng, 1, 20000), _log_int(rng, 1, 3000), new, kt, vt, ragged=rng.random() < 0.7)
        else:
            case = _paging("", kind, _log_int(rng, 1, 3000), rng.choice([16, 32, 64, 128, 48]), _log_int(rng, 1, 9000),
                           1 if rng.random() < 0.3 else _log_int(rng, 1, 5000), rng.random() < 0.2)
        del case["name"]
        w = work(case)
        if w["flops"] <= 9e11 and w["bytes"] <= 3e8 and _memory(case) <= 16e9:
            return case


def _memory(case):
    """Bytes of the largest score tensor's batch in the plain form."""
    if case["op"] not in ("packed", "paged", "prefix"):
        return 0
    lq, lk = _lengths(case)
    if case["op"] == "packed":
        return 4.0 * case["nq"] // case["nkv"] * len(lq) * max(lq) * max(lk)
    g = case["heads"] // case["N"]
    if case["op"] == "paged":
        return 4.0 * g * len(lq) * max(lq) * min(max(lk), case["sinks"] + case["window"] + max(lq))
    return 4.0 * g * len(lq) * max(lq) * (case["prefix"] + max(lk))


# ---------------------------------------------------------------- lengths and work
def _split(rng, total, n):
    """n lengths that add up to total, of very different sizes."""
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _lengths(case):
    """(query tokens, key tokens) of each sequence, from the case alone; of the paging calls
    (tokens more, or less; tokens held)."""
    rng = random.Random("%(op)s %(B)d" % case + " %d" % (case.get("q") or case["ctx"]))
    B = case["B"]
    if case["op"] == "packed":
        lq = _split(rng, case["q"], B) if case["ragged"] else [case["q"] // B] * B
        return lq, lq
    if case["op"] in ("paged", "prefix"):
        ctx, new = case["ctx"], min(case["new"], case["ctx"])
        if not case["ragged"]:
            return [new] * B, [ctx] * B
        lk = [ctx if b == 0 else rng.randint(max(1, ctx // 4), ctx) for b in range(B)]
        return [min(k, new if b == 0 else rng.randint((new + 1) // 2, new)) for b, k in enumerate(lk)], lk
    held = [rng.randint(0, case["ctx"]) for _ in range(B)]
    if case["op"] == "slots":
        return [0] * B, held
    if case["op"] == "truncate":
        return [rng.choice([h, rng.randint(0, min(h, case["new"]))]) for h in held], held
    return [case["new"] if case["new"] == 1 else rng.randint(0, case["new"]) for _ in range(B)], held


def _pages(n, bs):
    return -(-n // bs)


def _window_pairs(a, n, window, sinks):
    """Visible (query, key) pairs of the last a of n positions (queries before position 0 see none)."""
    p = torch.arange(n - a, n, dtype=torch.int64).clamp_(min=-1) + 1     # keys up to the query's own
    return int((p.clamp(max=window) + (p - window).clamp(min=0, max=sinks)).sum())


def _window_rows(a, n, window, sinks):
    """Positions that some of the last a of n positions sees."""
    lo = max(0, n - a - window + 1)
    return n - lo + min(sinks, lo)


def work(case):
    op = case["op"]
    lq, lk = _lengths(case)
    if op == "packed":
        d, pairs = case["d"], sum(_window_pairs(a, n, case["window"], case["sinks"]) for a, n in zip(lq, lk))
        return {"bytes": 2 * d * (2 * sum(lq) * case["nq"] + 2 * sum(lk) * case["nkv"]), "flops": 4 * d * case["nq"] * pairs}
    if op in ("paged", "prefix"):
        kw, vw = (case["R"], case["Dv"]) if case["variant"] == 1 else (case["Dkv"], case["Dv"])
        if op == "paged":
            rows = sum(_window_rows(a, n, case["window"], case["sinks"]) for a, n in zip(lq, lk))
            pairs = sum(_window_pairs(a, n, case["window"], case["sinks"]) for a, n in zip(lq, lk))
        else:
            rows = case["prefix"] + sum(lk)
            pairs = case["prefix"] * sum(lq) + sum(_window_pairs(a, n, n, 0) for a, n in zip(lq, lk))
        return {"bytes": rows * case["N"] * (kw * SIZE[case["kt"]] + vw * SIZE[case["vt"]])
                + 2 * sum(lq) * case["heads"] * (case["Dkv"] + case["Dv"]),
                "flops": 2 * (case["Dkv"] + case["Dv"]) * case["heads"] * pairs}
    B, bs = case["B"], case["bs"]
    if op == "extend":
        taken = sum(_pages(h + n, bs) - _pages(h, bs) for n, h in zip(lq, lk))
        return {"bytes": 8 * sum(lq) + 8 * taken + 16 * B, "flops": sum(lq)}
    if op == "slots":
        return {"bytes": 8 * sum(lk) + 4 * sum(_pages(h, bs) for h in lk) + 8 * B, "flops": sum(lk)}
    back = sum(_pages(h, bs) - _pages(h - n, bs) for n, h in zip(lq, lk))
    return {"bytes": 8 * back + 12 * B, "flops": back}


# ---------------------------------------------------------------- inputs
def _starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _cache(gen, case, shape, width, stored):
    """A cache of normed rows (unit rms times a gamma), stored as kv_rms_norm_rope_cache
    stores them, with the scale and offset of its quantisation ([N, D], or [D] in V1)."""
    per = (case["N"], width) if case["variant"] == 2 else (width,)
    gamma = torch.empty(width, device="cuda").uniform_(0.5, 1.5, generator=gen)
    rows = torch.randn(shape, device="cuda", generator=gen) * gamma
    if stored in HALF:
        return rows.to(HALF[stored]), None, None
    scale = torch.empty(per, device="cuda").uniform_(10.0, 40.0, generator=gen)
    offset = torch.empty(per, device="cuda").uniform_(-2.0, 2.0, generator=gen)
    s, o = scale, offset
    if case["variant"] == 2 and case["mode"] != "PA":       # heads before slots in the cache
        s, o = scale[:, None], offset[:, None]
    codes = rows.mul_(s).add_(o)
    if stored == "int8":
        return codes.round_().clamp_(-128, 127).to(torch.int8), scale, offset
    return codes.clamp_(-448, 448).to(STORED[stored]), scale, offset


def _table(gen, pages, block_num):
    """Pages given out at random: [B, most pages] with -1 behind each sequence's last, and
    the pages that are left."""
    ids = torch.randperm(block_num, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(pages), max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(table.shape[1], device="cuda") < torch.tensor(pages, device="cuda")[:, None]
    table[held] = ids[:sum(pages)]
    return table, ids[sum(pages):].clone()


def _prepare_paging(case, gen):
    (new, held), bs, B = _lengths(case), case["bs"], case["B"]
    pages = [_pages(h, bs) for h in held]
    after = [_pages(h + n, bs) for n, h in zip(new, held)] if case["op"] == "extend" else pages
    wanted = sum(after) - sum(pages)
    spare = wanted // 2 if case["short"] else wanted + 5
    block_num = sum(pages) + max(1, spare)
    table, free = _table(gen, pages, block_num)
    stack = torch.full((block_num,), -1, dtype=torch.int32, device="cuda")
    stack[:free.numel()] = free
    wide = torch.full((B, max(1, max(after))), -1, dtype=torch.int32, device="cuda")
    wide[:, :min(wide.shape[1], table.shape[1])] = table[:, :wide.shape[1]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    state = {"case": case, "table": wide, "free": stack, "count": i32([free.numel()]), "lens": i32(held), "new": i32(new),
             "block_num": block_num, "lens_out": torch.empty(B, dtype=torch.int32, device="cuda"),
             "count_out": torch.empty(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "truncate":
        state["keep"] = state["lens"] - state["new"]
        state["tokens"] = 1
        return state
    # room for a few tokens more than there are: a captured step's buffers have a fixed size
    state["tokens"] = (sum(new) if case["op"] == "extend" else sum(held)) + 7
    state["index"] = torch.empty(state["tokens"], dtype=torch.int64, device="cuda")
    state["cu"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] not in ("packed", "paged", "prefix"):
        return _prepare_paging(case, gen)
    state = {"case": case, "window": case.get("window"), "sinks": case.get("sinks")}
    lq, lk = _lengths(case)
    dt = HALF[case["dtype"]]
    if case["op"] == "packed":
        nq, nkv, d = case["nq"], case["nkv"], case["d"]
        if case["layout"] == "NBSD":
            qkv = torch.randn(nq + 2 * nkv, sum(lq), d, device="cuda", generator=gen).to(dt).transpose(0, 1)
        else:
            qkv = torch.randn(sum(lq), nq + 2 * nkv, d, device="cuda", generator=gen).to(dt)
        state["q"], state["k"], state["v"] = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
        state["out"] = torch.empty(sum(lq), nq, d, dtype=dt, device="cuda")
        state["starts_q"] = _starts(lq)
        state["lens"] = state["starts_q"].diff()
        state["scale"] = d ** -0.5
    else:
        bs, N, v1 = case["bs"], case["N"], case["variant"] == 1
        kw, vw = (case["R"], case["Dv"]) if v1 else (case["Dkv"], case["Dv"])
        if case["mode"] == "Norm":
            shape = (case["B"], N, case["ctx"])
        else:
            pages = [_pages(n, bs) for n in lk]
            ahead = _pages(case["prefix"], bs) if case["op"] == "prefix" else 0
            block_num = sum(pages) + ahead + 3
            shape = (block_num, bs, N) if case["mode"] == "PA" else (block_num, N, bs)
            state["table"], free = _table(gen, pages, block_num)
            if case["op"] == "prefix":
                state["prefix_table"] = free[:ahead].clone()
                state["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
        state["k_cache"], state["ks"], state["ko"] = _cache(gen, case, shape + (kw,), kw, case["kt"])
        state["v_cache"], state["vs"], state["vo"] = _cache(gen, case, shape + (vw,), vw, case["vt"])
        state["q"] = torch.randn(sum(lq), case["heads"], case["Dkv"], device="cuda", generator=gen).to(dt)
        state["out"] = torch.empty(sum(lq), case["heads"], vw, dtype=dt, device="cuda")
        state["starts_q"] = _starts(lq)
        state["lens"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
        # V1's absorbed heads keep the scale of the 128 + R channels they stand for
        state["scale"] = ((128 + case["R"]) if v1 else case["Dkv"]) ** -0.5
    state["longest_q"], state["longest_k"] = max(1, max(lq)), max(1, max(lk))
    state["tokens"] = sum(lq)
    return state


# ---------------------------------------------------------------- the plain forms
def _query_rows(state):
    """q as [B, longest, heads, Dk] in 32 bits, where its real rows are and whence they came."""
    q, starts = state["q"], state["starts_q"]
    pos = torch.arange(state["longest_q"], device=q.device)
    held = pos < starts.diff()[:, None]
    at = (starts[:-1, None].long() + pos).clamp_(max=q.shape[0] - 1)
    return q[at].float(), held, at


def _softmax_rows(s, seen):
    """Scores [..., Lk] to weights and their sum, where `seen`; a row that sees none gives zeros."""
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total.masked_fill(total == 0, 1.0)


def _plain_window(state, k, v, pos, held_k):
    """k [B, Lk, N, Dk] and v of the positions pos [B, Lk], of which held_k exist."""
    scale, window, sinks = state["scale"], state["window"], state["sinks"]
    out = torch.empty_like(state["out"])
    q, held, at = _query_rows(state)
    (B, Lq, heads), Lk, N = q.shape[:3], k.shape[1], k.shape[2]
    g = heads // N
    own_pos = torch.arange(Lq, device=q.device) + (state["lens"] - state["starts_q"].diff())[:, None]
    key, query = pos[:, None, :], own_pos[:, :, None]
    seen = (held_k[:, None, :] & (key <= query) & ((key > query - window) | (key < sinks)))[:, None, None]
    step = max(1, SCORES // (B * g * Lq * Lk))
    for n in range(0, N, step):
        h = slice(n * g, min(N, n + step) * g)
        kn, vn = k[:, :, n:n + step].float().permute(0, 2, 3, 1), v[:, :, n:n + step].float().transpose(1, 2)
        m = kn.shape[1]
        qn = q[:, :, h].reshape(B, Lq, m, g, -1).permute(0, 2, 3, 1, 4).reshape(B, m, g * Lq, -1)
        p, total = _softmax_rows((qn @ kn).mul_(scale).view(B, m, g, Lq, Lk), seen)
        o = (p.view(B, m, g * Lq, Lk) @ vn).view(B, m, g, Lq, -1) / total
        out[:, h][at[held]] = o.permute(0, 3, 1, 2, 4).reshape(B, Lq, m * g, -1)[held].to(out.dtype)
    return out


def _dequantised(x, scale, offset):
    """(code - offset) / scale in 32 bits; x [..., N, D]."""
    return x.float() if scale is None else (x.float() - offset) / scale


def _cached(state, cache, rows, pos):
    """Cached rows as [..., N, D] by page (or sequence) and place in it."""
    mode = state["case"]["mode"]
    if cache.dtype in (torch.float8_e4m3fn, torch.float8_e5m2):
        kind, cache = cache.dtype, cache.view(torch.uint8)
        return (cache[rows, pos] if mode == "PA" else cache[rows, :, pos]).view(kind)
    return cache[rows, pos] if mode == "PA" else cache[rows, :, pos]


def _keys_values(state, table, pos):
    """K and V [B, L, N, D] in 32 bits at the positions pos [B, L] of each sequence."""
    case = state["case"]
    if case["mode"] == "Norm":
        at = (torch.arange(case["B"], device="cuda")[:, None], pos)
    else:
        at = (table.gather(1, pos // case["bs"]).long().clamp_(min=0), pos % case["bs"])
    k = _dequantised(_cached(state, state["k_cache"], *at), state["ks"], state["ko"])
    v = _dequantised(_cached(state, state["v_cache"], *at), state["vs"], state["vo"])
    return (torch.cat([v, k], -1) if case["variant"] == 1 else k), v


def _plain_packed(state):
    starts, longest = state["starts_q"], state["longest_k"]
    pos = torch.arange(longest, device="cuda").expand(len(starts) - 1, -1)
    at = (starts[:-1, None].long() + pos).clamp_(max=state["k"].shape[0] - 1)
    return _plain_window(state, state["k"][at], state["v"][at], pos, pos < state["lens"][:, None])


def _plain_paged(state):
    """The first tokens and the windows' span of each sequence, gathered."""
    lens, lq = state["lens"].long(), state["starts_q"].diff().long()
    lo = (lens - lq - state["window"] + 1).clamp_(min=state["sinks"])
    first = torch.arange(min(state["sinks"], state["longest_k"]), device="cuda").expand(len(lens), -1)
    span = min(state["longest_k"], state["window"] + state["longest_q"])
    pos = torch.cat([first, lo[:, None] + torch.arange(span, device="cuda")], 1)
    held = pos < lens[:, None]
    k, v = _keys_values(state, state.get("table"), pos.where(held, 0))
    return _plain_window(state, k, v, pos, held)


def _plain_prefix(state):
    case, scale, out = state["case"], state["scale"], torch.empty_like(state["out"])
    P, lens = case["prefix"], state["lens"]
    q, held, at = _query_rows(state)
    (B, Lq, heads), N = q.shape[:3], case["N"]
    g = heads // N
    kp, vp = _keys_values(state, state["prefix_table"][None], torch.arange(P, device="cuda")[None])
    pos = torch.arange(state["longest_k"], device="cuda").expand(B, -1)
    ko, vo = _keys_values(state, state["table"], pos.where(pos < lens[:, None], 0))
    own_pos = torch.arange(Lq, device="cuda") + (lens - state["starts_q"].diff())[:, None]
    seen = (pos < lens[:, None])[:, None, :] & (pos[:, None, :] <= own_pos[:, :, None])
    seen = torch.cat([seen.new_ones(B, Lq, P), seen], -1)[:, None]
    for n in range(N):
        qn = q[:, :, n * g:(n + 1) * g].transpose(1, 2).reshape(B, g * Lq, -1)
        s = torch.cat([qn @ kp[0, :, n].T, qn @ ko[:, :, n].transpose(1, 2)], -1).mul_(scale)
        p, total = _softmax_rows(s.view(B, g, Lq, -1), seen)
        p = p.view(B, g * Lq, -1)
        o = (p[..., :P] @ vp[0, :, n] + p[..., P:] @ vo[:, :, n]).view(B, g, Lq, -1) / total
        out[:, n * g:(n + 1) * g][at[held]] = o.transpose(1, 2)[held].to(out.dtype)
    return out


def _spans_to_slots(state, first, n, served, table):
    """Slots of positions first .. first + n - 1 of each request in turn (-1: not served, or
    behind the last), and where each request's tokens start."""
    bs, T = state["case"]["bs"], state["tokens"]
    ends = n.long().cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    there = b < len(n)
    b = b.clamp_(max=len(n) - 1)
    pos = first.long()[b] + t - cu[b]
    there &= served[b] & (pos < table.shape[1] * bs)
    page = table[b, (pos // bs).where(there, 0)].long()
    there &= (page >= 0) & (page < state["block_num"])
    return torch.where(there, page * bs + pos % bs, -1), cu.clamp(max=T).to(torch.int32)


def _plain_extend(state):
    bs, table, lens, new = state["case"]["bs"], state["table"], state["lens"], state["new"]
    have, count = (lens + bs - 1) // bs, state["count"]
    fits = (lens + new <= table.shape[1] * bs) & (new.long().cumsum(0) <= state["tokens"])
    need = torch.where(fits, (lens + new + bs - 1) // bs - have, 0)
    upto = need.long().cumsum(0)
    served = fits & ((need == 0) | (upto <= count))
    taken = torch.where(served, upto, 0).amax()
    # page i of those that are taken is the i-th from the top of the free list
    column = torch.arange(table.shape[1], device="cuda") - have[:, None]
    fresh = served[:, None] & (column >= 0) & (column < need[:, None])
    from_top = (count - 1 - (upto - need)[:, None] - column).clamp_(min=0, max=state["free"].numel() - 1)
    table = torch.where(fresh, state["free"][from_top], table)
    index, cu = _spans_to_slots(state, lens, new, served, table)
    return [index, cu, lens + torch.where(served, new, 0), table, (count - taken).to(torch.int32)]


def _plain_slots(state):
    lens = state["lens"]
    return list(_spans_to_slots(state, torch.zeros_like(lens), lens, torch.ones_like(lens, dtype=torch.bool), state["table"]))


def _plain_truncate(state):
    bs, table, lens, count = state["case"]["bs"], state["table"], state["lens"], state["count"]
    keep = torch.minimum(state["keep"].clamp(min=0), lens)
    column = torch.arange(table.shape[1], device="cuda")
    back = table[(column >= ((keep + bs - 1) // bs)[:, None]) & (column < ((lens + bs - 1) // bs)[:, None])]
    free = state["free"].clone()
    free[count.long() + torch.arange(back.numel() - 1, -1, -1, device="cuda")] = back
    return [keep, free, count + back.numel()]


# ---------------------------------------------------------------- the library's calls
def _cache_params(native, case, state):
    half = {"bf16": native.RA_BF16, "fp16": native.RA_FP16}
    kind = {**half, "int8": native.RA_INT8, "e4m3": native.RA_FP8_E4M3, "e5m2": native.RA_FP8_E5M2}
    mode = {"Norm": native.RA_CACHE_NORM, "PA": native.RA_CACHE_PA, "PA_BNSD": native.RA_CACHE_PA_BNSD}[case["mode"]]
    paged = mode != native.RA_CACHE_NORM
    return native.KvRmsNormRopeCacheParams(
        B=case["B"], N=case["N"], S=1, Dkv=case["Dkv"], Dv=case["Dv"], rope_size=case["R"],
        variant=case["variant"], cache_mode=mode, block_num=state["k_cache"].shape[0] if paged else 0,
        block_size=case["bs"] if paged else 0, kv_dtype=half[case["dtype"]], k_cache_dtype=kind[case["kt"]],
        ckv_cache_dtype=kind[case["vt"]], epsilon=1e-5, cache_seq_len=0 if paged else case["ctx"])


def _handle(state):
    """The parameter structs and the workspace, which a program makes once and keeps."""
    from rope_attention_gb300 import native
    case, op = state["case"], state["case"]["op"]
    if op == "packed":
        params = native.packed_attention_params(state["q"], state["k"], state["v"], state["out"], B=case["B"], causal=True,
                                                softmax_scale=state["scale"])
    elif op in ("paged", "prefix"):
        state["cache"] = _cache_params(native, case, state)
        params = native.PagedAttentionParams(B=case["B"], total_q=state["tokens"], num_heads=case["heads"], causal=1,
                                             softmax_scale=state["scale"], max_seq_len=case["ctx"])
        if "table" in state:
            params.block_table_stride = state["table"].shape[1]
    else:
        params = native.KvCachePagingParams(B=case["B"], block_num=state["block_num"], block_size=case["bs"],
                                            block_table_stride=state["table"].shape[1], max_tokens=state["tokens"])
    room = WORKSPACE_BYTES
    if op == "prefix":
        state["prefix"] = native.AttentionPrefix(max_prefix_len=case["prefix"], table_entries=state["prefix_table"].numel())
        room = native.paged_prefix_attention_workspace_bytes(state["cache"], params, state["prefix"])
    elif op in ("packed", "paged"):
        state["visible"] = native.AttentionWindow(window=case["window"], sinks=case["sinks"])
    if op in ("packed", "paged", "prefix"):
        state["workspace"] = torch.zeros(room, dtype=torch.uint8, device="cuda")
    state["params"] = params


def _own(state):
    from rope_attention_gb300 import native
    if "params" not in state:
        _handle(state)
    case, op, params = state["case"], state["case"]["op"], state["params"]
    if op == "packed":
        starts = state["starts_q"] if case["ragged"] else None
        native.packed_window_attention(params, state["visible"], state["q"], state["k"], state["v"], state["out"],
                                       state["workspace"], cu_seqlens_q=starts, cu_seqlens_k=starts)
        return state["out"]
    if op == "paged":
        native.paged_window_attention(state["cache"], params, state["visible"], state["q"], state["k_cache"], state["v_cache"],
                                      state["lens"], state["out"], state["workspace"], block_table=state.get("table"),
                                      cu_seqlens_q=state["starts_q"], k_rope_scale=state["ks"], c_kv_scale=state["vs"],
                                      k_rope_offset=state["ko"], c_kv_offset=state["vo"])
        return state["out"]
    if op == "prefix":
        native.paged_prefix_attention(state["cache"], params, state["prefix"], state["q"], state["k_cache"], state["v_cache"],
                                      state["prefix_len"], state["prefix_table"], state["lens"], state["table"], state["out"],
                                      state["workspace"], cu_seqlens_q=state["starts_q"], k_rope_scale=state["ks"],
                                      c_kv_scale=state["vs"], k_rope_offset=state["ko"], c_kv_offset=state["vo"])
        return state["out"]
    if op == "extend":
        native.kv_cache_extend(params, state["new"], state["lens"], state["table"], state["free"], state["count"],
                               state["index"], state["cu"], state["lens_out"], state["count_out"])
        return [state[x] for x in ("index", "cu", "lens_out", "table", "count_out")]
    if op == "slots":
        native.kv_cache_slots(params, state["lens"], state["table"], state["index"], state["cu"])
        return [state["index"], state["cu"]]
    native.kv_cache_truncate(params, state["lens"], state["table"], state["free"], state["count"], state["lens_out"],
                             state["count_out"], keep=state["keep"])
    return [state[x] for x in ("lens_out", "free", "count_out")]


def run(state):
    if own:
        return _own(state)
    return {"packed": _plain_packed, "paged": _plain_paged, "prefix": _plain_prefix, "extend": _plain_extend,
            "slots": _plain_slots, "truncate": _plain_truncate}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _row(cache, mode, page, slot):
    """The rows of one run of slots of one page, [n, N, D] in 64 bits."""
    part = cache[page, slot] if mode == "PA" else cache[page][:, slot].float().transpose(0, 1)
    return part.double()


def _sequence(state, name, pages, b, n):
    """The first n cached rows of a sequence, [n, N, D] in 64 bits, page by page."""
    case, cache = state["case"], state[name + "_cache"]
    if case["mode"] == "Norm":
        rows = _row(cache, "Norm", b, slice(0, n))
    else:
        bs = case["bs"]
        rows = torch.cat([_row(cache, case["mode"], page, slice(0, min(bs, n - i * bs)))
                          for i, page in enumerate(pages[:_pages(n, bs)].tolist())])
    if state[name + "s"] is not None:
        rows = (rows - state[name + "o"].double()) / state[name + "s"].double()
    return rows


def _attend(q, k, v, first, window, sinks, scale):
    """One sequence: q [Lq, heads, Dk], k [Lk, N, Dk], v [Lk, N, Dv]; query i stands at first + i.
    In blocks of queries, each against the stretch of keys that it can see."""
    Lq, g = q.shape[0], q.shape[1] // k.shape[1]
    out = torch.zeros(Lq, q.shape[1], v.shape[2], dtype=torch.float64, device=q.device)
    block = 1024
    for i in range(0, Lq, block):
        n = min(block, Lq - i)
        hi = min(k.shape[0], first + i + n)
        lo = max(0, first + i - window + 1)
        j = torch.arange(max(0, hi), device=q.device)
        j = j[(j >= lo) | (j < sinks)]
        if j.numel() == 0:
            continue
        place = (first + torch.arange(i, i + n, device=q.device))[:, None]
        hidden = (j > place) | ((place - j >= window) & (j >= sinks))
        for h in range(q.shape[1]):
            s = torch.einsum("id,jd->ij", q[i:i + n, h].double(), k[j, h // g]) * scale
            weight = torch.softmax(torch.where(hidden, -math.inf, s), dim=1)
            out[i:i + n, h] = torch.nan_to_num(weight, nan=0.0) @ v[j, h // g]
    return out


def _exact_paging(case, state):
    """On the host, request by request."""
    bs, B, op, T = case["bs"], case["B"], case["op"], state["tokens"]
    lens, table, free, count = (state[x].tolist() for x in ("lens", "table", "free", "count"))
    count = count[0]
    if op == "truncate":
        keep, back = [max(0, min(k, n)) for k, n in zip(state["keep"].tolist(), lens)], []
        for b in range(B):
            back += table[b][_pages(keep[b], bs):_pages(lens[b], bs)]
        free[count:count + len(back)] = back[::-1]
        return [torch.tensor(x) for x in (keep, free, [count + len(back)])]
    index, cu, asked, out = [], [0], 0, list(lens)
    new = state["new"].tolist() if op == "extend" else lens
    for b in range(B):
        first, served = (lens[b], False) if op == "extend" else (0, True)
        if op == "extend":
            want = _pages(lens[b] + new[b], bs) - _pages(lens[b], bs)
            asked += want
            served = want == 0 or asked <= state["count"].item()
            if served:
                out[b] = lens[b] + new[b]
                for i in range(want):
                    count -= 1
                    table[b][_pages(lens[b], bs) + i] = free[count]
        index += [table[b][p // bs] * bs + p % bs if served else -1 for p in range(first, first + new[b])]
        cu.append(len(index))
    index += [-1] * (T - len(index))
    if op == "slots":
        return [torch.tensor(index), torch.tensor(cu)]
    return [torch.tensor(x) for x in (index, cu, out, table, [count])]


def exact(case, seed):
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    state = prepare(case, seed)
    if case["op"] not in ("packed", "paged", "prefix"):
        return _exact_paging(case, state)
    lq, lk = _lengths(case)
    prefix = case.get("prefix", 0)
    if prefix:
        kp, vp = (_sequence(state, x, state["prefix_table"], 0, prefix) for x in "kv")
    outs, start = [], 0
    for b, (a, n) in enumerate(zip(lq, lk)):
        q = state["q"][start:start + a]
        if case["op"] == "packed":
            k, v = (state[x][start:start + n].double() for x in "kv")
        else:
            pages = state["table"][b] if "table" in state else None
            k, v = (_sequence(state, x, pages, b, n) for x in "kv")
            if prefix:
                k, v = torch.cat([kp, k]), torch.cat([vp, v])
            if case["variant"] == 1:
                k = torch.cat([v, k], -1)
        n += prefix
        outs.append(_attend(q, k, v, n - a, state["window"] or n, state["sinks"] or 0, state["scale"]))
        start += a
    return torch.cat(outs)
