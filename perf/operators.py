"""Cases, plain forms and 64-bit values of the attention operators that follow the prologue.

Three operators: ``packed_attention`` (attention over whole prompts whose Q, K and V are
columns of the projection's output), ``paged_attention`` (new tokens, one or a chunk per
sequence, against the paged caches that kv_rms_norm_rope_cache writes) and
``kv_cache_read`` (cached rows gathered by slot and dequantised).

``own`` chooses what ``run`` does: the plain torch form (false) or the calls of this
repository's library (true).
"""
import math
import random

import torch

own = False

WORKSPACE_BYTES = 64 << 20       # what every attention call here is content with
SCORES = 1 << 30                 # score elements that the plain form holds at a time
EXACT_FLOPS = 4e12               # beyond this the 64-bit value takes too long

HALF = {"bf16": torch.bfloat16, "fp16": torch.float16}
STORED = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, **HALF}
SIZE = {"bf16": 2, "fp16": 2, "int8": 1, "e4m3": 1, "e5m2": 1}


# ---------------------------------------------------------------- cases
def _packed(name, B, q, kv, nq, nkv, d, causal, ragged, dtype="bf16", layout="BSD"):
    """B sequences, q query and kv key tokens in all (kv 0: self-attention, one buffer)."""
    return {"op": "packed", "name": name, "B": B, "q": q, "kv": kv, "nq": nq, "nkv": nkv, "d": d,
            "causal": causal, "ragged": ragged, "dtype": dtype, "layout": layout}


def _paged(name, variant, B, N, heads, Dkv, Dv, R, mode, bs, ctx, new, kt, vt, dtype="bf16", causal=True, ragged=True):
    """B sequences of up to ctx cached tokens, the last up to `new` of them attending."""
    return {"op": "paged", "name": name, "variant": variant, "B": B, "N": N, "heads": heads, "Dkv": Dkv, "Dv": Dv,
            "R": R, "mode": mode, "bs": bs, "ctx": ctx, "new": new, "kt": kt, "vt": vt, "dtype": dtype,
            "causal": causal, "ragged": ragged}


def _read(name, variant, B, N, S, Dkv, Dv, R, mode, bs, kt, vt, dtype="bf16"):
    """B x S tokens read back through their slots."""
    return {"op": "read", "name": name, "variant": variant, "B": B, "N": N, "S": S, "Dkv": Dkv, "Dv": Dv, "R": R,
            "mode": mode, "bs": bs, "kt": kt, "vt": vt, "dtype": dtype}


def listed():
    return [
        # the tiny self-attention layer (two heads of 64, 128 tokens): latency of one call
        _packed("prompt_tiny", 1, 128, 0, 2, 2, 64, False, False),
        # packed prompts of different lengths, grouped heads, causal: a language model's prefill
        _packed("prompt_packed_gqa", 7, 9001, 0, 32, 8, 128, True, True),
        # Wan 480p self-attention: every token of the latent grid against every other
        _packed("wan480_self", 1, 32760, 0, 40, 40, 128, False, False),
        # Wan 480p cross-attention: image tokens against 512 text tokens
        _packed("wan480_cross", 1, 32760, 512, 40, 40, 128, False, False),
        # one token for each of 8 sequences, V2 int8 cache: an ordinary decode step
        _paged("decode_v2_int8", 2, 8, 8, 64, 192, 128, 64, "PA_BNSD", 128, 4096, 1, "int8", "int8"),
        # a short chat: one sequence, one token, few cached rows; latency
        _paged("decode_v2_short", 2, 1, 2, 8, 192, 128, 64, "PA", 16, 333, 1, "bf16", "bf16"),
        # the MLA cache of 32 sequences, 128 query heads over one latent row
        _paged("decode_mla", 1, 32, 1, 128, 576, 512, 64, "PA_BNSD", 128, 4096, 1, "bf16", "bf16"),
        # one sequence with a long context: the length is all there is to split
        _paged("decode_mla_long_int8", 1, 1, 1, 16, 576, 512, 64, "PA_BNSD", 128, 131072, 2, "int8", "int8",
               ragged=False),
        # chunked prefill: new tokens over long contexts, 16-bit cache
        _paged("chunk_v2", 2, 4, 8, 32, 192, 128, 64, "PA_BNSD", 128, 16384, 512, "bf16", "bf16"),
        # the same over an FP8 cache, one length, fp16 around it
        _paged("chunk_v2_fp8", 2, 2, 4, 32, 128, 128, 64, "PA", 64, 8192, 777, "e4m3", "e4m3", dtype="fp16",
               ragged=False),
        # the whole int8 MLA cache read back
        _read("read_mla_int8", 1, 32, 1, 4096, 576, 512, 64, "PA_BNSD", 128, "int8", "int8"),
        # a short V2 sequence read back, FP8 keys beside 16-bit values
        _read("read_v2_short", 2, 1, 4, 801, 192, 128, 64, "PA", 32, "e4m3", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["packed", "packed", "paged", "paged", "paged", "read"])
    while True:
        if kind == "packed":
            B = rng.choice([1, 1, 2, 3, 5, 8, 17])
            nkv = rng.choice([1, 2, 4, 5, 8])
            case = _packed("", B, B * _log_int(rng, 1, 9000 // B), 0, nkv * rng.choice([1, 1, 2, 4, 7, 8]), nkv,
                           rng.choice([64, 128, 128, 80, 96, 16, 112]), rng.random() < 0.6, rng.random() < 0.6,
                           rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["BSD", "BSD", "NBSD"]))
            if rng.random() < 0.25:
                case["kv"] = B * _log_int(rng, 1, 4000 // B)
        elif kind == "paged":
            variant = rng.choice([1, 2, 2])
            kt, vt = rng.choice(["int8", "bf16", "e4m3", "e5m2"]), rng.choice(["int8", "bf16", "e4m3"])
            kt, vt = (kt, kt) if rng.random() < 0.7 else (kt, vt)
            N = 1 if variant == 1 else rng.choice([1, 2, 4, 8])
            Dkv, Dv, R = (576, 512, 64) if variant == 1 else rng.choice([(192, 128, 64), (128, 128, 64), (64, 64, 32), (96, 80, 32)])
            mode = rng.choice(["PA", "PA_BNSD", "PA_BNSD"] + (["Norm"] if variant == 2 else []))
            group = rng.choice([16, 32, 64, 128, 5]) if variant == 1 else rng.choice([1, 2, 4, 8, 16, 3])
            case = _paged("", variant, rng.choice([1, 1, 2, 4, 7, 16, 32, 61]), N, N * group, Dkv, Dv, R, mode,
                          rng.choice([32, 64, 96, 128, 256]), _log_int(rng, 1, 40000),
                          1 if rng.random() < 0.5 else _log_int(rng, 1, 900), kt, vt, "bf16",
                          rng.random() < 0.8, rng.random() < 0.7)
        else:
            variant = rng.choice([1, 2])
            kt, vt = rng.choice(["int8", "bf16", "e4m3", "e5m2"]), rng.choice(["int8", "bf16", "e4m3"])
            N = 1 if variant == 1 else rng.choice([1, 2, 4, 8])
            Dkv, Dv, R = (576, 512, 64) if variant == 1 else rng.choice([(192, 128, 64), (128, 128, 64), (96, 80, 32)])
            case = _read("", variant, rng.choice([1, 2, 8, 32]), N, _log_int(rng, 1, 4096), Dkv, Dv, R,
                         rng.choice(["PA", "PA_BNSD"]), rng.choice([32, 64, 128, 160]), kt, vt)
        del case["name"]
        w = work(case)
        if w["flops"] <= 2e14 and w["bytes"] <= 4e9 and _memory(case) <= 12e9:
            return case


def _memory(case):
    """Bytes of the largest score tensor's batch in the plain form."""
    if case["op"] == "read":
        return 0
    (lq, lk), heads = _lengths(case), case.get("nq") or case["heads"]
    per_head = heads // (case.get("nkv") or case["N"]) * len(lq) * max(lq) * max(lk)
    return 4.0 * per_head


# ---------------------------------------------------------------- lengths and work
def _split(rng, total, n):
    """n lengths that add up to total, of very different sizes."""
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _lengths(case):
    """(query tokens, key tokens) of each sequence, from the case alone."""
    rng = random.Random("%(op)s %(B)d" % case + " %d" % (case.get("q") or case["ctx"]))
    B = case["B"]
    if case["op"] == "packed":
        lq = _split(rng, case["q"], B) if case["ragged"] else [case["q"] // B] * B
        if not case["kv"]:
            return lq, lq
        return lq, _split(rng, case["kv"], B) if case["ragged"] else [case["kv"] // B] * B
    ctx, new = case["ctx"], min(case["new"], case["ctx"])
    if not case["ragged"]:
        return [new] * B, [ctx] * B
    lk = [ctx if b == 0 else rng.randint(max(1, ctx // 4), ctx) for b in range(B)]
    return [min(k, new if b == 0 else rng.randint((new + 1) // 2, new)) for b, k in enumerate(lk)], lk


def _pairs(lq, lk, causal):
    """Visible (query, key) pairs: query i of lq sees keys up to i + lk - lq."""
    if not causal:
        return sum(a * b for a, b in zip(lq, lk))
    total = 0
    for a, b in zip(lq, lk):
        n = min(a, b)                         # rows that see anything
        total += n * b - n * (n - 1) // 2     # the last row sees b, the one before b - 1, ...
    return total


def work(case):
    if case["op"] == "read":
        rows = case["B"] * case["S"] * case["N"]
        kw, vw = (case["R"], case["Dv"]) if case["variant"] == 1 else (case["Dkv"], case["Dv"])
        return {"bytes": rows * (kw * (SIZE[case["kt"]] + 2) + vw * (SIZE[case["vt"]] + 2)) + case["B"] * case["S"] * 8,
                "flops": 2 * rows * (kw + vw)}
    lq, lk = _lengths(case)
    pairs = _pairs(lq, lk, case["causal"])
    if case["op"] == "packed":
        d = case["d"]
        return {"bytes": 2 * d * (2 * sum(lq) * case["nq"] + 2 * sum(lk) * case["nkv"]), "flops": 4 * d * case["nq"] * pairs}
    kw, vw = (case["R"], case["Dv"]) if case["variant"] == 1 else (case["Dkv"], case["Dv"])
    return {"bytes": sum(lk) * case["N"] * (kw * SIZE[case["kt"]] + vw * SIZE[case["vt"]])
            + 2 * sum(lq) * case["heads"] * (case["Dkv"] + case["Dv"]),
            "flops": 2 * (case["Dkv"] + case["Dv"]) * case["heads"] * pairs}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "packed":
        lq, lk = _lengths(case)
        nq, nkv, d, dt = case["nq"], case["nkv"], case["d"], HALF[case["dtype"]]

        def projected(tokens, heads):       # a projection's output, as [tokens, heads, d]
            if case["layout"] == "NBSD":
                return torch.randn(heads, tokens, d, device="cuda", generator=gen).to(dt).transpose(0, 1)
            return torch.randn(tokens, heads, d, device="cuda", generator=gen).to(dt)

        if case["kv"]:
            state["q"] = projected(sum(lq), nq)
            state["k"], state["v"] = projected(sum(lk), nkv), projected(sum(lk), nkv)
        else:
            qkv = projected(sum(lq), nq + 2 * nkv)
            state["q"], state["k"], state["v"] = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
        state["out"] = torch.empty(sum(lq), nq, d, dtype=dt, device="cuda")
        state["starts_q"] = _starts(lq)
        state["starts_k"] = state["starts_q"] if not case["kv"] else _starts(lk)
        state["lens"] = state["starts_k"].diff()
        state["scale"] = d ** -0.5
    else:
        bs, N, v1 = case["bs"], case["N"], case["variant"] == 1
        kw, vw = (case["R"], case["Dv"]) if v1 else (case["Dkv"], case["Dv"])
        lk = _lengths(case)[1] if case["op"] == "paged" else [case["S"]] * case["B"]
        pages = [-(-n // bs) for n in lk]
        if case["mode"] == "Norm":
            shape = (case["B"], N, case["ctx"])
        else:
            block_num = sum(pages) + 3
            shape = (block_num, bs, N) if case["mode"] == "PA" else (block_num, N, bs)
            ids = torch.randperm(block_num, device="cuda", generator=gen).to(torch.int32)
            table = torch.full((case["B"], max(pages)), -1, dtype=torch.int32, device="cuda")
            held = torch.arange(max(pages), device="cuda") < torch.tensor(pages, device="cuda")[:, None]
            table[held] = ids[:sum(pages)]
            state["table"] = table
        state["k_cache"], state["ks"], state["ko"] = _cache(gen, case, shape + (kw,), kw, case["kt"])
        state["v_cache"], state["vs"], state["vo"] = _cache(gen, case, shape + (vw,), vw, case["vt"])
        dt = HALF[case["dtype"]]
        if case["op"] == "read":
            s = torch.arange(case["S"], device="cuda")
            state["index"] = (table[:, s // bs].long() * bs + s % bs).reshape(-1)
            state["k"] = torch.empty(case["B"], N, case["S"], kw, dtype=dt, device="cuda")
            state["v"] = torch.empty(case["B"], N, case["S"], vw, dtype=dt, device="cuda")
            return state
        lq = _lengths(case)[0]
        state["q"] = torch.randn(sum(lq), case["heads"], case["Dkv"], device="cuda", generator=gen).to(dt)
        state["out"] = torch.empty(sum(lq), case["heads"], vw, dtype=dt, device="cuda")
        state["starts_q"] = _starts(lq)
        state["lens"] = torch.tensor(lk, dtype=torch.int32, device="cuda")
        # V1's absorbed heads keep the scale of the 128 + R channels they stand for
        state["scale"] = ((128 + case["R"]) if v1 else case["Dkv"]) ** -0.5
    state["longest_q"], state["longest_k"], state["causal"] = max(1, max(lq)), max(1, max(lk)), case["causal"]
    state["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return state


# ---------------------------------------------------------------- the plain forms
def _padded(x, starts, longest):
    """[tokens, ...] -> [B, longest, ...] and the mask of its real rows."""
    pos = torch.arange(longest, device=x.device)
    held = pos < starts.diff()[:, None]
    at = (starts[:-1, None].long() + pos).clamp_(max=x.shape[0] - 1)
    return x[at], held, at


def _plain_attention(state, k, v):
    """q [tokens, heads, Dk]; k [B, Lk, N, Dk] and v [B, Lk, N, Dv], of any finite value beyond each length."""
    q, nk, causal, scale, out = (state[x] for x in ("q", "lens", "causal", "scale", "out"))
    N, heads, out = k.shape[2], q.shape[1], torch.empty_like(out)
    qp, held, at = _padded(q, state["starts_q"], state["longest_q"])
    B, Lq, Lk, g = qp.shape[0], qp.shape[1], k.shape[1], heads // N
    nq = state["starts_q"].diff()
    key = torch.arange(Lk, device=q.device)
    seen = (key < nk[:, None])[:, None, :].expand(B, Lq, Lk)
    if causal:
        last = torch.arange(Lq, device=q.device) + (nk - nq)[:, None]
        seen = seen & (key <= last[:, :, None])
    step = max(1, SCORES // (B * g * Lq * Lk))
    for n in range(0, N, step):
        h = slice(n * g, min(N, n + step) * g)
        kn, vn = k[:, :, n:n + step].float().permute(0, 2, 3, 1), v[:, :, n:n + step].float().transpose(1, 2)
        m = kn.shape[1]
        qn = qp[:, :, h].float().reshape(B, Lq, m, g, -1).permute(0, 2, 3, 1, 4).reshape(B, m, g * Lq, -1)
        s = (qn @ kn).mul_(scale).view(B, m, g, Lq, Lk)
        s.masked_fill_(~seen[:, None, None], -math.inf)
        top = s.amax(-1, keepdim=True).clamp_(min=-3e38)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p.view(B, m, g * Lq, Lk) @ vn).view(B, m, g, Lq, -1)
        o = o / total.masked_fill(total == 0, 1.0)
        out[:, h][at[held]] = o.permute(0, 3, 1, 2, 4).reshape(B, Lq, m * g, -1)[held].to(out.dtype)
    return out


def _dequantised(x, scale, offset):
    """(code - offset) / scale in 32 bits; x [..., N, D]."""
    return x.float() if scale is None else (x.float() - offset) / scale


def _cached(state, cache, at):
    """Cached rows as [..., N, D] by (sequence or page, position) indices."""
    mode = state["case"]["mode"]
    rows, pos = at
    if cache.dtype in (torch.float8_e4m3fn, torch.float8_e5m2):
        kind, cache = cache.dtype, cache.view(torch.uint8)
        got = (cache[rows, pos] if mode == "PA" else cache[rows, :, pos]).view(kind)
    else:
        got = cache[rows, pos] if mode == "PA" else cache[rows, :, pos]
    return got


def _plain_packed(state):
    k, v = (_padded(state[x], state["starts_k"], state["longest_k"])[0] for x in "kv")
    return _plain_attention(state, k, v)


def _plain_paged(state):
    case = state["case"]
    pos = torch.arange(state["longest_k"], device="cuda")
    if case["mode"] == "Norm":
        at = (torch.arange(case["B"], device="cuda")[:, None], pos[None])
    else:
        at = (state["table"][:, pos // case["bs"]].long().clamp_(min=0), (pos % case["bs"])[None])
    k = _dequantised(_cached(state, state["k_cache"], at), state["ks"], state["ko"])
    v = _dequantised(_cached(state, state["v_cache"], at), state["vs"], state["vo"])
    if case["variant"] == 1:
        k = torch.cat([v, k], -1)
    return _plain_attention(state, k, v)


def _plain_read(state):
    case = state["case"]
    at = (state["index"] // case["bs"], state["index"] % case["bs"])
    read = []
    for cache, scale, offset, out in (("k_cache", "ks", "ko", "k"), ("v_cache", "vs", "vo", "v")):
        rows = _dequantised(_cached(state, state[cache], at), state[scale], state[offset])
        rows = rows.view(case["B"], case["S"], case["N"], -1).transpose(1, 2)
        read.append(rows.to(state[out].dtype).contiguous())
    return read


# ---------------------------------------------------------------- the library's calls
def _cache_params(native, case, state):
    half = {"bf16": native.RA_BF16, "fp16": native.RA_FP16}
    kind = {**half, "int8": native.RA_INT8, "e4m3": native.RA_FP8_E4M3, "e5m2": native.RA_FP8_E5M2}
    mode = {"Norm": native.RA_CACHE_NORM, "PA": native.RA_CACHE_PA, "PA_BNSD": native.RA_CACHE_PA_BNSD}[case["mode"]]
    paged = mode != native.RA_CACHE_NORM
    return native.KvRmsNormRopeCacheParams(
        B=case["B"], N=case["N"], S=case.get("S", 1), Dkv=case["Dkv"], Dv=case["Dv"], rope_size=case["R"],
        variant=case["variant"], cache_mode=mode, block_num=state["k_cache"].shape[0] if paged else 0,
        block_size=case["bs"] if paged else 0, kv_dtype=half[case["dtype"]], k_cache_dtype=kind[case["kt"]],
        ckv_cache_dtype=kind[case["vt"]], epsilon=1e-5, cache_seq_len=0 if paged else case["ctx"])


def _own(state):
    from rope_attention_gb300 import native
    case = state["case"]
    if case["op"] == "packed":
        params = native.packed_attention_params(state["q"], state["k"], state["v"], state["out"], B=case["B"],
                                                causal=case["causal"], softmax_scale=state["scale"])
        ragged = case["ragged"]
        native.packed_attention(params, state["q"], state["k"], state["v"], state["out"], state["workspace"],
                                cu_seqlens_q=state["starts_q"] if ragged else None,
                                cu_seqlens_k=state["starts_k"] if ragged else None)
        return state["out"]
    cache = _cache_params(native, case, state)
    if case["op"] == "paged":
        params = native.PagedAttentionParams(B=case["B"], total_q=state["q"].shape[0], num_heads=case["heads"],
                                             causal=1 if case["causal"] else 0, softmax_scale=state["scale"],
                                             max_seq_len=case["ctx"])
        native.paged_attention(cache, params, state["q"], state["k_cache"], state["v_cache"], state["lens"],
                               state["out"], state["workspace"], block_table=state.get("table"),
                               cu_seqlens_q=state["starts_q"], k_rope_scale=state["ks"], c_kv_scale=state["vs"],
                               k_rope_offset=state["ko"], c_kv_offset=state["vo"])
        return state["out"]
    native.kv_cache_read(cache, state["index"], state["k_cache"], state["v_cache"], state["k"], state["v"],
                         k_rope_scale=state["ks"], c_kv_scale=state["vs"], k_rope_offset=state["ko"],
                         c_kv_offset=state["vo"])
    return [state["k"], state["v"]]


def run(state):
    if own:
        return _own(state)
    return {"packed": _plain_packed, "paged": _plain_paged, "read": _plain_read}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _row(cache, mode, page, slot):
    """The rows of one run of slots of one page, [n, N, D] in 64 bits."""
    part = cache[page, slot] if mode == "PA" else cache[page][:, slot].float().transpose(0, 1)
    return part.double()


def _sequence(state, cache, scale, offset, b, n):
    """The first n cached rows of sequence b, [n, N, D] in 64 bits, page by page."""
    case = state["case"]
    if case["mode"] == "Norm":
        rows = _row(cache, "Norm", b, slice(0, n))
    else:
        bs = case["bs"]
        rows = torch.cat([_row(cache, case["mode"], page, slice(0, min(bs, n - i * bs)))
                          for i, page in enumerate(state["table"][b, :-(-n // bs)].tolist())])
    if scale is not None:
        rows = (rows - offset.double()) / scale.double()
    return rows


def _softmax_sum(q, k, v, causal, scale):
    """One sequence: q [Lq, heads, Dk], k [Lk, N, Dk], v [Lk, N, Dv], head by head."""
    Lq, Lk, g = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    out = torch.zeros(Lq, q.shape[1], v.shape[2], dtype=torch.float64, device=q.device)
    if Lk == 0:
        return out
    hidden = torch.ones(Lq, Lk, dtype=torch.bool, device=q.device).triu(Lk - Lq + 1) if causal else None
    for h in range(q.shape[1]):
        s = torch.einsum("id,jd->ij", q[:, h].double(), k[:, h // g]) * scale
        if causal:
            s = torch.where(hidden, -math.inf, s)
        weight = torch.softmax(s, dim=1)
        out[:, h] = torch.nan_to_num(weight, nan=0.0) @ v[:, h // g]
    return out


def exact(case, seed):
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    state = prepare(case, seed)
    if case["op"] == "read":
        k, v = [], []
        for b in range(case["B"]):
            k.append(_sequence(state, state["k_cache"], state["ks"], state["ko"], b, case["S"]).transpose(0, 1))
            v.append(_sequence(state, state["v_cache"], state["vs"], state["vo"], b, case["S"]).transpose(0, 1))
        return [torch.stack(k), torch.stack(v)]
    lq, lk = _lengths(case)
    outs, start_q, start_k = [], 0, 0
    for b, (a, n) in enumerate(zip(lq, lk)):
        q = state["q"][start_q:start_q + a]
        if case["op"] == "packed":
            k, v = (state[x][start_k:start_k + n].double() for x in "kv")
        elif n:
            k = _sequence(state, state["k_cache"], state["ks"], state["ko"], b, n)
            v = _sequence(state, state["v_cache"], state["vs"], state["vo"], b, n)
            if case["variant"] == 1:
                k = torch.cat([v, k], -1)
        outs.append(_softmax_sum(q, k, v, case["causal"], state["scale"]))
        start_q, start_k = start_q + a, start_k + n
    return torch.cat(outs)
