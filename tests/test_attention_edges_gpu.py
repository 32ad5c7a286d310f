"""Calls of the attention operators at the edge of what the header allows, on the GPU:
workspaces that start on any 16 bytes, waits of the shortest time limit, codes beside their
zero point, weights far below a row's largest, scales near the least, and batches of very
different lengths."""
import numpy as np
import pytest
import torch

import oracle
from attention_util import HALF_STEP, TORCH
from rope_attention_gb300 import native
from test_attention_use import DEFAULT_WAIT_NS, Packed, Paged

pytestmark = pytest.mark.gpu

CODE = {"bf16": native.RA_BF16, "fp16": native.RA_FP16, "int8": native.RA_INT8, "e4m3": native.RA_FP8_E4M3,
        "e5m2": native.RA_FP8_E5M2}


@pytest.mark.parametrize("at", [0, 16])
def test_workspace_on_any_16_bytes(at):
    """Items of one or two pieces and more, whose pieces pass through the workspace."""
    for x in (Packed(1, [2000, 700], 2, 1, 128, True), Paged(2, [2500], [80], 4, N=2), Paged(3, [2500], [1], 4, N=2),
              Paged(4, [2500], [80], 4, N=2, quant=True)):
        n = (x.ws if isinstance(x, Packed) else x.run_.workspace).numel()
        pool = torch.zeros(n + 64, dtype=torch.uint8, device="cuda")
        pool[at + n:] = 77
        ws = pool[at:at + n]
        assert ws.data_ptr() % 32 == at
        if isinstance(x, Packed):
            x.ws = ws
        else:
            x.run_.workspace = ws
            x.kv.run()
        x.run()
        torch.cuda.synchronize()
        assert x.status() == 0 and (pool[:at] == 0).all() and (pool[at + n:] == 77).all()
        x.check("workspace at " + str(at))


SHORT_WAITS = {
    "packed": lambda: Packed(5, [40] * 50 + [600], 16, 4, 128, True),
    "decode": lambda: Paged(6, [700, 90, 333, 1] * 8, [1, 1, 1, 1] * 8, 16, N=4),
    "decode_int8": lambda: Paged(7, [700, 90, 333, 1] * 8, [1, 1, 1, 1] * 8, 16, N=4, quant=True),
    "decode_v1": lambda: Paged(8, [700, 90, 333] * 8, [1, 2, 1] * 8, 16, variant=1),
    "decode_v1_int8": lambda: Paged(9, [700, 90, 333] * 8, [1, 2, 1] * 8, 16, variant=1, quant=True),
    "chunk": lambda: Paged(10, [700, 90, 333] * 8, [80, 90, 33] * 8, 8, N=4),
    "chunk_int8": lambda: Paged(11, [700, 90, 333] * 8, [80, 90, 33] * 8, 8, N=4, quant=True),
    "chunk_int8_short": lambda: Paged(12, [90, 40, 65] * 20, [90, 40, 33] * 20, 64, N=8, quant=True),
}


@pytest.mark.parametrize("name", SHORT_WAITS)
def test_waits_that_run_out_anywhere(name):
    """A limit of a microsecond, about a load's latency, runs out in any of the pipelines' waits,
    in any of the warps, at any point of a run over several pieces: every block still leaves
    with its copies landed, and the calls behind it are right."""
    x = SHORT_WAITS[name]()
    if isinstance(x, Paged):
        x.kv.run()
    torch.cuda.synchronize()
    gave_up = 0
    try:
        for limit in (1000, 2000, 4000, 8000) * 5:
            native.ra_set_wait_timeout_ns(limit)
            x.run()
            torch.cuda.synchronize()
            gave_up += x.status() != 0
            native.ra_set_wait_timeout_ns(DEFAULT_WAIT_NS)
            x.out.fill_(7.0)
            x.run()
            torch.cuda.synchronize()
            assert x.status() == 0
    finally:
        native.ra_set_wait_timeout_ns(DEFAULT_WAIT_NS)
    x.check(f"behind {gave_up} calls that gave up")


def rounded_between(x, slack, dtype):
    """The 16-bit numbers that x (1 - slack) and x (1 + slack) round to, in order."""
    a, b = (torch.from_numpy(x * f).to(TORCH[dtype]).double().numpy() for f in (1 - slack, 1 + slack))
    return np.minimum(a, b), np.maximum(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["int8", "e4m3", "e5m2"])
def test_read_near_the_zero_point(kind, dtype):
    """Codes at and beside their offset: (code - offset) / scale as one difference, one
    reciprocal and one product in fp32, at most 3 half steps (and their products) of the
    result, then one rounding.  A code equal to its offset is zero."""
    B, N, S, D, bs = 2, 2, 64, 64, 32
    g = np.random.default_rng(21)
    codes = g.integers(-128, 128, (4, N, bs, D)).astype(np.float64)
    if kind != "int8":
        t = torch.from_numpy(codes).to({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[kind])
        codes = t.double().numpy()
    scale = g.uniform(10, 40, (N, D)).astype(np.float32)
    offset = codes[0, :, 0].astype(np.float32)                     # integers, each some code's value
    offset[:, ::3] += np.float32(0.37)                              # and numbers beside one
    codes[:, :, ::2] = codes[0, :, 0][None, :, None]                # every second row: the offset's own code
    cache = torch.from_numpy(codes.astype(np.int8)).cuda() if kind == "int8" else \
        torch.from_numpy(codes).to({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[kind]).cuda()
    p = native.KvRmsNormRopeCacheParams(B=B, N=N, S=S, Dkv=D, Dv=D, rope_size=32, variant=2, cache_mode=native.RA_CACHE_PA_BNSD,
                                        block_num=4, block_size=bs, kv_dtype=CODE[dtype], k_cache_dtype=CODE[kind],
                                        ckv_cache_dtype=CODE[kind], epsilon=1e-5)
    sd, od = torch.from_numpy(scale).cuda(), torch.from_numpy(offset).cuda()
    outs = [torch.full((B, N, S, D), 7.0, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    native.kv_cache_read(p, torch.arange(B * S, device="cuda"), cache, cache, *outs, sd, sd, od, od)
    rows = codes.reshape(B, 2, N, bs, D).transpose(0, 2, 1, 3, 4).reshape(B, N, S, D)
    want = (rows - offset.astype(np.float64)[None, :, None]) / scale.astype(np.float64)[None, :, None]
    lo, hi = rounded_between(want, 3.01 * 2.0 ** -24, dtype)
    assert (want == 0).mean() > 0.25
    for out in outs:
        got = out.double().cpu().numpy()
        assert (got[want == 0] == 0).all()
        assert ((lo <= got) & (got <= hi)).all(), float(((got < lo) | (got > hi)).mean())


@pytest.mark.parametrize("variant,quant", [(2, False), (2, True), (1, False), (1, True)])
def test_rows_of_a_serving_cache_read_back(variant, quant):
    """Every row of a cache that the writer filled and attention reads: the bytes that are there,
    dequantised, within three half steps of fp32 and the last rounding."""
    x = Paged(23, [130, 130], [100, 100], 4, variant=variant, quant=quant)
    x.kv.run()
    x.run()
    c = x.kv.case
    read = [torch.full((c.B, c.N, c.S, w), 7.0, dtype=torch.bfloat16, device="cuda") for w in (c.k_width, c.ckv_width)]
    native.kv_cache_read(x.kv.params, x.kv.index, x.kv.k_cache, x.kv.ckv_cache, *read, x.kv.k_scale, x.kv.v_scale,
                         x.kv.k_offset, x.kv.v_offset)
    torch.cuda.synchronize()
    for got, cache, scale, offset, kind in ((read[0], x.kv.k_cache, c.k_scale, c.k_offset, c.k_qtype),
                                            (read[1], x.kv.ckv_cache, c.v_scale, c.v_offset, c.v_qtype)):
        host = cache.cpu().numpy() if quant else cache.view(torch.int16).cpu().numpy().view(np.uint16)
        want, bad = oracle.attention.kv_cache_read(c.index, host, B=c.B, N=c.N, S=c.S, cache_mode=c.cache_mode,
                                                   block_size=c.block_size, stored=kind if quant else "bf16", scale=scale,
                                                   offset=offset)
        lo, hi = rounded_between(want, 3.01 * 2.0 ** -24 if quant else 0.0, "bf16")
        got = got.double().cpu().numpy()
        assert bad == 0 and np.abs(want).mean() > 0.1 and ((lo <= got) & (got <= hi)).all()


def one_cache(lens, kt, dtype, variant=2):
    """Zeroed caches of one kv head in pages of 64, their parameters, the table and, over codes,
    scales of 2 for keys and 1 for values.  Keys and values 64 wide, V1's with 16 rotated channels."""
    bs, pages = 64, [-(-n // 64) for n in lens]
    n_pages = sum(pages)
    Dkv, Dv, R = (64, 64, 32) if variant == 2 else (80, 64, 16)
    kw = Dkv if variant == 2 else R
    tt = {**TORCH, "int8": torch.int8, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[kt]
    kc = torch.zeros(n_pages, 1, bs, kw, device="cuda").to(tt)
    vc = torch.zeros(n_pages, 1, bs, Dv, device="cuda").to(tt)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    quant = kt not in TORCH
    p = native.KvRmsNormRopeCacheParams(B=len(lens), N=1, S=1, Dkv=Dkv, Dv=Dv, rope_size=R, variant=variant,
                                        cache_mode=native.RA_CACHE_PA_BNSD, block_num=n_pages, block_size=bs,
                                        kv_dtype=CODE[dtype], k_cache_dtype=CODE[kt], ckv_cache_dtype=CODE[kt], epsilon=1e-5)
    scales = dict(k_rope_scale=torch.full((1, kw) if variant == 2 else (kw,), 2.0, device="cuda"),
                  c_kv_scale=torch.full((1, Dv) if variant == 2 else (Dv,), 1.0, device="cuda")) if quant else {}
    return p, kc, vc, table.cuda(), scales


def attend_cache(p, kc, vc, table, scales, q, lens, scale, causal=0):
    params = native.PagedAttentionParams(B=len(lens), total_q=q.shape[0], num_heads=q.shape[1], causal=causal, softmax_scale=scale,
                                         max_seq_len=max(lens), block_table_stride=table.shape[1])
    out = torch.full((q.shape[0], q.shape[1], p.Dv), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.zeros(native.paged_attention_workspace_bytes(p, params), dtype=torch.uint8, device="cuda")
    native.paged_attention(p, params, q, kc, vc, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws, table, lse=lse, **scales)
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0
    return out, lse


def attend_prompt(q, k, v, scale):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    p = native.packed_attention_params(q, k, v, out, softmax_scale=scale)
    ws = torch.zeros(native.packed_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    native.packed_attention(p, q, k, v, out, ws, lse)
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("new", [1, 90], ids=["step", "chunk"])
@pytest.mark.parametrize("kt,dtype,variant", [("fp16", "fp16", 2), ("int8", "bf16", 2), ("e4m3", "bf16", 2), ("int8", "fp16", 2),
                                              ("int8", "bf16", 1), ("int8", "fp16", 1), ("prompt", "fp16", 0)])
def test_a_tail_far_below_a_sink(kt, dtype, variant, new):
    """One key holds nearly all of the weight and has the value 0; 299 keys 17.5 nats (2^-25.2)
    below it have the value 100 (E4M3, of three bits: 18 and 96).  What is left of them is the result.  An fp16 weight is held
    with 2^7 (the largest one between 2^7 and 2^15), so each is off by half of fp16's least
    number at most: 2^-25 / 2^7 of the largest one."""
    n = 300
    q = torch.zeros(new, 2, 80 if variant == 1 else 64, dtype=TORCH[dtype], device="cuda")
    if kt == "prompt":
        q[..., 0] = 1
        k, v = torch.zeros(n, 1, 64, dtype=q.dtype, device="cuda"), torch.full((n, 1, 64), 100.0, dtype=q.dtype, device="cuda")
        k[0, 0, 0], v[0] = 17.5, 0
        out, lse = attend_prompt(q, k, v, 1.0)
    else:
        p, kc, vc, table, scales = one_cache([n], kt, dtype, variant)
        q[..., 64 if variant == 1 else 0] = 1  # (V1's latent channels, a part of the key, meet zeros)
        kc[0, 0, 0, 0] = torch.tensor({"int8": 35.0, "e4m3": 36.0}.get(kt, 17.5), device="cuda").to(kc.dtype)
        vc.copy_(torch.full(vc.shape, 96.0 if kt == "e4m3" else 100.0, device="cuda").to(vc.dtype))
        vc[0, 0, 0] = torch.zeros(vc.shape[-1], device="cuda").to(vc.dtype)
        out, lse = attend_cache(p, kc, vc, table, scales, q, [n], 1.0)
    top, value = (18.0, 96.0) if kt == "e4m3" else (17.5, 100.0)
    total = 1 + (n - 1) * np.exp(-top)
    want = (n - 1) * np.exp(-top) * value / total
    tol = (n - 1) * 2.0 ** -32 * value + 2 * HALF_STEP[dtype] * want
    err = (out.double() - want).abs().max().item()
    assert err <= tol, (err / want, tol / want)
    assert (lse.double() - (top + np.log(total))).abs().max() <= 2.0 ** -17 * (1 + top)


@pytest.mark.parametrize("new", [1, 90], ids=["step", "chunk"])
@pytest.mark.parametrize("kt,variant", [("bf16", 2), ("int8", 2), ("int8", 1), ("bf16", 1), ("prompt", 0)])
@pytest.mark.parametrize("scale,zero_q", [(1e-38, False), (1e-9, True)], ids=["least_scale", "zero_queries"])
def test_scores_that_are_all_alike(scale, zero_q, kt, variant, new):
    """A softmax scale near fp32's least normal number, or queries of zeros under a small one:
    every weight is alike, the result is the mean of the values and the lse log(n); with an
    item in one piece (n = 50) and in many (n = 5000)."""
    for n in (50, 5000):
        g = torch.Generator(device="cuda").manual_seed(22)
        Dk = 80 if variant == 1 else 64
        q = torch.randn(new, 2, Dk, device="cuda", generator=g).bfloat16()
        if zero_q:
            q.zero_()
        rnd = lambda shape: torch.randint(-100, 100, shape, device="cuda", generator=g).float()
        if kt == "prompt":
            k, v = rnd((n, 1, 64)).bfloat16(), rnd((n, 1, 64)).bfloat16()
            values = v[:, 0]
            out, lse = attend_prompt(q, k, v, scale)
        else:
            p, kc, vc, table, scales = one_cache([n], kt, "bf16", variant)
            kc.copy_(rnd(kc.shape).to(kc.dtype))
            vc.copy_(rnd(vc.shape).to(vc.dtype))
            values = vc[:, 0].reshape(-1, 64)[:n]
            out, lse = attend_cache(p, kc, vc, table, scales, q, [n], scale)
        values = values.double()
        mean, spread = values.mean(0), values.abs().mean(0)
        assert ((out.double() - mean).abs() <= HALF_STEP["bf16"] * (mean.abs() + spread) + 2.0 ** -17 * spread).all()
        assert (lse.double() - np.log(n)).abs().max() <= 2.0 ** -17 * (1 + np.log(n))


@pytest.mark.parametrize("lens,heads,N,variant,quant", [
    ([900, 3, 64, 700, 1, 128, 450, 65, 333, 899] * 2, 8, 8, 2, False),        # one whole item a block
    ([900, 3, 64, 700, 1, 128, 450, 65, 333, 899] * 4, 8, 8, 2, True),         # whole items, two or three a block
    ([9000] + [130] * 30, 8, 1, 1, False),                                     # one cut into many pieces among whole ones
    ([9000] + [130] * 30, 16, 8, 2, True),
], ids=["whole", "whole_int8", "long_v1", "long_int8"])
def test_decode_batches_of_very_different_lengths(lens, heads, N, variant, quant):
    x = Paged(24, lens, [1] * len(lens), heads, N=N, variant=variant, quant=quant)
    x.kv.run()
    x.run()
    torch.cuda.synchronize()
    assert x.status() == 0
    x.check("lengths")
