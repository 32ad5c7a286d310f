"""The boundary of packed_attention, paged_attention and kv_cache_read, on the CPU: every
rejection with its status, the workspace sizes, the binding's own refusals (shapes, strides,
types, short tensors), the kernels' register budgets, and the oracle against closed forms.
Every call runs under the validate-only hook: no placeholder address reaches a kernel."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
from attention_util import half_values
from rope_attention_gb300 import build, native, runner, synth
from test_kernel_resources import ptxas_report

A16 = 0x10000  # 16-byte aligned placeholder address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = native.load()
    lib.ra_test_validate_only(1)
    yield lib
    lib.ra_test_validate_only(0)


def packed(**kw):
    base = dict(B=2, total_q=100, total_k=100, num_heads=4, num_kv_heads=2, head_dim=64, dtype=native.RA_BF16, causal=1,
                softmax_scale=0.125, q_token_stride=512, q_head_stride=64, k_token_stride=512, k_head_stride=64,
                v_token_stride=512, v_head_stride=64, out_token_stride=256, out_head_stride=64)
    base.update(kw)
    return native.PackedAttentionParams(**base)


def call_packed(L, p=None, **over):
    a = dict(q=A16, k=A16, v=A16, out=A16, lse=None, cq=None, ck=None, ws=A16, n=64 << 20)
    a.update(over)
    st = L.packed_attention(ctypes.byref(p or packed()), a["q"], a["k"], a["v"], a["out"], a["lse"], a["cq"], a["ck"],
                            a["ws"], a["n"], None)
    return st, L.ra_last_error().decode()


def test_packed_accepts(L):
    assert call_packed(L) == (0, "")
    assert call_packed(L, packed(total_q=101), cq=A16) == (0, "")
    assert call_packed(L, packed(num_heads=65535, num_kv_heads=1, out_token_stride=65535 * 64)) == (0, "")
    # NBSd strides: heads outside tokens
    assert call_packed(L, packed(q_token_stride=64, q_head_stride=6400, out_token_stride=64, out_head_stride=6400)) == (0, "")


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -1), (dict(total_q=0), -1), (dict(total_k=0), -1), (dict(total_q=1 << 31), -1), (dict(num_heads=3), -1),
    (dict(num_kv_heads=0), -1), (dict(num_heads=65536), -1), (dict(head_dim=24), -1), (dict(head_dim=0), -1),
    (dict(head_dim=144), -2), (dict(dtype=native.RA_FP32), -1), (dict(causal=2), -1), (dict(softmax_scale=0.0), -1),
    (dict(softmax_scale=-1.0), -1), (dict(softmax_scale=float("nan")), -1), (dict(softmax_scale=float("inf")), -1),
    (dict(q_token_stride=-8), -1), (dict(k_head_stride=60), -3), (dict(v_token_stride=0), -1),
    (dict(k_token_stride=1 << 39), -1), (dict(out_token_stride=64), -1), (dict(out_head_stride=32), -1),
    (dict(total_q=101), -1), (dict(total_k=101), -1),
])
def test_packed_params_rejected(L, kw, code):
    st, msg = call_packed(L, packed(**kw))
    assert st == code and msg


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(q=A16 + 2), -3), (dict(k=A16 + 8), -3), (dict(v=A16 + 4), -3), (dict(out=A16 + 8), -3), (dict(lse=A16 + 2), -3),
    (dict(cq=A16 + 1), -3), (dict(ck=A16 + 2), -3), (dict(ws=A16 + 4), -3), (dict(n=100), -4),
])
def test_packed_call_rejected(L, over, code):
    st, msg = call_packed(L, **over)
    assert st == code and msg


def cache(**kw):
    base = dict(B=2, N=2, S=1, Dkv=192, Dv=128, rope_size=64, variant=2, cache_mode=native.RA_CACHE_PA_BNSD, block_num=8,
                block_size=32, kv_dtype=native.RA_BF16, k_cache_dtype=native.RA_BF16, ckv_cache_dtype=native.RA_BF16,
                epsilon=1e-5)
    base.update(kw)
    return native.KvRmsNormRopeCacheParams(**base)


def paged(**kw):
    base = dict(B=2, total_q=6, num_heads=4, causal=1, softmax_scale=0.1, max_seq_len=100, block_table_stride=4)
    base.update(kw)
    return native.PagedAttentionParams(**base)


def call_paged(L, c=None, p=None, **over):
    a = dict(q=A16, kc=A16, vc=A16, lens=A16, table=A16, cq=None, ks=None, vs=None, ko=None, vo=None, out=A16, lse=None,
             err=None, ws=A16, n=64 << 20)
    a.update(over)
    st = L.paged_attention(ctypes.byref(c or cache()), ctypes.byref(p or paged()), a["q"], a["kc"], a["vc"], a["lens"],
                           a["table"], a["cq"], a["ks"], a["vs"], a["ko"], a["vo"], a["out"], a["lse"], a["err"], a["ws"],
                           a["n"], None)
    return st, L.ra_last_error().decode()


V1 = dict(variant=1, N=1, Dkv=576, Dv=512)


def test_paged_accepts(L):
    assert call_paged(L) == (0, "")
    assert call_paged(L, cache(**V1)) == (0, "")
    assert call_paged(L, cache(k_cache_dtype=native.RA_INT8), ks=A16) == (0, "")
    norm = dict(cache_mode=native.RA_CACHE_NORM, block_num=0, block_size=0, cache_seq_len=64)
    assert call_paged(L, cache(**norm), paged(block_table_stride=0), table=None) == (0, "")


@pytest.mark.parametrize("c,p,over,code", [
    (dict(variant=3), {}, {}, -1), (dict(N=3), {}, {}, -1), (dict(variant=1, N=2), {}, {}, -1), (dict(Dkv=12), {}, {}, -1),
    (dict(variant=1, N=1, Dkv=576, Dv=500), {}, {}, -1), (dict(kv_dtype=native.RA_FP32), {}, {}, -1),
    (dict(k_cache_dtype=native.RA_INT8), {}, {}, -1), ({}, {}, dict(ks=A16), -1), ({}, {}, dict(ko=A16), -1),
    (dict(cache_mode=native.RA_CACHE_PA_NZ), {}, {}, -2), (dict(cache_mode=9), {}, {}, -1), (dict(block_num=0), {}, {}, -1),
    (dict(block_size=24), {}, {}, -1), (dict(k_cache_dtype=native.RA_INT8, block_size=16), {}, dict(ks=A16), -1),
    (dict(k_quant_scalar=1), {}, {}, -1), (dict(Dkv=272), {}, {}, -2), (dict(Dv=264), {}, {}, -2), (dict(Dkv=200), {}, {}, -2),
    (dict(variant=1, N=1, Dkv=640, Dv=576), {}, {}, -2), (dict(variant=1, N=1, Dkv=544, Dv=480), {}, {}, -2),
    (dict(variant=1, N=1, Dkv=640, Dv=512, rope_size=128), {}, {}, -2),
    ({}, dict(B=0), {}, -1), ({}, dict(total_q=0), {}, -1), ({}, dict(num_heads=5), {}, -1), ({}, dict(causal=-1), {}, -1),
    ({}, dict(softmax_scale=float("nan")), {}, -1), ({}, dict(max_seq_len=-1), {}, -1), ({}, dict(max_seq_len=1 << 31), {}, -1),
    ({}, dict(block_table_stride=0), {}, -1), ({}, dict(reserved=1), {}, -1), ({}, dict(total_q=7), {}, -1),
    ({}, dict(total_q=1 << 30), {}, -1),
    ({}, {}, dict(q=None), -1), ({}, {}, dict(kc=None), -1), ({}, {}, dict(vc=None), -1), ({}, {}, dict(lens=None), -1),
    ({}, {}, dict(table=None), -1), ({}, {}, dict(out=None), -1), ({}, {}, dict(ws=None), -1), ({}, {}, dict(q=A16 + 8), -3),
    ({}, {}, dict(kc=A16 + 8), -3), ({}, {}, dict(lens=A16 + 2), -3), ({}, {}, dict(err=A16 + 1), -3),
    ({}, {}, dict(ws=A16 + 8), -3), ({}, {}, dict(n=300), -4), ({}, dict(max_seq_len=1000), dict(n=4096), -4),
    (dict(cache_mode=native.RA_CACHE_NORM, cache_seq_len=64, B=3), dict(block_table_stride=0), dict(table=None), -1),
    (dict(cache_mode=native.RA_CACHE_NORM, cache_seq_len=64), dict(block_table_stride=0), {}, -1),
    (dict(cache_mode=native.RA_CACHE_NORM, cache_seq_len=0), dict(block_table_stride=0), dict(table=None), -1),
])
def test_paged_rejected(L, c, p, over, code):
    st, msg = call_paged(L, cache(**c), paged(**p), **over)
    assert st == code and msg


def test_paged_workspace_stays_within_its_bound(L):
    n = ctypes.c_size_t()
    for c in (cache(), cache(**V1), cache(Dkv=256, Dv=256), cache(**V1, ckv_cache_dtype=native.RA_INT8)):
        for q in (2, 64, 5000):
            p = paged(total_q=q, num_heads=128 if c.variant == 1 else 64, max_seq_len=1 << 20, block_table_stride=1 << 15)
            assert L.paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(p), ctypes.byref(n)) == 0
            assert 256 < n.value <= 64 << 20
            big = n.value
            p.max_seq_len = 10
            assert L.paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(p), ctypes.byref(n)) == 0 and n.value <= big
    assert L.paged_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(paged()), None) == -1
    assert L.packed_attention_workspace_bytes(ctypes.byref(packed()), None) == -1
    assert L.packed_attention_workspace_bytes(ctypes.byref(packed()), ctypes.byref(n)) == 0 and 0 < n.value <= 64 << 20


def call_read(L, c=None, **over):
    a = dict(index=A16, kc=A16, vc=A16, ks=None, vs=None, ko=None, vo=None, k=A16, v=A16, err=None)
    a.update(over)
    st = L.kv_cache_read(ctypes.byref(c or cache(S=5)), a["index"], a["kc"], a["vc"], a["ks"], a["vs"], a["ko"], a["vo"],
                         a["k"], a["v"], a["err"], None)
    return st, L.ra_last_error().decode()


@pytest.mark.parametrize("c,over,code", [
    ({}, {}, 0), ({}, dict(k=None), 0), ({}, dict(v=None, vc=None), 0), (dict(cache_mode=native.RA_CACHE_PA_BLK_BNSD), {}, 0),
    (dict(S=0), {}, -1), (dict(B=0), {}, -1), ({}, dict(index=None), -1), ({}, dict(k=None, v=None), -1),
    ({}, dict(kc=None), -1), ({}, dict(index=A16 + 4), -3), ({}, dict(k=A16 + 8), -3), ({}, dict(err=A16 + 2), -3),
    (dict(k_cache_dtype=native.RA_INT8), dict(ks=A16 + 4), -3), (dict(Dv=2048), {}, -1), (dict(rope_size=12), {}, -1),
    (dict(cache_mode=native.RA_CACHE_PA_BLK_NZ), {}, -2),
])
def test_read_checks(L, c, over, code):
    st, msg = call_read(L, cache(**{"S": 5, **c}), **over)
    assert st == code and bool(msg) == (code != 0)


def test_status_checks(L):
    v = ctypes.c_int32(5)
    assert L.attention_status(None, None, ctypes.byref(v)) == -1
    assert L.attention_status(A16 + 4, None, ctypes.byref(v)) == -3
    assert L.attention_status(A16, None, None) == -1
    assert L.attention_status(A16, None, ctypes.byref(v)) == 0 and v.value == 0


# ---------------------------------------------------------------- the binding
def test_packed_params_from_projection_views():
    T, nq, nk, d = 6, 4, 2, 64
    bsd = torch.zeros(T, (nq + 2 * nk) * d, dtype=torch.bfloat16).view(T, nq + 2 * nk, d)
    out = torch.zeros(T, nq, d, dtype=torch.bfloat16)
    p = native.packed_attention_params(bsd[:, :nq], bsd[:, nq:nq + nk], bsd[:, nq + nk:], out, B=2, causal=True)
    assert (p.total_q, p.total_k, p.num_heads, p.num_kv_heads, p.head_dim) == (T, T, nq, nk, d)
    assert (p.q_token_stride, p.q_head_stride, p.v_token_stride, p.out_token_stride) == (512, 64, 512, 256)
    assert p.softmax_scale == pytest.approx(0.125) and p.causal == 1
    nbsd = torch.zeros(nq + 2 * nk, T, d, dtype=torch.bfloat16).transpose(0, 1)
    p = native.packed_attention_params(nbsd[:, :nq], nbsd[:, nq:nq + nk], nbsd[:, nq + nk:], out)
    assert (p.k_token_stride, p.k_head_stride) == (64, T * 64)
    # a storage one element short of what those strides address
    ws = torch.zeros(256, dtype=torch.uint8)
    need = ((T - 1) * 64 + (nq - 1) * T * 64 + 64) * 2
    short = torch.zeros(need // 2 - 1, dtype=torch.bfloat16).view(1, 1, -1)
    with pytest.raises(ValueError, match=f"^q: the call needs {need} bytes, the tensor's storage holds {need - 2}"):
        native.packed_attention(p, short, nbsd[:, nq:nq + nk], nbsd[:, nq + nk:], out, ws)


def test_packed_binding_refusals():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    good = (t(5, 4, 64), t(7, 2, 64), t(7, 2, 64), t(5, 4, 64))
    for i, x, msg in ((1, t(7, 2, 32), "k"), (2, t(6, 2, 64), "v"), (3, t(5, 4, 64, dt=torch.float16), "out"),
                      (0, t(5, 64), "q"), (1, t(7, 2, 128)[..., ::2], "k"), (3, t(4, 4, 64), "out")):
        bad = list(good)
        bad[i] = x
        with pytest.raises(ValueError, match=f"^{msg}: "):
            native.packed_attention_params(*bad)
    with pytest.raises(ValueError, match="^q: "):
        native.packed_attention_params(*(x.float() for x in good))
    p = native.packed_attention_params(*good)
    ws = torch.zeros(256, dtype=torch.uint8)
    short = t(4, 4, 64)
    with pytest.raises(ValueError, match=r"^q: the call needs 2560 bytes"):
        native.packed_attention(p, short, *good[1:], ws)
    with pytest.raises(ValueError, match=r"^lse: the call needs 80 bytes"):
        native.packed_attention(p, *good, ws, lse=torch.zeros(19))
    with pytest.raises(ValueError, match=r"^cu_seqlens_k: the call needs 8 bytes"):
        native.packed_attention(p, *good, ws, cu_seqlens_k=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match=r"expected a CUDA tensor"):
        native.packed_attention(p, *good, ws)
    with pytest.raises(TypeError, match="^v: expected a tensor"):
        native.packed_attention(p, *good[:2], None, good[3], ws)
    with pytest.raises(TypeError, match="^params: "):
        native.packed_attention(cache(), *good, ws)
    with pytest.raises(TypeError):
        native.packed_attention_params(*good, B="two")


def test_paged_and_read_binding_refusals():
    c, p = cache(), paged()
    half = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    kc, vc = half(8, 2, 32, 192), half(8, 2, 32, 128)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = dict(q=half(6, 4, 192), k_cache=kc, ckv_cache=vc, seq_lens=i32(2), out=half(6, 4, 128),
                workspace=torch.zeros(1 << 20, dtype=torch.uint8), block_table=i32(2, 4))
    for name, x, msg in (("q", half(5, 4, 192), "the call needs"), ("k_cache", kc[:-1], "the call needs"),
                         ("ckv_cache", vc[:-1], "the call needs"), ("seq_lens", i32(1), "the call needs"),
                         ("block_table", i32(1, 4), "expected"), ("block_table", i32(8), "expected"),
                         ("block_table", i32(2, 3), "the call needs"), ("out", half(6, 4, 127), "the call needs"),
                         ("q", good["q"].half(), "expected torch.bfloat16"), ("k_cache", kc.half(), "expected"),
                         ("k_cache", torch.zeros(8, 2, 32, 384, dtype=torch.int8), "expected")):
        with pytest.raises(ValueError, match=f"^{name}: {msg}"):
            native.paged_attention(c, p, **{**good, name: x})
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        native.paged_attention(c, p, **good)
    c = cache(S=5)
    good = dict(index=torch.zeros(10, dtype=torch.int64), k_cache=kc, ckv_cache=vc, k_out=half(2, 2, 5, 192),
                c_kv_out=half(2, 2, 5, 128))
    for name, x in (("index", good["index"][:9]), ("k_out", good["k_out"][:1]), ("c_kv_out", good["c_kv_out"][:1])):
        with pytest.raises(ValueError, match=f"^{name}: the call needs"):
            native.kv_cache_read(c, **{**good, name: x})
    with pytest.raises(ValueError, match="^k_out: expected"):
        native.kv_cache_read(c, **{**good, "k_out": good["k_out"].half()})


# ---------------------------------------------------------------- kernels
@pytest.mark.parametrize("file,kernel,budget", [
    # the tile kernel launches 384 threads (2 x 216 + 72 = 3 x 168), with converters 512 (2 x 192 + 2 x 64 = 4 x 128)
    ("packed_attention.cu", "tile_attention_kernel", {168: 4}),
    ("paged_tile.cu", "tile_attention_kernel", {168: 4, 128: 4}),
    ("paged_attention.cu", "paged_attention_kernel", {128: 4}),   # 2 x 160 + 120 + 72 = 4 x 128
    ("cache_read.cu", "cache_read_kernel", {64: 2}),              # four blocks of 256 threads an SM
])
def test_register_budgets(file, kernel, budget, tmp_path):
    """The attention kernels move registers between their warpgroups: what they give out must
    be what they were launched with, or a warpgroup waits for ever."""
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    rep = ptxas_report(file, str(tmp_path))
    hits = [v for n, v in rep.items() if kernel in n]
    assert {r: sum(h[0] == r for h in hits) for r in {h[0] for h in hits}} == budget, hits
    # the softmax warps run with more registers than ptxas was given: a few words that live
    # across their loops may spill
    assert all(spill <= (384 if 128 in budget and 168 in budget else 160) for _, spill in hits), hits
    # four blocks of 256 threads an SM, or two
    assert all((regs <= 64 and spill <= 128) if "Li4" in n else (regs <= 128 and spill == 0)
               for n, (regs, spill) in rep.items() if "attention_join_kernel" in n)


# ---------------------------------------------------------------- the oracle
def test_oracle_attend_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((5, 3))
    o, lse, _ = oracle.attention.attend(np.zeros((2, 4)), rng.standard_normal((5, 4)), v, 1.0, False)
    assert np.allclose(o, v.mean(0)) and np.allclose(lse, np.log(5))
    # one key far above the others takes everything
    k = np.zeros((5, 4))
    k[3, 0] = 1000.0
    o, _, _ = oracle.attention.attend(np.eye(1, 4), k, v, 1.0, False)
    assert np.allclose(o[0], v[3])
    # causal with two more queries than keys: the first two rows see nothing, the third key 0
    o, lse, _ = oracle.attention.attend(rng.standard_normal((7, 4)), rng.standard_normal((5, 4)), v, 1.0, True)
    assert np.all(o[:2] == 0) and np.all(lse[:2] == -np.inf) and np.allclose(o[2], v[0])


def test_oracle_attention_against_torch():
    q, k, v = (half_values(3, i, s, "bf16")[1] for i, s in enumerate([(9, 4, 16), (9, 2, 16), (9, 2, 16)]))
    res = oracle.attention.packed_attention(q, k, v, starts_q=[0, 4, 9], starts_k=[0, 4, 9], scale=0.25, causal=True)
    for a, z in ((0, 4), (4, 9)):
        t = lambda x: torch.from_numpy(x[a:z]).transpose(0, 1)
        want = torch.nn.functional.scaled_dot_product_attention(t(q), t(k).repeat_interleave(2, 0), t(v).repeat_interleave(2, 0),
                                                                is_causal=True, scale=0.25)
        assert np.allclose(res["out"][a:z], want.transpose(0, 1).numpy(), atol=1e-12)


def test_oracle_paged_equals_packed_through_any_table():
    kb, k = half_values(4, 0, (40, 2, 32), "bf16")
    vb, v = half_values(4, 1, (40, 2, 16), "bf16")
    q = half_values(4, 2, (3, 4, 32), "bf16")[1]
    want = oracle.attention.packed_attention(q, k, v, starts_q=[0, 3], starts_k=[0, 40], scale=0.2, causal=True)
    table = np.array([[4, 0, 2]])
    for mode in ("PA", "PA_BNSD"):
        kc = np.zeros((5, 16, 2, 32), np.uint16)
        vc = np.zeros((5, 16, 2, 16), np.uint16)
        for j in range(40):
            kc[table[0, j // 16], j % 16], vc[table[0, j // 16], j % 16] = kb[j], vb[j]
        if mode == "PA_BNSD":
            kc, vc = kc.transpose(0, 2, 1, 3), vc.transpose(0, 2, 1, 3)
        got = oracle.attention.paged_attention(q, kc, vc, variant=2, seq_lens=[40], starts_q=[0, 3], scale=0.2, causal=True,
                                               cache_mode=mode, block_size=16, table=table)
        assert np.allclose(got["out"], want["out"]) and np.allclose(got["lse"], want["lse"])


def test_oracle_read_inverts_the_writer():
    c = synth.make_kv("pin", 5, variant=2, B=2, N=2, S=9, Dkv=32, Dv=16, rope_size=8, block_size=32, block_num=2, quant_k=True,
                      skip_frac=0.2)
    r = oracle.kv_rms_norm_rope_cache(c.kv, c.gamma, c.cos, c.sin, c.index, c.k_cache, c.ckv_cache, variant=2, rope_size=8,
                                      block_size=32, k_scale=c.k_scale, k_offset=c.k_offset, v=c.v, is_output_kv=True)
    got, bad = oracle.attention.kv_cache_read(c.index, r["k_cache"], B=2, N=2, S=9, cache_mode="PA_BNSD", block_size=32,
                                              stored="int8", scale=c.k_scale, offset=c.k_offset)
    keep = (c.index != -1).reshape(2, 9)
    step = 0.5 / c.k_scale[None, :, None, :]     # half a code
    inside = np.abs(r["k_rope"] * c.k_scale[None, :, None, :] + c.k_offset[None, :, None, :]) < 127
    ok = (np.abs(got - r["k_rope"]) <= step * 1.001) | ~inside
    assert bad == 0 and ok[keep[:, None, :].repeat(2, 1)].all()
    assert (got[~keep[:, None, :].repeat(2, 1)] == 0).all()
