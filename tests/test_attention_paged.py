"""paged_attention on the GPU against the fp64 oracle: both variants, every cache mode and
stored type, single tokens and chunks, row counts around the tile sizes, lengths around the
key tiles and pages (none at all among them), bad pages, and rows outside every sequence."""
import numpy as np
import pytest
import torch

import oracle
from attention_util import TORCH, check_attention, half_values
from rope_attention_gb300 import native, synth

pytestmark = pytest.mark.gpu

CODE = {"bf16": native.RA_BF16, "fp16": native.RA_FP16, "int8": native.RA_INT8, "e4m3": native.RA_FP8_E4M3,
        "e5m2": native.RA_FP8_E5M2}


def stored(seed, k, shape, kind, params_shape, offsets=True, scale_range=(10.0, 40.0)):
    """A cache's host array with its scale and offset; unused rows are made NaN by the caller."""
    if kind in TORCH:
        return half_values(seed, k, shape, kind)[0], None, None
    scale = synth.stream(seed, k + 1).uniform(*scale_range, params_shape).astype(np.float32)
    offset = synth.stream(seed, k + 2).uniform(-2, 2, params_shape).astype(np.float32) if offsets else None
    if kind == "int8":
        return synth.stream(seed, k).integers(-128, 128, shape).astype(np.int8), scale, offset
    x = synth.stream(seed, k).standard_normal(shape, dtype=np.float32) * 30
    t = torch.from_numpy(x).clamp(-448, 448).to({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[kind])
    return t.view(torch.uint8).numpy(), scale, offset


def device(x, kind):
    if x is None:
        return None
    if kind in TORCH:
        return torch.from_numpy(x.view(np.int16)).cuda().view(TORCH[kind])
    return torch.from_numpy(x).cuda()


def run_case(seed, *, variant, lens, news, heads, N=1, Dkv=192, Dv=128, R=64, mode="PA_BNSD", bs=32, kt="bf16", vt="bf16",
             dtype="bf16", causal=True, scalar=False, offsets=True, tail=0, bad_pages=(), std=1.0, max_len=None,
             scale_range=(10.0, 40.0), given_starts=True):
    B = len(lens)
    kw, vw = (R, Dv) if variant == 1 else (Dkv, Dv)
    pages = [-(-n // bs) for n in lens]
    n_pages = sum(pages) + 2
    if mode == "Norm":
        cap = max(max(lens), 1) + 5
        shape = (B, N, cap)
    else:
        shape = (n_pages, bs, N) if mode == "PA" else (n_pages, N, bs)
    ps = lambda w: ((1,) if scalar else (w,)) if variant == 1 else (N, w)
    kc, ks, ko = stored(seed, 10, shape + (kw,), kt, ps(kw), offsets, scale_range)
    vc, vs, vo = stored(seed, 20, shape + (vw,), vt, ps(vw), offsets, scale_range)
    table = None
    used = np.zeros(shape[:2] if mode == "PA" else (shape[0], shape[2]), bool)
    if mode == "Norm":
        for b, n in enumerate(lens):
            used[b, :n] = True
    else:
        ids = synth.stream(seed, 1).permutation(n_pages)
        table = np.full((B, max(max(pages), 1) + 1), 1 << 30, np.int32)
        at = 0
        for b, n in enumerate(lens):
            table[b, :pages[b]] = ids[at:at + pages[b]]
            at += pages[b]
            for j in range(n):
                used[table[b, j // bs], j % bs] = True
        for b, i, value in bad_pages:
            table[b, i] = value
    # slots that no sequence has hold NaN (bf16 0x7FBF is one, fp16's too, and FP8's 0x7F)
    for c, kind in ((kc, kt), (vc, vt)):
        fill = {"int8": -77, "e4m3": 0x7F, "e5m2": 0x7F}.get(kind, 0x7FBF)
        if mode == "PA":
            c[~used] = fill
        else:
            np.moveaxis(c, 1, 2)[~used] = fill
    starts = [0] + list(np.cumsum(news))
    qb, q = half_values(seed, 0, (starts[-1] + tail, heads, Dkv), dtype, std)
    qd = torch.from_numpy(qb.view(np.int16)).cuda().view(TORCH[dtype])
    out = torch.full((starts[-1] + tail, heads, vw), 7.0, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((starts[-1] + tail, heads), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = native.KvRmsNormRopeCacheParams(
        B=B, N=N, S=1, Dkv=Dkv, Dv=Dv, rope_size=R, variant=variant, cache_mode=synth.CACHE_MODES[mode],
        block_num=0 if mode == "Norm" else n_pages, block_size=0 if mode == "Norm" else bs, kv_dtype=CODE[dtype],
        k_cache_dtype=CODE[kt], ckv_cache_dtype=CODE[vt], epsilon=1e-5, cache_seq_len=cap if mode == "Norm" else 0,
        k_quant_scalar=1 if scalar and ks is not None else 0, c_kv_quant_scalar=1 if scalar and vs is not None else 0)
    scale = Dkv ** -0.5
    p = native.PagedAttentionParams(B=B, total_q=starts[-1] + tail, num_heads=heads, causal=1 if causal else 0,
                                    softmax_scale=scale, max_seq_len=max_len or max(lens))
    p.block_table_stride = 0 if table is None else table.shape[1]
    ws = torch.zeros(native.paged_attention_workspace_bytes(cache, p), dtype=torch.uint8, device="cuda")
    dev = lambda x: None if x is None else torch.from_numpy(np.asarray(x)).cuda()
    args = dict(block_table=dev(table), cu_seqlens_q=torch.tensor(starts, dtype=torch.int32, device="cuda") if given_starts else None,
                k_rope_scale=dev(ks), c_kv_scale=dev(vs), k_rope_offset=dev(ko), c_kv_offset=dev(vo), lse=lse,
                dev_error_count=err)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kd, vd = device(kc, kt), device(vc, vt)
    native.paged_attention(cache, p, qd, kd, vd, lens_d, out, ws, **args)
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0
    ref = oracle.attention.paged_attention(
        q, kc, vc, variant=variant, seq_lens=lens, starts_q=starts, scale=scale, causal=causal, cache_mode=mode,
        block_size=bs, table=table, k_type=kt if ks is not None else dtype, v_type=vt if vs is not None else dtype,
        k_scale=ks, k_offset=ko, v_scale=vs, v_offset=vo)
    quant_k = ks is not None or (variant == 1 and vs is not None)
    per_head = (lambda x: None if x is None else np.repeat(x, heads // N, axis=0) if x.ndim == 2 else x)
    worst = check_attention(out, lse, ref, f"{variant} {mode} {kt} {vt} {lens} {news}", dtype=dtype, Dk=Dkv,
                            p_type="fp16" if vs is not None else dtype, q_step=2.0 ** -11 if quant_k else 0.0,
                            v_scale=per_head(vs), v_offset=per_head(vo), keys=max(lens + [1]))
    assert (int(err) > 0) == bool(bad_pages)
    if tail and given_starts:
        assert (out[starts[-1]:] == 7).all() and (lse[starts[-1]:] == 7).all()
    # the same call again, on a workspace that holds the first one's partial results
    again = torch.full_like(out, 7.0)
    args["lse"] = None
    native.paged_attention(cache, p, qd, kd, vd, lens_d, again, ws, **args)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    return worst


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 128, 129, 300, 1000])
def test_decode_lengths(n):
    run_case(1, variant=2, lens=[n], news=[1], heads=8, N=2)


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD", "Norm"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("e4m3", "e4m3"), ("e5m2", "e5m2"),
                                   ("int8", "bf16"), ("bf16", "e4m3")])
def test_v2_types_and_modes(mode, kt, vt):
    run_case(2, variant=2, lens=[150, 40, 333], news=[1, 3, 20], heads=12, N=4, mode=mode, kt=kt, vt=vt)


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("e4m3", "e5m2"), ("int8", "bf16"),
                                   ("bf16", "int8")])
def test_v1_types_and_modes(mode, kt, vt):
    run_case(3, variant=1, lens=[150, 40, 333], news=[1, 2, 5], heads=16, Dkv=576, Dv=512, mode=mode, kt=kt, vt=vt)


@pytest.mark.parametrize("scalar,offsets", [(True, True), (False, False)])
def test_v1_quantisation_forms(scalar, offsets):
    run_case(4, variant=1, lens=[100, 65], news=[1, 1], heads=8, Dkv=576, Dv=512, kt="int8", vt="int8", scalar=scalar,
             offsets=offsets)


def test_v1_norm_and_small_widths():
    run_case(5, variant=1, lens=[70, 90], news=[2, 1], heads=5, Dkv=80, Dv=64, R=16, mode="Norm")


@pytest.mark.parametrize("dims", [(16, 16, 8), (64, 64, 32), (96, 80, 32), (128, 128, 64), (256, 256, 64), (80, 208, 16)])
@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_v2_widths(dims, kt):
    run_case(6, variant=2, lens=[100, 200], news=[1, 30], heads=6, N=2, Dkv=dims[0], Dv=dims[1], R=dims[2], kt=kt, vt=kt)


@pytest.mark.parametrize("heads", [1, 3, 15, 16, 17, 33, 64, 65, 128])
def test_v1_head_counts(heads):
    run_case(7, variant=1, lens=[130, 20], news=[1, 1], heads=heads, Dkv=576, Dv=512)


@pytest.mark.parametrize("new", [1, 2, 15, 16, 17, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_chunks(new, causal):
    run_case(8, variant=2, lens=[400, max(new, 40)], news=[new, min(new, 40)], heads=4, N=2, causal=causal)


def test_more_queries_than_keys():
    run_case(9, variant=2, lens=[20, 0, 3], news=[50, 4, 7], heads=2, N=1, causal=True)
    run_case(9, variant=2, lens=[20, 0, 3], news=[50, 4, 7], heads=2, N=1, causal=False)


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_split_over_blocks_and_empty_sequences(kt):
    run_case(10, variant=2, lens=[5000, 0, 1, 1500, 64], news=[1, 1, 1, 4, 0], heads=8, N=2, kt=kt, vt=kt, tail=3)
    run_case(11, variant=1, lens=[4100], news=[2], heads=16, Dkv=576, Dv=512, kt=kt, vt=kt, bs=64)


def test_many_sequences_more_than_threads():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 90, 601)]
    run_case(12, variant=2, lens=lens, news=[1] * 601, heads=2, N=1, Dkv=64, Dv=64, R=32)


@pytest.mark.parametrize("kt", ["bf16", "e4m3"])
def test_bad_pages_are_left_out(kt):
    run_case(13, variant=2, lens=[300, 100], news=[5, 1], heads=4, N=2, kt=kt, vt=kt, bad_pages=[(0, 1, -1), (0, 4, 1 << 20)])


def test_every_page_bad():
    run_case(14, variant=2, lens=[40], news=[2], heads=4, N=2, bad_pages=[(0, 0, -7), (0, 1, -7)])


def test_fp16_and_scales_far_from_one():
    run_case(15, variant=2, lens=[200, 100], news=[3, 1], heads=4, N=2, dtype="fp16", kt="fp16", vt="fp16")
    run_case(16, variant=2, lens=[200, 100], news=[3, 1], heads=4, N=2, dtype="fp16", kt="int8", vt="int8")
    run_case(17, variant=2, lens=[200, 100], news=[3, 1], heads=4, N=2, kt="int8", vt="int8", scale_range=(2e4, 9e4))


def test_equal_tokens_without_starts():
    run_case(18, variant=2, lens=[100, 130, 9], news=[3, 3, 3], heads=4, N=2, given_starts=False)


def test_large_scores():
    run_case(19, variant=2, lens=[900], news=[40], heads=4, N=2, std=20.0)


# ---------------------------------------------------------------- many rows per sequence and kv head
@pytest.mark.parametrize("dims", [(64, 64, 32), (96, 80, 32), (128, 128, 64), (160, 48, 64), (192, 128, 64), (16, 16, 8)])
@pytest.mark.parametrize("kt", ["bf16", "int8", "e4m3", "e5m2"])
def test_chunk_widths_and_types(dims, kt):
    run_case(20, variant=2, lens=[300, 90, 0], news=[150, 90, 3], heads=4, N=2, Dkv=dims[0], Dv=dims[1], R=dims[2], kt=kt, vt=kt)


@pytest.mark.parametrize("mode,bs", [("PA", 16), ("PA", 96), ("PA_BNSD", 32), ("PA_BNSD", 64), ("PA_BNSD", 128), ("PA_BNSD", 160),
                                     ("PA_BNSD", 256), ("Norm", 0)])
@pytest.mark.parametrize("kt,Dkv", [("bf16", 128), ("bf16", 192), ("int8", 128), ("int8", 192)])
def test_chunk_pages(mode, bs, kt, Dkv):
    if kt == "int8" and bs == 16:
        bs = 32
    run_case(21, variant=2, lens=[400, 129], news=[100, 129], heads=6, N=2, Dkv=Dkv, mode=mode, bs=bs or 32, kt=kt, vt=kt)


@pytest.mark.parametrize("g", [1, 3, 7, 64, 100, 128, 130])
def test_chunk_groups(g):
    run_case(22, variant=2, lens=[200, 40], news=[80 if g < 8 else 5, 40 if g < 8 else 3], heads=2 * g, N=2)


@pytest.mark.parametrize("kt", ["bf16", "int8"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_chunk_split_over_blocks(kt, causal):
    run_case(23, variant=2, lens=[4500, 0, 70, 1], news=[40, 2, 70, 9], heads=2, N=1, kt=kt, vt=kt, tail=5, causal=causal)


@pytest.mark.parametrize("kt", ["bf16", "e4m3"])
def test_chunk_bad_pages(kt):
    run_case(24, variant=2, lens=[300, 200], news=[80, 70], heads=4, N=2, kt=kt, vt=kt, bad_pages=[(0, 1, -1), (0, 4, 1 << 20), (1, 0, -3)])


def test_chunk_more_queries_than_keys():
    run_case(25, variant=2, lens=[60, 0, 3], news=[300, 100, 90], heads=2, N=1)


def test_chunk_fp16_and_far_scales():
    run_case(26, variant=2, lens=[200], news=[100], heads=4, N=2, dtype="fp16", kt="fp16", vt="fp16")
    run_case(27, variant=2, lens=[200], news=[100], heads=4, N=2, dtype="fp16", kt="int8", vt="e4m3")
    run_case(28, variant=2, lens=[200], news=[100], heads=4, N=2, kt="int8", vt="int8", scale_range=(2e4, 9e4), std=30.0)
    run_case(29, variant=2, lens=[200], news=[100], heads=4, N=2, kt="int8", vt="int8", offsets=False)


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_cut_runs_over_more_sequences_than_a_warp_holds(kt):
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 1500, 70)]
    run_case(30, variant=2, lens=lens, news=[1] * 70, heads=2, N=1, Dkv=64, Dv=64, R=32, kt=kt, vt=kt, max_len=5000)
    news = [int(min(n, x)) for n, x in zip(lens, rng.integers(0, 120, 70))]
    run_case(31, variant=2, lens=lens, news=news, heads=4, N=2, Dkv=64, Dv=64, R=32, kt=kt, vt=kt, tail=2)
