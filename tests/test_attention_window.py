"""packed_window_attention and paged_window_attention on the GPU against the fp64 oracle: windows and
sinks around the key tiles, rows that see nothing, every cache mode and stored type, decode steps and
chunks, pages that left the window and were given away, cut items, and a window that hides nothing."""
import numpy as np
import pytest
import torch

import oracle
from attention_util import TORCH, check_attention, half_values
from paged_forms_util import Case
from rope_attention_gb300 import native

pytestmark = pytest.mark.gpu


def run_packed(seed, lens_q, lens_k, nq, nkv, d, window, sinks, dtype="bf16", layout="BSD", tail_q=0, tail_k=0, std=1.0,
               given_starts=True):
    """Tokens of the sequences, then tail rows of NaN that belong to none."""
    starts = lambda lens: [0] + list(np.cumsum(lens))
    sq, sk = starts(lens_q), starts(lens_k)
    dev, vals = {}, {}
    for i, (name, total, heads, tail) in enumerate((("q", sq[-1], nq, tail_q), ("k", sk[-1], nkv, tail_k), ("v", sk[-1], nkv, tail_k))):
        bits, vals[name] = half_values(seed, i, (total + tail, heads, d), dtype, std if name != "v" else 1.0)
        t = torch.from_numpy(bits.view(np.int16)).cuda().view(TORCH[dtype]).clone()
        t[total:] = float("nan")
        dev[name] = t if layout == "BSD" else t.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full_like(dev["q"], 7.0)
    lse = torch.full((sq[-1] + tail_q, nq), 7.0, device="cuda")
    p = native.packed_attention_params(dev["q"], dev["k"], dev["v"], out, B=len(lens_q), causal=True)
    ws = torch.zeros(native.packed_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    cu = lambda s: torch.tensor(s, dtype=torch.int32, device="cuda") if given_starts else None
    w = native.AttentionWindow(window=window, sinks=sinks)
    call = lambda o, l: native.packed_window_attention(p, w, dev["q"], dev["k"], dev["v"], o, ws, l, cu(sq), cu(sk))
    call(out, lse)
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0
    ref = oracle.attention.packed_attention(vals["q"], vals["k"], vals["v"], starts_q=sq, starts_k=sk, scale=p.softmax_scale,
                                            causal=True, window=window, sinks=sinks)
    check_attention(out, lse, ref, str((lens_q, lens_k, nq, nkv, d, window, sinks)), dtype=dtype, Dk=d)
    if tail_q:
        assert (out[sq[-1]:] == 7).all() and (lse[sq[-1]:] == 7).all()
    again = torch.full_like(out, 7.0)
    call(again, None)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    return out, lse, p, dev, ws


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 200, 256, 400])
@pytest.mark.parametrize("sinks", [0, 1, 4, 64, 127, 128, 130])
def test_windows_and_sinks(window, sinks):
    run_packed(1, [700], [700], 2, 1, 64, window, sinks)


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 385, 600])
def test_lengths(n):
    run_packed(2, [n], [n], 1, 1, 128, 100, 3)


@pytest.mark.parametrize("d", [16, 48, 80, 112, 128])
def test_head_dims(d):
    run_packed(3, [300], [300], 4, 2, d, 40, 5)


@pytest.mark.parametrize("lq,lk", [(1, 700), (5, 400), (300, 1), (300, 128), (257, 90), (129, 513)])
def test_cross_lengths(lq, lk):
    # more queries than keys: the first rows see nothing
    run_packed(4, [lq], [lk], 2, 2, 64, 70, 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["BSD", "NBSD"])
def test_packed_ragged_with_tails(dtype, layout):
    run_packed(5, [70, 0, 1, 300, 129], [70, 5, 0, 411, 129], 6, 2, 128, 50, 7, dtype, layout, tail_q=9, tail_k=133)
    run_packed(6, [200, 200], [200, 200], 4, 4, 64, 33, 0, dtype, layout, given_starts=False)


def test_many_items_and_cut_ones():
    run_packed(7, [40] * 20, [40] * 20, 128, 32, 64, 9, 2)                    # strided whole items
    run_packed(8, [9, 300, 0, 33] * 30, [9, 300, 0, 33] * 30, 32, 8, 64, 20, 1)  # runs of whole items
    run_packed(9, [3], [9000], 1, 1, 128, 5000, 300)                          # few rows, many keys: cut
    run_packed(10, [300], [6000], 1, 1, 128, 2500, 0)
    run_packed(11, [200], [200], 2, 2, 64, 30, 4, std=12.0)


def test_a_window_that_hides_nothing_is_packed_attention():
    for window, sinks in ((700, 0), (1 << 40, 0), (1, 700), (1, 1 << 50)):
        out, lse, p, dev, ws = run_packed(12, [700], [700], 2, 1, 128, window, sinks)
        want, want_lse = torch.empty_like(out), torch.empty_like(lse)
        native.packed_attention(p, dev["q"], dev["k"], dev["v"], want, ws, want_lse)
        assert torch.equal(want.view(torch.int16), out.view(torch.int16)) and torch.equal(want_lse, lse)


# ---------------------------------------------------------------- over the paged caches
@pytest.mark.parametrize("window", [1, 31, 32, 63, 64, 65, 100, 128, 300])
@pytest.mark.parametrize("sinks", [0, 4, 64, 65, 200])
def test_decode_windows(window, sinks):
    Case(20, variant=2, lens=[500, 64, 65, 130, 3], news=[1] * 5, heads=8, N=2, window=window, sinks=sinks).run_and_check()


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD", "Norm"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("e4m3", "e5m2"), ("int8", "bf16")])
def test_v2_types_and_modes(mode, kt, vt):
    Case(21, variant=2, lens=[250, 40, 333, 0], news=[1, 3, 20, 2], heads=12, N=4, mode=mode, kt=kt, vt=vt, window=50, sinks=5,
         tail=2).run_and_check()


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("bf16", "int8")])
def test_v1_types_and_modes(mode, kt, vt):
    Case(22, variant=1, lens=[350, 40, 333], news=[1, 2, 5], heads=16, Dkv=576, Dv=512, mode=mode, kt=kt, vt=vt, window=90,
         sinks=3).run_and_check()


@pytest.mark.parametrize("window", [1, 60, 96, 128, 200])
@pytest.mark.parametrize("sinks", [0, 5, 96, 140])
@pytest.mark.parametrize("kt,Dkv", [("bf16", 192), ("int8", 192), ("bf16", 128), ("e4m3", 128)])
def test_chunk_windows(window, sinks, kt, Dkv):
    Case(23, variant=2, lens=[700, 129], news=[150, 129], heads=4, N=2, Dkv=Dkv, kt=kt, vt=kt, window=window, sinks=sinks).run_and_check()


@pytest.mark.parametrize("mode,bs", [("PA", 16), ("PA", 96), ("PA_BNSD", 64), ("PA_BNSD", 160), ("PA_BNSD", 256), ("Norm", 0)])
@pytest.mark.parametrize("new", [1, 100])
def test_pages(mode, bs, new):
    Case(24, variant=2, lens=[900, 150], news=[new, new], heads=6, N=2, mode=mode, bs=bs or 32, window=130, sinks=20).run_and_check()


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_decode_split_over_blocks(kt):
    Case(25, variant=2, lens=[9000, 0, 1, 4000, 64], news=[1, 1, 1, 4, 0], heads=8, N=2, kt=kt, vt=kt, window=3333, sinks=100,
         tail=3).run_and_check()
    Case(26, variant=1, lens=[6100], news=[2], heads=16, Dkv=576, Dv=512, kt=kt, vt=kt, bs=64, window=4500, sinks=70).run_and_check()


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_chunk_split_over_blocks_and_more_queries_than_keys(kt):
    Case(27, variant=2, lens=[4500, 0, 70, 1], news=[40, 2, 70, 9], heads=2, N=1, kt=kt, vt=kt, window=2000, sinks=33, tail=5).run_and_check()
    Case(28, variant=2, lens=[60, 0, 3], news=[300, 100, 90], heads=2, N=1, kt=kt, vt=kt, window=20, sinks=2).run_and_check()


@pytest.mark.parametrize("kt", ["bf16", "e4m3"])
def test_bad_pages_in_the_window_are_left_out(kt):
    Case(29, variant=2, lens=[300, 100], news=[5, 1], heads=4, N=2, kt=kt, vt=kt, window=100, sinks=40,
         bad_pages=[(0, 0, -1), (0, 8, 1 << 20)]).run_and_check()
    Case(30, variant=2, lens=[300, 200], news=[80, 70], heads=4, N=2, kt=kt, vt=kt, window=90, sinks=10,
         bad_pages=[(0, 7, 1 << 20), (1, 0, -3)]).run_and_check()


def test_many_sequences():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 400, 601)]
    Case(31, variant=2, lens=lens, news=[1] * 601, heads=2, N=1, Dkv=64, Dv=64, R=32, window=77, sinks=3).run_and_check()
    news = [int(min(n, x)) for n, x in zip(lens[:70], rng.integers(0, 120, 70))]
    Case(32, variant=2, lens=lens[:70], news=news, heads=4, N=2, Dkv=64, Dv=64, R=32, window=50, sinks=0, tail=2).run_and_check()


def test_fp16_and_large_scores():
    for kt in ("fp16", "int8"):
        for news in ([3, 1], [90, 70]):
            Case(33, variant=2, lens=[200, 100], news=news, heads=4, N=2, dtype="fp16", kt=kt, vt=kt, window=60, sinks=9).run_and_check()
    Case(34, variant=2, lens=[900], news=[40], heads=4, N=2, std=20.0, window=300, sinks=50).run_and_check()


def test_a_window_that_hides_nothing_is_paged_attention():
    # to the bit where both calls run the same kernel (V2 with up to 16 rows has one of its own here, which
    # sums in another order: the other tests hold it to the oracle)
    for variant, news, kt in ((2, [100, 60], "int8"), (1, [2, 1], "int8")):
        dims = dict(Dkv=576, Dv=512, N=1) if variant == 1 else dict(N=2)
        c = Case(35, variant=variant, lens=[333, 150], news=news, heads=8, kt=kt, vt=kt, window=1 << 33, sinks=0, **dims)
        c.run_and_check()
        want, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
        native.paged_attention(c.cache, c.params, c.q, c.kd, c.vd, c.lens_d, want, c.ws, lse=lse, **c.args)
        assert torch.equal(want.view(torch.int16), c.out.view(torch.int16)) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("at", [0, 16])
@pytest.mark.parametrize("heads,N,B,new,Dv", [(6, 2, 1, 2, 16), (3, 1, 2, 2, 48), (13, 1, 1, 1, 128), (6, 1, 3, 1, 32), (5, 1, 1, 3, 16),
                                              (24, 8, 2, 2, 16)])
def test_small_items_stay_in_their_workspace(at, heads, N, B, new, Dv):
    c = Case(36, variant=2, lens=[512] * B, news=[new] * B, heads=heads, N=N, Dkv=32, Dv=Dv, R=16, window=500, sinks=2)
    n = c.ws.numel()
    room = torch.zeros(at + n + 4096, dtype=torch.uint8, device="cuda")
    room[at + n:] = 77
    room[:at] = 77
    c.ws = room[at:at + n]
    c.run_and_check()
    assert (room[:at] == 77).all() and (room[at + n:] == 77).all()
