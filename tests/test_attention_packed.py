"""packed_attention on the GPU against the fp64 oracle: head sizes, grouped heads, strides of
both projection layouts, packed sequences (empty ones too), causal masks that leave rows
without keys, rows outside every sequence, and non-finite rows behind a sequence's end."""
import numpy as np
import pytest
import torch

import oracle
from attention_util import TORCH, check_attention, half_values
from rope_attention_gb300 import native

pytestmark = pytest.mark.gpu


def run_case(seed, lens_q, lens_k, nq, nkv, d, causal, dtype="bf16", layout="BSD", std=1.0, tail_q=0, tail_k=0,
             scale=None, given_starts=True):
    """Tokens of the sequences, then tail rows of NaN that belong to none."""
    starts = lambda lens: [0] + list(np.cumsum(lens))
    sq, sk = starts(lens_q), starts(lens_k)
    dev = {}
    vals = {}
    for i, (name, total, heads, tail) in enumerate((("q", sq[-1], nq, tail_q), ("k", sk[-1], nkv, tail_k),
                                                    ("v", sk[-1], nkv, tail_k))):
        bits, val = half_values(seed, i, (total + tail, heads, d), dtype, std if name != "v" else 1.0)
        t = torch.from_numpy(bits.view(np.int16)).cuda().view(TORCH[dtype]).clone()
        t[total:] = float("nan")
        dev[name] = t if layout == "BSD" else t.transpose(0, 1).contiguous().transpose(0, 1)
        vals[name] = val
    out = torch.full_like(dev["q"], 7.0)
    lse = torch.full((sq[-1] + tail_q, nq), 7.0, device="cuda")
    p = native.packed_attention_params(dev["q"], dev["k"], dev["v"], out, B=len(lens_q), causal=causal, softmax_scale=scale)
    ws = torch.zeros(native.packed_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    cu = lambda s: torch.tensor(s, dtype=torch.int32, device="cuda") if given_starts else None
    native.packed_attention(p, dev["q"], dev["k"], dev["v"], out, ws, lse, cu(sq), cu(sk))
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0
    ref = oracle.attention.packed_attention(vals["q"], vals["k"], vals["v"], starts_q=sq, starts_k=sk,
                                            scale=p.softmax_scale, causal=causal)
    worst = check_attention(out, lse, ref, str((lens_q, lens_k, nq, nkv, d, causal)), dtype=dtype, Dk=d)
    if tail_q:
        assert (out[sq[-1]:] == 7).all() and (lse[sq[-1]:] == 7).all()
    return worst


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("d", [16, 48, 64, 80, 112, 128])
def test_head_dims(d, causal):
    run_case(1, [130], [130], 2, 1, d, causal)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385, 600])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_lengths(n, causal):
    run_case(2, [n], [n], 1, 1, 128, causal)


@pytest.mark.parametrize("lq,lk", [(1, 700), (5, 129), (300, 1), (300, 128), (257, 90), (129, 513), (512, 256)])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_cross_lengths(lq, lk, causal):
    # causal with more queries than keys: the first rows see nothing
    run_case(3, [lq], [lk], 2, 2, 64, causal)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["BSD", "NBSD"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_packed_ragged_with_tails(dtype, layout, causal):
    run_case(4, [70, 0, 1, 300, 129], [70, 5, 0, 411, 129], 6, 2, 128, causal, dtype, layout, tail_q=9, tail_k=133)


def test_many_sequences():
    lens = [(7 * i) % 23 for i in range(75)]
    run_case(5, lens, lens, 2, 1, 64, True)


def test_equal_lengths_without_starts():
    run_case(6, [150] * 3, [70] * 3, 4, 4, 64, False, given_starts=False)


@pytest.mark.parametrize("std", [6.0, 0.01])
def test_score_ranges(std):
    # scores of several hundred: the running maximum grows again and again
    run_case(7, [300], [900], 1, 1, 128, False, std=std)


def test_growing_scores_rescale():
    """Keys whose scores grow tile after tile, beyond what is left unscaled."""
    d, L = 64, 700
    q = torch.zeros(4, 1, d, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(L, 1, d, device="cuda", dtype=torch.bfloat16)
    q[:, 0, 0] = torch.tensor([1.0, -1.0, 0.25, 2.0])
    k[:, 0, 0] = torch.arange(L, device="cuda") / 4
    v = torch.randn(L, 1, d, device="cuda").bfloat16()
    out = torch.empty_like(q)
    lse = torch.empty(4, 1, device="cuda")
    p = native.packed_attention_params(q, k, v, out, softmax_scale=1.0)
    ws = torch.zeros(native.packed_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    native.packed_attention(p, q, k, v, out, ws, lse)
    ref = oracle.attention.packed_attention(*(x.double().cpu().numpy() for x in (q, k, v)), starts_q=[0, 4],
                                            starts_k=[0, L], scale=1.0, causal=False)
    check_attention(out, lse, ref, "growing", dtype="bf16", Dk=d)
    assert native.attention_status(ws) == 0
