"""paged_prefix_attention on the GPU against the fp64 oracle: prefixes around the key tiles and pages
(none at all among them), every stored type of both variants, single tokens and chunks, sequences
without positions or tokens of their own, bad pages, and rows outside every sequence.  Short prefixes
and few sequences are served by one call with the prefix ahead of each sequence, many rows behind a
longer one by two that share its reads: the tests from `MANY` on have sizes of the second sort."""
import numpy as np
import pytest
import torch

from paged_forms_util import Case
from rope_attention_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 63, 64, 65, 96, 128, 129, 300, 1000])
@pytest.mark.parametrize("heads", [4, 32])
def test_prefix_lengths(prefix, heads):
    Case(1, variant=2, lens=[70, 1, 40, 130], news=[1] * 4, heads=heads, N=2, prefix=prefix).run_and_check()


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("e4m3", "e4m3"), ("e5m2", "e5m2"), ("int8", "bf16"),
                                   ("bf16", "e4m3")])
@pytest.mark.parametrize("news", [[1, 1, 1], [1, 3, 20], [150, 40, 90]], ids=["decode", "few", "chunk"])
def test_v2_types(mode, kt, vt, news):
    Case(2, variant=2, lens=[150, 40, 333], news=news, heads=12, N=4, mode=mode, kt=kt, vt=vt, prefix=200).run_and_check()


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("e4m3", "e5m2"), ("int8", "bf16"), ("bf16", "int8")])
def test_v1_types(mode, kt, vt):
    Case(3, variant=1, lens=[150, 40, 333], news=[1, 2, 5], heads=16, Dkv=576, Dv=512, mode=mode, kt=kt, vt=vt, prefix=130).run_and_check()


@pytest.mark.parametrize("scalar,offsets", [(True, True), (False, False)])
def test_v1_quantisation_forms(scalar, offsets):
    Case(4, variant=1, lens=[100, 65], news=[1, 1], heads=8, Dkv=576, Dv=512, kt="int8", vt="int8", scalar=scalar, offsets=offsets,
         prefix=90).run_and_check()


@pytest.mark.parametrize("heads", [1, 5, 17, 64, 128])
def test_v1_head_counts(heads):
    Case(5, variant=1, lens=[30, 20, 0], news=[1, 1, 1], heads=heads, Dkv=576, Dv=512, prefix=150).run_and_check()


@pytest.mark.parametrize("dims", [(16, 16, 8), (64, 64, 32), (96, 80, 32), (128, 128, 64), (256, 256, 64), (80, 208, 16)])
@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_v2_widths(dims, kt):
    Case(6, variant=2, lens=[100, 200], news=[1, 30], heads=6, N=2, Dkv=dims[0], Dv=dims[1], R=dims[2], kt=kt, vt=kt, prefix=170).run_and_check()


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_sequences_without_positions_or_tokens(causal, kt):
    # a sequence without positions of its own sees the prefix; one without tokens is left out
    Case(7, variant=2, lens=[0, 20, 0, 3, 64], news=[4, 50, 1, 7, 0], heads=4, N=2, causal=causal, kt=kt, vt=kt, prefix=100,
         tail=5).run_and_check()
    Case(8, variant=2, lens=[0, 0], news=[1, 1], heads=4, N=2, causal=causal, kt=kt, vt=kt, prefix=40).run_and_check()
    Case(9, variant=2, lens=[0, 0], news=[1, 90], heads=4, N=2, causal=causal, kt=kt, vt=kt, prefix=0).run_and_check()


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_split_over_blocks(kt):
    Case(10, variant=2, lens=[500, 0, 1, 1500, 64], news=[1, 1, 1, 4, 0], heads=8, N=2, kt=kt, vt=kt, prefix=5000, tail=3).run_and_check()
    Case(11, variant=1, lens=[410, 33], news=[2, 1], heads=16, Dkv=576, Dv=512, kt=kt, vt=kt, bs=64, prefix=4100).run_and_check()
    Case(12, variant=2, lens=[3000, 200], news=[100, 200], heads=2, N=1, kt=kt, vt=kt, prefix=3000).run_and_check()


@pytest.mark.parametrize("bs", [16, 48, 96, 128, 256])
def test_pages(bs):
    Case(13, variant=2, lens=[400, 129], news=[100, 1], heads=6, N=2, bs=bs, prefix=333).run_and_check()


@pytest.mark.parametrize("kt", ["bf16", "e4m3"])
def test_bad_pages_are_left_out(kt):
    Case(14, variant=2, lens=[300, 100], news=[5, 1], heads=4, N=2, kt=kt, vt=kt, prefix=200, bad_pages=[(0, 1, -1)],
         bad_prefix=[(2, 1 << 20)]).run_and_check()
    Case(15, variant=2, lens=[40], news=[60], heads=4, N=2, kt=kt, vt=kt, prefix=64, bad_prefix=[(0, -1), (1, -1)]).run_and_check()


def test_many_sequences():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 90, 601)]
    Case(16, variant=2, lens=lens, news=[1] * 601, heads=2, N=1, Dkv=64, Dv=64, R=32, prefix=150).run_and_check()


def test_fp16_and_large_scores():
    for kt in ("fp16", "int8"):
        for news in ([3, 1], [90, 70]):
            Case(17, variant=2, lens=[200, 100], news=news, heads=4, N=2, dtype="fp16", kt=kt, vt=kt, prefix=150).run_and_check()
    Case(18, variant=2, lens=[300], news=[40], heads=4, N=2, std=20.0, prefix=300).run_and_check()


def test_equal_tokens_without_starts():
    Case(19, variant=2, lens=[100, 130, 9], news=[3, 3, 3], heads=4, N=2, given_starts=False, prefix=77).run_and_check()


def test_a_longer_bound_and_a_wider_table_change_nothing():
    a = Case(20, variant=2, lens=[100, 30], news=[1, 1], heads=4, N=2, prefix=77)
    b = Case(20, variant=2, lens=[100, 30], news=[1, 1], heads=4, N=2, prefix=77, spare=4)
    for c in (a, b):
        c.run_and_check()
    # a length beyond the bound is clamped to it
    b.form.max_prefix_len = 77
    b.prefix_len.fill_(79)
    first = b.out.clone()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), b.out.view(torch.int16))


# ---------------------------------------------------------------- many rows behind one prefix
MANY = dict(variant=2, lens=[(7 * i) % 40 for i in range(96)], news=[1] * 96, heads=16, N=8, prefix=1100)


def tokens_of(lens, most):
    return [min(max(n, 1), 1 + i % most) for i, n in enumerate(lens)]


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD"])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("e4m3", "e5m2"), ("int8", "bf16"), ("bf16", "e4m3")])
def test_many_sequences_share_v2(mode, kt, vt):
    Case(21, mode=mode, kt=kt, vt=vt, tail=3, **MANY).run_and_check()


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_many_sequences_share_other_widths_and_tokens(kt):
    for dims in ((64, 64, 32), (96, 80, 32), (128, 128, 64), (256, 208, 64)):
        case = {**MANY, "Dkv": dims[0], "Dv": dims[1], "R": dims[2], "kt": kt, "vt": kt, "news": tokens_of(MANY["lens"], 3)}
        Case(22, **case).run_and_check()
    # one row tile for the batch's rows of a kv head, and chunks
    Case(23, variant=2, lens=[3, 0], news=[1, 1], heads=8, N=8, prefix=40000, kt=kt, vt=kt).run_and_check()
    Case(24, variant=2, lens=[40] * 40, news=[18] * 40, heads=16, N=8, prefix=2000, kt=kt, vt=kt).run_and_check()


@pytest.mark.parametrize("prefix", [1100, 4000])
@pytest.mark.parametrize("kt,vt", [("bf16", "bf16"), ("int8", "int8"), ("int8", "bf16"), ("bf16", "e5m2")])
def test_many_sequences_share_v1(kt, vt, prefix):
    lens = [(5 * i) % 30 for i in range(150)]
    Case(25, variant=1, lens=lens, news=tokens_of(lens, 2), heads=16, Dkv=576, Dv=512, kt=kt, vt=vt,
         prefix=prefix).run_and_check()


def test_many_sequences_share_fp16_bad_pages_and_no_prefix_after_all():
    for kt in ("fp16", "int8"):
        Case(26, dtype="fp16", kt=kt, vt=kt, **MANY).run_and_check()
    Case(27, bad_pages=[(5, 0, -1)], bad_prefix=[(2, 1 << 20), (30, -4)], **MANY).run_and_check()
    Case(28, causal=False, given_starts=False, std=8.0, **MANY).run_and_check()
    # sized for a long prefix, called with a short one and with none
    c = Case(29, spare=1100, **{**MANY, "prefix": 1})
    c.run_and_check()
    c.prefix_len.fill_(0)
    c.ref_args["prefix_len"] = 0
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    c.check("no prefix")


@pytest.mark.parametrize("kt", ["bf16", "int8"])
def test_two_calls_in_one_launch_sized_for_a_longer_prefix(kt):
    # the latent: each of the prefix's row tiles is cut over many blocks, or is one block's where it is short
    for B, prefix in ((150, 1), (8, 65), (9, 16000), (5, 130), (61, 64)):
        lens = [(11 * i) % 90 for i in range(B)]
        c = Case(30, variant=1, lens=lens, news=tokens_of(lens, 2), heads=16, Dkv=576, Dv=512, kt=kt, vt=kt, prefix=prefix,
                 spare=20000 - prefix, tail=2)
        c.run_and_check()
        c.prefix_len.fill_(0)
        c.ref_args["prefix_len"] = 0
        c.run()
        torch.cuda.synchronize()
        assert c.status() == 0
        c.check("no prefix")
    Case(31, variant=2, lens=[40] * 61, news=[1] * 61, heads=16, N=4, Dkv=256, Dv=208, R=64, kt=kt, vt=kt, prefix=9000).run_and_check()


@pytest.mark.parametrize("kt,heads,window", [("bf16", 8, None), ("int8", 16, None), ("bf16", 8, 2500), ("int8", 16, 3000), ("bf16", 32, 2000)])
def test_many_passes_give_the_same_bits(kt, heads, window):
    # long runs of tiles from pages all over the cache, whose copies land in any order
    lens = [(397 * i) % 3000 + 1 for i in range(61)]
    form = dict(window=window, sinks=4) if window else dict(prefix=9000)
    c = Case(32, variant=2, lens=lens, news=[1] * 61, heads=heads, N=2, Dkv=128, Dv=128, bs=128, kt=kt, vt=kt, **form)
    c.run_and_check()
    out = torch.full_like(c.out, 7.0)
    for _ in range(20):
        for _ in range(150):
            c.run(out=out, lse=None)
        torch.cuda.synchronize()
        assert c.status() == 0
        assert torch.equal(out.view(torch.int16), c.out.view(torch.int16))
