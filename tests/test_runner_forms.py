"""The forms of a runner's call, on the CPU: what it refuses before it allocates or launches anything."""
import pytest
import torch

from rope_attention_gb300 import native, runner, synth


def test_a_window_behind_a_prefix_is_refused():
    case = synth.make_kv("forms", 1, variant=2, B=2, N=2, S=8, Dkv=64, Dv=64, rope_size=32, block_size=16, block_num=4)
    kv = runner.KvRun(case, device="cpu")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    table, window = [[0, 1], [2, 3]], native.AttentionWindow(window=4, sinks=1)
    with pytest.raises(ValueError, match="window and prefix"):
        runner.PagedAttentionRun(kv, q, [5, 7], table, window=window, prefix=(8, [0]))
    # each by itself is one
    assert runner.PagedAttentionRun(kv, q, [5, 7], table, window=window).prefix is None
    assert runner.PagedAttentionRun(kv, q, [5, 7], table, prefix=(8, [0])).window is None
