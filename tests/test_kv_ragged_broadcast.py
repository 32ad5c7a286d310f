"""kv_rms_norm_rope_cache with cos/sin broadcast over S, where the last tile of rows is not full, on
shared memory that holds large numbers from the kernel before: rows that do not exist look up
nothing."""
import pytest
import torch

from parity_util import check_kv
from rope_attention_gb300 import native, runner, synth

pytestmark = pytest.mark.gpu


def fill_shared_memory():
    """Attention over values whose bits are large as integers, on every SM."""
    x = torch.full((4096, 16, 128), 1.5, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    params = native.packed_attention_params(x, x, x, out, causal=False)
    ws = torch.zeros(native.packed_attention_workspace_bytes(params), dtype=torch.uint8, device="cuda")
    native.packed_attention(params, x, x, x, out, ws)
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0


@pytest.mark.parametrize("S", [1, 3, 17, 29, 33])
@pytest.mark.parametrize("kw", [dict(variant=2, N=8, Dkv=192, Dv=128, block_size=32, block_num=4, quant_k=True, quant_v=True),
                                dict(variant=2, N=1, Dkv=192, Dv=128, cache_mode="Norm", cache_seq=40),
                                dict(variant=1, N=1, Dkv=576, Dv=512, block_size=32, block_num=4, quant_v=True),
                                dict(variant=1, N=1, Dkv=576, Dv=512, cache_mode="Norm", cache_seq=40, dtype="fp16")],
                         ids=["v2", "v2_norm", "v1", "v1_norm"])
def test_rows_behind_the_last(kw, S):
    case = synth.make_kv("ragged", 70 + S, B=3, S=S, rope_broadcast=True, **kw)
    r = runner.KvRun(case)
    for _ in range(3):
        fill_shared_memory()
        r.err.zero_()
        r.run()
        torch.cuda.synchronize()
    assert native.kv_rms_norm_rope_cache_status() == 0
    check_kv(case, r, "ragged broadcast")
