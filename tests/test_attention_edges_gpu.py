"""Calls of the attention operators at the edge of what the header allows, on the GPU:
workspaces that start on any 16 bytes, waits of the shortest time limit."""
import pytest
import torch

from rope_attention_gb300 import native
from test_attention_use import DEFAULT_WAIT_NS, Packed, Paged

pytestmark = pytest.mark.gpu


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
