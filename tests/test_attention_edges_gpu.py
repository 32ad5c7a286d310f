"""Calls of the attention operators at the edge of what the header allows, on the GPU:
workspaces that start on any 16 bytes."""
import pytest
import torch

from test_attention_use import Packed, Paged

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
