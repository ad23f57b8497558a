"""The status word of the dispatch's workspace, as of every other call's."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_gpu_block import gen_for, rnd  # noqa: E402
from test_gpu_exchange import routing  # noqa: E402

pytestmark = pytest.mark.gpu


# one launch, and a count before it
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (300, 16, 4), (5000, 64, 4)])
def test_a_workspace_that_held_something_else(T, E, k):
    gen = gen_for(T, E, k)
    ids, x = routing(gen, T, E, k), rnd(gen, T, 64)
    cfg = moe.exchange_cfg(64, E, k)
    ws = torch.full((moe.moe_dispatch_workspace_bytes(cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
    for source in (x, None):
        ws.fill_(0xFF)
        moe.moe_dispatch_forward(cfg, source, ids, ws=ws)
        assert moe.moe_device_status(ws) == (moe.MOE_OK, 0)
