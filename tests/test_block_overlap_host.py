"""Outputs that share memory with what a call still reads are refused before anything is
enqueued.  Addresses are never read: on a machine without a GPU a call that is let through ends
in the launch's error."""
import pytest

torch = pytest.importorskip("torch")
moe = pytest.importorskip("sparse_moe_ffn_route_gb300")
from test_block_host import INVALID, ref, three  # noqa: E402

T, D, FF = 4, 64, 128
ROWS, MATRIX = T * D * 2, D * FF * 2
BASE = {n: 0x1000000 * (i + 1) for i, n in enumerate(
    ("x", "dy", "gate", "up", "down", "saved", "dx", "dgate", "dup", "ddown", "ws"))}


def backward(**at):
    p = {**BASE, **at}
    c = moe.glu_cfg(D, FF)
    ws, saved = moe.moe_glu_workspace_bytes(c, T), moe.moe_glu_saved_bytes(c, T)
    return moe._lib.moe_glu_backward(ref(c), p["x"], T, ref(three(p["gate"], p["up"], p["down"])), p["saved"], saved,
                                     p["dy"], p["dx"], ref(three(p["dgate"], p["dup"], p["ddown"])), p["ws"], ws, None)


CASES = [("dx", "dy", 0), ("dx", "x", 0), ("dx", "x", ROWS - 16), ("dy", "dx", 16), ("dgate", "gate", 0),
         ("ddown", "down", MATRIX - 16), ("dup", "dgate", 0), ("dx", "saved", 256), ("ws", "x", -16), ("saved", "ws", 512),
         ("dup", "dy", -MATRIX + 16)]


@pytest.mark.parametrize("moved,onto,by", CASES)
def test_backward_outputs_apart(moved, onto, by):
    assert backward(**{moved: BASE[onto] + by}) == INVALID


@pytest.mark.parametrize("by", [0, 16, -16])
def test_w4_output_apart_from_its_input(by):
    c = moe.w4_cfg(64, 64, 32)
    at = BASE["x"]
    assert moe._lib.moe_w4_linear(ref(c), at, T, ref(three(BASE["gate"], BASE["up"], None)), at + by, None) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is let through reads its addresses")
def test_neighbours_are_let_through():
    assert backward() != INVALID
    assert backward(dx=BASE["x"] + ROWS) != INVALID and backward(dup=BASE["dgate"] + MATRIX) != INVALID
    c = moe.w4_cfg(64, 64, 32)
    at = BASE["x"]
    assert moe._lib.moe_w4_linear(ref(c), at, T, ref(three(BASE["gate"], BASE["up"], None)), at + T * 64 * 2, None) != INVALID
