"""Every byte of packed weights and of saved inputs that later calls read is written: scale bytes are read by 16 rows
(include/deft.h), past the last row, too."""
import pytest
import torch

from irregular_gather_cnn_amd.pointwise import Pointwise8
from test_pointwise import LAYOUTS, inputs


def parts(at, rows, depth):
    """Where a matrix's codes and its scale bytes lie in a buffer, and where the next matrix starts."""
    blocks, scale_rows = -(-depth // 128), -(-rows // 16) * 16
    scales = -(-(at + blocks * rows * 128) // 256) * 256
    end = scales + blocks * scale_rows
    return (slice(at, at + blocks * rows * 128), slice(scales, end)), -(-end // 256) * 256


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,c_in,s,c_out", [(1, 1, 1, 1), (2, 130, 41, 77), (1, 129, 20, 300), (3, 16, 64, 250)])
def test_nothing_is_left_of_what_was_there(n, c_in, s, c_out, layout, dtype):
    print("pw8 scales", n, c_in, s, c_out, layout, dtype, flush=True)
    x, w, b, dy = inputs(n, c_in, s, c_out, layout, dtype, seed=9)
    h = Pointwise8(n, c_in, s, c_out, layout=layout, dtype=dtype, training=True)
    runs = []
    for fill in (0, 0xff):
        packed, saved = (torch.full((size,), fill, dtype=torch.uint8, device="cuda") for size in (h.packed_bytes, h.saved_bytes))
        h.ws.fill_(fill)
        h.pack(w, out=packed)
        y, _ = h.forward(x, packed, b, saved=saved)
        h.ws.fill_(fill)
        g = h.backward(saved, packed, dy)
        runs.append((packed, saved, y, g["dx"], g["dw"], g["db"]))
    rows, turned_at = parts(0, c_out, c_in)
    turned, end = parts(turned_at, c_in, c_out)
    assert end == h.packed_bytes
    kept, end = parts(0, c_in, n * s)
    assert end == h.saved_bytes
    for part in rows + turned:
        assert torch.equal(runs[0][0][part], runs[1][0][part])
    for part in kept:
        assert torch.equal(runs[0][1][part], runs[1][1][part])
    for got, want in zip(runs[0][2:], runs[1][2:]):
        assert torch.equal(got, want) and torch.isfinite(got).all()
