"""Rows whose length is no multiple of 16 bytes in a pitch that is one: tensor maps can describe them, and a
store through a map writes the whole of the 16 bytes that a row ends in. What lies behind a row's end is not the library's:
outputs leave it as it is, and inputs may hold anything there."""
import math

import pytest
import torch

import objective_ref as ref
import pack_virtual_rank_gb300 as rv
from test_head_gpu import PAD, Call, check, inputs, targets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 140])
@pytest.mark.parametrize("dim,pitch", [(1, 8), (3, 8), (7, 8), (11, 16), (30, 32), (33, 40), (63, 64), (66, 72), (130, 136), (363, 368)])
@pytest.mark.parametrize("piece_bytes", [0, 1])
def test_nothing_behind_a_row_is_touched(piece_bytes, dim, pitch, tokens, dtype):
    rows = [70, 1, 301]
    g, h, ws, rw = inputs(tokens, dim, rows, dtype, 31)
    t = targets(g, tokens, sum(rows), 0.2 if tokens > 3 else 0.0)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    c = Call(h, ws, rw, piece_bytes=piece_bytes, extra=pitch - dim)
    for x in [c.hidden] + c.weights:                        # inputs hold NaN behind their rows
        full = torch.as_strided(x, (x.shape[0], pitch), (pitch, 1))
        full[:, dim:] = math.nan
    check(c.xent(t), want)                                  # (looks at what lies around every output)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 140])
def test_views_of_odd_width(tokens, dtype):
    """The weight's gradient beside another matrix in the rows of one buffer."""
    dim, pitch = 21, 64
    g, h, ws, rw = inputs(tokens, dim, [333], dtype, 32)
    t = targets(g, tokens, 333, 0.2 if tokens > 3 else 0.0)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    c = Call(h, ws, rw)
    buf = torch.full((333, pitch), PAD, dtype=h.dtype, device="cuda")
    for at in (0, 16, 32):
        buf.fill_(PAD)
        view = buf[:, at:at + dim]
        rv.relay_linear_xent(rv.make_head(c.hidden, c.weights, c.dh, [view]), t.cuda(), c.loss[:tokens], row_weight=c.rw)
        torch.cuda.synchronize()
        ref.close("d_weight", view, want["d_weight"], want["d_weight_b"])
        buf[:, at:at + dim] = PAD
        assert bool((buf == PAD).all()), at
