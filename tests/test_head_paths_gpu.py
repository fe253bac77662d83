"""Ways through the losses that the other tests do not take, against the definition: distillation and confident rows
over several pieces of the vocabulary, more columns in one piece than one block of the scaling pass has, and more row tiles
than are walked together."""
import pytest
import torch

import objective_ref as ref
from test_head_gpu import Call, check, inputs, targets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("piece_bytes", [1, 2 * 2 * 256 * 256])
@pytest.mark.parametrize("top,tau", [(1, 4.0), (33, 0.5), (128, 2.0)])
@pytest.mark.parametrize("tokens", [60, 300])
def test_distillation_over_pieces(tokens, top, tau, piece_bytes, dtype):
    rows = [700, 0, 513]
    V = sum(rows)
    g, h, ws, rw = inputs(tokens, 104, rows, dtype, 21)
    index = torch.randint(0, V, (tokens, top), generator=g, dtype=torch.int32)
    if top > 3:
        index[:, 1] = index[:, 0]                          # ids given twice, and three times
        index[::2, 3] = index[::2, 0]
    gone = torch.rand(tokens, top, generator=g) < 0.2
    index[gone] = torch.tensor([-1, V], dtype=torch.int32)[torch.arange(int(gone.sum())) % 2]
    index[::7] = -1
    logits = torch.randn(tokens, top, generator=g) * 3
    want = ref.head(h, ws, index, logits, rw, tau)
    check(Call(h, ws, rw, piece_bytes=piece_bytes).distill(logits, index, tau), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [100, 300])
def test_confident_rows_over_pieces(tokens, dtype):
    g, h, ws, rw = inputs(tokens, 128, [600], dtype, 22, scale=1.0)
    t = torch.randint(0, 600, (tokens,), generator=g, dtype=torch.int32)
    h = (h.float() + 18.0 * ws[0][t.long()].float()).to(h.dtype)
    want = ref.head(h, ws, t[:, None], None, rw, 1.0)
    assert want["loss"].median() < 1e-3
    check(Call(h, ws, rw, piece_bytes=1).xent(t), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [70, 300])
@pytest.mark.parametrize("rows", [[8192], [8193], [8000, 5000, 7001]])
def test_more_columns_than_a_block_scales(rows, tokens, dtype):
    V = sum(rows)
    g, h, ws, rw = inputs(tokens, 40, rows, dtype, 23)
    t = targets(g, tokens, V)
    check(Call(h, ws, rw).xent(t), ref.head(h, ws, t[:, None], None, rw, 1.0))
    index = torch.randint(-V // 5, V, (tokens, 19), generator=g, dtype=torch.int32)
    index[:, 2] = index[:, 11]
    logits = torch.randn(tokens, 19, generator=g)
    check(Call(h, ws, rw).distill(logits, index, 2.0), ref.head(h, ws, index, logits, rw, 2.0))


@pytest.mark.parametrize("dtype,tokens", [("bf16", 2100), ("f32", 600)])
@pytest.mark.parametrize("piece_bytes", [0, 1])
def test_more_row_tiles_than_are_walked_together(piece_bytes, dtype, tokens):
    """Rows of 16384 elements: 64 MiB of packed hidden are 8 row tiles of a bf16 head, 2 of an fp32 head."""
    g, h, ws, rw = inputs(tokens, 16384, [300, 250], dtype, 24)
    t = targets(g, tokens, 550, 0.01)
    check(Call(h, ws, rw, piece_bytes=piece_bytes).xent(t), ref.head(h, ws, t[:, None], None, rw, 1.0))
