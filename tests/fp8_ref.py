"""Plain 64-bit forms of the 8-bit quantization and product."""
import math

import torch

F, U = 2.0 ** -24, 2.0 ** -8
BLOCK = 128


def round_e4m3(x):
    """float64 to the nearest e4m3 value (ties to even), |x| <= 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(2.0, e - 3)
    return torch.round(x / step) * step


def scale_of(top):
    """The least 2^k >= 2^-126 with top / 2^k <= 448; 1 for 0; NaN for what is not finite."""
    if math.isnan(top) or math.isinf(top):
        return math.nan
    if top == 0:
        return 1.0
    k = -126
    while top / 2.0 ** k > 448:
        k += 1
    return 2.0 ** k


def scales(x, tile):
    """Row-scaled: [blocks of columns, rows]; tiles: [blocks of rows, blocks of columns]."""
    r, c = x.shape
    rb, cb = -(-r // BLOCK), -(-c // BLOCK)
    a = x.double().abs()
    a[torch.isnan(a)] = math.inf
    if tile:
        s = [[scale_of(float(a[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK].max())) for j in range(cb)] for i in range(rb)]
    else:
        s = [[scale_of(float(v)) for v in a[:, j * BLOCK:(j + 1) * BLOCK].amax(dim=1)] for j in range(cb)]
    return torch.tensor(s, dtype=torch.float64).reshape((rb, cb) if tile else (cb, r))


def spread(s, shape, tile):
    """A scale for every value."""
    s = s.double() if tile else s.double().t()
    s = s.repeat_interleave(BLOCK, dim=1)[:, :shape[1]]
    return s.repeat_interleave(BLOCK, dim=0)[:shape[0]] if tile else s


def quantize(x, tile):
    """8-bit values (float64) and scales of x [rows, cols]."""
    s = scales(x, tile)
    q = x.double() / spread(s, x.shape, tile)
    return torch.where(torch.isnan(q), q, round_e4m3(q.nan_to_num(0.0))), s


def matmul(a, a_s, b, b_s, wide):
    """Row-scaled a times tile-scaled b, and how far a result may be off: in a block, each of four products
    of 32 cuts its terms and the sum so far to 24 bits (33 cuts of 2^-23 of the block's size); each block adds one
    rounding, and the scales' product one; the result rounds once."""
    fa, fb = a.double() * spread(a_s, a.shape, False), b.double() * spread(b_s, b.shape, True)
    y, size = fa @ fb.t(), fa.abs() @ fb.abs().t()
    blocks = -(-a.shape[1] // BLOCK)
    return y, (132 * 2 * F + (blocks + 2) * F) * size + (F if wide else U) * y.abs() + 1e-37
