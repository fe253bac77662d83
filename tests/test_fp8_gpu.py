"""Quantization to 8 bits and products with a scale for each block of 128, against their 64-bit forms: every width of the kernel,
odd sizes, strides, groups with and without rows, empty and special blocks, captured calls, other streams."""
import math

import pytest
import torch

import fp8_ref as ref
import pack_virtual_rank_gb300 as rv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def q_of(rows, cols, tiles=False, batch=None):
    q, s = rv.alloc_fp8(rows, cols, "cuda", tiles=tiles, batch=batch)
    q.view(torch.uint8).fill_(0x31)
    s.fill_(7.0)
    return q, s


def data(rows, cols, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 2) * scale
    if x.numel() > 3:
        x[rows // 2, cols // 2] = 0.0
    return x.to(DT[dtype])


def same_values(q, want):
    got = q.float().cpu().double()
    return torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9))


# ------------------------------------------------------------------------- quantization --

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 257), (200, 1000), (77, 16), (300, 9), (256, 384), (200, 256)])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_is_exact(rows, cols, dtype, tiles):
    x = data(rows, cols, dtype)
    for extra in (0, 3, 8):                                # row strides on and off the 16-byte grid
        buf = torch.full((rows, cols + extra), 9.0, dtype=DT[dtype], device="cuda")
        xc = buf[:, :cols]
        xc.copy_(x)
        q, s = q_of(rows, cols, tiles)
        qt, st = q_of(cols, rows, not tiles)
        rv.relay_quantize_fp8(xc, q, s, qt, st, tiles=tiles, tiles_t=not tiles)
        want, want_s = ref.quantize(x, tiles)
        want_t, want_st = ref.quantize(x.t(), not tiles)
        assert torch.equal(s.cpu().double(), want_s) and same_values(q, want)
        assert torch.equal(st.cpu().double(), want_st) and same_values(qt, want_t)
        only, s1 = q_of(rows, cols, tiles)
        rv.relay_quantize_fp8(xc, only, s1, tiles=tiles)
        assert torch.equal(only.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, s)
        only, s1 = q_of(cols, rows, not tiles)
        rv.relay_quantize_fp8(xc, qt=only, scale_t=s1, tiles_t=not tiles)
        assert torch.equal(only.view(torch.uint8), qt.view(torch.uint8)) and torch.equal(s1, st)


def test_bytes_behind_a_row_stay():
    x = torch.randn(200, 130, device="cuda").bfloat16()
    whole = torch.full((200, 160), 0x55, dtype=torch.uint8, device="cuda")
    q = whole.view(torch.float8_e4m3fn)[:, :130]
    turned = torch.full((130, 224), 0x55, dtype=torch.uint8, device="cuda")
    qt = turned.view(torch.float8_e4m3fn)[:, :200]
    rv.relay_quantize_fp8(x, q, torch.empty(2, 200, device="cuda"), qt, torch.empty(2, 130, device="cuda"))
    assert bool((whole[:, 130:] == 0x55).all()) and bool((turned[:, 200:] == 0x55).all())
    assert same_values(q, ref.quantize(x.cpu(), False)[0]) and same_values(qt, ref.quantize(x.cpu().t(), False)[0])


def test_ends_of_the_range():
    rows = [[0.0] * 128, [448.0] + [1.0] * 127, [449.0] + [0.1] * 127, [1e-45] * 128, [3e38, -3e38] + [1e30] * 126,
            [2.0 ** -126, 2.0 ** -133] * 64, [-0.0] * 128, [224.0, 225.0] * 64, [1.0, 2.0 ** -17] * 64, [2.0 ** -118] * 128,
            [1.75 * 2.0 ** -118, 2.0 ** -126] * 64]
    rows += [[0.0] * 127 + [v] for v in (math.nan, math.inf, -math.inf)]
    x = torch.tensor(rows)
    q, s = q_of(*x.shape)
    qt, st = q_of(128, len(rows), tiles=True)
    rv.relay_quantize_fp8(x.cuda(), q, s, qt, st, tiles_t=True)
    want, want_s = ref.quantize(x, False)
    assert torch.equal(s.cpu().double().nan_to_num(9.0), want_s.nan_to_num(9.0)) and same_values(q, want)
    assert bool(torch.isnan(st).all()) and bool(torch.isnan(qt.float()).all())


@pytest.mark.parametrize("rows,cols,n", [(100, 200, 3), (128, 128, 1), (257, 129, 4), (256, 384, 2)])
def test_quantize_a_batch(rows, cols, n):
    x = torch.stack([data(rows, cols, "bf16", seed=i) for i in range(n)])
    q, s = q_of(rows, cols, True, n)
    qt, st = q_of(cols, rows, True, n)
    rv.relay_quantize_fp8(x.cuda(), q, s, qt, st, tiles=True, tiles_t=True)
    for i in range(n):
        want, want_s = ref.quantize(x[i], True)
        assert torch.equal(s[i].cpu().double(), want_s) and same_values(q[i], want)
        assert torch.equal(st[i].cpu().double(), want_s.t()) and same_values(qt[i], want.t())


GROUPS = [[5], [0], [128, 128], [0, 1, 0, 127, 129, 0], [300, 0, 0, 2], [1] * 40, [130, 7] * 20]


def offsets(lengths, skip=0):
    return torch.tensor([skip] + [skip + sum(lengths[:i + 1]) for i in range(len(lengths))], dtype=torch.int32)


@pytest.mark.parametrize("lengths", GROUPS)
@pytest.mark.parametrize("cols", [150, 256])
@pytest.mark.parametrize("tiles_t", [False, True])
def test_quantize_groups(lengths, tiles_t, cols):
    skip, behind = 3, 5
    rows = skip + sum(lengths) + behind
    x = data(rows, cols, "bf16")
    x[:skip] = math.nan                                   # no group's rows: not looked at
    x[skip + sum(lengths):] = math.nan
    off = offsets(lengths, skip)
    q, s = q_of(rows, cols)
    depth = rv.fp8_depth(rows, len(lengths))
    qt, st = q_of(cols, depth, tiles_t)
    rv.relay_quantize_fp8(x.cuda(), q, s, qt, st, tiles_t=tiles_t, offset=off.cuda())
    at = 0
    for i, n in enumerate(lengths):
        part = x[off[i]:off[i + 1]]
        want, want_s = ref.quantize(part, False)
        assert torch.equal(s[:, off[i]:off[i + 1]].cpu().double(), want_s) and same_values(q[off[i]:off[i + 1]], want)
        full = torch.zeros(-(-n // 128) * 128, cols)
        full[:n] = part
        want, want_s = ref.quantize(full.t(), tiles_t)
        got_s = st[:, at // 128:(at + len(full)) // 128] if tiles_t else st[at // 128:(at + len(full)) // 128]
        assert torch.equal(got_s.cpu().double(), want_s) and same_values(qt[:, at:at + len(full)], want)
        at += len(full)
    assert bool((q.view(torch.uint8)[:skip] == 0x31).all()) and bool((q.view(torch.uint8)[skip + sum(lengths):] == 0x31).all())
    assert bool((qt.view(torch.uint8)[:, at:] == 0x31).all())


# -------------------------------------------------------------------------------- products --

def operands(rows, cols, depth, seed=0, batch=None):
    """8-bit matrices and scales that are not powers of two."""
    g = torch.Generator().manual_seed(seed + rows + 7 * cols + 31 * depth)
    a, a_s = q_of(rows, depth)
    b, b_s = q_of(cols, depth, True, batch)
    for q, s in ((a, a_s), (b, b_s)):
        q.copy_((torch.randn(q.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn))
        s.copy_(torch.exp(torch.randn(s.shape, generator=g)))
    return a, a_s, b, b_s


def check(out, a, a_s, b, b_s):
    y, bound = ref.matmul(a.float().cpu(), a_s.cpu(), b.float().cpu(), b_s.cpu(), out.dtype is torch.float32)
    off = (out.double().cpu() - y).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("rows", [1, 2, 15, 17, 33, 64, 100, 128, 129, 300, 600])
@pytest.mark.parametrize("cols,depth", [(1, 1), (8, 16), (127, 130), (128, 128), (260, 1000), (1544, 640), (130, 4096)])
def test_product(rows, cols, depth):
    a, a_s, b, b_s = operands(rows, cols, depth)
    for dtype, extra in ((torch.bfloat16, 0), (torch.float32, 3)):
        buf = torch.full((rows, cols + extra), 9.0, dtype=dtype, device="cuda")
        rv.relay_matmul_fp8(a, a_s, b, b_s, buf[:, :cols])
        rv.device_status()
        check(buf[:, :cols], a, a_s, b, b_s)
        assert bool((buf[:, cols:] == 9.0).all())


# What each kernel of relay_matmul_fp8 is chosen for: pairs of CTAs, 128, 64, 32 and 16 rows to a tile, the depth whole and split two, four
# and eight ways.
FORMS = [(3000, 1000, 200), (3000, 2056, 640), (3000, 2051, 640), (3001, 2060, 300), (400, 4096, 1024), (390, 4090, 500), (300, 1030, 6000),
         (300, 512, 4096), (40, 3000, 3000), (40, 2051, 4000), (200, 2051, 700), (16, 8192, 4096), (9, 520, 4096), (16, 12000, 9000)]


@pytest.mark.parametrize("rows,cols,depth", FORMS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_every_form_of_the_product(rows, cols, depth, out):
    a, a_s, b, b_s = operands(rows, cols, depth)
    y, bound = ref.matmul(a.float(), a_s, b.float(), b_s, out is torch.float32)
    for extra, skip in ((0, 0), (24, 8), (1, 1)):          # rows on the 16-byte grid, views of wider rows, rows off it
        buf = torch.full((rows, cols + extra), 9.0, dtype=out, device="cuda")
        got = buf[:, skip:skip + cols]
        rv.relay_matmul_fp8(a, a_s, b, b_s, got)
        rv.device_status()
        assert bool(((got.double() - y).abs() <= bound).all())
        assert bool((buf[:, :skip] == 9.0).all()) and bool((buf[:, skip + cols:] == 9.0).all())


@pytest.mark.parametrize("lengths,cols,depth", [
    ([3000, 1, 0, 2500, 3499], 520, 384), ([255, 257, 256, 4000, 31, 4201], 514, 300), ([64] * 32, 1408, 512),
    ([700, 0, 33, 64, 65, 1, 137] + [0] * 25, 1000, 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_every_form_of_the_product_of_groups(lengths, cols, depth, out):
    skip, rows, n = 5, sum(lengths) + 9, len(lengths)
    a, a_s, b, b_s = operands(rows, cols, depth, batch=n)
    off = offsets(lengths, skip)
    got = torch.full((rows, cols), 9.0, dtype=out, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, got, offset=off.cuda())
    rv.device_status()
    for i in range(n):
        part = slice(int(off[i]), int(off[i + 1]))
        y, bound = ref.matmul(a[part].float(), a_s[:, part], b[i].float(), b_s[i], out is torch.float32)
        assert bool(((got[part].double() - y).abs() <= bound).all())
    assert bool((got[:skip] == 9.0).all()) and bool((got[int(off[-1]):] == 9.0).all())


@pytest.mark.parametrize("cols", [1040, 1041])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_pairs_by_depth(cols, out):
    rows, lengths = 1100, [300, 0, 1000, 7]
    depth = rv.fp8_depth(sum(lengths), 4)
    a, a_s, b, b_s = operands(rows, cols, depth)
    got = torch.full((4, rows, cols), 9.0, dtype=out, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, got, offset=offsets(lengths).cuda(), by_depth=True)
    rv.device_status()
    at = 0
    for i, m in enumerate(lengths):
        end = at + -(-m // 128) * 128
        if m == 0:
            assert bool((got[i] == 0).all())
            continue
        ks = slice(at // 128, end // 128)
        y, bound = ref.matmul(a[:, at:end].float(), a_s[ks], b[:, at:end].float(), b_s[:, ks], out is torch.float32)
        assert bool(((got[i].double() - y).abs() <= bound).all())
        at = end


def test_product_without_depth():
    out = torch.full((5, 7), 9.0, device="cuda")
    a, a_s = rv.alloc_fp8(5, 0, "cuda")
    b, b_s = rv.alloc_fp8(7, 0, "cuda", tiles=True)
    rv.relay_matmul_fp8(a, a_s, b, b_s, out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("lengths", GROUPS + [[700, 3, 0, 90], [64] * 9, [300] * 5])
@pytest.mark.parametrize("cols,depth", [(130, 256), (40, 1000)])
def test_product_of_groups(lengths, cols, depth):
    skip, behind, n = 2, 3, len(lengths)
    rows = skip + sum(lengths) + behind
    a, a_s, b, b_s = operands(rows, cols, depth, batch=n)
    off = offsets(lengths, skip)
    out = torch.full((rows, cols), 9.0, dtype=torch.float32, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, out, offset=off.cuda())
    rv.device_status()
    for i in range(n):
        part = slice(int(off[i]), int(off[i + 1]))
        check(out[part], a[part], a_s[:, part], b[i], b_s[i])
    assert bool((out[:skip] == 9.0).all()) and bool((out[skip + sum(lengths):] == 9.0).all())


@pytest.mark.parametrize("lengths", GROUPS + [[700, 3, 0, 90], [64] * 9])
@pytest.mark.parametrize("rows,cols", [(20, 300), (130, 200), (400, 130)])
def test_product_by_depth(lengths, rows, cols):
    tokens, n = sum(lengths) + 4, len(lengths)
    depth = rv.fp8_depth(tokens, n)
    a, a_s, b, b_s = operands(rows, cols, depth)
    off = offsets(lengths, 1)
    out = torch.full((n, rows, cols), 9.0, dtype=torch.float32, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, out, offset=off.cuda(), by_depth=True)
    rv.device_status()
    at = 0
    for i, m in enumerate(lengths):
        end = at + -(-m // 128) * 128
        if m == 0:
            assert bool((out[i] == 0).all())
        else:
            ks = slice(at // 128, end // 128)
            check(out[i], a[:, at:end], a_s[ks], b[:, at:end], b_s[:, ks])
        at = end


@pytest.mark.parametrize("rows,cols,depth", [(20, 300, 40), (300, 130, 1000)])
def test_product_by_depth_without_groups(rows, cols, depth):
    """The whole depth is one group, of any length."""
    a, a_s, b, b_s = operands(rows, cols, depth)
    out = torch.full((1, rows, cols), 9.0, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, out, by_depth=True)
    check(out[0], a, a_s, b, b_s)
    flat = torch.full((rows, cols), 9.0, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, flat, by_depth=True)
    assert torch.equal(flat, out[0])


def test_offsets_beyond_32_bits():
    """More than 2^31 values in an operand and in the result."""
    rows, cols, depth = 270000, 8192, 128
    a, a_s, b, b_s = operands(rows, cols, depth)
    out = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    rv.relay_matmul_fp8(a, a_s, b, b_s, out)
    rv.device_status()
    for part in (slice(0, 50), slice(262100, 262200), slice(rows - 40, rows)):
        check(out[part], a[part], a_s[:, part], b, b_s)
    del out
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda") % 256 - 128
    q, s = q_of(rows, cols)
    rv.relay_quantize_fp8(x, q, s)
    want, want_s = ref.quantize(x[-1:].cpu(), False)
    assert same_values(q[-1:], want) and torch.equal(s[:, -1:].cpu().double(), want_s)
    assert bool((q[-2].view(torch.uint8) == 0).all())


@pytest.mark.parametrize("rows", [4, 60, 200, 9000])
def test_offsets_that_are_wrong_stay_in_range(rows):
    """Unspecified results, no access out of range: what lies around the output stays."""
    a, a_s, b, b_s = operands(rows, 130, 256, batch=6)
    x = torch.randn(rows, 130, device="cuda")
    for bad in ([0, -5, 10 ** 9, 3, rows, rows + 7, 1], [2 ** 31 - 1] * 7, [-2 ** 31] * 7, [0, rows, 0, rows, 0, rows, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf = torch.full((rows + 2, 130), 9.0, device="cuda")
        rv.relay_matmul_fp8(a, a_s, b, b_s, buf[1:-1], offset=off)
        depth = rv.fp8_depth(rows, 6)
        qt, st = q_of(130, depth)
        rv.relay_quantize_fp8(x, qt=qt, scale_t=st, offset=off)
        g, g_s, h, h_s = operands(140, 130, depth)
        deep = torch.full((8, 140, 130), 9.0, device="cuda")
        rv.relay_matmul_fp8(g, g_s, h, h_s, deep[1:-1], offset=off, by_depth=True)
        torch.cuda.synchronize()
        rv.device_status()
        assert bool((buf[0] == 9.0).all()) and bool((buf[-1] == 9.0).all())
        assert bool((deep[0] == 9.0).all()) and bool((deep[-1] == 9.0).all())


def test_a_block_that_is_not_finite_shows_in_its_rows():
    x, w = torch.randn(70, 300), torch.randn(260, 300)
    x[3, 200], x[5, 0] = math.nan, math.inf
    xq, xs = q_of(70, 300)
    wq, ws = q_of(260, 300, True)
    rv.relay_quantize_fp8(x.cuda(), xq, xs)
    rv.relay_quantize_fp8(w.cuda(), wq, ws, tiles=True)
    out = torch.empty(70, 260, device="cuda")
    rv.relay_matmul_fp8(xq, xs, wq, ws, out)
    nan = torch.isnan(out).cpu()
    assert bool(nan[[3, 5]].all()) and int(nan.sum()) == 2 * 260


@pytest.mark.parametrize("rows", [3, 50, 500, 9000])
def test_equal_calls_equal_bits_and_captured(rows):
    x, w = torch.randn(rows, 520, device="cuda").bfloat16(), torch.randn(2, 390, 520, device="cuda").bfloat16()
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    xq, xs = q_of(rows, 520)
    wq, ws = q_of(390, 520, True, 2)
    out = torch.empty(rows, 390, dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        rv.relay_quantize_fp8(w, wq, ws, tiles=True, stream=stream)
        rv.relay_quantize_fp8(x, xq, xs, stream=stream)
        rv.relay_matmul_fp8(xq, xs, wq, ws, out, offset=off, stream=stream)
    step()
    first = out.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    step(stream)
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    off.copy_(torch.tensor([0, rows, rows], dtype=torch.int32))      # the groups are read when the call runs
    x.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    y, bound = ref.matmul(xq.float(), xs, wq[0].float(), ws[0], False)
    assert bool(((out.double() - y).abs() <= bound).all())


@pytest.mark.parametrize("lengths", [[200], [100, 0, 333, 50]])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_a_layer_forward_and_backward(lengths, out):
    """Quantize, multiply, and both gradients, as a training step calls them: against the products of the 64-bit
    quantized matrices."""
    n, d, c = len(lengths), 300, 280
    rows = sum(lengths)
    g = torch.Generator().manual_seed(rows)
    x, dy = torch.randn(rows, d, generator=g).bfloat16(), (torch.randn(rows, c, generator=g) * 1e-3).bfloat16()
    w = (torch.randn(n, c, d, generator=g) * 0.1).bfloat16()
    off = offsets(lengths).cuda()
    deep = rv.fp8_depth(rows, n)
    wq, ws = q_of(c, d, True, n)
    wt, wts = q_of(d, c, True, n)
    xq, xs = q_of(rows, d)
    xt, xts = q_of(d, deep, True)
    gq, gs = q_of(rows, c)
    gt, gts = q_of(c, deep)
    y, dx, dw = (torch.full(s, 9.0, dtype=out, device="cuda") for s in ((rows, c), (rows, d), (n, c, d)))
    rv.relay_quantize_fp8(w.cuda(), wq, ws, wt, wts, tiles=True, tiles_t=True)
    rv.relay_quantize_fp8(x.cuda(), xq, xs, xt, xts, tiles_t=True, offset=off)
    rv.relay_matmul_fp8(xq, xs, wq, ws, y, offset=off)
    rv.relay_quantize_fp8(dy.cuda(), gq, gs, gt, gts, offset=off)
    rv.relay_matmul_fp8(gq, gs, wt, wts, dx, offset=off)
    rv.relay_matmul_fp8(gt, gts, xt, xts, dw, offset=off, by_depth=True)
    rv.device_status()
    at, wide = 0, out is torch.float32
    for i, m in enumerate(lengths):
        part = slice(at, at + m)
        at += m
        for got, a, b in ((y[part], x[part], w[i]), (dx[part], dy[part], w[i].t()), (dw[i], dy[part].t(), x[part].t())):
            if m == 0:
                assert bool((got == 0).all())
                continue
            want, bound = ref.matmul(*ref.quantize(a, False), *ref.quantize(b, True), wide)
            assert bool(((got.double().cpu() - want).abs() <= bound).all())
    # the quantized gradient is the gradient: off by the two roundings to a 3-bit fraction, 2^-4 of each factor at most
    want = torch.cat([dy[off[i]:off[i + 1]].double() @ w[i].double() for i in range(n)])
    size = torch.cat([dy[off[i]:off[i + 1]].double().abs() @ w[i].double().abs() for i in range(n)])
    small = 300 * 2.0 ** -10 * 448 * 448 * 2.0 ** -20                # values below the normal range of their block
    assert bool(((dx.double().cpu() - want).abs() <= 0.14 * size + small).all())


@pytest.mark.parametrize("rows", [4, 100, 300, 9000])
def test_waits_run_out_and_are_reported(rows):
    """The stage barriers expect more bytes than the loads bring: the kernel gives up, says so, and the context stays
    usable."""
    L = rv.lib()
    rv.device_status()
    a, a_s, b, b_s = operands(rows, 300, 1500)
    out = torch.empty(rows, 300, device="cuda")
    words = rv._binding._matmul_fp8_words(a, a_s, b, b_s, out, None, False)
    for extra, status in ((0, rv.OK), (16, rv.ERR_CUDA), (0, rv.OK)):
        assert L.relay_test_fp8_wait(words, extra, None) == rv.OK
        torch.cuda.synchronize()
        assert L.relay_device_status() == status
        if status != rv.OK:
            assert b"gave up" in L.relay_last_error()
            assert L.relay_device_status() == rv.OK
    y, bound = ref.matmul(a.float(), a_s, b.float(), b_s, True)
    assert bool(((out.double() - y).abs() <= bound).all())
