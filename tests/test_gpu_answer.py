"""The operators between a model's last hidden state and text on the GPU,
against plain 64-bit forms (tests/answers.py)."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import answers

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bpe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bpe_merge_amd
    return bpe_merge_amd


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _same(a, b):
    return torch.equal(a.cpu().view(torch.uint8) if a.dtype == E4M3 else a.cpu(),
                       b.cpu().view(torch.uint8) if b.dtype == E4M3 else b.cpu())


# ---------------------------------------------------------------- norm

def _check_norm(q, scales, h, x, r, w, eps):
    y, h64 = answers.norm(x, r, w, eps)
    # h: one f32 addition, then one rounding to x's type
    step = answers.half_step(x.dtype) + (2.0 ** -24 if x.dtype != torch.float32 else 0.0)
    small = torch.finfo(x.dtype).tiny * answers.half_step(x.dtype) * 2
    assert np.all(np.abs(h.double().cpu().numpy() - h64) <= step * np.abs(h64) + small)
    # y in f32: the addition (in y and, halved twice, in its root), the root's
    # rounding and two products: 5 half steps; its block's scale one more
    s = scales.double().cpu().numpy()
    want = np.maximum(answers.block_max(y) / 448.0, answers.TINY)
    assert np.all(np.abs(s - want) <= 8 * 2.0 ** -24 * want)
    # e4m3: half a step of 2^-3, or half the smallest step 2^-9
    sw = answers.spread(s, *y.shape, False)
    got = q.float().double().cpu().numpy() * sw
    assert np.all(np.abs(got - y) <= (2.0 ** -4 * np.abs(y) + 2.0 ** -10 * sw) * (1 + 2.0 ** -18))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, d", [(1, 1), (1, 7), (3, 8), (5, 127), (2, 128), (9, 129), (4, 512), (7, 513), (6, 1000),
                                     (3, 1024), (2, 1031), (3, 2048), (5, 2049), (2, 4096), (3, 5000), (2, 8192),
                                     (2, 8200), (1, 20001), (1, 65536)])
def test_norm_quant(bpe, dtype, rows, d):
    x = (_randn(rows * d, rows, d) * 2).to(dtype).cuda()
    r = (_randn(rows * d + 1, rows, d) * 5).to(dtype).cuda()
    w = (1 + 0.3 * _randn(d, d)).to(dtype).cuda()
    _check_norm(*bpe.norm_quant(x, w, residual=r, eps=1e-5), x, r, w, 1e-5)
    q, s, h = bpe.norm_quant(x, w, eps=1e-2)
    _check_norm(q, s, h, x, None, w, 1e-2)
    assert _same(h, x)


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_quant_in_place_strided_and_more_dimensions(bpe, dtype):
    rows, d = 10, 700
    wide = _randn(1, rows, 1501).to(dtype).cuda()
    x, r = wide[:, 1:701], _randn(2, rows, d).to(dtype).cuda()
    w = (1 + 0.3 * _randn(3, d)).to(dtype).cuda()
    want = bpe.norm_quant(x.contiguous(), w, residual=r)
    assert all(_same(a, b) for a, b in zip(bpe.norm_quant(x, w, residual=r), want))
    before = wide.clone()
    held = r.clone()
    got = bpe.norm_quant(x, w, residual=held, sum_out=held)
    assert got[2] is held and all(_same(a, b) for a, b in zip(got, want)) and _same(wide, before)
    got = bpe.norm_quant(x, w, residual=r, sum_out=x)
    assert all(_same(a, b) for a, b in zip(got, want)) and _same(wide[:, 701:], before[:, 701:]) and _same(wide[:, 0], before[:, 0])
    q, s, h = bpe.norm_quant(before[:, 1:701].reshape(2, 5, d), w, residual=r.reshape(2, 5, d))
    assert q.shape == (2, 5, d) and s.shape == (2, 5, 6) and _same(q.reshape(rows, d), want[0]) and _same(s.reshape(rows, 6), want[1])
    assert [t.shape for t in bpe.norm_quant(x[:0], w)] == [(0, d), (0, 6), (0, d)]
    q, s, h = bpe.norm_quant(r[3], w)
    assert q.shape == (d,) and s.shape == (6,)


def test_no_gradients_pass_through(bpe):
    x = _randn(1, 3, 256).cuda().requires_grad_()
    w = torch.ones(256).cuda().requires_grad_()
    q, s, h = bpe.norm_quant(x, w, residual=x)
    b, sb = bpe.quant_weight(x)
    logits = bpe.matmul_scaled(q, s, b, sb, out_dtype=torch.float32)
    ids, logp = bpe.sample(logits.requires_grad_(), torch.rand(3).cuda())
    assert not any(t.requires_grad for t in (q, s, h, b, sb, ids, logp))


def test_norm_quant_of_zeros_extremes_and_no_numbers(bpe):
    d = 300
    w = torch.ones(d).cuda()
    x = _randn(5, 6, d)
    x[0] = 0.0
    x[1, 7] = math.nan
    x[2, 200] = math.inf
    x[3] = x[3] * 1e30          # squares past the f32 range
    x[4, :128] = 0.0            # a block of zeros beside others
    x[5] = x[5] * 1e-25
    q, s, h = (t.float().cpu().numpy() for t in bpe.norm_quant(x.cuda(), w, eps=1e-12))
    assert not q[0].any() and np.all(s[0] == np.float32(answers.TINY))
    assert np.isnan(q[1]).all() and np.isnan(s[1]).all()
    assert np.isnan(q[2, 200]) and np.isnan(s[2, 1]) and not q[2, :128].any() and not q[2, 256:].any()
    for i in (3, 4, 5):
        _check_norm(*bpe.norm_quant(x[i:i + 1].cuda(), w, eps=1e-12), x[i:i + 1], None, w, 1e-12)
    w[130] = math.nan
    q, s, _ = (t.float().cpu().numpy() for t in bpe.norm_quant(x[4:5].cuda(), w))
    assert np.isnan(s[0]).tolist() == [False, True, False] and np.isnan(q[0, 128:256]).all() and not np.isnan(q[0, 256:]).any()


@pytest.mark.parametrize("d", [40, 700, 3000, 20001])
def test_norm_quant_of_tiny_rows_without_eps(bpe, d):
    """Root mean squares from the smallest f32 numbers on: y is of the
    weight's size all the same."""
    w = (1 + 0.3 * _randn(d, d)).cuda()
    x = _randn(d + 1, 6, d) * torch.tensor([2.0 ** -149, 2.0 ** -140, 2.0 ** -128, 2.0 ** -126, 2.0 ** -100, 1.0])[:, None].double()
    x = x.float()
    x[0] = 0.0
    x[0, d // 2] = 2.0 ** -149
    _check_norm(*bpe.norm_quant(x.cuda(), w, eps=0.0), x, None, w, 0.0)
    x = x.bfloat16()
    x[0, d // 3] = 2.0 ** -133
    q, s, h = (t.cpu() for t in bpe.norm_quant(x.cuda(), w.bfloat16(), eps=0.0))
    some = (x != 0).any(1)  # the second row's numbers are too small for bfloat16: 0 / 0
    assert some.tolist() == [True, False, True, True, True, True]
    _check_norm(q[some], s[some], h[some], x[some], None, w.bfloat16(), 0.0)
    assert bool(q[1].float().isnan().all()) and bool(s[1].isnan().all()) and not bool(h[1].any())


def test_norm_quant_of_more_rows_than_a_launch_takes(bpe):
    """2^26 rows of up to 1,024 columns are more threads than a launch has."""
    rows = (1 << 26) + 5
    x = torch.randn(rows, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    w = torch.tensor([1.5]).bfloat16().cuda()
    q, s, h = bpe.norm_quant(x, w, residual=x, eps=0.5)
    step = 1 << 24
    for at in range(0, rows, step):
        part = slice(at, min(rows, at + step))
        for got, want in zip((q, s, h), bpe.norm_quant(x[part], w, residual=x[part], eps=0.5)):
            assert torch.equal(got[part].view(torch.uint8), want.view(torch.uint8))
    _check_norm(q[-9:], s[-9:], h[-9:], x[-9:], x[-9:], w, 0.5)


# ---------------------------------------------------------------- product

def _operand(seed, rows, k, rows_too):
    """e4m3 values over their whole range, and scales of very different sizes."""
    v = _randn(seed, rows, k) * torch.exp2(torch.randint(-6, 6, (rows, 1), generator=torch.Generator().manual_seed(seed)).float())
    q = v.clamp(-448, 448).to(E4M3)
    blocks = -(-k // 128)
    s = torch.exp2(_randn(seed + 1, -(-rows // 128) if rows_too else rows, blocks) * 2)
    return q, s


def _check_product(out, a, sa, b, sb):
    want, size = answers.product(a, sa, b, sb)
    off = np.abs(out.double().cpu().numpy() - want)
    tol = answers.product_tolerance(size, sa.shape[1]) + answers.half_step(out.dtype) * np.abs(want)
    if out.dtype != torch.float32 and out.shape[0] > 64:  # the e4m3 instructions' own sums
        tol += answers.product_dropped(a, sa, b, sb)
    tol *= 1 + 2.0 ** -8  # the second rounding is of the first one's result
    if out.dtype == torch.float16:
        tol += 2.0 ** -25
    bad = off > tol
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), off[bad][:5], want[bad][:5])


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 100, 5), (2, 17, 130), (16, 300, 256), (17, 129, 384), (5, 70, 1000), (32, 65, 512),
          (33, 200, 272), (64, 128, 128), (64, 33, 2048), (65, 127, 256), (100, 300, 640), (128, 129, 144), (129, 257, 512),
          (200, 456, 1000), (256, 512, 1024), (300, 1000, 387), (513, 260, 128)]


@pytest.mark.parametrize("m, n, k", SHAPES)
def test_matmul_scaled(bpe, m, n, k):
    a, sa = _operand(m + k, m, k, False)
    b, sb = _operand(n + 2 * k, n, k, True)
    sa, sb = sa * 2.0 ** -6, sb * 2.0 ** -8
    ac, sac, bc, sbc = (t.cuda() for t in (a, sa, b, sb))
    for dtype in TYPES:
        # f16: kept inside its range
        f = 2.0 ** -8 if dtype == torch.float16 else 1.0
        _check_product(bpe.matmul_scaled(ac, sac * f, bc, sbc, out_dtype=dtype), a, sa * f, b, sb)


# by the tile that each takes: 128 x 64 (whole and short last blocks), 256 x
# 256, 256 x 128 (short), 128 x 128 (short), streams over more than 64 rows;
# rows that go through registers: 128 x 64 and 128 x 128, of a block or more
# and of less
@pytest.mark.parametrize("m, n, k", [(5, 6200, 256), (64, 6200, 400), (33, 6150, 144), (520, 16640, 384), (260, 40000, 272),
                                     (515, 8000, 528), (130, 456, 2064), (33, 16100, 401), (2, 30050, 129), (64, 12500, 255),
                                     (515, 8000, 529), (70, 3300, 1023), (64, 1700, 2064), (600, 456, 2049), (64, 12500, 127), (9, 48100, 5),
                                     (300, 700, 100), (515, 8000, 63), (65, 500, 1)])
def test_matmul_scaled_of_every_tile(bpe, m, n, k):
    """Large results, looked at in whole blocks of columns: the first two, one
    in the middle and the last two."""
    a, sa = _operand(m, m, k, False)
    b, sb = _operand(n, n, k, True)
    last = (n - 1) // 128
    take = sorted({0, 1, last // 2, last - 1, last})
    columns = [c for block in take for c in range(block * 128, min(n, block * 128 + 128))]
    rows = sorted({0, 1, m // 2, m - 2, m - 1} | set(range(0, m, max(1, m // 40))))
    for dtype in (torch.float32, torch.bfloat16):
        out = bpe.matmul_scaled(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
        want, size = answers.product(a[rows], sa[rows], b[columns], sb[take])
        got = out[rows][:, columns].double().cpu().numpy()
        tol = answers.product_tolerance(size, sa.shape[1]) + answers.half_step(dtype) * np.abs(want)
        if dtype != torch.float32 and m > 64:
            tol += answers.product_dropped(a[rows], sa[rows], b[columns], sb[take])
        assert np.all(np.abs(got - want) <= tol * (1 + 2.0 ** -8))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m, n, k", [(16, 40, 128), (64, 6200, 256), (65, 300, 128), (130, 300, 272), (130, 300, 257),
                                     (600, 8256, 1024), (520, 16640, 384), (789, 9244, 128), (130, 456, 2048)])
def test_matmul_scaled_of_sums_that_cancel(bpe, dtype, m, n, k):
    """Two of the groups of 8 columns hold one product of 2^16 and seven of
    7.5, just below 2^-13 of it; the large ones cancel. f32 sums leave 105;
    bfloat16 results of more than 64 rows are allowed to lose the small ones."""
    row = torch.zeros(2, k)
    for at, large in ((0, 256.0), (64, -256.0)):
        row[0, at:at + 8], row[1, at:at + 8] = 2.0, 3.75
        row[0, at + 3], row[1, at + 3] = 256.0, large
    a, b = row[:1].expand(m, k).to(E4M3).contiguous(), row[1:].expand(n, k).to(E4M3).contiguous()
    blocks = -(-k // 128)
    sa, sb = torch.ones(m, blocks), torch.ones(-(-n // 128), blocks)
    out = bpe.matmul_scaled(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype).double()
    want, size = answers.product(a[:1], sa[:1], b[:1], sb[:1])
    assert want[0, 0] == 105.0
    tol = answers.product_tolerance(size, blocks) + answers.half_step(dtype) * want
    if dtype == torch.bfloat16 and m > 64:
        tol += answers.product_dropped(a[:1], sa[:1], b[:1], sb[:1])
    assert float((out - 105.0).abs().max()) <= tol[0, 0] * (1 + 2.0 ** -8)


@pytest.mark.parametrize("m, n, k, pad", [(3, 50, 256, 16), (3, 50, 256, 3), (40, 100, 384, 16), (40, 100, 384, 1), (150, 140, 256, 48),
                                          (150, 140, 256, 5), (3, 50, 90, 7), (70, 7000, 2064, 1),
                                          (3, 9000, 6800, 1)])
def test_matmul_scaled_of_rows_in_wider_buffers(bpe, m, n, k, pad):
    """What lies beside the rows is NaN: it must neither count nor change."""
    def wide(t, pad, fill):
        w = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=torch.float32).to(t.dtype).cuda()
        w[:, :t.shape[1]] = t.cuda()
        return w
    a, sa = _operand(1, m, k, False)
    b, sb = _operand(2, n, k, True)
    aw, bw = wide(a, pad, math.nan), wide(b, pad, math.nan)
    saw, sbw = wide(sa, 3, math.nan), wide(sb, 2, math.nan)
    ow = torch.full((m, n + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    blocks = sa.shape[1]
    out = bpe.matmul_scaled(aw[:, :k], saw[:, :blocks], bw[:, :k], sbw[:, :blocks], out=ow[:, :n])
    assert out.data_ptr() == ow.data_ptr() and bool((ow[:, n:] == 7.0).all())
    _check_product(out, a, sa, b, sb)
    if pad > 5:  # rows that begin inside a buffer
        _check_product(bpe.matmul_scaled(aw[1:, :k], saw[1:, :blocks], bw[:, :k], sbw[:, :blocks]), a[1:], sa[1:], b, sb)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m, n, k", answers.PRODUCTS)
def test_matmul_scaled_by_every_kernel(bpe, dtype, m, n, k):
    """Looked at as in the test of every tile, in every type."""
    a, sa = _operand(m, m, k, False)
    b, sb = _operand(n, n, k, True)
    if dtype == torch.float16:  # kept inside its range
        sa, sb = sa * 2.0 ** -14, sb * 2.0 ** -8
    last = (n - 1) // 128
    take = sorted({0, 1, last // 2, last - 1, last})
    columns = [c for block in take for c in range(block * 128, min(n, block * 128 + 128))]
    rows = sorted({0, m // 2, m - 1} | set(range(0, m, max(1, m // 40))))
    out = bpe.matmul_scaled(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=dtype)
    want, size = answers.product(a[rows], sa[rows], b[columns], sb[take])
    got = out[rows][:, columns].double().cpu().numpy()
    tol = answers.product_tolerance(size, sa.shape[1]) + answers.half_step(dtype) * np.abs(want)
    if dtype == torch.bfloat16 and m > 64:
        tol += answers.product_dropped(a[rows], sa[rows], b[columns], sb[take])
    tol = tol * (1 + 2.0 ** -8) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert dtype != torch.float16 or np.abs(want).max() < 65504
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("far", ["a", "b", "both"])
def test_matmul_scaled_of_rows_far_apart(bpe, dtype, far):
    """Rows 2^23 bytes apart and more, which leave a tile's 32-bit offsets."""
    m, n, k = 70, 20, 300
    a, sa = _operand(3, m, k, False)
    b, sb = _operand(4, n, k, True)

    def spread(t, wide):
        if not wide:
            return t.cuda()
        f = torch.full(((t.shape[0] - 1) * ((1 << 23) + 48) + t.shape[1],), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
        v = f.as_strided(t.shape, ((1 << 23) + 48, 1))
        v.copy_(t)
        return v
    out = bpe.matmul_scaled(spread(a, far != "b"), sa.cuda() * 2.0 ** -8, spread(b, far != "a"), sb.cuda() * 2.0 ** -8, out_dtype=dtype)
    _check_product(out, a, sa * 2.0 ** -8, b, sb * 2.0 ** -8)


def test_matmul_scaled_of_more_rows_than_a_launch_takes(bpe):
    """2^16 workgroups of 64 rows of a, by two rows of b 2^23 bytes apart."""
    m, n, k = (1 << 22) + 70, 2, 16
    a, sa = _operand(3, 4096, k, False)
    b, sb = _operand(4, n, k, True)
    at = torch.randint(0, 4096, (m,), generator=torch.Generator().manual_seed(5))
    f = torch.zeros((1 << 23) + k, dtype=torch.uint8, device="cuda").view(E4M3)
    bw = f.as_strided((n, k), (1 << 23, 1))
    bw.copy_(b)
    few = bpe.matmul_scaled(a.cuda(), sa.cuda(), bw, sb.cuda(), out_dtype=torch.float32)
    _check_product(few, a, sa, b, sb)
    many = bpe.matmul_scaled(a.view(torch.uint8)[at].view(E4M3).cuda(), sa[at].cuda(), bw, sb.cuda(), out_dtype=torch.float32)
    assert torch.equal(many, few[at.cuda()])


def test_matmul_scaled_rows_do_not_depend_on_one_another(bpe):
    a, sa = (t.cuda() for t in _operand(5, 200, 512, False))
    b, sb = (t.cuda() for t in _operand(6, 300, 512, True))
    want = bpe.matmul_scaled(a, sa, b, sb, out_dtype=torch.float32)
    bad = a.float()
    bad[7] = math.nan
    sa2 = sa.clone()
    sa2[100] = math.inf
    got = bpe.matmul_scaled(bad.to(E4M3), sa2, b, sb, out_dtype=torch.float32)
    keep = [i for i in range(200) if i not in (7, 100)]
    assert _same(got[keep], want[keep]) and bool(got[7].isnan().all()) and not bool(got[100].isfinite().any())
    assert _same(bpe.matmul_scaled(a, sa, b, sb, out_dtype=torch.float32), want)


def test_matmul_scaled_past_the_end_of_short_rows(bpe):
    """NaN right behind the last row of either operand, where a short last
    block's copies must not reach."""
    for m, n, k in ((70, 300, 400), (20, 6200, 144), (300, 300, 272)):
        a, sa = _operand(1, m, k, False)
        b, sb = _operand(2, n, k, True)

        def fenced(t):
            f = torch.full((t.numel() + 512,), math.nan).to(E4M3).cuda()
            v = f[256:256 + t.numel()].view(t.shape)
            v.copy_(t)
            return v
        for dtype in (torch.float32, torch.bfloat16):
            _check_product(bpe.matmul_scaled(fenced(a), sa.cuda(), fenced(b), sb.cuda(), out_dtype=dtype), a, sa, b, sb)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, k", [(1, 1), (3, 130), (128, 128), (129, 127), (300, 1000)])
def test_quant_weight(bpe, dtype, n, k):
    w = (_randn(n + k, n, k + 5) * 0.02).to(dtype)
    q, s = bpe.quant_weight(w.cuda()[:, 2:k + 2])
    y = w[:, 2:k + 2].double().numpy()
    want = np.maximum(answers.block_max(y, True) / 448.0, answers.TINY)
    got_s = s.double().cpu().numpy()
    assert np.all(np.abs(got_s - want) <= 2.0 ** -24 * want)
    sw = answers.spread(got_s, n, k, True)
    off = np.abs(q.float().double().cpu().numpy() * sw - y)
    assert np.all(off <= (2.0 ** -4 * np.abs(y) + 2.0 ** -10 * sw) * (1 + 2.0 ** -18))


def _by_division(y, s):
    """e4m3 codes of the f32 quotients y / s."""
    return torch.from_numpy(y.float().cpu().numpy() / s.astype(np.float32)).to(E4M3)


@pytest.mark.parametrize("dtype", TYPES)
def test_quant_weight_divides(bpe, dtype):
    """Values of 8 to 12 bits often lie half way between two codes of their
    block's scale: the quotient has to be rounded once."""
    n, k = 515, 1030
    w = _randn(7, n, k) * 0.02
    w[130:300] *= torch.exp2(-135 * torch.rand(170, 1, generator=torch.Generator().manual_seed(1)))
    w[300:, :500] *= 1e37
    w[5, 100:200] = torch.tensor([0.0, -0.0] * 50)
    w = w.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)
    q, s = bpe.quant_weight(w.cuda())
    assert _same(q, _by_division(w, answers.spread(s.cpu().numpy(), n, k, True)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [500, 1024, 2000, 4096, 8192, 65536])
def test_norm_quant_divides(bpe, dtype, d):
    """Rows of 1 and -1 have a norm of exactly 1, so that y is the weight."""
    sign = torch.sign(_randn(d, 3, d)).to(dtype)
    w = (1 + 0.3 * _randn(d + 1, d)).to(dtype)
    w[7:9] = torch.tensor([0.0, -0.0])
    w[256:400] *= 2.0 ** -120 if dtype != torch.float16 else 2.0 ** -14
    q, s, _ = bpe.norm_quant(sign.cuda(), w.cuda(), eps=0.0)
    assert _same(q, _by_division(sign * w, answers.spread(s.cpu().numpy(), 3, d, False)))


# ---------------------------------------------------------------- sampling

def _check_sample(ids, logp, x, u, settings):
    xs = x.float().cpu().numpy()
    for i in range(len(xs)):
        s = [float(np.float32(v if not isinstance(v, (list, np.ndarray)) else v[i])) for v in settings]
        want, share = answers.draw(xs[i], float(u[i]), s[0], int(s[1]), s[2], s[3])
        assert int(ids[i]) == want, (i, int(ids[i]), want, s)
        got = float(logp[i])
        # one f32 rounding; weights are off by half a unit of 2^-43 each
        assert got == share or abs(got - share) <= 2.0 ** -24 * abs(share) + xs.shape[1] * 2.0 ** -43, (i, got, share)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.8, 50, 0.95, 0.0), (1.3, 0, 1.0, 0.05),
            (1.0, 200, 0.8, 0.02), (0.0, 5, 0.9, 0.0), (1.0, 1, 1.0, 0.0), (5.0, 1000, 0.99, 0.0), (1.0, 0, 0.999, 0.0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1, 2, 3, 5, 64, 257, 1023, 1025, 4100, 8192, 8193, 32256, 40001, 65536, 65541])
def test_sample(bpe, dtype, v):
    rows = 6
    g = torch.Generator().manual_seed(v)
    x = (2.5 * torch.randn(rows, v, generator=g)).to(dtype)
    for k, s in enumerate(SETTINGS):
        u = torch.rand(rows, generator=g)
        ids, logp = bpe.sample(x.cuda(), u.cuda(), *s)
        _check_sample(ids.cpu(), logp.cpu(), x, u, s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [6000, 32256, 40001, 65536, 70001])
def test_sample_of_cuts_past_a_list(bpe, dtype, v):
    """More kept than a list holds, by count, by weight and by both, with and
    without a least weight, and the lowest kept id."""
    rows = 5
    g = torch.Generator().manual_seed(v + 1)
    x = (1.5 * torch.randn(rows, v, generator=g)).to(dtype)
    x[3] = x[3].abs().neg()        # a steep edge at the largest
    x[4, ::3] = -math.inf
    for s in ((1.0, 5000, 1.0, 0.0), (1.0, 5000, 0.9, 0.0), (1.0, 0, 0.97, 0.0), (0.6, 3000, 0.99, 0.01), (2.0, 4000, 0.5, 0.1),
              (1.0, 0, 1.0, 0.003), (1.0, 0, 0.9999, 0.0), (0.3, 2000, 0.8, 0.0)):
        for u in (torch.rand(rows, generator=g), torch.zeros(rows), torch.full((rows,), 1 - 2.0 ** -24)):
            ids, logp = bpe.sample(x.cuda(), u.cuda(), *s)
            _check_sample(ids.cpu(), logp.cpu(), x, u, s)


@pytest.mark.parametrize("v", [300, 9000, 50000])
def test_sample_with_settings_for_each_row(bpe, v):
    rows = 40
    g = torch.Generator().manual_seed(v)
    x = 3 * torch.randn(rows, v + 3, generator=g)
    r = np.random.RandomState(v)
    s = [r.choice([0.0, 0.5, 1.0, -1.0, math.nan], rows).astype(np.float32), r.choice([0, 1, 7, 100, -5, 1 << 30], rows).astype(np.int32),
         r.choice([1.0, 0.9, 0.5, 0.0, 2.0, 0.01], rows).astype(np.float32), r.choice([0.0, 0.1, 1.0, 3.0, -1.0], rows).astype(np.float32)]
    u = torch.rand(rows, generator=g)
    ids, logp = bpe.sample(x.cuda()[:, 2:v + 2], u.cuda(), *(torch.from_numpy(t).cuda() for t in s))
    s[2] = np.where(s[2] >= 1, 1, s[2])
    _check_sample(ids.cpu(), logp.cpu(), x[:, 2:v + 2], u, s)


def test_sample_of_equal_logits_is_exact(bpe):
    """Equal weights: the id is the whole part of u times what is kept, and of
    equal logits the lowest ids are kept."""
    for v in (7, 1000, 32256, 65536):
        x = torch.full((8, v), -3.25, device="cuda")
        u = torch.tensor([0.0, 2.0 ** -24, 0.25, 0.5, 0.75, 0.9, 1 - 2.0 ** -24, 0.3])
        for top_k, top_p in ((0, 1.0), (5, 1.0), (v - 1, 1.0), (0, 0.5), (v // 2 + 1, 0.5)):
            keep = top_k or v
            if top_p < 1:
                keep = math.ceil(top_p * keep)
            ids, logp = bpe.sample(x, u.cuda(), top_k=top_k, top_p=top_p)
            assert ids.tolist() == [int(float(t) * keep) for t in u], (v, top_k, top_p)
            assert np.allclose(logp.cpu().numpy(), -math.log(keep), rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("dtype", TYPES)
def test_sample_of_masked_rows(bpe, dtype):
    """Masks of -inf and of the type's lowest value, NaN, +inf, rows with
    nothing left, and steps that need many turns of the search."""
    v = 20000
    low = torch.finfo(dtype).min
    x = (2 * _randn(9, 12, v)).to(dtype)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 100:] = -math.inf
    x[3, 100:] = low
    x[4] = low
    x[5, 5:19990] = math.nan
    x[6, [77, 19999]] = math.inf
    x[7] = x[7].round()                                   # few distinct values
    x[8] = -torch.exp2(torch.arange(v) % 16).to(dtype)     # spacings that double
    x[9, ::2] = 0.0
    x[9, 1::2] = -0.0
    x[10, 3:] = -math.inf
    x[10, :3] = low
    x[11, 1:] = -math.inf
    g = torch.Generator().manual_seed(3)
    for s in SETTINGS + [(1e-3, 500, 0.9, 0.0), (1e6, 3000, 0.7, 0.0), (1.0, 150, 0.9999, 0.0)]:
        for u in (torch.rand(12, generator=g), torch.zeros(12), torch.ones(12), torch.full((12,), math.nan)):
            ids, logp = bpe.sample(x.cuda(), u.cuda(), *s)
            if s[0] != 1e6:
                _check_sample(ids.cpu(), logp.cpu(), x, u, s)
            else:  # weights nearly all equal: compare what does not hang on their 40th bit
                _check_sample(ids.cpu()[[0, 1, 10, 11]], logp.cpu()[[0, 1, 10, 11]], x[[0, 1, 10, 11]], u[[0, 1, 10, 11]], s)


def test_sample_of_more_rows_than_a_launch_takes(bpe):
    """2^24 rows in workgroups of 256 threads, each row with settings."""
    rows = (1 << 24) + 3
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, 2, device="cuda", generator=g)
    x[::7, 0] = -math.inf
    x[::21, 1] = -math.inf
    u = torch.rand(rows, device="cuda", generator=g)
    k = torch.arange(rows, device="cuda", dtype=torch.int32) % 3  # off, the largest, both
    ids, logp = bpe.sample(x, u, top_k=k)
    share = torch.softmax(x.double(), 1)
    want = torch.where(k == 1, x[:, 1] > x[:, 0], u.double() >= share[:, 0]).int()
    sure = (share[:, 0] - u.double()).abs() > 2.0 ** -40  # not on the border itself
    want[::21] = -1
    sure[::21] = True
    assert torch.equal(ids[sure], want[sure])
    assert torch.equal(logp == -math.inf, ids < 0)
    step = 1 << 22
    for at in range(0, rows, step):
        part = slice(at, min(rows, at + step))
        some = bpe.sample(x[part], u[part], top_k=k[part])
        assert torch.equal(ids[part], some[0]) and torch.equal(logp[part], some[1])


# ---------------------------------------------------------------- decoding

@pytest.fixture(scope="module")
def vocabulary():
    merges = answers.merge_list(5000, 4, longest=40)
    return merges, answers.strings(merges)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 2047, 2048, 2049, 4096, 100003, 300007])
def test_decode(bpe, vocabulary, n):
    merges, text = vocabulary
    r = np.random.RandomState(n)
    ids = r.randint(0, len(text), n)
    tagged = np.where(r.rand(n) < 0.3, ids | 0x10000, ids).astype(np.int32)
    tagged[r.rand(n) < 0.01] = -1
    parts = [text[t & 0xFFFF] if t >= 0 else b"" for t in tagged.tolist()]
    want = b"".join(parts)
    with bpe.Decoder(torch.from_numpy(merges)) as d:
        assert d.info() == (5256, max(len(t) for t in text))
        got, places = d.decode(torch.from_numpy(tagged).cuda(), offsets=True)
        assert got.cpu().numpy().tobytes() == want
        assert places.tolist() == [0] + np.cumsum([len(p) for p in parts]).tolist()
        # into a longer buffer, from any alignment: nothing past the text changes
        for skew in (0, 1, 13):
            out = torch.full((len(want) + 64,), 0xAB, dtype=torch.uint8, device="cuda")
            got = d.decode(torch.from_numpy(tagged).cuda(), out=out[skew:])
            assert got.cpu().numpy().tobytes() == want
            rest = out.cpu().numpy()
            assert np.all(rest[:skew] == 0xAB) and np.all(rest[skew + len(want):] == 0xAB)
        # host memory through the C ABI
        host, n_bytes = np.zeros(len(want) + 8, dtype=np.uint8), ctypes.c_size_t(0)
        places = np.zeros(n + 1, dtype=np.int64)
        st = bpe._lib.bpe_decoder_decode(d._h, tagged.ctypes.data if n else None, n, None, host.ctypes.data, host.size,
                                         places.ctypes.data, ctypes.byref(n_bytes))
        assert st == bpe.OK and host[:n_bytes.value].tobytes() == want and places[-1] == len(want)


def test_decode_of_long_strings(bpe):
    """Strings far past an entry and past a tile's staging."""
    merges = [(97 + i, 98 + i, 1) for i in range(4)]
    for k in range(4, 22):
        merges.append((255 + k, 256 + k - 4, 1))
    merges = np.array(merges, dtype=np.int32)
    text = answers.strings(merges)
    r = np.random.RandomState(0)
    for n in (5, 300, 3000):
        ids = r.randint(0, len(text), n).astype(np.int32)
        want = b"".join(text[i] for i in ids.tolist())
        with bpe.Decoder(merges) as d:
            got = d.decode(torch.from_numpy(ids).cuda())
            assert got.cpu().numpy().tobytes() == want
            host, n_bytes = np.zeros(len(want), dtype=np.uint8), ctypes.c_size_t(0)
            assert bpe._lib.bpe_decoder_decode(d._h, ids.ctypes.data, n, None, host.ctypes.data, host.size, None,
                                               ctypes.byref(n_bytes)) == bpe.OK
            assert host.tobytes() == want
            assert bpe._lib.bpe_decoder_decode(d._h, ids.ctypes.data, n, None, host.ctypes.data, host.size - 1, None,
                                               ctypes.byref(n_bytes)) == bpe.EINVAL and n_bytes.value == len(want)
            assert bpe._lib.bpe_decoder_decode(d._h, ids.ctypes.data, n, None, None, 0, None,
                                               ctypes.byref(n_bytes)) == bpe.OK and n_bytes.value == len(want)


def test_decode_refuses_bad_tokens_and_small_buffers(bpe, vocabulary):
    merges, text = vocabulary
    with bpe.Decoder(merges) as d:
        for n in (10, 5000):
            for bad in (5256, 0x20000, 0x7FFFFFFF, -2):
                ids = torch.zeros(n, dtype=torch.int32, device="cuda")
                ids[n - 3] = bad
                ids[n - 1] = bad
                out = torch.full((n + 5,), 7, dtype=torch.uint8, device="cuda")
                with pytest.raises(bpe.BpeError, match="token %d" % (n - 3)):
                    d.decode(ids, out=out)
                assert bool((out == 7).all())
            ids = torch.full((n,), 300, dtype=torch.int32, device="cuda")
            size = n * len(text[300])
            out = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
            with pytest.raises(bpe.BpeError, match="%d bytes" % size):
                d.decode(ids, out=out[:size - 1])
            assert bool((out == 7).all())
            assert d.decode(ids, out=out).cpu().numpy().tobytes() == text[300] * n
        with pytest.raises(TypeError):
            d.decode(torch.zeros(4, dtype=torch.int64, device="cuda"))


def test_decode_refuses_arrays_that_share_memory(bpe, vocabulary):
    merges, _ = vocabulary
    with bpe.Decoder(merges) as d:
        for n in (10, 5000):
            held = torch.zeros(3 * n + 8, dtype=torch.int32, device="cuda")
            ids, memory = held[:n], held.view(torch.uint8)
            for out in (memory, memory[:n], memory[4 * n - 1:], ids[n // 2:].view(torch.uint8)):
                with pytest.raises(bpe.BpeError, match="share"):
                    d.decode(ids, out=out)
            n_bytes = ctypes.c_size_t(0)
            places = held.data_ptr() + 8 * (n // 4)
            for args in ((None, 0, places), (held.data_ptr() + 8 * n, n, held.data_ptr() + 4 * n)):
                assert bpe._lib.bpe_decoder_decode(d._h, ids.data_ptr(), n, None, *args, ctypes.byref(n_bytes)) == bpe.EINVAL
            assert not bool(held.any())
            # side by side is fine
            assert d.decode(ids, out=memory[4 * n:]).tolist() == [0] * n


def test_decode_of_the_whole_id_space(bpe):
    merges = answers.merge_list(65280, 9, longest=15)
    text = answers.strings(merges)
    ids = np.random.RandomState(1).permutation(65536).astype(np.int32)
    with bpe.Decoder(merges) as d:
        assert d.info()[0] == 65536
        want = b"".join(text[i] for i in ids.tolist())
        assert d.decode(torch.from_numpy(ids).cuda()).cpu().numpy().tobytes() == want
        # more text than was made room for at first
        many = torch.full((5000,), int(np.argmax([len(t) for t in text])), dtype=torch.int32, device="cuda")
        assert d.decode(many).cpu().numpy().tobytes() == max(text, key=len) * 5000


def test_decode_from_several_threads(bpe, vocabulary):
    """Texts of different lengths through one decoder, by one pass and by two."""
    merges, text = vocabulary
    failed = []
    with bpe.Decoder(merges) as d:
        def work(seed):
            try:
                with torch.cuda.stream(torch.cuda.Stream()):
                    r = np.random.RandomState(seed)
                    for n in (5, 3000, 60, 20000, 1, 2500) * 4:
                        ids = r.randint(0, len(text), n).astype(np.int32)
                        got, places = d.decode(torch.from_numpy(ids).cuda(), offsets=True)
                        assert got.cpu().numpy().tobytes() == b"".join(text[i] for i in ids.tolist())
                        assert int(places[-1]) == got.numel()
            except Exception as e:
                failed.append(e)
        threads = [threading.Thread(target=work, args=(seed,)) for seed in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not failed, failed


def test_decode_gives_encoded_text_back(bpe):
    import corpus
    data = corpus.generate(corpus.CONFIGS[2].scaled(200_001, seed=11))
    d = torch.from_numpy(data.copy()).cuda()
    merges, tokens = bpe.train(d, 500)
    with bpe.Decoder(merges) as dec, bpe.Encoder(merges) as enc, bpe.Trie(merges) as trie:
        for t in (tokens, enc.encode(d), trie.encode(d)):
            assert torch.equal(dec.decode(t), d)


# ---------------------------------------------------------------- together

def _step(bpe, x, r, w, b, sb, u):
    q, s, h = bpe.norm_quant(x, w, residual=r)
    logits = bpe.matmul_scaled(q, s, b, sb, out_dtype=torch.float32)
    ids, logp = bpe.sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)
    return q, s, h, logits, ids, logp


def _inputs(seed, rows, d=512, v=3256):
    x, r, u = _randn(seed, rows, d).bfloat16(), _randn(seed + 1, rows, d).bfloat16(), torch.rand(rows, generator=torch.Generator().manual_seed(seed))
    return x.cuda(), r.cuda(), u.cuda()


@pytest.mark.parametrize("rows", [1, 20, 130])
def test_a_captured_step_replays(bpe, rows):
    w = (1 + 0.1 * _randn(1, 512)).bfloat16().cuda()
    b, sb = bpe.quant_weight((_randn(2, 3256, 512) * 0.2).cuda())
    x, r, u = _inputs(10, rows)
    _step(bpe, x, r, w, b, sb, u)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(bpe, x, r, w, b, sb, u)
    for seed in (20, 30, 40, 50):
        nx, nr, nu = _inputs(seed, rows)
        x.copy_(nx), r.copy_(nr), u.copy_(nu)
        graph.replay()
        torch.cuda.synchronize()
        want = _step(bpe, nx, nr, w, b, sb, nu)
        assert all(_same(a, c) for a, c in zip(out, want)), seed


def test_another_stream_and_its_order(bpe):
    w = torch.ones(512).bfloat16().cuda()
    b, sb = bpe.quant_weight((_randn(2, 3256, 512) * 0.2).cuda())
    x, r, u = _inputs(7, 64)
    want = _step(bpe, x, r, w, b, sb, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late = torch.zeros_like(x)
        for _ in range(20):
            late.add_(1.0)
        late.copy_(x)
        got = _step(bpe, late, r, w, b, sb, u)
        with bpe.Decoder(answers.merge_list(3000, 1)) as d:
            text = d.decode(got[4])
    side.synchronize()
    assert all(_same(a, c) for a, c in zip(got, want))
    words = answers.strings(answers.merge_list(3000, 1))
    assert text.cpu().numpy().tobytes() == b"".join(words[i] for i in want[4].tolist())


def test_the_example_generates_text(bpe):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "answer.py")
    spec = importlib.util.spec_from_file_location("example_answer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    ids, texts, merges = example.main(["--bytes", "200000", "--merges", "300", "--rows", "3", "--steps", "25"])
    words = answers.strings(merges.cpu().numpy())
    assert ids.shape == (3, 26) and texts == [b"".join(words[i] for i in row) for row in ids.tolist()]
