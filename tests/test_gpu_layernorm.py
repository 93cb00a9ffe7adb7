"""Layer norm (forward, backward, and into 8 bits) and the 8-bit row quantizer against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_18_b200 as nv
from i8_ref import HALF, i8_quantize, layernorm, layernorm_backward

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD8, GUARD = 85, -77.0


def guarded(rows, cols, dtype, gap, fill=GUARD):
    """A rows x cols matrix inside a buffer with `gap` extra columns and one extra row, and the buffer."""
    buf = torch.full((rows + 1, cols + gap), fill, dtype=dtype, device="cuda")
    return buf[:rows, :cols], buf


def untouched(buf, rows, cols, fill=GUARD):
    b = buf.float()
    return bool((b[rows:] == fill).all() and (b[:, cols:] == fill).all())


def inputs(rows, cols, dtype, seed=0, gap=0, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x[:, ::37] *= 30.0
    x += shift * torch.randn(cols, generator=g)
    if rows > 2:
        x[1] = 0.0                      # an empty row
        x[2] = 3.25                     # a constant row
    t, _ = guarded(rows, cols, dtype, gap)
    t.copy_(x.to(dtype))
    return t, t.float().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


SIZES = [(1, 16), (3, 48), (5, 256), (1, 4096), (149, 1008), (7, 8192), (33, 8208), (3, 14336), (2, 33040), (300, 5120),
         (1, 131056), (446, 5120), (460, 8192), (450, 10240), (445, 14352), (4100, 4096)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [0, 16])
def test_i8_quantize(rows, cols, dtype, gap):
    x, xn = inputs(rows, cols, dtype, rows + cols, gap)
    codes, buf = guarded(rows, cols, torch.int8, gap, GUARD8)
    scales, st = torch.empty(rows, device="cuda"), status()
    nv.nvfp4_i8_quantize(x, codes, scales, dev_status=st)
    rc, rs = i8_quantize(xn)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    assert st.item() == 0 and untouched(buf, rows, cols, GUARD8)


def test_i8_quantize_edges():
    """Ties, the largest and smallest magnitudes, and rows with NaN and infinities beside finite ones."""
    x = torch.zeros(9, 64)
    x[0, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])              # scale 1: ties to even
    x[1, 0] = 3.3e38
    x[2, 0] = 2.0 ** -110
    x[2, 1] = -(2.0 ** -111)
    x[3, 0] = 2.0 ** -111                                          # below the smallest amax: an empty row
    x[4, 5] = float("nan")
    x[5, 63] = float("inf")
    x[6, 0] = -float("inf")
    x[7, :] = -1.0
    x[8, 3] = 1e-40                                                # subnormal: an empty row
    for dtype in (F32, BF):
        t = x.to(dtype).cuda()
        codes, scales, st = torch.empty(9, 64, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda"), status()
        nv.nvfp4_i8_quantize(t, codes, scales, dev_status=st)
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        good = [0, 1, 2, 3, 7, 8]
        rc, rs = i8_quantize(t.float().cpu().numpy()[good])
        np.testing.assert_array_equal(c[good], rc)
        np.testing.assert_array_equal(s[good], rs)
        assert list(c[0, :4]) == [127, 0, 2, -2] and s[3] == 0 and s[8] == 0
        assert np.isnan(s[4:7]).all() and not c[4:7].any()
        assert st.item() == 5                                      # NVFP4_ERR_NONFINITE


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,pdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_layernorm(rows, cols, dtype, pdt):
    gap = 16 if rows % 2 else 0
    x, xn = inputs(rows, cols, dtype, rows + cols, gap)
    g = torch.Generator().manual_seed(cols)
    gamma = (1 + 0.2 * torch.randn(cols, generator=g)).to(pdt).cuda()
    beta = (0.1 * torch.randn(cols, generator=g)).to(pdt).cuda()
    y, buf = guarded(rows, cols, dtype, gap)
    mean, rstd, st = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), status()
    nv.nvfp4_layernorm(x, y, gamma, beta, mean=mean, rstd=rstd, dev_status=st)
    ry, rm, rr = layernorm(xn, gamma.float().cpu().numpy(), beta.float().cpu().numpy())
    # the sums agree to far below half a step of fp32, so each statistic is the reference's or its neighbour
    np.testing.assert_allclose(mean.cpu().numpy(), rm, rtol=2 * HALF, atol=0)
    np.testing.assert_allclose(rstd.cpu().numpy(), rr, rtol=2 * HALF, atol=0)
    # and, from the statistics returned, y is the same chain of fp32 steps
    want = (xn - mean.cpu().numpy()[:, None]) * rstd.cpu().numpy()[:, None] * gamma.float().cpu().numpy() + beta.float().cpu().numpy()
    assert want.dtype == np.float32
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(dtype))
    assert st.item() == 0 and untouched(buf, rows, cols)
    # into 8 bits: the quantizer on the fp32 result
    codes, cbuf = guarded(rows, cols, torch.int8, 16, GUARD8)
    scales = torch.empty(rows, device="cuda")
    nv.nvfp4_layernorm_i8_quantize(x, codes, scales, gamma, beta, dev_status=st)
    rc, rs = i8_quantize(want)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    assert st.item() == 0 and untouched(cbuf, rows, cols, GUARD8)


@pytest.mark.parametrize("with_gamma,with_beta", [(True, False), (False, True), (False, False)])
def test_layernorm_without_parameters(with_gamma, with_beta):
    x, xn = inputs(37, 1024, BF, 3)
    gamma = (torch.rand(1024) + 0.5).cuda() if with_gamma else None
    beta = torch.randn(1024).cuda() if with_beta else None
    y = torch.empty(37, 1024, dtype=BF, device="cuda")
    nv.nvfp4_layernorm(x, y, gamma, beta, eps=1e-3)
    ry, _, _ = layernorm(xn, None if gamma is None else gamma.cpu().numpy(), None if beta is None else beta.cpu().numpy(), 1e-3)
    assert torch.equal(y.cpu(), torch.from_numpy(ry).to(BF))


@pytest.mark.parametrize("rows", [65, 700])
def test_layernorm_in_place(rows):
    x, xn = inputs(rows, 8192, F32, 5)
    ry, _, _ = layernorm(xn)
    nv.nvfp4_layernorm(x, x)
    assert torch.equal(x.cpu(), torch.from_numpy(ry))


@pytest.mark.parametrize("shift", [100.0, 3000.0])
def test_layernorm_far_from_zero(shift):
    """Rows whose mean is far larger than their spread: the fp32 chain from mean and rstd, and the statistics in 64 bits."""
    g = torch.Generator().manual_seed(11)
    x = (torch.randn(40, 2048, generator=g) + shift).cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    nv.nvfp4_layernorm(x, y, mean=mean, rstd=rstd)
    ry, rm, rr = layernorm(x.cpu().numpy())
    np.testing.assert_array_equal(mean.cpu().numpy(), rm)
    np.testing.assert_array_equal(rstd.cpu().numpy(), rr)
    np.testing.assert_array_equal(y.cpu().numpy(), ry)


@pytest.mark.parametrize("scale,eps", [(1e20, 1e-5), (1e-20, 0.0), (1e-20, 1e-38), (1e15, 0.0)])
@pytest.mark.parametrize("rows,cols", [(7, 512), (500, 4096)])
def test_layernorm_far_scales(rows, cols, scale, eps):
    """Variances far outside the range of usual ones: the same statistics and results."""
    x = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(7)) * scale).cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    nv.nvfp4_layernorm(x, y, eps=eps, mean=mean, rstd=rstd)
    ry, rm, rr = layernorm(x.cpu().numpy(), eps=eps)
    np.testing.assert_array_equal(mean.cpu().numpy(), rm)
    np.testing.assert_array_equal(rstd.cpu().numpy(), rr)
    np.testing.assert_array_equal(y.cpu().numpy(), ry)


def test_layernorm_nonfinite_rows():
    x = torch.randn(6, 512, device="cuda")
    x[1, 7], x[3, 0], x[4, 511] = float("nan"), float("inf"), -float("inf")
    y, st = torch.empty_like(x), status()
    nv.nvfp4_layernorm(x, y, dev_status=st)
    ry, _, _ = layernorm(x.cpu().numpy()[[0, 2, 5]])
    assert torch.isnan(y[[1, 3, 4]]).all() and st.item() == 5
    np.testing.assert_array_equal(y.cpu().numpy()[[0, 2, 5]], ry)
    codes, scales, st = torch.empty(6, 512, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda"), status()
    nv.nvfp4_layernorm_i8_quantize(x, codes, scales, dev_status=st)
    rc, rs = i8_quantize(ry)
    assert st.item() == 5 and torch.isnan(scales[[1, 3, 4]]).all() and not codes[[1, 3, 4]].any()
    np.testing.assert_array_equal(codes.cpu().numpy()[[0, 2, 5]], rc)
    # a constant row with eps = 0 has no norm
    st = status()
    nv.nvfp4_layernorm(torch.ones(2, 64, device="cuda"), y[:2, :64], eps=0.0, dev_status=st)
    assert st.item() == 5 and torch.isnan(y[:2, :64]).all()


BWD = [(1, 16), (2, 48), (5, 256), (333, 1024), (149, 8208), (700, 4096), (4, 14336), (2, 33040), (1000, 80), (3, 8192),
       (2100, 272), (2500, 1024), (1300, 8192), (600, 10256), (2049, 64), (500, 16384)]


@pytest.mark.parametrize("rows,cols", BWD)
@pytest.mark.parametrize("dtype,pdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_layernorm_backward(rows, cols, dtype, pdt):
    gap = 16 if rows % 2 else 0
    x, xn = inputs(rows, cols, dtype, rows + cols, gap)
    g = torch.Generator().manual_seed(cols)
    dy, _ = guarded(rows, cols, dtype, gap)
    dy.copy_(torch.randn(rows, cols, generator=g).to(dtype))
    gamma = (1 + 0.2 * torch.randn(cols, generator=g)).to(pdt).cuda()
    _, mean, rstd = layernorm(xn)
    m, r = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    (rx, rg, rb), (mx, mg, mb) = layernorm_backward(dy.float().cpu().numpy(), xn, mean, rstd, gamma.float().cpu().numpy())
    ws = nv.LayerNormWorkspace(rows, cols)
    outs = []
    for _ in range(2):
        dx, buf = guarded(rows, cols, dtype, gap)
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        ws.buf.fill_(255)                                   # no initialisation needed (all bytes 255 read as NaN)
        nv.nvfp4_layernorm_backward(dy, x, m, r, dx, gamma, dg, db, ws)
        assert untouched(buf, rows, cols)
        outs.append((dx, dg, db))
    for a, b in zip(*outs):
        assert torch.equal(a, b)                            # a fixed order of summation
    # fp32 sums: a term passes through at most `deep` additions, each off by half a step of what it has summed; 6 more
    # for the products and differences around them.  Row sums: K / 16 serial terms of a thread at the very most.
    deep_row, deep_col = min(cols, 64 + cols // 256) + 16, rows + 6
    eps_out = HALF if dtype == F32 else 2.0 ** -8
    assert (np.abs(dx.double().cpu().numpy() - rx) <= deep_row * HALF * mx + eps_out * (np.abs(rx) + deep_row * HALF * mx) + 1e-38).all()
    assert (np.abs(dg.double().cpu().numpy() - rg) <= deep_col * HALF * mg + 1e-38).all()
    assert (np.abs(db.double().cpu().numpy() - rb) <= deep_col * HALF * mb + 1e-38).all()


@pytest.mark.parametrize("rows", [300, 2300])
def test_layernorm_backward_parts(rows):
    """Any of the three gradients alone is the one of the full call; without a gain it is one."""
    x, xn = inputs(rows, 512, F32, 2)
    dy = torch.randn(rows, 512, device="cuda")
    _, mean, rstd = layernorm(xn)
    m, r = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    ws = nv.LayerNormWorkspace(rows, 512)

    def grads(gamma, want):
        t = [torch.empty(rows, 512, device="cuda"), torch.empty(512, device="cuda"), torch.empty(512, device="cuda")]
        a = [v if w else None for v, w in zip(t, want)]
        nv.nvfp4_layernorm_backward(dy, x, m, r, a[0], gamma, a[1], a[2], ws if want[1] or want[2] else None)
        return a

    gamma = torch.rand(512, device="cuda") + 0.5
    full = grads(gamma, (1, 1, 1))
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)):
        for got, ref in zip(grads(gamma, want), full):
            assert got is None or torch.equal(got, ref)
    for got, ref in zip(grads(None, (1, 1, 1)), grads(torch.ones(512, device="cuda"), (1, 1, 1))):
        assert torch.equal(got, ref)


def test_layernorm_gradient_is_the_slope():
    """Central differences of the 64-bit layer norm along random directions, against dx, dgamma and dbeta."""
    rng = np.random.default_rng(4)
    M, K, eps = 6, 96, 1e-5
    x = rng.standard_normal((M, K)).astype(np.float32)
    gamma, beta = (1 + 0.3 * rng.standard_normal(K)).astype(np.float32), rng.standard_normal(K).astype(np.float32)
    dy = rng.standard_normal((M, K)).astype(np.float32)

    def loss(x, gamma, beta):
        mean = x.mean(1, keepdims=True)
        var = ((x - mean) ** 2).mean(1, keepdims=True)
        return float((dy * ((x - mean) / np.sqrt(var + eps) * gamma + beta)).sum())

    t = [torch.from_numpy(v).cuda() for v in (x, gamma, beta, dy)]
    y, mean, rstd = torch.empty(M, K, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    nv.nvfp4_layernorm(t[0], y, t[1], t[2], eps=eps, mean=mean, rstd=rstd)
    dx, dg, db = torch.empty(M, K, device="cuda"), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    nv.nvfp4_layernorm_backward(t[3], t[0], mean, rstd, dx, t[1], dg, db, nv.LayerNormWorkspace(M, K))
    point = [v.astype(np.float64) for v in (x, gamma, beta)]
    for i, grad in enumerate((dx, dg, db)):
        for _ in range(3):
            way = rng.standard_normal(point[i].shape)
            h = 1e-5
            up, down = list(point), list(point)
            up[i], down[i] = point[i] + h * way, point[i] - h * way
            slope = (loss(*up) - loss(*down)) / (2 * h)
            got = float((grad.double().cpu().numpy() * way).sum())
            # differences: h^2 times the third derivative (order 10 per element of the sum) and 2^-53 |loss| / h;
            # gradients: 64 half steps of fp32 of the summed magnitudes
            scale = float(np.abs(grad.double().cpu().numpy() * way).sum()) + float(np.abs(dy).sum())
            assert abs(slope - got) <= scale * (64 * HALF + 100 * h * h + 2.0 ** -50 / h)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(3, 64), (500, 16384)])
def test_layernorm_differences_beyond_fp32(rows, cols, dtype):
    """A finite row whose largest difference from its mean overflows fp32 has no norm, and that is reported."""
    x = torch.randn(rows, cols, device="cuda").to(dtype)
    x[1] = -3e38
    x[1, 5] = 3e38
    y, st = torch.empty_like(x), status()
    nv.nvfp4_layernorm(x, y, dev_status=st)
    assert st.item() == 5 and torch.isnan(y[1, 5])
    assert torch.isfinite(y[torch.arange(rows) != 1]).all()
    codes, scales, st = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda"), status()
    nv.nvfp4_layernorm_i8_quantize(x, codes, scales, dev_status=st)
    assert st.item() == 5 and torch.isnan(scales[1]) and not codes[1].any()
    assert torch.isfinite(scales[torch.arange(rows) != 1]).all()


@pytest.mark.parametrize("rows,cols", [(4100, 6672), (500, 9232), (4097, 5648)])
@pytest.mark.parametrize("dtype,pdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_layernorm_ragged_rows(rows, cols, dtype, pdt):
    """Long rows that leave lanes of their last warp idle, in every kernel that takes them."""
    test_layernorm(rows, cols, dtype, pdt)
