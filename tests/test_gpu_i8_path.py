"""The layer norm and the 8-bit linear as they are used together: chains, streams, captured graphs, long strides,
timeouts, and beside the 4-bit path."""
import time

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_18_b200 as nv
from gpu_util import rel_fro, run_quantize
from i8_ref import i8_gemm, i8_quantize, layernorm, layernorm_backward

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


class Block:
    """norm -> 8-bit linear with a bias -> 8-bit linear, weights quantized by the same row quantizer."""

    def __init__(self, K, N, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.gamma, self.beta = (1 + 0.1 * torch.randn(K, generator=g)).cuda(), (0.1 * torch.randn(K, generator=g)).cuda()
        self.bias = torch.randn(N, generator=g).cuda()
        self.w = []
        for n, k in ((N, K), (K, N)):
            w = (0.05 * torch.randn(n, k, generator=g)).cuda()
            c, s = torch.empty(n, k, dtype=I8, device="cuda"), torch.empty(n, device="cuda")
            nv.nvfp4_i8_quantize(w, c, s)
            self.w.append((c, s))
        self.K, self.N = K, N

    def buffers(self, M):
        e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        return dict(c0=e(M, self.K, dtype=I8), s0=e(M), h=e(M, self.N, dtype=BF), c1=e(M, self.N, dtype=I8), s1=e(M), y=e(M, self.K))

    def run(self, x, b, stream=None):
        nv.nvfp4_layernorm_i8_quantize(x, b["c0"], b["s0"], self.gamma, self.beta, stream=stream)
        nv.nvfp4_i8_gemm(b["c0"], b["s0"], *self.w[0], b["h"], bias=self.bias, stream=stream)
        nv.nvfp4_i8_quantize(b["h"], b["c1"], b["s1"], stream=stream)
        nv.nvfp4_i8_gemm(b["c1"], b["s1"], *self.w[1], b["y"], stream=stream)
        return b["y"]

    def want(self, x):
        n = lambda t: t.float().cpu().numpy()  # noqa: E731
        y, _, _ = layernorm(n(x), n(self.gamma), n(self.beta))
        c, s = i8_quantize(y)
        w = [(c_.cpu().numpy(), n(s_)) for c_, s_ in self.w]
        h = torch.from_numpy(i8_gemm(c, s, *w[0], n(self.bias))).to(BF).float().numpy()
        c, s = i8_quantize(h)
        return torch.from_numpy(i8_gemm(c, s, *w[1]))


def rows(M, K, seed=0, dtype=BF):
    return torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("M", [1, 3, 4, 5, 16, 33, 64, 100, 128, 129, 250, 520])
def test_chain(M):
    """Every kernel of the product in its place in a chain; back to back calls whose operands the call before wrote."""
    blk = Block(1024, 2560)
    b = blk.buffers(M)
    xs = [rows(M, 1024, s, BF if M % 2 else F32) for s in range(4)]
    got = [blk.run(x, b).clone() for x in xs for _ in range(3)]
    for i, x in enumerate(xs):
        want = blk.want(x)
        for j in range(3):
            assert torch.equal(got[3 * i + j].cpu(), want)


@pytest.mark.parametrize("M", [1, 4, 16, 64, 300])
def test_chain_in_a_graph(M):
    """Captured once, replayed on new inputs; two graphs over the same buffers, replayed in turn."""
    blk = Block(512, 1024, 1)
    b, x = blk.buffers(M), rows(M, 512, 0)
    blk.run(x, b)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            blk.run(x, b)
        graphs.append(g)
    for s in range(1, 5):
        fresh = rows(M, 512, s)
        x.copy_(fresh)
        graphs[s % 2].replay()
        assert torch.equal(b["y"].cpu(), blk.want(fresh))


def test_two_streams_at_once():
    """Independent calls overlap on two streams: each has its own buffers, none shares state."""
    blk = Block(1024, 1536, 2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sizes = (70, 300)
    bufs, xs = [blk.buffers(m) for m in sizes], [rows(m, 1024, m) for m in sizes]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, b, x in zip(streams, bufs, xs):
            blk.run(x, b, stream=s)                       # explicit
    with torch.cuda.stream(streams[0]):
        blk.run(xs[0], bufs[0])                            # the current one
    torch.cuda.synchronize()
    for b, x in zip(bufs, xs):
        assert torch.equal(b["y"].cpu(), blk.want(x))


def test_training_step_and_graph():
    """Forward and backward through the norm; the backward pass captured into a graph that shares its workspace with
    an eager call and with a second graph."""
    M, K = 260, 768
    x, dy = rows(M, K, 3, F32), rows(M, K, 4, F32)
    gamma, beta = torch.rand(K, device="cuda") + 0.5, torch.randn(K, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    ws = nv.LayerNormWorkspace(M, K)
    out = [torch.empty_like(x), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")]

    def step():
        nv.nvfp4_layernorm(x, y, gamma, beta, mean=mean, rstd=rstd)
        nv.nvfp4_layernorm_backward(dy, x, mean, rstd, out[0], gamma, out[1], out[2], ws)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in out]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for g in (graphs[0], None, graphs[1], graphs[0]):
        for t in out:
            t.fill_(float("nan"))
        step() if g is None else g.replay()
        for a, b in zip(out, first):
            assert torch.equal(a, b)
    (rx, rg, rb), (mx, mg, mb) = layernorm_backward(dy.cpu().numpy(), x.cpu().numpy(), mean.cpu().numpy(), rstd.cpu().numpy(),
                                                    gamma.cpu().numpy())
    for got, ref, mag, deep in zip(out, (rx, rg, rb), (mx, mg, mb), (128, M + 6, M + 6)):
        assert (np.abs(got.double().cpu().numpy() - ref) <= deep * 2.0 ** -24 * (mag + np.abs(ref))).all()


def test_beside_the_four_bit_path():
    """The layer norm feeds the NVFP4 linear, and the 8-bit linear computes the same layer closer to fp64."""
    M, K, N = 64, 1024, 512
    x = rows(M, K, 5, F32) * 3 + 1
    gamma, beta = torch.rand(K, device="cuda") + 0.5, torch.randn(K, device="cuda")
    w = 0.05 * torch.randn(N, K, device="cuda")
    y = torch.empty_like(x)
    nv.nvfp4_layernorm(x, y, gamma, beta)
    q4, w4 = run_quantize(y, nv.SF_TILED), run_quantize(w, nv.SF_TILED)
    o4, o8 = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    nv.nvfp4_gemm(q4, w4, o4)
    c, s = torch.empty(M, K, dtype=I8, device="cuda"), torch.empty(M, device="cuda")
    wc, wsc = torch.empty(N, K, dtype=I8, device="cuda"), torch.empty(N, device="cuda")
    nv.nvfp4_layernorm_i8_quantize(x, c, s, gamma, beta)
    nv.nvfp4_i8_quantize(w, wc, wsc)
    nv.nvfp4_i8_gemm(c, s, wc, wsc, o8)
    # the fused call is the two calls on an fp32 norm
    c2, s2 = torch.empty_like(c), torch.empty_like(s)
    nv.nvfp4_i8_quantize(y, c2, s2)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    ref = y.double().cpu().numpy() @ w.double().cpu().numpy().T
    # each operand is off by at most half a step of 1/127 of its row's largest value: with normal rows (largest about
    # 4 sigma) 4 / 254 / sqrt(3) = 0.9% a factor, 1.3% both; 4-bit values are off by up to a quarter of themselves
    assert rel_fro(o8.cpu().numpy(), ref) < 0.02 < rel_fro(o4.cpu().numpy(), ref) < 0.3


def test_offsets_beyond_32_bits():
    """Rows that start 2^31 elements and more into their buffers."""
    ld = 1 << 30
    M, K, N = 3, 64, 40
    buf = torch.empty(2 * ld + K, dtype=BF, device="cuda")
    x = buf.as_strided((M, K), (ld, 1))
    x.copy_(rows(M, K, 1))
    cbuf = torch.empty(2 * ld + K, dtype=I8, device="cuda")
    c, s = cbuf.as_strided((M, K), (ld, 1)), torch.empty(M, device="cuda")
    nv.nvfp4_i8_quantize(x, c, s)
    rc, rs = i8_quantize(x.float().cpu().numpy())
    np.testing.assert_array_equal(c.cpu().numpy(), rc)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    ybuf = torch.empty(2 * ld + K, dtype=BF, device="cuda")
    y, mean, rstd = ybuf.as_strided((M, K), (ld, 1)), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    nv.nvfp4_layernorm(x, y, mean=mean, rstd=rstd)
    ry, _, _ = layernorm(x.float().cpu().numpy())
    assert torch.equal(y.cpu(), torch.from_numpy(ry).to(BF))
    dx, dg = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(K, device="cuda")
    nv.nvfp4_layernorm_backward(y, x, mean, rstd, dx, None, dg, None, nv.LayerNormWorkspace(M, K))
    d2, g2 = torch.empty_like(dx), torch.empty_like(dg)
    nv.nvfp4_layernorm_backward(y.contiguous(), x.contiguous(), mean, rstd, d2, None, g2, None, nv.LayerNormWorkspace(M, K))
    assert torch.equal(dx, d2) and torch.equal(dg, g2)
    w = torch.randint(-127, 128, (N, K), dtype=I8, device="cuda")
    ws = torch.rand(N, device="cuda")
    for out_rows in (3, 5, 130):                            # each kernel of the product, its operand and output far apart
        a = c if out_rows == 3 else torch.randint(-127, 128, (out_rows, K), dtype=I8, device="cuda")
        sa = s if out_rows == 3 else torch.rand(out_rows, device="cuda")
        far = (2 * ld) // (out_rows - 1) // 16 * 16 + 16
        o = torch.empty(far * (out_rows - 1) + N, dtype=BF, device="cuda").as_strided((out_rows, N), (far, 1))
        nv.nvfp4_i8_gemm(a, sa, w, ws, o)
        want = i8_gemm(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy())
        assert torch.equal(o.cpu(), torch.from_numpy(want).to(BF))


def test_many_rows():
    """More rows than one wave holds, and than 16 bits count."""
    M, K = 70001, 32
    x = rows(M, K, 9)
    c, s = torch.empty(M, K, dtype=I8, device="cuda"), torch.empty(M, device="cuda")
    nv.nvfp4_i8_quantize(x, c, s)
    rc, rs = i8_quantize(x.float().cpu().numpy())
    np.testing.assert_array_equal(c.cpu().numpy(), rc)
    w, ws = torch.randint(-127, 128, (48, K), dtype=I8, device="cuda"), torch.rand(48, device="cuda")
    y = torch.empty(M, 48, device="cuda")
    nv.nvfp4_i8_gemm(c, s, w, ws, y)
    np.testing.assert_array_equal(y.cpu().numpy(), i8_gemm(rc, rs, w.cpu().numpy(), ws.cpu().numpy()))
    yt = torch.empty(48, M, dtype=BF, device="cuda")          # the same with many output channels
    nv.nvfp4_i8_gemm(w, ws, c, s, yt)
    assert torch.equal(yt.cpu(), torch.from_numpy(i8_gemm(w.cpu().numpy(), ws.cpu().numpy(), rc, rs)).to(BF))
    one = torch.empty(1, M, device="cuda")
    nv.nvfp4_i8_gemm(w[:1], ws[:1], c, s, one)
    np.testing.assert_array_equal(one.cpu().numpy(), i8_gemm(w[:1].cpu().numpy(), ws[:1].cpu().numpy(), rc, rs))


@pytest.mark.parametrize("M,N,K", [(16, 256, 2048), (64, 640, 4096), (128, 256, 4096), (200, 512, 8192), (300, 700, 1024)])
def test_timeout_is_reported_and_recovered_from(M, N, K):
    """With its loads withheld a call gives up after the limit, reports it, and leaves the context usable."""
    rng = np.random.default_rng(0)
    a, w = (torch.from_numpy(rng.integers(-127, 128, s, dtype=np.int8)).cuda() for s in ((M, K), (N, K)))
    sa, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    y, st = torch.empty(M, N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    nv.nvfp4_i8_gemm(a, sa, w, sw, y, dev_status=st)
    good = y.clone()
    torch.cuda.synchronize()
    nv.nvfp4_test_wait_fault(20_000_000, True)
    try:
        t0 = time.perf_counter()
        nv.nvfp4_i8_gemm(a, sa, w, sw, y, dev_status=st)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        nv.nvfp4_test_wait_fault(0, False)
    assert st.item() == 6 and dt < 2.0, (st.item(), dt)
    st.zero_()
    nv.nvfp4_i8_gemm(a, sa, w, sw, y, dev_status=st)
    assert st.item() == 0 and torch.equal(y, good)
