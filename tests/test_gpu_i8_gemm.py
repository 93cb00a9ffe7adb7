"""The 8-bit integer linear: exact int32 sums, so its output is the plain form's, bit for bit."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_18_b200 as nv
from i8_ref import i8_gemm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def codes(rng, rows, cols, gap=0):
    c = rng.integers(-128, 128, (rows, cols), dtype=np.int8)
    buf = torch.full((rows, cols + gap), 99, dtype=torch.int8, device="cuda")
    buf[:, :cols] = torch.from_numpy(c).cuda()
    return c, buf[:, :cols]


def case(M, N, K, out, bias=True, gap=0, seed=0, ygap=0):
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    a, at = codes(rng, M, K, gap)
    w, wt = codes(rng, N, K, gap)
    sa, sw = (rng.uniform(0.001, 0.1, n).astype(np.float32) for n in (M, N))
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    y = torch.full((M + 1, N + ygap), -77.0, dtype=out, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    nv.nvfp4_i8_gemm(at, torch.from_numpy(sa).cuda(), wt, torch.from_numpy(sw).cuda(), y[:M, :N],
                     None if b is None else torch.from_numpy(b).cuda(), dev_status=st)
    want = torch.from_numpy(i8_gemm(a, sa, w, sw, b)).to(out)
    assert st.item() == 0
    got = y.cpu()
    assert torch.equal(got[:M, :N], want)
    assert (got[M:] == -77.0).all() and (got[:, N:] == -77.0).all()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 61, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 48), (64, 128), (100, 144), (256, 1024), (257, 272), (300, 4096)])
def test_i8_gemm(M, N, K):
    out = BF if (M + N) % 2 else F32
    case(M, N, K, out, bias=M % 3 != 0, gap=16 * (M % 2), ygap=(0, 1, 16)[M % 3])


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 1000, 14336), (16, 5120, 1040), (61, 640, 27648),
                                   (128, 11008, 512), (777, 1500, 4096), (2048, 2100, 528), (1031, 4096, 2064)])
def test_i8_gemm_larger(M, N, K, out):
    case(M, N, K, out)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_i8_gemm_extreme_sums(M):
    """All codes -128 (and 127) at the longest K: sums next to the ends of int32."""
    K, N = nv.NVFP4_I8_MAX_K, 40
    at = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wt = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wt[1::2] = 127
    y = torch.empty(M, N, device="cuda")
    nv.nvfp4_i8_gemm(at, torch.ones(M, device="cuda"), wt, torch.ones(N, device="cuda"), y)
    want = np.where(np.arange(N) % 2 == 0, np.float32(K * 16384), np.float32(-K * 16256))
    np.testing.assert_array_equal(y.cpu().numpy(), np.broadcast_to(want, (M, N)))


def test_i8_gemm_one_hot():
    """Row m of A picks column k(m) of W: every operand element at its place."""
    M, N, K = 300, 500, 656
    rng = np.random.default_rng(1)
    pick = rng.integers(0, K, M)
    a = np.zeros((M, K), np.int8)
    a[np.arange(M), pick] = 1
    w, wt = codes(rng, N, K)
    for m in (1, 16, 100, 300):
        y = torch.empty(m, N, device="cuda")
        nv.nvfp4_i8_gemm(torch.from_numpy(a[:m]).cuda(), torch.ones(m, device="cuda"), wt, torch.ones(N, device="cuda"), y)
        np.testing.assert_array_equal(y.cpu().numpy(), w[:, pick[:m]].T.astype(np.float32))


def test_i8_gemm_nan_scale_stays_in_its_row():
    a = torch.ones(20, 64, dtype=torch.int8, device="cuda")
    w = torch.ones(33, 64, dtype=torch.int8, device="cuda")
    sa = torch.ones(20, device="cuda")
    sa[3] = float("nan")
    y = torch.empty(20, 33, device="cuda")
    nv.nvfp4_i8_gemm(a, sa, w, torch.ones(33, device="cuda"), y)
    assert torch.isnan(y[3]).all() and (y[torch.arange(20) != 3] == 64).all()
