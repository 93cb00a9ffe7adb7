"""The tensor-core kernels of the 8-bit integer linear: the tile kernel's waits, widths and order of tiles, and the splits of
K, at shapes that reach each of them."""
import time

import pytest
import torch

import nvfp4_block_scaled_18_b200 as nv
from i8_cases import GROUPS, SPLITS, TILES

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
ERR_TIMEOUT = 6


def operands(M, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randint(-128, 128, (M, K), dtype=I8, device="cuda", generator=g)
    w = torch.randint(-128, 128, (N, K), dtype=I8, device="cuda", generator=g)
    sa, sw = (0.01 + torch.rand(n, device="cuda", generator=g) for n in (M, N))
    return a, sa, w, sw


@pytest.mark.parametrize("M,N,K", [(700, 9000, 256), (777, 11008, 4096), (5000, 6000, 256)])
def test_one_warp_that_gives_up_stops_no_other(M, N, K):
    """One output warp of each CTA gives up at its first of several tiles, the others go on: the launch ends, says so,
    and the next call is right."""
    a, sa, w, sw = operands(M, N, K)
    y, st = torch.empty(M, N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    nv.nvfp4_i8_gemm(a, sa, w, sw, y, dev_status=st)
    good = y.clone()
    torch.cuda.synchronize()
    assert st.item() == 0
    nv.nvfp4_test_wait_fault(20_000_000, 2)
    try:
        t0 = time.perf_counter()
        nv.nvfp4_i8_gemm(a, sa, w, sw, y, dev_status=st)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        nv.nvfp4_test_wait_fault(0, 0)
    assert st.item() == ERR_TIMEOUT and dt < 2.0, (st.item(), dt)
    st.zero_()
    nv.nvfp4_i8_gemm(a, sa, w, sw, y, dev_status=st)
    assert st.item() == 0 and torch.equal(y, good)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (4, 100, 64), (16, 300, 1024), (100, 300, 2048), (200, 512, 8192),
                                   (300, 500, 256), (1031, 4096, 2064)])
def test_without_a_bias_nothing_is_added(M, N, K, out):
    """A product of -0 stays -0 in every kernel: fl32(acc) = +0, times a negative channel scale."""
    a, sa, w, sw = operands(M, N, K)
    y = torch.empty(M, N, dtype=out, device="cuda")
    nv.nvfp4_i8_gemm(torch.zeros_like(a), sa, w, -sw, y)
    assert (y == 0).all() and torch.signbit(y).all()
    nv.nvfp4_i8_gemm(torch.zeros_like(a), sa, w, -sw, y, bias=torch.zeros(N, device="cuda"))
    assert (y == 0).all() and not torch.signbit(y).any()          # -0 + 0


def plain(a, sa, w, sw, bias):
    """float32 result before the rounding to the output type: sums in 64 bits over runs of K, exact."""
    acc = torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for k in range(0, a.shape[1], 8192):
        acc += a[:, k:k + 8192].double() @ w[:, k:k + 8192].double().T
    y = acc.float() * sa[:, None] * sw
    return y if bias is None else y + bias


def check(M, N, K, out, with_bias, pad):
    """Exact, and nothing written beside the output; rows of Y `pad` elements further apart than they are long."""
    a, sa, w, sw = operands(M, N, K, M + N + K)
    bias = torch.randn(N, device="cuda") if with_bias else None
    buf, st = torch.full((M + 1, N + pad), -77.0, dtype=out, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    nv.nvfp4_i8_gemm(a, sa, w, sw, buf[:M, :N], bias, dev_status=st)
    assert torch.equal(buf[:M, :N], plain(a, sa, w, sw, bias).to(out)) and st.item() == 0
    assert (buf[M:] == -77.0).all() and (buf[:, N:] == -77.0).all()


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K,bn,swap", TILES)
def test_every_width(M, N, K, bn, swap, out):
    check(M, N, K, out, M % 2 == 0, -N % 8 if M % 3 else 3)


@pytest.mark.parametrize("M,N,K,tok,group", GROUPS)
def test_groups_of_tokens(M, N, K, tok, group):
    check(M, N, K, BF, True, 0)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K,ks", SPLITS)
def test_split_of_k_for_many_tokens(M, N, K, ks, out):
    check(M, N, K, out, N % 2 == 0, M % 3)


@pytest.mark.parametrize("M", [13, 30, 50, 100])
@pytest.mark.parametrize("row_tiles", [3, 20, 40, 45, 47, 60, 80, 120, 160])
def test_split_of_k_for_few_tokens(M, row_tiles):
    """Every split for every padding of the tokens, and row tiles that leave none."""
    for K in (912, 3088, 9008):
        check(M, 128 * row_tiles - 5, K, BF if K == 3088 else F32, M % 4 == 0, 0)
