"""Refusals of the layer norm and 8-bit linear entry points: on the host, before any CUDA call."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_18_b200 as nv

OK16, EPS = 1 << 20, ctypes.c_float(1e-5)      # a fake, never dereferenced, aligned device address
INVALID, ALIGNMENT, UNSUPPORTED, WORKSPACE = 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_18_b200 import build
    build.build()
    return nv.load_library()


def test_i8_quantize_refusals(lib):
    def call(x=OK16, dt=1, M=4, K=64, ldx=64, codes=OK16, ldc=64, scales=OK16):
        return lib.nvfp4_i8_quantize(x, dt, M, K, ldx, codes, ldc, scales, None, None)

    for bad in (dict(x=None), dict(dt=2), dict(M=0), dict(M=-1), dict(K=0), dict(K=72), dict(ldx=48), dict(codes=None),
                dict(scales=None), dict(ldc=48)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=OK16 + 8), dict(ldx=68), dict(codes=OK16 + 8), dict(ldc=72), dict(scales=OK16 + 2)):
        assert call(**bad) == ALIGNMENT, bad
    K = nv.NVFP4_I8_MAX_K + 16
    assert call(K=K, ldx=K, ldc=K) == UNSUPPORTED


def test_layernorm_refusals(lib):
    def call(x=OK16, dt=1, M=4, K=64, ldx=64, gamma=OK16, beta=OK16, pdt=0, eps=1e-5, y=OK16, ldy=64, mean=OK16, rstd=OK16):
        return lib.nvfp4_layernorm(x, dt, M, K, ldx, gamma, beta, pdt, ctypes.c_float(eps), y, ldy, mean, rstd, None, None)

    for bad in (dict(x=None), dict(y=None), dict(dt=5), dict(pdt=5), dict(M=0), dict(K=40), dict(ldy=32),
                dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(gamma=OK16 + 4), dict(beta=OK16 + 4), dict(y=OK16 + 2), dict(ldy=68), dict(mean=OK16 + 1), dict(rstd=OK16 + 2)):
        assert call(**bad) == ALIGNMENT, bad
    K = nv.NVFP4_I8_MAX_K + 16
    assert call(K=K, ldx=K, ldy=K) == UNSUPPORTED

    def quant(gamma=OK16, pdt=1, eps=0.0, codes=OK16, ldc=64, scales=OK16):
        return lib.nvfp4_layernorm_i8_quantize(OK16, 1, 4, 64, 64, gamma, None, pdt, ctypes.c_float(eps), codes, ldc, scales,
                                               None, None)

    assert quant(codes=None) == INVALID and quant(scales=None) == INVALID and quant(eps=-1e-9) == INVALID
    assert quant(ldc=16) == INVALID and quant(pdt=9) == INVALID
    assert quant(ldc=65) == ALIGNMENT and quant(gamma=OK16 + 8) == ALIGNMENT


def test_layernorm_backward_refusals(lib):
    need = nv.nvfp4_layernorm_workspace_size(4, 64)
    assert need > 0 and need % 4 == 0 and nv.nvfp4_layernorm_workspace_size(0, 64) == 0
    assert nv.nvfp4_layernorm_workspace_size(1 << 20, 4096) == nv.nvfp4_layernorm_workspace_size(1 << 21, 4096)

    def call(dy=OK16, lddy=64, x=OK16, M=4, gamma=OK16, pdt=1, mean=OK16, rstd=OK16, dx=OK16, lddx=64, dg=OK16, db=OK16,
             ws=OK16, ws_n=need):
        return lib.nvfp4_layernorm_backward(dy, lddy, x, 64, 1, M, 64, gamma, pdt, mean, rstd, dx, lddx, dg, db, ws, ws_n, None)

    for bad in (dict(dy=None), dict(x=None), dict(M=0), dict(pdt=3), dict(mean=None), dict(rstd=None), dict(lddy=32),
                dict(lddx=32), dict(dx=None, dg=None, db=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dy=OK16 + 2), dict(dx=OK16 + 2), dict(lddx=68), dict(dg=OK16 + 2), dict(db=OK16 + 1),
                dict(mean=OK16 + 1), dict(ws=OK16 + 8), dict(gamma=OK16 + 2)):
        assert call(**bad) == ALIGNMENT, bad
    for bad in (dict(ws=None), dict(ws_n=need - 1)):
        assert call(**bad) == WORKSPACE, bad


def test_i8_gemm_refusals(lib):
    def call(a=OK16, lda=64, sa=OK16, w=OK16, ldw=64, sw=OK16, bias=OK16, M=4, N=32, K=64, y=OK16, dt=0, ldy=32):
        return lib.nvfp4_i8_gemm(a, lda, sa, w, ldw, sw, bias, M, N, K, y, dt, ldy, None, None)

    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(dt=4), dict(M=0), dict(N=0),
                dict(K=0), dict(K=56), dict(lda=48), dict(ldw=48), dict(ldy=31)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(a=OK16 + 8), dict(w=OK16 + 8), dict(lda=72), dict(ldw=72), dict(y=OK16 + 2), dict(y=OK16 + 1, dt=1),
                dict(sa=OK16 + 2), dict(sw=OK16 + 2), dict(bias=OK16 + 2)):
        assert call(**bad) == ALIGNMENT, bad
    K = nv.NVFP4_I8_MAX_K + 16
    assert call(K=K, lda=K, ldw=K) == UNSUPPORTED
    assert call(M=2 ** 31) == UNSUPPORTED and call(N=2 ** 31 - 1, ldy=2 ** 31) == UNSUPPORTED
    assert call(lda=1 << 40) == UNSUPPORTED


def test_binding_refusals(lib):
    """Shapes, dtypes and devices, before the library is called."""
    x, c, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    v = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_i8_quantize(x, c, s)
    with pytest.raises(ValueError, match="codes"):
        nv.nvfp4_i8_quantize(x, c.float(), s)
    with pytest.raises(ValueError, match="codes"):
        nv.nvfp4_i8_quantize(x, c[:3], s)
    with pytest.raises(ValueError, match="scales"):
        nv.nvfp4_i8_quantize(x, c, s[:3])
    with pytest.raises(ValueError, match="row-major"):
        nv.nvfp4_i8_quantize(torch.zeros(64, 4).T, c, s)
    with pytest.raises(ValueError, match="y must"):
        nv.nvfp4_layernorm(x, x.bfloat16(), v, v)
    with pytest.raises(ValueError, match="beta"):
        nv.nvfp4_layernorm(x, x, v, v.bfloat16())
    with pytest.raises(ValueError, match="gamma"):
        nv.nvfp4_layernorm_i8_quantize(x, c, s, v[:32])
    with pytest.raises(ValueError, match="mean"):
        nv.nvfp4_layernorm_backward(x, x, s[:2], s, x)
    with pytest.raises(ValueError, match="dgamma"):
        nv.nvfp4_layernorm_backward(x, x, s, s, x, v, v.double())
    with pytest.raises(ValueError, match="w_codes"):
        nv.nvfp4_i8_gemm(c, s, torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="y must"):
        nv.nvfp4_i8_gemm(c, s, c, s, torch.zeros(4, 5))
    with pytest.raises(ValueError, match="bias"):
        nv.nvfp4_i8_gemm(c, s, c, s, torch.zeros(4, 4), bias=torch.zeros(3))
    with pytest.raises(TypeError):
        nv.nvfp4_i8_gemm(c, s, c, s, torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(TypeError):
        nv.nvfp4_layernorm(x.half(), x.half())
