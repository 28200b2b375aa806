"""What the MXFP4 entry points refuse, checked on the host before anything touches a GPU."""
import ctypes

import pytest
import torch

NEW = {"wq_quantize_mxfp4", "wq_gemm_mxfp4_workspace_bytes", "wq_gemm_mxfp4", "wq_gemm_mxfp4_bf16",
       "wq_gemm_mxfp4_experts", "wq_gemm_mxfp4_experts_bf16"}


@pytest.fixture
def host():
    """A 16-byte aligned host address: what is not device memory."""
    buf = (ctypes.c_uint8 * 256)()
    return ctypes.c_void_p((ctypes.addressof(buf) + 15) // 16 * 16), buf


def test_exports(wq):
    assert NEW <= set(wq.header_functions())
    for n in NEW:
        assert hasattr(wq._lib, n)


def test_quantize_refusals(wq, host):
    p, lib = host[0], wq._lib
    assert lib.wq_quantize_mxfp4(p, 2, 4, 64, p, p, p, p, None) == wq.WQ_EINVAL and "dtype" in wq.last_error()
    for n, k in [(0, 32), (4, 0), (4, 16), (4, 48), (4, -32), (1 << 31, 32)]:
        assert lib.wq_quantize_mxfp4(p, 0, n, k, p, p, p, p, None) == wq.WQ_EINVAL, (n, k)
    assert lib.wq_quantize_mxfp4(None, 0, 4, 32, p, p, p, p, None) == wq.WQ_EINVAL
    assert lib.wq_quantize_mxfp4(ctypes.c_void_p(p.value + 2), 0, 4, 32, p, p, p, p, None) == wq.WQ_EALIGN
    assert lib.wq_quantize_mxfp4(p, 0, 4, 32, p, p, p, p, None) == wq.WQ_EINVAL      # host memory


def test_weight_descriptor(wq, host):
    p, lib = host[0], wq._lib
    d = wq.WqWeight(wq.FMT_MXFP4, 64, 4, 64, p.value, p.value)
    assert lib.wq_dequant(ctypes.byref(d), p, None) == wq.WQ_EUNSUPPORTED and "32" in wq.last_error()
    d = wq.WqWeight(wq.FMT_MXFP4, 32, 4, 48, p.value, p.value)
    assert lib.wq_gemv_w4a16(ctypes.byref(d), p, 1, p, None) == wq.WQ_EINVAL


def test_product_refusals(wq, host):
    p, lib, by = host[0], wq._lib, ctypes.byref
    good = wq.WqWeight(wq.FMT_MXFP4, 32, 4, 64, p.value, p.value)
    dyadic = wq.WqWeight(wq.FMT_DYADIC4, 32, 4, 64, p.value, p.value)
    odd = wq.WqWeight(wq.FMT_MXFP4, 32, 4, 96, p.value, p.value)
    assert lib.wq_gemm_mxfp4(None, by(good), p, None) == wq.WQ_EINVAL
    assert lib.wq_gemm_mxfp4(by(good), None, p, None) == wq.WQ_EINVAL
    assert lib.wq_gemm_mxfp4(by(dyadic), by(good), p, None) == wq.WQ_EINVAL and "MXFP4" in wq.last_error()
    assert lib.wq_gemm_mxfp4(by(odd), by(odd), p, None) == wq.WQ_EINVAL
    assert lib.wq_gemm_mxfp4(by(good), by(good), p, None) == wq.WQ_EINVAL            # host memory
    assert lib.wq_gemm_mxfp4_bf16(by(good), p, 0, p, p, 1 << 20, None) == wq.WQ_EINVAL
    for e in (0, -1, 4097):
        assert lib.wq_gemm_mxfp4_experts(by(good), e, p, by(good), p, None) == wq.WQ_EINVAL
        assert "experts" in wq.last_error() or "device memory" in wq.last_error() or "Attributes" in wq.last_error()
        assert lib.wq_gemm_mxfp4_experts_bf16(by(good), e, p, p, 3, p, p, 1 << 20, None) == wq.WQ_EINVAL


def test_workspace_bytes(wq):
    f = wq.gemm_mxfp4_workspace_bytes
    # codes rounded up to 256 bytes, then the scale rows of whole 16 bytes
    assert f(100, 4096) == 100 * 2048 + 100 * 128
    assert f(33, 64) == 1280 + 33 * 16
    assert f(8, 4096) == f(1, 64) == 0 and f(9, 4096) == 9 * 2048 + 9 * 128
    assert f(8, 4096, 2) == f(32, 4096, 64) == 0 and f(33, 4096, 64) == f(33, 4096)
    assert wq._lib.wq_gemm_mxfp4_workspace_bytes(0, 64, 0) == 0
    assert wq._lib.wq_gemm_mxfp4_workspace_bytes(64, 64, -1) == 0


def test_binding_refusals(wq):
    """Tensors on the CPU, of another type or shape, never reach the library."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        wq.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        wq.fake_quant_mxfp4(x)
    z = torch.zeros(0, dtype=torch.uint8)
    w = wq.PackedWeight(wq.FMT_MXFP4, 32, 8, 64, z, z)
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(w, x)
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(wq.PackedWeight(wq.FMT_DYADIC4, 32, 8, 64, z, z), w)
    # scale bytes without the rows' padding
    with pytest.raises(ValueError):
        wq.PackedWeight(wq.FMT_MXFP4, 32, 8, 64, torch.zeros((8, 32), dtype=torch.uint8),
                        torch.zeros((8, 2), dtype=torch.uint8)).desc()
    wq.PackedWeight(wq.FMT_MXFP4, 32, 8, 64, torch.zeros((8, 32), dtype=torch.uint8),
                    torch.zeros((8, 16), dtype=torch.uint8)).desc()
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(w, wq.PackedWeight(wq.FMT_MXFP4, 32, 4, 128, z, z))
    with pytest.raises(ValueError):
        wq.gemm_experts_mxfp4(w, x, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        wq.gemm_experts_mxfp4(w, x, None)
