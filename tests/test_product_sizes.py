"""The products refuse sizes whose whole tiles and steps would pass 2^31 (32-bit row and column
numbers in the kernels), before any pointer is looked at."""
import ctypes

import pytest

LIMIT = 2 ** 31 - 1024
FORMATS = [("DYADIC4", 64), ("DYADIC4", 32), ("LLOYD8S", 32), ("LUT16", 64), ("MXFP4", 32)]


@pytest.fixture
def host():
    """A 16-byte aligned host address: what is not device memory."""
    buf = (ctypes.c_uint8 * 256)()
    return ctypes.c_void_p((ctypes.addressof(buf) + 15) // 16 * 16), buf


def calls(wq, d, p):
    lib, by = wq._lib, ctypes.byref(d)
    plan = ctypes.c_void_p(None)
    one = (ctypes.c_void_p * 1)(p.value)
    out = [lambda: lib.wq_gemv_w4a16(by, p, 1, p, None),
           lambda: lib.wq_gemv_w4a16_grouped((wq.WqWeight * 1)(d), one, one, 1, 1, None),
           lambda: lib.wq_gemv_plan_create((wq.WqWeight * 1)(d), one, one, 1, 1, ctypes.byref(plan)),
           lambda: lib.wq_gemm_w4a16(by, p, 32, p, p, 1 << 40, None)]
    if d.fmt == wq.FMT_MXFP4:
        out += [lambda: lib.wq_gemm_mxfp4(by, by, p, None),
                lambda: lib.wq_gemm_mxfp4_bf16(by, p, 32, p, p, 1 << 40, None),
                lambda: lib.wq_gemm_mxfp4_experts(by, 1, p, by, p, None),
                lambda: lib.wq_gemm_mxfp4_experts_bf16(by, 1, p, p, 32, p, p, 1 << 40, None)]
    return out


@pytest.mark.parametrize("fmt, group", FORMATS)
@pytest.mark.parametrize("n, k", [(1, 2 ** 31 - 64), (1, 2 ** 31 - 512), (2 ** 31 - 1, 64), (LIMIT + 1, 64)])
def test_refused(wq, host, fmt, group, n, k):
    d = wq.WqWeight(getattr(wq, "FMT_" + fmt), group, n, k, host[0].value, host[0].value)
    for call in calls(wq, d, host[0]):
        assert call() == wq.WQ_EINVAL and "2^31 - 1024" in wq.last_error()


@pytest.mark.parametrize("fmt, group", FORMATS)
@pytest.mark.parametrize("n, k", [(1, LIMIT), (LIMIT, 64)])
def test_the_largest_sizes_are_not(wq, host, fmt, group, n, k):
    """They get as far as the pointers (host memory here)."""
    d = wq.WqWeight(getattr(wq, "FMT_" + fmt), group, n, k, host[0].value, host[0].value)
    for call in calls(wq, d, host[0]):
        assert call() == wq.WQ_EINVAL and "weight.packed" in wq.last_error()
