"""The W4A16 products refuse activations and outputs that are smaller than what the kernels read and
write: the binding compares their shapes with the weight's before any launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def made(wq, fmt, n=128, k=256):
    w = torch.randn((n, k), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    if fmt == "mxfp4":
        return wq.quantize_mxfp4(w)[0]
    if fmt == "dyadic":
        return wq.quantize_dyadic(w)[0]
    return wq.quantize_lloyd(w, mode=wq.LLOYD_G32_WARM if fmt == "lloyd8s" else wq.LLOYD_KMEANS16, rounds=1)[0]


def x_of(*shape):
    return torch.ones(shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("fmt", ["mxfp4", "dyadic", "lloyd8s", "lut16"])
def test_refused(wq, fmt):
    w = made(wq, fmt)
    for call in (wq.gemv, lambda w, x, out=None: wq.gemv_grouped([w], [x], None if out is None else [out]),
                 lambda w, x, out=None: wq.GroupedGemv([w], [x], [x_of(4, 128) if out is None else out]),
                 wq.gemm, wq.gemm_static):
        with pytest.raises(ValueError):
            call(w, x_of(4, 224))
        with pytest.raises(ValueError):
            call(w, x_of(2, 2, 256))
        with pytest.raises(ValueError):
            call(w, x_of(4, 256), out=x_of(3, 128))
        with pytest.raises(TypeError):
            call(w, x_of(4, 256), out=torch.empty((4, 128), dtype=torch.uint8, device="cuda"))
        with pytest.raises(ValueError):
            call(w, x_of(4, 256), out=x_of(4, 256)[:, ::2])
    with pytest.raises(ValueError):
        wq.gemv_grouped([w, w], [x_of(4, 256), x_of(3, 256)])
    with pytest.raises(ValueError):
        wq.gemv_grouped([w, w], [x_of(4, 256)])
    with pytest.raises(ValueError):
        wq.GroupedGemv([], [], [])


@pytest.mark.parametrize("fmt", ["mxfp4", "dyadic", "lloyd8s", "lut16"])
def test_taken(wq, fmt):
    """Shapes that hold what is read and written: a vector, a row too many in `out`."""
    w, x = made(wq, fmt), x_of(4, 256)
    y = wq.gemv(w, x)
    assert torch.equal(wq.gemv(w, x[0]), wq.gemv(w, x[:1])[0])
    for call in (wq.gemv, wq.gemm, wq.gemm_static):
        out = torch.full((5, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        assert call(w, x, out=out) is out
        assert torch.equal(out[:4], y) and (out[4] == 9.0).all()
    out = torch.full((5, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    plan = wq.GroupedGemv([w], [x.view(4, 1, 256)], [out])
    plan()
    assert torch.equal(out[:4], y) and (out[4] == 9.0).all()
    plan.close()


def test_coded_activations_on_the_host(wq):
    w = made(wq, "mxfp4")
    x = wq.PackedWeight(wq.FMT_MXFP4, 32, 4, 256, torch.zeros((4, 128), dtype=torch.uint8),
                        torch.zeros((4, 16), dtype=torch.uint8))
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(w, x)
