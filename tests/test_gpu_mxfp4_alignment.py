"""MXFP4 quantisation on buffers that begin at any multiple of 16 bytes, bit for bit: the alignment
every pointer of the library is promised, and no more."""
import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu


def at(shape, dtype, skip, fill):
    """A contiguous tensor `skip` bytes into a larger buffer filled with `fill`, and that buffer."""
    size = torch.empty(0, dtype=dtype).element_size()
    numel = shape[0] * shape[1]
    buf = torch.full((numel + 2 * 128 // size,), fill, dtype=dtype, device="cuda")
    t = buf[skip // size:skip // size + numel].view(shape)
    assert t.data_ptr() % 128 == skip and t.is_contiguous()
    return t, buf


def rows(n, k, seed, dtype):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal((n, k)) * np.exp2(g.integers(-8, 8, (n, 1)))).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("skip", [0, 16, 32, 48, 112])
@pytest.mark.parametrize("n, k", [(1, 32), (3, 544), (129, 96), (700, 2080)])
def test_a_matrix_inside_a_flat_buffer(wq, n, k, skip, dtype):
    """One parameter of a flat buffer through the binding: codes, scale bytes and values."""
    want = rows(n, k, n + k, dtype)
    x, _ = at((n, k), dtype, skip, 1e30)
    x.copy_(want)
    codes, scale = mx.quantize(want.double().numpy())
    pw, c = wq.quantize_mxfp4(x, codes=True)
    q, pw2 = wq.fake_quant_mxfp4(x, packed=True)
    assert np.array_equal(pw.aux.cpu().numpy(), scale) and torch.equal(pw2.aux, pw.aux)
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(pw.packed.cpu().numpy(), codes[:, 0::2] | codes[:, 1::2] << 4)
    assert torch.equal(pw2.packed, pw.packed)
    assert np.array_equal(q.cpu().double().numpy(), mx.values(codes, scale))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("skips", [(0, 16, 0, 0, 0), (16, 0, 0, 0, 0), (16, 48, 16, 48, 112), (32, 96, 80, 16, 48)])
def test_every_output_at_an_offset_of_its_own(wq, skips, dtype):
    """The C entry with x, q, scale, codes and packed at these offsets; what lies around the
    outputs is left as it was."""
    n, k = 37, 1056
    want = rows(n, k, 5, dtype)
    x, _ = at((n, k), dtype, skips[0], 1e30)
    x.copy_(want)
    q, qb = at((n, k), dtype, skips[1], 7.0)
    s, sb = at((n, wq.mx_pitch(k)), torch.uint8, skips[2], 201)
    c, cb = at((n, k), torch.uint8, skips[3], 202)
    p, pb = at((n, k // 2), torch.uint8, skips[4], 203)
    wq._check(wq._lib.wq_quantize_mxfp4(x.data_ptr(), wq.F32 if dtype == torch.float32 else wq.BF16, n, k, s.data_ptr(),
                                        c.data_ptr(), p.data_ptr(), q.data_ptr(),
                                        torch.cuda.current_stream().cuda_stream))
    codes, scale = mx.quantize(want.double().numpy())
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(p.cpu().numpy(), codes[:, 0::2] | codes[:, 1::2] << 4)
    assert np.array_equal(q.cpu().double().numpy(), mx.values(codes, scale))
    for buf, t, fill in ((qb, q, 7.0), (sb, s, 201), (cb, c, 202), (pb, p, 203)):
        lo = (t.data_ptr() - buf.data_ptr()) // t.element_size()
        assert (buf[:lo] == fill).all() and (buf[lo + t.numel():] == fill).all()


def test_chunk_numbers_of_64_bits_at_an_offset(wq):
    """69 GB of fp32 at an offset of 16 bytes: the rows at its start, its middle and its end."""
    n, k = (1 << 19) + 9, 32800
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free memory")
    x = torch.empty((n * k + 8,), dtype=torch.float32, device="cuda")[4:4 + n * k].view(n, k)
    at_rows = [0, 131073, 262144, n - 2, n - 1]
    for i, r in enumerate(at_rows):
        x[r] = rows(1, k, i, torch.float32)[0].cuda()
    pw, _ = wq.quantize_mxfp4(x)
    for i, r in enumerate(at_rows):
        codes, scale = mx.quantize(rows(1, k, i, torch.float32).double().numpy())
        assert np.array_equal(pw.aux[r].cpu().numpy(), scale[0])
        assert np.array_equal(pw.packed[r].cpu().numpy(), codes[0, 0::2] | codes[0, 1::2] << 4)
    del x, pw
    torch.cuda.empty_cache()
