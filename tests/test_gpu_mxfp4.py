"""MXFP4 on the GPU against the fp64 oracle: quantisation and reconstruction bit for bit, the
W4A16 products and the block-scaled products within tolerance and exactly where every sum is."""
import numpy as np
import pytest
import torch

import oracle
from oracle import mx
from _util import f32, matmul_tolerance, to_dev, to_dev_bits

pytestmark = pytest.mark.gpu


def weights(n, k, seed, lo=-6, hi=3):
    """Codes and scale bytes drawn at random (scales 2^lo .. 2^hi, every code), padding at 255."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (n, k), dtype=np.uint8)
    scale = np.full((n, mx.pitch(k)), 255, np.uint8)
    scale[:, :k // 32] = g.integers(127 + lo, 128 + hi, (n, k // 32))
    return codes, scale


def packed(wq, codes, scale):
    n, k = codes.shape
    return wq.PackedWeight(wq.FMT_MXFP4, 32, n, k, to_dev(codes[:, 0::2] | codes[:, 1::2] << 4), to_dev(scale))


def acts(m, k, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal((m, k)) * np.exp(0.5 * g.standard_normal(k))).astype(np.float32)).bfloat16()


def one_hot(m, k, seed):
    """Rows of zeros with one 1 each, and its columns."""
    at = np.random.default_rng(seed).integers(0, k, m)
    x = np.zeros((m, k), np.float32)
    x[np.arange(m), at] = 1.0
    return torch.from_numpy(x).bfloat16(), at


def check(y, xv, wv):
    ref, bound = mx.product(xv, wv)
    err = np.abs(f32(y) - ref)
    assert (err <= matmul_tolerance(ref, bound)).all(), float((err / np.maximum(bound, 1e-300)).max())


# --- quantisation ------------------------------------------------------------------------

def check_quantise(wq, x):
    codes, scale = mx.quantize(x.double().numpy())
    pw, c = wq.quantize_mxfp4(x.cuda(), codes=True)
    q, pw2 = wq.fake_quant_mxfp4(x.cuda(), packed=True)
    assert np.array_equal(pw.aux.cpu().numpy(), scale)
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(pw.packed.cpu().numpy(), codes[:, 0::2] | codes[:, 1::2] << 4)
    assert torch.equal(pw2.packed, pw.packed) and torch.equal(pw2.aux, pw.aux)
    v = mx.values(codes, scale)
    assert q.dtype == x.dtype and np.array_equal(q.cpu().double().numpy(), v, equal_nan=True)
    neg = ~np.isnan(v)
    assert np.array_equal(np.signbit(q.cpu().float().numpy())[neg], np.signbit(v)[neg])
    d = wq.dequant(pw)
    assert np.array_equal(d.cpu().double().numpy(), v, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n, k", [(1, 32), (1, 64), (3, 512), (5, 544), (7, 2080), (129, 96), (1000, 4096)])
def test_quantise_shapes(wq, n, k, dtype):
    g = np.random.default_rng(n * 7 + k)
    x = g.standard_normal((n, k)) * np.exp2(g.integers(-8, 8, (n, 1)))
    check_quantise(wq, torch.from_numpy(x.astype(np.float32)).to(dtype))


def test_quantise_every_bf16_pattern(wq):
    """Every bf16 value beside a largest one of each of its binade's neighbours."""
    bits = np.arange(65536, dtype=np.uint16).reshape(-1, 16)
    top = (bits & 0x7FFF).max(1, keepdims=True).astype(np.int64)
    rows = []
    for up in (0, 1, 2, 3, 5):
        lead = np.minimum(top + (up << 7), 0x7F7F).astype(np.uint16)
        rows.append(np.concatenate([bits, np.repeat(lead, 16, 1)], 1))
    x = torch.from_numpy(np.concatenate(rows).view(np.int16)).view(torch.bfloat16)
    check_quantise(wq, x.contiguous())


def test_quantise_fp32_ties_and_ends(wq):
    """Every midpoint and its neighbours at many scales, subnormals, the largest values, blocks
    with NaN and infinities, zeros of both signs."""
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    pts = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9)), mx.LEVELS[1:]])
    pts = np.concatenate([pts, [4.0, 6.5, 7.99]]).astype(np.float32)[:31]
    rows = []
    for e in (-149, -140, -127, -126, -125, -100, -3, 0, 9, 90, 125):
        with np.errstate(over="ignore", under="ignore"):
            b = np.ldexp(np.concatenate([pts, [4.0]]).astype(np.float64), e).astype(np.float32)
        rows += [b, -b]
    z = np.zeros(32, np.float32)
    rows += [z, -z]
    for bad in (np.nan, np.inf, -np.inf):
        b = np.ones(32, np.float32)
        b[17] = bad
        rows.append(b)
    check_quantise(wq, torch.from_numpy(np.stack(rows)))


def test_dequant_at_the_ends_of_the_scales(wq):
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scale = np.zeros((256, 16), np.uint8)
    scale[:, 0] = np.arange(256)
    v = mx.values(codes, scale)
    d = wq.dequant(packed(wq, codes, scale)).cpu().double().numpy()
    v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)   # past bf16's largest
    assert np.array_equal(d, v, equal_nan=True)


# --- W4A16 products ----------------------------------------------------------------------

@pytest.mark.parametrize("n, k", [(1, 32), (17, 96), (128, 256), (300, 2080), (1003, 544), (2048, 4096)])
@pytest.mark.parametrize("m", [1, 3, 8, 9, 16])
def test_gemv(wq, m, n, k):
    codes, scale = weights(n, k, n + k)
    x = acts(m, k, m)
    check(wq.gemv(packed(wq, codes, scale), x.cuda()), x.double().numpy(), mx.values(codes, scale))


@pytest.mark.parametrize("m, n, k", [(17, 130, 64), (33, 1003, 1088), (64, 256, 4096), (100, 300, 192),
                                     (128, 512, 512), (129, 257, 576), (512, 1024, 2048), (600, 640, 320)])
def test_gemm(wq, m, n, k):
    codes, scale = weights(n, k, n + k)
    x = acts(m, k, m)
    check(wq.gemm(packed(wq, codes, scale), x.cuda()), x.double().numpy(), mx.values(codes, scale))


@pytest.mark.parametrize("m", [1, 7, 16, 48, 128, 300])
def test_w4a16_one_hot_is_exact_at_every_scale(wq, m):
    n, k = 256, 512
    codes, scale = weights(n, k, 5, lo=-127, hi=124)
    x, at = one_hot(m, k, m)
    y = wq.gemm(packed(wq, codes, scale), x.cuda())
    assert np.array_equal(f32(y), mx.values(codes, scale)[:, at].T)


def test_gemv_grouped_and_plan(wq):
    shapes = [(100, 512), (64, 96), (700, 1056)]
    ws, xs, refs = [], [], []
    for i, (n, k) in enumerate(shapes):
        codes, scale = weights(n, k, i)
        ws.append(packed(wq, codes, scale))
        x = acts(4, k, i)
        xs.append(x.cuda())
        refs.append((x.double().numpy(), mx.values(codes, scale)))
    for y, r in zip(wq.gemv_grouped(ws, xs), refs):
        check(y, *r)
    ys = [torch.empty((4, n), dtype=torch.bfloat16, device="cuda") for n, _ in shapes]
    plan = wq.GroupedGemv(ws, xs, ys)
    plan()
    torch.cuda.synchronize()
    for y, r in zip(ys, refs):
        check(y, *r)
    plan.close()


def test_overlapped_plans_behind_a_quantisation_of_their_weights(wq):
    """The kernel just before the last plan does not write its weights, the one before that does."""
    g = torch.Generator(device="cuda").manual_seed(5)
    w = [torch.randn((8192, 8192), generator=g, device="cuda").bfloat16() for _ in range(2)]
    x = torch.randn((1, 8192), generator=g, device="cuda").bfloat16()
    want = [wq.gemv(wq.quantize_mxfp4(v)[0], x) for v in w]
    pw, _ = wq.quantize_mxfp4(w[0])
    small, _ = wq.quantize_mxfp4(w[0][:64])
    plans, ys = [], []
    for p in (small, pw):
        ys.append(torch.empty((1, p.n), dtype=torch.bfloat16, device="cuda"))
        plans.append(wq.GroupedGemv([p], [x], [ys[-1]], overlap=True))
    s = torch.cuda.current_stream().cuda_stream
    for i in (1, 0, 1, 0):
        wq._check(wq._lib.wq_quantize_mxfp4(w[i].data_ptr(), wq.BF16, 8192, 8192, pw.aux.data_ptr(), None,
                                            pw.packed.data_ptr(), None, s))
        for p in plans:
            p()
        assert torch.equal(ys[1], want[i])
    for p in plans:
        p.close()


@pytest.mark.parametrize("m", [40, 200])
def test_gemm_static(wq, m):
    """The GEMM on the library's own scratch takes the format, too."""
    n, k = 512, 4096
    codes, scale = weights(n, k, 5)
    x = acts(m, k, m)
    check(wq.gemm_static(packed(wq, codes, scale), x.cuda()), x.double().numpy(), mx.values(codes, scale))


# --- block-scaled products ---------------------------------------------------------------

@pytest.mark.parametrize("m", [1, 16, 17, 40, 70, 130, 300])
def test_product_one_hot_is_exact(wq, m):
    """x picks columns of W: the scale byte of every block of W, then of x, reaches its rows."""
    n, k = 300, 1088
    codes, scale = weights(n, k, 3, lo=-100, hi=90)
    x, at = one_hot(m, k, m)
    y = wq.gemm_mxfp4(packed(wq, codes, scale), x.cuda())
    assert np.array_equal(f32(y), mx.values(codes, scale)[:, at].T)
    # and the other way round: one-hot weights, every scale of the activations
    xc, xs = weights(m, k, 4, lo=-100, hi=90)
    w, at = one_hot(n, k, 9)
    wc, wsc = mx.quantize(w.double().numpy())
    y = wq.gemm_mxfp4(packed(wq, wc, wsc), packed(wq, xc, xs))
    assert np.array_equal(f32(y), mx.values(xc, xs)[:, at])
    assert wq.device_error() == 0


@pytest.mark.parametrize("k", [64, 128, 192, 448, 512, 576, 1024, 2112, 4096])
@pytest.mark.parametrize("m, n", [(1, 1), (1, 300), (5, 128), (16, 129), (31, 260), (64, 64), (65, 200)])
def test_product(wq, m, n, k):
    codes, scale = weights(n, k, n + k)
    x = acts(m, k, m)
    xc, xs = mx.quantize(x.double().numpy())
    pw = packed(wq, codes, scale)
    y = wq.gemm_mxfp4(pw, x.cuda())
    check(y, mx.values(xc, xs), mx.values(codes, scale))
    assert torch.equal(y, wq.gemm_mxfp4(pw, packed(wq, xc, xs)))
    assert wq.device_error() == 0


@pytest.mark.parametrize("m, n, k", [(1, 20000, 512), (5, 20000, 2112), (8, 19000, 576), (9, 20000, 1088)])
def test_product_of_few_rows_over_all_of_k(wq, m, n, k):
    """So many weight rows that no CTA splits K: one to five scale stages each."""
    codes, scale = weights(n, k, n + k)
    x = acts(m, k, m)
    xc, xs = mx.quantize(x.double().numpy())
    check(wq.gemm_mxfp4(packed(wq, codes, scale), x.cuda()), mx.values(xc, xs), mx.values(codes, scale))
    assert wq.device_error() == 0


@pytest.mark.parametrize("m, n, k", [(127, 300, 832), (128, 128, 4096), (129, 500, 1088), (255, 129, 320),
                                     (256, 256, 2048), (257, 1003, 2112), (1000, 640, 512), (4096, 384, 1024)])
def test_product_large(wq, m, n, k):
    codes, scale = weights(n, k, n + k)
    x = acts(m, k, m)
    xc, xs = mx.quantize(x.double().numpy())
    check(wq.gemm_mxfp4(packed(wq, codes, scale), x.cuda()), mx.values(xc, xs), mx.values(codes, scale))
    assert wq.device_error() == 0


# --- grouped by expert -------------------------------------------------------------------

def experts_ref(xv, wv, off, n):
    y = np.zeros((xv.shape[0], n))
    b = np.zeros((xv.shape[0], n))
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        y[r], b[r] = mx.product(xv[r], wv[e * n:(e + 1) * n])
    return y, b


@pytest.mark.parametrize("counts, n, k", [
    ([1], 128, 64), ([3], 100, 512), ([0, 1], 7, 64), ([1, 0, 0, 2], 130, 576), ([0, 0, 5, 0], 257, 128),
    ([16, 17, 1, 0, 15, 33], 200, 1088), ([130, 0, 1, 257, 64], 300, 192), ([500, 3], 129, 1024),
    ([1] * 70, 64, 256), ([0] * 40 + [2] + [0] * 30 + [9], 33, 320), ([300, 0, 290, 310], 384, 512),
    ([0, 3, 0] * 100 + [40] + [1] * 33, 16, 64), ([0] * 500 + [5] + [0] * 523, 8, 64), ([200] * 40, 24, 64),
    ([0] * 20 + [37] + [0] * 80 + [18] + [0] * 40, 200, 1088), ([8], 130, 2112), ([9], 130, 2112), ([4, 4], 20, 576),
])
def test_experts(wq, counts, n, k):
    e, t = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    codes, scale = weights(e * n, k, n + k)
    x = acts(t, k, t)
    xc, xs = mx.quantize(x.double().numpy())
    pw = packed(wq, codes, scale)
    y = wq.gemm_experts_mxfp4(pw, x.cuda(), to_dev(off))
    ref, bound = experts_ref(mx.values(xc, xs), mx.values(codes, scale), off, n)
    assert (np.abs(f32(y) - ref) <= matmul_tolerance(ref, bound)).all()
    assert torch.equal(y, wq.gemm_experts_mxfp4(pw, packed(wq, xc, xs), to_dev(off)))
    assert wq.device_error() == 0


def test_experts_leave_other_rows_alone(wq):
    """Rows before the first and behind the last expert's keep what they held, whatever x holds there."""
    n, k, t = 200, 576, 50
    off = np.array([7, 7, 20, 41], np.int32)
    codes, scale = weights(3 * n, k, 1)
    x = acts(t, k, 2)
    x[:7] = float("nan")
    x[41:] = float("inf")
    out = torch.full((t, n), 3.5, dtype=torch.bfloat16, device="cuda")
    y = wq.gemm_experts_mxfp4(packed(wq, codes, scale), x.cuda(), to_dev(off), out=out)
    assert y is out and (y[:7] == 3.5).all() and (y[41:] == 3.5).all()
    xc, xs = mx.quantize(np.nan_to_num(x.double().numpy(), posinf=0.0))
    ref, bound = experts_ref(mx.values(xc, xs), mx.values(codes, scale), off, n)
    r = slice(7, 41)
    assert (np.abs(f32(y) - ref)[r] <= matmul_tolerance(ref, bound)[r]).all()


def test_experts_with_no_rows_at_all(wq):
    codes, scale = weights(4 * 64, 128, 1)
    pw = packed(wq, codes, scale)
    out = torch.full((9, 64), -2.0, dtype=torch.bfloat16, device="cuda")
    wq.gemm_experts_mxfp4(pw, acts(9, 128, 1).cuda(), torch.full((5,), 4, dtype=torch.int32, device="cuda"), out=out)
    assert (out == -2.0).all()
    y = wq.gemm_experts_mxfp4(pw, torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                              torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 64)


# --- as they are used --------------------------------------------------------------------

@pytest.mark.parametrize("m, n, k", [(3, 200, 576), (40, 130, 1088), (100, 260, 512), (300, 264, 320), (260, 131, 320)])
def test_nothing_outside_the_output_is_written(wq, m, n, k):
    codes, scale = weights(n, k, 1)
    pw = packed(wq, codes, scale)
    x = acts(m, k, 2)
    pad = 24
    buf = torch.full((m + 2 * pad, n), 7.25, dtype=torch.bfloat16, device="cuda")
    lo = next(r for r in range(pad) if (r * n * 2) % 16 == 0 and r > 0) if (n * 2) % 16 else pad
    out = buf[lo:lo + m]
    wq.gemm_mxfp4(pw, x.cuda(), out=out)
    assert (buf[:lo] == 7.25).all() and (buf[lo + m:] == 7.25).all()
    xc, xs = mx.quantize(x.double().numpy())
    check(out, mx.values(xc, xs), mx.values(codes, scale))


@pytest.mark.parametrize("n", [121, 250, 251, 252, 253, 254, 255, 256, 257, 319, 321])
def test_rows_of_every_alignment_in_wide_tiles(wq, n):
    """Rows of y that begin at any multiple of two bytes, last rows of an expert inside a tile of 32."""
    k, off = 320, np.array([1, 301, 302, 302, 595], np.int32)
    codes, scale = weights(4 * n, k, n)
    x = acts(600, k, 3)
    xc, xs = mx.quantize(x.double().numpy())
    out = torch.full((600, n), 7.25, dtype=torch.bfloat16, device="cuda")
    wq.gemm_experts_mxfp4(packed(wq, codes, scale), x.cuda(), to_dev(off), out=out)
    assert (out[:1] == 7.25).all() and (out[595:] == 7.25).all()
    ref, bound = experts_ref(mx.values(xc, xs), mx.values(codes, scale), off, n)
    r = slice(1, 595)
    assert (np.abs(f32(out) - ref)[r] <= matmul_tolerance(ref, bound)[r]).all()
    y = wq.gemm_mxfp4(packed(wq, codes[:n], scale[:n]), x.cuda())
    check(y, mx.values(xc, xs), mx.values(codes[:n], scale[:n]))
    assert wq.device_error() == 0


def test_nan_blocks_reach_their_rows_and_columns_only(wq):
    """A NaN scale byte of x makes one row of y NaN, one of w a column; few rows (quantised by the
    product), some, and many."""
    n, k = 260, 576
    codes, scale = weights(n, k, 1)
    scale[77, 3] = 255
    pw = packed(wq, codes, scale)
    for m in (5, 9, 50, 300):
        x = acts(m, k, m)
        x[m // 2, 100] = float("inf")
        y = wq.gemm_mxfp4(pw, x.cuda()).float().cpu().numpy()
        bad = np.zeros((m, n), bool)
        bad[m // 2] = True
        bad[:, 77] = True
        assert np.array_equal(np.isnan(y), bad)


@pytest.mark.parametrize("m, experts", [(5, 0), (48, 0), (300, 0), (40, 4), (700, 3)])
def test_captured_and_replayed(wq, m, experts):
    """One capture, replayed on new activations (and offsets), gives what eager calls give; two
    graphs, each with buffers of its own, replayed at once on two streams, too."""
    n, k = 256, 640
    codes, scale = weights(max(1, experts) * n, k, 3)
    pw = packed(wq, codes, scale)

    def call(x, off, out):
        return wq.gemm_experts_mxfp4(pw, x, off, out=out) if experts else wq.gemm_mxfp4(pw, x, out=out)

    def offsets(seed):
        cut = np.sort(np.random.default_rng(seed).integers(0, m + 1, experts - 1)) if experts else []
        return torch.tensor([0, *cut, m], dtype=torch.int32, device="cuda")

    graphs = []
    for g in range(2):
        x, off = acts(m, k, g).cuda(), offsets(g)
        out = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(x, off, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(x, off, out)
        graphs.append((graph, x, off, out, s))
    for step in range(3):
        want = []
        for g, (graph, x, off, out, s) in enumerate(graphs):
            x.copy_(acts(m, k, 10 * step + g))
            off.copy_(offsets(10 * step + g))
            out.zero_()
            want.append(call(x, off, torch.zeros_like(out)))
        torch.cuda.synchronize()
        for graph, x, off, out, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (graph, x, off, out, s), w in zip(graphs, want):
            assert torch.equal(out, w)
    assert wq.device_error() == 0


def test_other_streams_and_a_workspace_of_the_callers(wq):
    """Inputs made on a side stream, the call on the same stream, no synchronisation between."""
    n, k, m = 384, 1024, 200
    codes, scale = weights(n, k, 3)
    pw = packed(wq, codes, scale)
    need = wq.gemm_mxfp4_workspace_bytes(m, k)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            x = acts(m, k, i).cuda(non_blocking=True) * 1.0
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            outs.append((wq.gemm_mxfp4(pw, x, workspace=ws), ws, x))
    torch.cuda.synchronize()
    for i, (y, _, x) in enumerate(outs):
        xc, xs = mx.quantize(x.double().cpu().numpy())
        check(y, mx.values(xc, xs), mx.values(codes, scale))


def test_calls_repeat_bit_for_bit(wq):
    for m, n, k in [(2, 300, 8192), (20, 512, 4096), (90, 200, 4096), (500, 640, 2048)]:
        codes, scale = weights(n, k, 3)
        pw, x = packed(wq, codes, scale), acts(m, k, 4).cuda()
        y = wq.gemm_mxfp4(pw, x)
        assert all(torch.equal(y, wq.gemm_mxfp4(pw, x)) for _ in range(5))


def test_binding_refuses_on_the_gpu(wq):
    codes, scale = weights(64, 128, 1)
    pw = packed(wq, codes, scale)
    x = acts(8, 128, 1).cuda()
    with pytest.raises(TypeError):
        wq.gemm_mxfp4(pw, x.float())
    with pytest.raises(TypeError):
        wq.quantize_mxfp4(x.half())
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(pw, x[:, :64])
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(pw, x.t().contiguous().t())
    with pytest.raises(ValueError):
        wq.gemm_mxfp4(pw, x, out=torch.empty((8, 63), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        wq.gemm_mxfp4(pw, x, out=torch.empty((8, 64), device="cuda"))
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        wq.gemm_experts_mxfp4(pw, x, off.long())
    with pytest.raises(ValueError):                      # 64 rows are no 3 experts'
        wq.gemm_experts_mxfp4(pw, x, torch.tensor([0, 1, 2, 8], dtype=torch.int32, device="cuda"))
    with pytest.raises(wq.WqError) as e:                 # offsets not 16-byte aligned
        wq.gemm_experts_mxfp4(pw, x, torch.zeros(8, dtype=torch.int32, device="cuda")[1:4])
    assert e.value.status == wq.WQ_EALIGN
    wq.debug_fail_next_launches(1)
    with pytest.raises(wq.WqError) as e:
        wq.gemm_mxfp4(pw, x)
    assert e.value.status == wq.WQ_ECUDA
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    d = pw.desc()
    import ctypes
    xx = acts(40, 128, 1).cuda()
    y = torch.empty((40, 64), dtype=torch.bfloat16, device="cuda")
    assert wq._lib.wq_gemm_mxfp4_bf16(ctypes.byref(d), xx.data_ptr(), 40, y.data_ptr(), small.data_ptr(), 16,
                                      None) == wq.WQ_EINVAL and "workspace" in wq.last_error()


def test_an_output_past_two_to_the_31_elements(wq):
    """y[m, n] of 2.2 G elements: rows at its start, its middle and its end, exactly (one-hot x)."""
    m, n, k = 67000, 32832, 64
    codes, scale = weights(n, k, 8)
    x, at = one_hot(m, k, 5)
    y = wq.gemm_mxfp4(packed(wq, codes, scale), x.cuda())
    v = mx.values(codes, scale)
    for r in (0, 1, 33000, 65407, 65408, 66815, m - 1):
        assert np.array_equal(f32(y[r]), v[:, at[r]]), r
    assert wq.device_error() == 0


def test_quantisation_past_two_to_the_35_elements(wq):
    """Chunk numbers that need 64 bits (70 GB of activations, checked at their end)."""
    n, k = 1 << 20, 32800
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB of free memory")
    x = torch.empty((n, k), dtype=torch.bfloat16, device="cuda")
    rows = [0, 500_000, n - 2, n - 1]
    for i, r in enumerate(rows):
        x[r] = acts(1, k, i)[0].cuda()
    pw, _ = wq.quantize_mxfp4(x)
    for i, r in enumerate(rows):
        codes, scale = mx.quantize(acts(1, k, i).double().numpy())
        assert np.array_equal(pw.aux[r].cpu().numpy(), scale[0])
        assert np.array_equal(pw.packed[r].cpu().numpy(), codes[0, 0::2] | codes[0, 1::2] << 4)
    del x, pw
    torch.cuda.empty_cache()


# --- together ----------------------------------------------------------------------------

def test_a_mixture_of_experts_layer(wq):
    """Coded projections and experts in a row, each against 64 bits on the inputs it was given: a
    router's top choice sorts the rows, up and gate (stacked) by expert, SwiGLU, down by expert,
    rows back in place, a dense projection behind; then one row of it by the W4A16 GEMV."""
    hidden, inner, e, t = 256, 448, 6, 75
    g = torch.Generator().manual_seed(3)

    def coded(rows, cols):
        w = (torch.randn((rows, cols), generator=g) * 0.1).bfloat16()
        codes, scale = mx.quantize(w.double().numpy())
        pw, _ = wq.quantize_mxfp4(w.cuda())
        assert np.array_equal(pw.aux.cpu().numpy(), scale)
        return pw, mx.values(codes, scale)

    up, upv = coded(e * 2 * inner, hidden)
    down, downv = coded(e * hidden, inner)
    head, headv = coded(320, hidden)
    x = torch.randn((t, hidden), generator=g).bfloat16().cuda()
    expert = (x @ torch.randn((hidden, e), generator=g).bfloat16().cuda()).argmax(1)
    order = expert.argsort(stable=True)
    off = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), torch.bincount(expert, minlength=e).cumsum(0)]).int()
    xs = x[order].contiguous()
    a = wq.gemm_experts_mxfp4(up, xs, off)
    act = (torch.nn.functional.silu(a[:, :inner].float()) * a[:, inner:].float()).bfloat16()
    b = wq.gemm_experts_mxfp4(down, act, off)
    back = torch.empty_like(b)
    back[order] = b
    y = wq.gemm_mxfp4(head, back)
    one = wq.gemv(head, back[:1].contiguous())
    torch.cuda.synchronize()
    offs = off.cpu().numpy()

    def coded_rows(v):
        return mx.values(*mx.quantize(v.double().cpu().numpy()))

    for got, rows, wv, n in ((a, xs, upv, 2 * inner), (b, act, downv, hidden)):
        ref, bound = experts_ref(coded_rows(rows), wv, offs, n)
        assert (np.abs(f32(got) - ref) <= matmul_tolerance(ref, bound)).all()
    check(y, coded_rows(back), headv)
    check(one, back[:1].double().cpu().numpy(), headv)


def test_fake_quantisation_in_a_training_step(wq):
    """Straight through: the forward value is the code value, the gradient reaches the latents as
    it is. Against the formula, and against differences of the loss in the code values."""
    class Straight(torch.autograd.Function):
        @staticmethod
        def forward(ctx, z):
            return wq.fake_quant_mxfp4(z.detach())[0]

        @staticmethod
        def backward(ctx, g):
            return g

    g = torch.Generator().manual_seed(1)
    z = torch.randn((24, 96), generator=g).cuda().requires_grad_()
    x = torch.randn((10, 96), generator=g).double().cuda()
    q = Straight.apply(z)
    codes, scale = mx.quantize(z.detach().double().cpu().numpy())
    v = mx.values(codes, scale)
    assert np.array_equal(q.detach().double().cpu().numpy(), v)
    loss = ((x @ q.double().T) ** 2).sum()
    loss.backward()
    xn = x.cpu().numpy()
    want = 2 * (v @ xn.T) @ xn
    got = z.grad.double().cpu().numpy()
    # the gradient is rounded to fp32 once
    assert (np.abs(got - want) <= 2.0 ** -23 * np.abs(want) + 1e-300).all()
    d = 1e-3
    for i, j in ((0, 0), (7, 50), (23, 95)):
        e = np.zeros_like(v)
        e[i, j] = d
        diff = (((xn @ (v + e).T) ** 2).sum() - ((xn @ (v - e).T) ** 2).sum()) / (2 * d)
        assert abs(diff - got[i, j]) <= 1e-6 * (np.abs(want).max() + 1)
