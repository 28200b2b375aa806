"""The MXFP4 products along the routes that larger calls take: one CTA a tile with K split over 2, 4
and 8 ranks at 33 to 128 rows, and pairs of CTAs at every tile width with several tiles a pair and 5
to 11 stages of 256 columns a tile, dense and by expert. Every row against 64 bits, and exactly."""
import numpy as np
import pytest
import torch

from oracle import mx
from _util import bf16_half_ulp, to_dev

SMS = 148


def pair_width(rows, columns):
    """Activation rows a tile of the pair kernel: fewest rounds of the grid times (width + 400)."""
    def cost(bn):
        return -(-columns * -(-rows // bn) // (SMS // 2)) * (bn + 400)
    return min(range(256, 31, -16), key=cost)


def ranks(m, n, k):
    """CTAs that split K in the kernel of one CTA a tile."""
    ctas, stages, cl = -(-m // (64 if m <= 64 else 128)) * -(-n // 128), -(-k // 256), 1
    while cl < 8 and ((2 * ctas * cl <= SMS and stages // (2 * cl) >= 2) or
                      (2 * ctas * cl <= 2 * SMS and stages // (2 * cl) >= 4)):
        cl *= 2
    return cl


# (ranks, m, n, k): a last rank with fewer columns and ranks with none (4160 columns are 17 stages,
# an even number a rank), weight rows that are no multiple of 4, a single row past a tile
SPLIT = [(8, 65, 130, 4160), (8, 128, 1003, 11008), (8, 100, 2050, 8192), (4, 65, 4100, 4160), (4, 128, 4701, 4160),
         (4, 100, 9001, 8192), (2, 128, 9500, 4160), (2, 65, 9601, 8192), (2, 100, 9474, 11008), (8, 33, 131, 4160),
         (8, 64, 1003, 8192), (4, 40, 4101, 4160), (2, 64, 9500, 4160), (2, 33, 9473, 8192)]
# (width, m, n, k), more tiles than pairs
DENSE = [(64, 64, 19300, 1280), (80, 75, 19201, 1344), (96, 96, 19210, 2624), (112, 101, 19300, 2048),
         (128, 1537, 2811, 1600), (144, 1795, 2555, 2112), (160, 2017, 2556, 1792), (176, 2242, 2555, 2368),
         (192, 2467, 2560, 1280), (208, 2497, 2811, 1344), (224, 2290, 3323, 2624), (240, 2467, 3328, 2304),
         (256, 250, 19201, 1344), (256, 1021, 9472, 1600)]
# (width, rows, experts, n, k)
EXPERTS = [(32, 320, 40, 300, 1280), (48, 960, 40, 264, 2624), (64, 1440, 40, 300, 1344), (80, 1760, 40, 261, 1600),
           (96, 2240, 40, 300, 2048), (112, 2720, 40, 272, 1280), (128, 3040, 40, 300, 2112), (144, 3520, 40, 264, 1344),
           (160, 4000, 40, 300, 2368), (176, 4320, 40, 263, 1280), (192, 4800, 40, 304, 1600), (208, 5280, 40, 300, 1344),
           (224, 5600, 40, 258, 1792), (240, 6080, 40, 264, 1280), (256, 6560, 40, 300, 1344), (96, 4480, 80, 264, 1280)]


def counts_of(rows, experts, seed):
    """Rows by expert: from none to about twice the average."""
    g = np.random.default_rng(seed)
    like = g.uniform(0.0, 2.0, experts)
    like[g.integers(0, experts, 3)] = 0.0
    return np.bincount(g.choice(experts, rows, p=like / like.sum()), minlength=experts)


def test_the_cases_take_these_routes():
    """The launch's rules at 148 SMs, written out again: a case that leaves its route is moved back."""
    for cl, m, n, k in SPLIT:
        assert 32 < m <= 128 and (k > 4096 or (m <= 64 and cl > 2)) and ranks(m, n, k) == cl
    for width, m, n, k in DENSE:
        tiles = -(-n // 256)
        assert m > 128 or (k <= 4096 and (m > 64 or ranks(m, n, k) <= 2))
        assert pair_width(m, tiles) == width and -(-m // width) * tiles > SMS // 2 and 5 <= -(-k // 256) <= 11
    for width, rows, experts, n, k in EXPERTS:
        tiles, mean = -(-n // 256), -(-rows // experts)
        assert rows > experts // 2 and pair_width(max(mean, min(mean + mean // 2, 256)), tiles * experts) == width
        full = sum(-(-int(c) // width) for c in counts_of(rows, experts, rows + k))
        assert full * tiles > 50 and 5 <= -(-k // 256) <= 11
    assert {c[0] for c in DENSE} == set(range(64, 257, 16)) and {c[0] for c in EXPERTS} == set(range(32, 257, 16))


def packed(wq, codes, scale):
    n, k = codes.shape
    return wq.PackedWeight(wq.FMT_MXFP4, 32, n, k, to_dev(codes[:, 0::2] | codes[:, 1::2] << 4), to_dev(scale))


def weights(n, k, seed, lo=-6, hi=3):
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (n, k), dtype=np.uint8)
    scale = np.full((n, mx.pitch(k)), 255, np.uint8)
    scale[:, :k // 32] = g.integers(127 + lo, 128 + hi, (n, k // 32))
    return codes, scale


def acts(m, k, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy((g.standard_normal((m, k)) * np.exp(0.5 * g.standard_normal(k))).astype(np.float32)).bfloat16()


def one_hot(m, k, seed):
    at = np.random.default_rng(seed).integers(0, k, m)
    x = np.zeros((m, k), np.float32)
    x[np.arange(m), at] = 1.0
    return torch.from_numpy(x).bfloat16(), at


def check(y, xv, wv):
    """All of y against 64-bit products, the tolerance of every product here: 2e-3 of the sum of
    magnitudes and the rounding to bf16."""
    x, w = to_dev(xv), to_dev(wv)
    ref, bound = (x @ w.T).cpu().numpy(), (x.abs() @ w.abs().T).cpu().numpy()
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= 2e-3 * bound + bf16_half_ulp(ref)).all(), float((err / np.maximum(bound, 1e-300)).max())


def check_dense(wq, m, n, k):
    codes, scale = weights(n, k, n + k)
    pw, x = packed(wq, codes, scale), acts(m, k, m)
    xc, xs = mx.quantize(x.double().numpy())
    px = packed(wq, xc, xs)
    y = wq.gemm_mxfp4(pw, x.cuda())
    check(y, mx.values(xc, xs), mx.values(codes, scale))
    for _ in range(3):
        assert torch.equal(y, wq.gemm_mxfp4(pw, px))
    # one column of the weights a row, at scales from end to end: exact
    codes, scale = weights(n, k, n + 1, lo=-100, hi=90)
    x, at = one_hot(m, k, m)
    y = wq.gemm_mxfp4(packed(wq, codes, scale), x.cuda())
    assert np.array_equal(y.double().cpu().numpy(), mx.values(codes, scale)[:, at].T)
    # and one column of the activations a weight row
    xc, xs = weights(m, k, m + 2, lo=-100, hi=90)
    codes, scale = np.zeros((n, k), np.uint8), np.zeros((n, mx.pitch(k)), np.uint8)
    at = np.random.default_rng(9).integers(0, k, n)
    codes[np.arange(n), at], scale[np.arange(n), at // 32] = 6, 125      # 4 times 2^-2
    y = wq.gemm_mxfp4(packed(wq, codes, scale), packed(wq, xc, xs))
    assert np.array_equal(y.double().cpu().numpy(), mx.values(xc, xs)[:, at])
    assert wq.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cl, m, n, k", SPLIT)
def test_one_cta_a_tile_with_k_split(wq, cl, m, n, k):
    check_dense(wq, m, n, k)


@pytest.mark.gpu
@pytest.mark.parametrize("width, m, n, k", DENSE)
def test_pairs_with_several_tiles(wq, width, m, n, k):
    check_dense(wq, m, n, k)


@pytest.mark.gpu
@pytest.mark.parametrize("width, rows, experts, n, k", EXPERTS)
def test_experts_with_several_tiles(wq, width, rows, experts, n, k):
    counts = counts_of(rows, experts, rows + k)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    of = np.repeat(np.arange(experts), counts)
    codes, scale = weights(experts * n, k, n + k)
    pw, x = packed(wq, codes, scale), acts(rows, k, rows)
    xc, xs = mx.quantize(x.double().numpy())
    y = wq.gemm_experts_mxfp4(pw, x.cuda(), to_dev(off))
    xv, wv = mx.values(xc, xs), mx.values(codes, scale)
    for e in range(experts):
        check(y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]], wv[e * n:(e + 1) * n])
    px = packed(wq, xc, xs)
    for _ in range(3):
        assert torch.equal(y, wq.gemm_experts_mxfp4(pw, px, to_dev(off)))
    codes, scale = weights(experts * n, k, n + 1, lo=-100, hi=90)
    x, at = one_hot(rows, k, rows)
    y = wq.gemm_experts_mxfp4(packed(wq, codes, scale), x.cuda(), to_dev(off))
    v = mx.values(codes, scale).reshape(experts, n, k)
    assert np.array_equal(y.double().cpu().numpy(), v[of, :, at])
    assert wq.device_error() == 0
