"""The MXFP4 operators as a benchmark: cases, inputs, plain forms and calls.

MXFP4 is the OCP microscaling format of 4-bit floating point: blocks of 32 consecutive values of a row share a power of
two 2^(s - 127) (an E8M0 byte s), each value is an E2M1 code (sign, two exponent bits, one mantissa bit). Operators:

  quantise  rows to MXFP4 and the values the codes stand for (fake quantisation of latents, coding of weights and
            activations);
  weights   y = x W^T for MXFP4 weights and bf16 activations (decode and prefill);
  product   y = x W^T for MXFP4 weights and bf16 activations that are coded as MXFP4 first;
  experts   the same for rows sorted by expert, each range of rows with its expert's weights.

Plain forms are elementary torch operations in 32 bits; exact() computes in 64 bits, apart from them.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # E2M1 magnitudes by code


def listed():
    return [
        # the activations of a decode batch in front of a projection (hidden size 4096): launch latency
        dict(name="quantise_decode", op="quantise", n=16, k=4096, dtype="bf16"),
        # one large projection coded offline: bandwidth
        dict(name="quantise_weight", op="quantise", n=8192, k=28672, dtype="bf16"),
        # a training step's latent weights, an odd number of rows and a row of 65 blocks
        dict(name="quantise_latent", op="quantise", n=8191, k=2080, dtype="fp32"),
        # decode of one token on a large projection: the weights' bytes
        dict(name="weights_decode", op="weights", m=1, n=8192, k=28672),
        # a small odd projection of a few tokens (ragged rows, a last block of 32)
        dict(name="weights_odd", op="weights", m=5, n=1003, k=2080),
        # prefill of a short prompt with bf16 activations
        dict(name="weights_prefill", op="weights", m=512, n=4096, k=11008),
        # one token through a coded product
        dict(name="product_token", op="product", m=1, n=4096, k=4096),
        # a ragged batch
        dict(name="product_odd", op="product", m=77, n=5003, k=2112),
        # prefill: the tensor cores' rate
        dict(name="product_prefill", op="product", m=4096, n=4096, k=11008),
        # mixture of experts, decode: 8 tokens of 4 experts each
        dict(name="experts_decode", op="experts", t=32, e=64, n=1408, k=2048, spread=1.0),
        # a ragged batch with empty experts and odd rows
        dict(name="experts_odd", op="experts", t=301, e=17, n=1003, k=1088, spread=2.0),
        # mixture of experts, prefill
        dict(name="experts_prefill", op="experts", t=8192, e=32, n=5632, k=2048, spread=0.5),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["quantise", "weights", "product", "experts"])
    if op == "quantise":
        n, k = size(1, 16384), 32 * size(1, 896)
        return dict(op=op, n=max(1, min(n, 8192 * 28672 // k)), k=k, dtype=rng.choice(["bf16", "fp32"]))
    if op == "weights":
        m = size(1, 512)
        return dict(op=op, m=m, n=size(16, 8192 if m <= 16 else 4096), k=(32 if m <= 16 else 64) * size(2, 172))
    if op == "product":
        return dict(op=op, m=size(1, 4096), n=size(16, 4096), k=64 * size(1, 172))
    return dict(op=op, t=size(1, 8192), e=size(2, 32), n=size(16, 5632), k=64 * size(1, 32),
                spread=round(rng.uniform(0.0, 2.0), 2))


# --- inputs --------------------------------------------------------------------------------

def _pow2(e):
    """2^e as fp32 for whole e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).to(torch.int32).view(torch.float32)


def _quantise(x):
    """Blocks of 32 of the rows of x: (signed E2M1 values fp32 [n, k/32, 32], exponents int32 [n, k/32])."""
    v = x.float().view(x.shape[0], -1, 32)
    top = v.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)             # floor(log2 top) - 2
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    v = v * _pow2(-e).unsqueeze(-1)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)                # round() takes ties to the even code
    return torch.copysign(q, v), e


def _pack(q):
    """Signed E2M1 values [n, blocks, 32] -> two codes a byte [n, k/2], the even column in the low half."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).view(q.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _weights(rows, k, gen):
    """A projection's weights, normal with a few outliers, coded: (packed [rows, k/2], scale bytes [rows, pitch]); the
    rows of scale bytes are padded to whole 16 bytes."""
    packed = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((rows, 16 * -(-k // 512)), dtype=torch.uint8, device="cuda")
    w = torch.randn((rows, k), generator=gen, device="cuda") * 0.02
    w *= torch.where(torch.rand((rows, k), generator=gen, device="cuda") < 0.001, 20.0, 1.0)
    q, e = _quantise(w.bfloat16())
    packed.copy_(_pack(q))
    scale[:, :k // 32] = (e + 127).to(torch.uint8)
    return packed, scale


def _activations(m, k, gen):
    """Hidden states: normal values, channels of unlike size."""
    x = torch.randn((m, k), generator=gen, device="cuda")
    return (x * torch.exp(0.5 * torch.randn((1, k), generator=gen, device="cuda"))).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantise":
        x = torch.randn((case["n"], case["k"]), generator=gen, device="cuda") * 0.02
        s["x"] = x if case["dtype"] == "fp32" else x.bfloat16()
        return s
    if case["op"] != "experts":
        s["packed"], s["scale"] = _weights(case["n"], case["k"], gen)
        s["x"] = _activations(case["m"], case["k"], gen)
        return s
    t, e = case["t"], case["e"]
    s["packed"], s["scale"] = _weights(e * case["n"], case["k"], gen)
    s["x"] = _activations(t, case["k"], gen)
    host = torch.Generator().manual_seed(seed)
    liked = torch.softmax(case["spread"] * torch.randn(e, generator=host), 0)
    count = torch.bincount(torch.multinomial(liked, t, replacement=True, generator=host), minlength=e)
    s["most"] = int(count.max())
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)]).to(torch.int32).cuda()
    return s


# --- one pass ------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return _plain(s)


def _own(s):
    import w4a16_matmul_b200 as wq

    if s["op"] == "quantise":
        q, coded = wq.fake_quant_mxfp4(s["x"], packed=True)
        return q, coded.aux[:, :s["k"] // 32]
    w = wq.PackedWeight(wq.FMT_MXFP4, 32, s["packed"].shape[0], s["k"], s["packed"], s["scale"])
    if s["op"] == "weights":
        return wq.gemv(w, s["x"]) if s["m"] <= 16 else wq.gemm(w, s["x"])
    if s["op"] == "product":
        return wq.gemm_mxfp4(w, s["x"])
    return wq.gemm_experts_mxfp4(w, s["x"], s["offsets"])


def _decode(packed, scale, k):
    """The values of packed codes, fp32 [rows, k]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=packed.device)
    v = grid[torch.stack([packed & 15, packed >> 4], -1).view(packed.shape[0], -1).int()]
    return (v.view(packed.shape[0], -1, 32) * _pow2(scale[:, :k // 32].int() - 127).unsqueeze(-1)).view(-1, k)


def _rounded(x):
    """x coded as MXFP4, as values in fp32."""
    q, e = _quantise(x)
    return (q * _pow2(e).unsqueeze(-1)).view(x.shape)


def _plain(s):
    if s["op"] == "quantise":
        q, e = _quantise(s["x"])
        return (q * _pow2(e).unsqueeze(-1)).view(s["x"].shape).to(s["x"].dtype), (e + 127).to(torch.uint8)
    w = _decode(s["packed"], s["scale"], s["k"])
    if s["op"] == "weights":
        return (s["x"].float() @ w.T).bfloat16()
    if s["op"] == "product":
        return (_rounded(s["x"]) @ w.T).bfloat16()
    t, off = s["t"], s["offsets"].long()
    rows = (off[:-1, None] + torch.arange(s["most"], device="cuda")).clamp(max=t - 1)
    y = torch.bmm(_rounded(s["x"])[rows], w.view(s["e"], s["n"], s["k"]).transpose(1, 2))
    at = torch.arange(t, device="cuda")
    e = torch.searchsorted(off, at, right=True) - 1
    return y[e, at - off[e]].bfloat16()


# --- 64 bits -------------------------------------------------------------------------------

def _nearest64(x):
    """MXFP4 of x by comparison with every level and every power of two: (values float64, scale bytes)."""
    v = x.double().view(x.shape[0], -1, 32)
    top = v.abs().amax(-1)
    powers = torch.tensor([2.0 ** p for p in range(-150, 129)], dtype=torch.float64, device=x.device)
    e = (torch.bucketize(top, powers, right=True) - 151 - 2).clamp(-127, 127)
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), e.double())
    a = (v / scale.unsqueeze(-1)).abs()
    code = torch.zeros(a.shape, dtype=torch.int8, device=x.device)
    for j in range(7):
        middle = (GRID[j] + GRID[j + 1]) / 2
        code += (a >= middle) if j % 2 else (a > middle)             # a tie goes to the even code
    level = torch.tensor(GRID, dtype=torch.float64, device=x.device)[code.int()]
    return (torch.where(v < 0, -level, level) * scale.unsqueeze(-1)).view(x.shape), (e + 127).to(torch.uint8)


def _values64(packed, scale, k):
    out = torch.empty((packed.shape[0], k), dtype=torch.float64, device=packed.device)
    for half in range(2):
        c = (packed >> (4 * half)) & 15
        ex, m = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(ex == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.pow(2.0, ex.double() - 1))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    s = torch.pow(2.0, scale[:, :k // 32].double() - 127)
    return (out.view(packed.shape[0], -1, 32) * s.unsqueeze(-1)).view(-1, k)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        return _nearest64(s["x"])
    w = _values64(s["packed"], s["scale"], case["k"])
    x = s["x"].double() if case["op"] == "weights" else _nearest64(s["x"])[0]
    if case["op"] != "experts":
        return x @ w.T
    y = torch.zeros((case["t"], case["n"]), dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist()
    for e in range(case["e"]):
        y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w[e * case["n"]:(e + 1) * case["n"]].T
    return y


# --- what a pass cannot do without ---------------------------------------------------------

def work(case):
    k = case["k"]
    code = k / 2 + k / 32                                            # bytes of a coded row
    if case["op"] == "quantise":
        held = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=case["n"] * (2 * held * k + code), flops=10 * case["n"] * k)
    if case["op"] != "experts":
        m, n = case["m"], case["n"]
        return dict(bytes=n * code + 2 * m * (k + n), flops=2 * m * n * k)
    t, e, n = case["t"], case["e"], case["n"]
    met = e * (1 - (1 - 1 / e) ** t)                                 # experts that have rows, were all liked alike
    return dict(bytes=met * n * code + 2 * t * (k + n), flops=2 * t * n * k)
