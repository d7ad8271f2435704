"""8-bit activations on a GPU: quantization, residual norm, gated SiLU and the
8-bit product, each against its formula in 64 bits.

Tolerances count roundings (a rounding to fp32 is off by at most u = 2^-24 of
the value, to bf16 2^-8, to fp16 2^-11):
  - codes lie within half a step of the exact value over the returned scale, to
    which the fp32 arithmetic before the rounding adds `rel` of the row's maximum;
  - int8 sums are exact; the result takes three fp32 roundings and one to Y's type;
  - an e4m3 product of two codes is exact in fp32, and each of the K additions
    is off by at most 2^-23 of the running sum of magnitudes (rounded or cut).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

Q8, E4M3 = 8, 3
TOP = {Q8: 127.0, E4M3: 448.0}
U = 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
RANGE = 9                                        # RT_ERR_OPERAND_RANGE


@pytest.fixture(scope="module", autouse=True)
def rtq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from int8_dequant_gemm_b200 import build
    build.build()
    import int8_dequant_gemm_b200 as r
    r.lib()
    assert r.device_status() == r.OK
    yield r
    torch.cuda.synchronize()
    assert r.device_status() == r.OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


def values(codes):
    """Codes as 64-bit numbers."""
    return codes.double() if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn).double()


def half_step(t, fmt):
    """Half the distance of neighbouring codes at |t|."""
    if fmt == Q8:
        return torch.full_like(t, 0.5)
    return torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 4)


def check_rows(fmt, codes, scales, y, rel):
    """codes * scales are the rows of y in 8 bits, y known to `rel` of its row's maximum."""
    y = y.double()
    top = y.abs().amax(dim=1)
    s = scales.double()
    assert bool(((s - top / TOP[fmt]).abs() <= (rel + 2 * U) * top / TOP[fmt]).all())
    live = s > 0
    assert bool((codes[~live].to(torch.int32) == 0).all()) and bool((top[~live] == 0).all())
    y, s, top, c = y[live], s[live][:, None], top[live][:, None], values(codes[live])
    edge = half_step(y.abs() * (1 + rel) / s, fmt) * s + (rel + 4 * U) * top
    assert bool(((c * s - y).abs() <= edge).all())


def rows_of(M, K, seed, dtype):
    """Rows of mixed size with a few large channels, a zero row among them."""
    x = randn(M, K, seed=seed) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=gen(seed + 1), device="cuda").float())
    x[:, :: max(1, K // 5)] *= 8
    if M > 2:
        x[M // 2] = 0
    return x.to(dtype)


# one token, odd row counts, every group width of the row kernels in 4-byte and 2-byte types
ROWS = [(1, 512), (1, 16), (3, 128), (7, 256), (80, 512), (131, 528), (33, 2048), (9, 1040),
        (5, 4096), (2, 8208), (3, 16384), (2, 16400), (2, 32768)]


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize(rtq, M, K, dtype):
    x = rows_of(M, K, 10 + K, dtype)
    c, s = rtq.quantize_a8(x, Q8)
    hc, hs = rtq.quantize_q8_row(x.float().cpu().numpy())
    assert np.array_equal(c.cpu().numpy(), hc) and np.array_equal(s.cpu().numpy(), hs)
    c, s = rtq.quantize_a8(x, E4M3)
    check_rows(E4M3, c, s, x, 0.0)


def test_quantize_borders_and_extremes(rtq):
    """Values on rounding borders, at both ends of fp32 and in its subnormals:
    the host quantizer's bits."""
    K = 64
    base = np.zeros((9, K), np.float32)
    half = np.float32(0.5)
    for i, top in enumerate((127.0, 254.0, 63.5, 1.0, 3.0e38, 1e-30, 1e-38, 1e-42, 1e-45)):
        t = np.float32(top)
        base[i, 0] = t
        k = np.arange(1, K, dtype=np.float32)
        base[i, 1:] = (k + half) * (t / np.float32(127)) * np.where(k % 2 == 0, 1, -1)
    base[3, 1:] = np.nextafter(base[3, 1:], np.float32(np.inf))
    c, s = rtq.quantize_a8(torch.from_numpy(base).cuda(), Q8)
    hc, hs = rtq.quantize_q8_row(base)
    assert np.array_equal(s.cpu().numpy(), hs)
    assert np.array_equal(c.cpu().numpy(), hc)
    x = torch.from_numpy(base[:6]).cuda()
    check_rows(E4M3, *rtq.quantize_a8(x, E4M3), x, 0.0)


# scale: h and h * g are rounded (2 u), the sum of squares runs over at most
# 32 values a thread and 10 levels (45 u, halved by the root), then the root,
# two quotients and a product: below 32 u
NORM_REL = 32 * U


def norm64(x, r, g, eps):
    h = x.double() + (0 if r is None else r.double())
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + eps)
    return h, y if g is None else y * g.double()


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_addnorm(rtq, M, K, dtype, fmt):
    x, r = rows_of(M, K, 20 + K, dtype), randn(M, K, seed=21, dtype=dtype)
    if M > 2:
        r[M // 2] = 0                             # a row of zeros
    g = 1 + 0.3 * randn(K, seed=22)
    c, s, h = rtq.addnorm_a8(x, g, fmt, residual=r, eps=1e-5)
    h64, y = norm64(x, r, g, 1e-5)
    check_rows(fmt, c, s, y, NORM_REL)
    assert torch.equal(h, (x.float() + r.float()).to(dtype))
    c2, s2, none = rtq.addnorm_a8(x, None, fmt)
    assert none is None
    check_rows(fmt, c2, s2, norm64(x, None, None, 1e-6)[1], NORM_REL)


@pytest.mark.parametrize("target", ["x", "residual"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_addnorm_in_place(rtq, dtype, target):
    M, K = 37, 1040
    x, r, g = randn(M, K, seed=1, dtype=dtype), randn(M, K, seed=2, dtype=dtype), randn(K, seed=3)
    want = rtq.addnorm_a8(x, g, Q8, residual=r)
    x2, r2 = x.clone(), r.clone()
    got = rtq.addnorm_a8(x2, g, Q8, residual=r2, H=x2 if target == "x" else r2)
    assert got[2] is (x2 if target == "x" else r2)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert torch.equal(r2 if target == "x" else x2, r if target == "x" else x)


def test_addnorm_range(rtq):
    """Rows whose squares leave fp32, whose values are tiny, and mixtures of
    both in one block: the norm is of the row's shape, not its size."""
    for K in (64, 512, 1024, 2048):
        x = randn(40, K, seed=K)
        size = torch.tensor([1.0, 1e30, 3e37, 1e-25, 1e-30], device="cuda").repeat(8)[:, None]
        # a power of two near each size, so that the scaled rows are exact
        size = torch.exp2(torch.round(torch.log2(size.double()))).float()
        g = 1 + 0.1 * randn(K, seed=5)
        for fmt in (Q8, E4M3):
            c, s, _ = rtq.addnorm_a8(x * size, g, fmt, eps=2e-38)
            check_rows(fmt, c, s, norm64(x * size, None, g, float(np.float32(2e-38)))[1], NORM_REL)
    big = torch.full((2, 64), 1e30, device="cuda")
    c, s, _ = rtq.addnorm_a8(big, torch.full((64,), 1e10, device="cuda"), Q8)
    check_rows(Q8, c, s, norm64(big, None, torch.full((64,), 1e10, device="cuda"), 1e-6)[1], NORM_REL)


def gate_rel(a):
    """exp is documented to 2 + 1.173 |a| units of 2^-23, its quotient to 2 units, then a product."""
    return (2 + 1.173 * float(a.abs().max()) + 2 + 1) * 2.0 ** -23


@pytest.mark.parametrize("M,F", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_gate(rtq, M, F, dtype, fmt):
    u = randn(M, 2 * F, seed=30 + F, dtype=dtype)
    u[:, : F : 7] *= 6
    if M > 2:
        u[M // 2, F:] = 0
    c, s = rtq.gate_a8(u, fmt)
    a, b = u.double().chunk(2, dim=1)
    check_rows(fmt, c, s, a * torch.sigmoid(a) * b, gate_rel(a))


def test_gate_far_values(rtq):
    a = torch.tensor([-200.0, -90.0, -60.0, -1.0, 0.0, 1.0, 60.0, 90.0] * 2, device="cuda")
    for row in (a, a[:4].repeat(4), torch.full_like(a, -60.0)):
        u = torch.cat([row, torch.linspace(-3, 3, 16, device="cuda")])[None]
        c, s = rtq.gate_a8(u, Q8)
        x, b = u.double().chunk(2, dim=1)
        check_rows(Q8, c, s, x * torch.sigmoid(x) * b, gate_rel(x))


@pytest.mark.parametrize("fmt", [Q8, E4M3])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("K", [64, 512, 1040, 4096])
def test_rows_that_are_not_finite(rtq, fmt, bad, K):
    """Such a row gets scale NaN and zero codes, the others their usual bits;
    the product then gives NaN for that row alone."""
    M, hit = 21, (3, 20)
    x = randn(M, K, seed=K)
    spoiled = x.clone()
    spoiled[hit[0], K - 1] = bad
    spoiled[hit[1], 0] = bad
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[list(hit)] = False
    u, us = torch.cat([x, x], 1), torch.cat([spoiled, x], 1)
    pairs = [(rtq.quantize_a8(x, fmt), rtq.quantize_a8(spoiled, fmt)),
             (rtq.addnorm_a8(x, None, fmt), rtq.addnorm_a8(spoiled, None, fmt)),
             (rtq.addnorm_a8(x, None, fmt, residual=x), rtq.addnorm_a8(x, None, fmt, residual=spoiled)),
             (rtq.gate_a8(u, fmt), rtq.gate_a8(us, fmt))]
    assert rtq.device_status() == RANGE
    for want, got in pairs:
        assert torch.equal(want[0][keep], got[0][keep]) and torch.equal(want[1][keep], got[1][keep])
        assert bool(got[1][~keep].isnan().all()) and bool((got[0][~keep].to(torch.int32) == 0).all())
    c, s = pairs[0][1]
    w, ws = rtq.quantize_a8(randn(40, K, seed=9), fmt)
    y = rtq.qgemm_a8(fmt, c, s, w, ws)
    assert rtq.device_status() == RANGE
    assert bool(y[~keep].isnan().all()) and bool(y[keep].isfinite().all())


@pytest.mark.parametrize("fmt", [Q8, E4M3])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dequant(rtq, fmt, dtype):
    for M, K in ((1, 16), (3, 528), (257, 2048)):
        c, s = rtq.quantize_a8(rows_of(M, K, 40, torch.float32), fmt)
        got = rtq.dequant_a8(fmt, c, s, dtype=dtype)
        assert torch.equal(got, (values(c).float() * s[:, None]).to(dtype))


# ---------------------------------------------------------------- the product
def codes_of(rows, K, fmt, seed):
    g = gen(seed)
    if fmt == Q8:
        return torch.randint(-128, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    bits = torch.randint(0, 256, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
    return torch.where((bits & 0x7F) == 0x7F, bits - 1, bits)          # no NaN codes


def product64(fmt, xc, xs, wc, ws, bias):
    """The product and the bound of its error before the rounding to Y's type."""
    xv, wv = values(xc), values(wc)
    K = xc.shape[1]
    scale = xs.double()[:, None] * (1 if ws is None else ws.double()[None])
    y = (xv @ wv.t()) * scale
    slack = 2.5 * U * y.abs()
    if fmt == E4M3:
        slack = slack + K * 2.0 ** -23 * (xv.abs() @ wv.abs().t()) * scale.abs()
    if bias is not None:
        y = y + bias.double()
    return y, slack + U * y.abs()


def check_product(Y, y, slack):
    info = torch.finfo(Y.dtype)
    edge = slack + (0 if Y.dtype == torch.float32 else info.eps / 2) * (y.abs() + slack) + info.tiny * info.eps
    assert Y.shape == y.shape and bool(((Y.double() - y).abs() <= edge).all())


def operands(fmt, M, N, K, seed, bias=True):
    xs = 0.5 + torch.rand(M, generator=gen(seed), device="cuda")
    ws = (0.5 + torch.rand(N, generator=gen(seed + 1), device="cuda")) * (2.0 ** -16)
    b = randn(N, seed=seed + 2) if bias else None
    return codes_of(M, K, fmt, seed + 3), xs, codes_of(N, K, fmt, seed + 4), ws, b


SIZES = [(1, 1, 16), (1, 4096, 512), (2, 7, 32), (15, 130, 144), (16, 128, 128), (17, 300, 272),
         (77, 200, 144), (80, 512, 2048), (80, 512, 512), (80, 2048, 512), (127, 1000, 400),
         (128, 129, 4112), (129, 300, 272), (130, 1, 16), (200, 2048, 512), (256, 256, 1024),
         (257, 513, 640), (300, 512, 2048), (513, 384, 128), (1000, 1003, 1040), (1024, 4096, 512),
         (2049, 512, 2064), (4096, 512, 512), (2500, 1000, 512), (3001, 2000, 400),
         (5003, 1003, 1040), (4100, 2200, 2048), (9000, 515, 256), (9, 5000, 2048), (520, 4999, 1024),
         (3, 4097, 512), (4, 131, 8208), (5, 512, 2048), (8, 515, 528), (8, 4100, 4096), (2, 6001, 1040), (6000, 2000, 400), (9000, 2048, 640),
         (9001, 2003, 1040), (7001, 2050, 512)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_product(rtq, M, N, K, fmt):
    xc, xs, wc, ws, b = operands(fmt, M, N, K, seed=M + N + K)
    y, slack = product64(fmt, xc, xs, wc, ws, b)
    for dtype in DTYPES:
        # guard bands on both sides of Y keep their bits
        buf = torch.full((M * N + 512,), 7.0, dtype=dtype, device="cuda")
        Y = buf[256:256 + M * N].view(M, N)
        rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b, Y=Y)
        check_product(Y, y, slack)
        assert bool((buf[:256] == 7).all()) and bool((buf[256 + M * N:] == 7).all())
    y, slack = product64(fmt, xc, xs, wc, ws, None)
    check_product(rtq.qgemm_a8(fmt, xc, xs, wc, ws), y, slack)


def test_product_sizes_take_every_plan(rtq):
    for fmt in (Q8, E4M3):
        plans = [rtq.a8_plan(*n, fmt) for n in SIZES]
        assert any(p["cores"] for p in plans) and {p["split"] for p in plans} >= {1, 2, 4, 8}
        assert any(not (p["walk"] or p["cores"]) and p["split"] == 1 for p in plans)
        assert any(p["walk"] and p["pair"] for p in plans)
        assert any(p["walk"] and not p["pair"] for p in plans)


@pytest.mark.parametrize("fmt", [Q8, E4M3])
@pytest.mark.parametrize("M", [128, 640])
def test_product_of_identity_codes(rtq, fmt, M):
    """One activation code a row picks one column of the weights: every code's
    value and place, bit for bit."""
    K = M
    one = 1 if fmt == Q8 else 0x38                # e4m3 1.0
    xc = torch.zeros(M, K, dtype=torch.int8 if fmt == Q8 else torch.uint8, device="cuda")
    xc.fill_diagonal_(one)
    wc = codes_of(256, K, fmt, seed=3)
    ones = torch.ones(max(M, 256), device="cuda")
    Y = rtq.qgemm_a8(fmt, xc, ones[:M].contiguous(), wc, ones[:256].contiguous())
    assert torch.equal(Y.double(), values(wc).t())


def test_int8_sum_is_exact_at_its_largest(rtq):
    """-128 * -128 over the longest K the call takes stays inside int32."""
    K = 131056
    for M, N in ((1, 3), (300, 130)):
        xc = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        wc = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        wc[-1] = 127
        one = torch.ones(max(M, N), device="cuda")
        Y = rtq.qgemm_a8(Q8, xc, one[:M].contiguous(), wc, one[:N].contiguous())
        assert float(Y[0, 0]) == float(np.float32(128 * 128 * K))
        assert float(Y[M - 1, N - 1]) == float(np.float32(-128 * 127 * K))


def test_e4m3_weights_without_scales(rtq):
    xc, xs, wc, _, b = operands(E4M3, 90, 200, 512, seed=5)
    xs = xs * 2.0 ** -16
    check_product(rtq.qgemm_a8(E4M3, xc, xs, wc, bias=b), *product64(E4M3, xc, xs, wc, None, b))


def test_int8_rows_do_not_depend_on_the_call(rtq):
    xc, xs, wc, ws, b = operands(Q8, 2500, 700, 1040, seed=6)
    Y = rtq.qgemm_a8(Q8, xc, xs, wc, ws, bias=b)
    for lo, hi in ((0, 1), (7, 90), (100, 400), (1000, 2500)):
        assert torch.equal(rtq.qgemm_a8(Q8, xc[lo:hi].contiguous(), xs[lo:hi].contiguous(), wc, ws, bias=b), Y[lo:hi])


@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_product_repeats_its_bits(rtq, fmt):
    for M, N, K in ((80, 512, 2048), (1000, 1003, 1040)):
        a = operands(fmt, M, N, K, seed=8)
        first = rtq.qgemm_a8(fmt, *a[:4], bias=a[4])
        for _ in range(3):
            assert torch.equal(rtq.qgemm_a8(fmt, *a[:4], bias=a[4]), first)


def test_results_beyond_the_output_type_are_reported(rtq):
    xc, xs, wc, ws, _ = operands(Q8, 33, 40, 512, seed=9)
    rtq.qgemm_a8(Q8, xc, xs, wc, ws, dtype=torch.float16)
    assert rtq.device_status() == rtq.OK
    Y = rtq.qgemm_a8(Q8, xc, xs * 1e8, wc, ws, dtype=torch.float16)
    assert bool(Y.isinf().any()) and rtq.device_status() == RANGE
    rtq.qgemm_a8(Q8, xc, xs * 1e8, wc, ws)
    assert rtq.device_status() == rtq.OK


@pytest.mark.parametrize("M,N,K", [(80, 130, 512), (80, 130, 2048), (2500, 1000, 512), (5003, 1003, 1040), (3, 130, 512)])
def test_only_results_that_exist_are_reported(rtq, M, N, K):
    """A bias beyond fp16 that the sums bring back into range: what a tile computes
    beyond the last row (0 + bias) is not an output."""
    xc = torch.full((M, K), 100, dtype=torch.int8, device="cuda")
    wc = torch.full((N, K), -100, dtype=torch.int8, device="cuda")
    one = torch.ones(max(M, N), device="cuda")
    b = torch.full((N,), 1e4 * K, device="cuda")
    Y = rtq.qgemm_a8(Q8, xc, one[:M].contiguous(), wc, one[:N].contiguous(), bias=b, dtype=torch.float16)
    assert bool((Y == 0).all()) and rtq.device_status() == rtq.OK


def test_offsets_beyond_32_bits(rtq):
    """Y and X of more than 2^31 elements, checked on the first, middle and last rows."""
    M, N, K = 600_000, 4096, 32
    xc, xs, wc, ws, b = operands(Q8, M, N, K, seed=11)
    Y = rtq.qgemm_a8(Q8, xc, xs, wc, ws, bias=b, dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, M // 2, 524_287, 524_288, M - 2, M - 1], device="cuda")
    check_product(Y[rows], *product64(Q8, xc[rows], xs[rows], wc, ws, b))
    del Y
    M, K = 300_000, 8192
    x = torch.randn(M, K, generator=gen(12), device="cuda", dtype=torch.float16)
    rows = torch.tensor([0, M // 2, 262_143, 262_144, M - 1], device="cuda")
    c, s, h = rtq.addnorm_a8(x, None, Q8, residual=x)
    check_rows(Q8, c[rows], s[rows], norm64(x[rows], x[rows], None, 1e-6)[1], NORM_REL)
    assert torch.equal(h[rows], x[rows] * 2)
    got = rtq.dequant_a8(Q8, c, s, out=h)
    assert torch.equal(got[rows], (values(c[rows]).float() * s[rows][:, None]).half())


# --------------------------------------------------------- used together
def feed_forward(rtq, fmt, x, r, g, w13, w2, dtype):
    c, s, h = rtq.addnorm_a8(x, g, fmt, residual=r)
    u = rtq.qgemm_a8(fmt, c, s, *w13, dtype=dtype)
    c2, s2 = rtq.gate_a8(u, fmt)
    return (c, s, h), u, (c2, s2), rtq.qgemm_a8(fmt, c2, s2, *w2, dtype=dtype)


@pytest.mark.parametrize("fmt", [Q8, E4M3])
@pytest.mark.parametrize("M", [1, 80, 1000])
def test_feed_forward_from_device_made_weights(rtq, fmt, M):
    """Norm, w1|w3, gate and w2 in one stream, weights quantized on the device
    just before; each stage against 64 bits from the codes it was given."""
    d, f = 512, 2048
    x, r, g = randn(M, d, seed=1), randn(M, d, seed=2), 1 + 0.1 * randn(d, seed=3)
    w13 = rtq.quantize_a8(randn(2 * f, d, seed=4) * d ** -0.5, fmt)
    w2 = rtq.quantize_a8(randn(d, f, seed=5) * f ** -0.5, fmt)
    for dtype in DTYPES:
        (c, s, h), u, (c2, s2), y = feed_forward(rtq, fmt, x.to(dtype), r.to(dtype), g, w13, w2, dtype)
        check_rows(fmt, c, s, norm64(x.to(dtype), r.to(dtype), g, 1e-6)[1], NORM_REL)
        check_product(u, *product64(fmt, c, s, *w13, None))
        a, b = u.double().chunk(2, dim=1)
        check_rows(fmt, c2, s2, a * torch.sigmoid(a) * b, gate_rel(a))
        check_product(y, *product64(fmt, c2, s2, *w2, None))


def test_device_made_weights_serve_the_weight_only_product(rtq):
    """quantize_a8's int8 rows are q8 weights: used at once by rt_qgemm_q8, with
    one of these operators in between, they give the host quantizer's results."""
    w, x = randn(512, 2048, seed=1), randn(300, 2048, seed=2)
    hc, hs = rtq.quantize_q8_row(w.cpu().numpy())
    want = rtq.qgemm_q8(x, torch.from_numpy(hc).cuda(), torch.from_numpy(hs).cuda())
    for _ in range(20):
        c, s = rtq.quantize_a8(w, Q8)
        a = rtq.quantize_a8(x, Q8)
        rtq.qgemm_a8(Q8, *a, *a)
        assert torch.equal(rtq.qgemm_q8(x, c, s), want)
        c.zero_(), s.zero_()


@pytest.mark.parametrize("M", [16, 600])
def test_captured_and_replayed(rtq, M):
    """Two graphs of the whole run, replayed on two streams at once with new
    inputs, give the eager calls' bits."""
    d, f, fmt = 256, 1024, Q8
    w13 = rtq.quantize_a8(randn(2 * f, d, seed=4), fmt)
    w2 = rtq.quantize_a8(randn(d, f, seed=5), fmt)
    g = randn(d, seed=6)
    sets = []
    for i in range(2):
        x, r = randn(M, d, seed=10 + i), randn(M, d, seed=20 + i)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            feed_forward(rtq, fmt, x, r, g, w13, w2, torch.float32)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = feed_forward(rtq, fmt, x, r, g, w13, w2, torch.float32)
        sets.append((x, r, stream, graph, out))
    for turn in range(3):
        for i, (x, r, stream, graph, out) in enumerate(sets):
            x.copy_(randn(M, d, seed=100 + 10 * turn + i))
            r.copy_(randn(M, d, seed=200 + 10 * turn + i))
        torch.cuda.synchronize()
        for x, r, stream, graph, out in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for x, r, stream, graph, out in sets:
            want = feed_forward(rtq, fmt, x, r, g, w13, w2, torch.float32)
            for a, b in zip((*want[0], want[1], *want[2], want[3]), (*out[0], out[1], *out[2], out[3])):
                assert torch.equal(a, b)


def test_explicit_stream_and_one_buffer_reused(rtq):
    """Calls on a stream that is not the current one, each overwriting what the
    one before still reads: stream order holds between overlapping launches."""
    s = torch.cuda.Stream()
    xs = [randn(700, 512, seed=i) for i in range(6)]
    w, ws = rtq.quantize_a8(randn(300, 512, seed=50), Q8)
    want = [rtq.qgemm_a8(Q8, *rtq.quantize_a8(x, Q8), w, ws) for x in xs]
    c, sc = rtq.quantize_a8(xs[0], Q8)
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for x in xs:
            rtq.quantize_a8(x, Q8, codes=c, scales=sc, stream=s)
            got.append(rtq.qgemm_a8(Q8, c, sc, w, ws, Y=torch.empty(700, 300, device="cuda"), stream=s))
        s.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(128, 129, 4112), (100, 30000, 128), (2500, 1000, 512), (5003, 1003, 1040),
                                   (4100, 2200, 2048), (9000, 2048, 640)])
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_injected_missing_box_times_out_and_recovers(rtq, M, N, K, fmt):
    xc, xs, wc, ws, b = operands(fmt, M, N, K, seed=13)
    want = rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b)
    rtq.debug_inject(1, 2_000_000)
    try:
        rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b)
        assert rtq.device_status() == rtq.RT_ERR_DEVICE_TIMEOUT
    finally:
        rtq.debug_inject(0, 0)
    assert rtq.device_status() == rtq.OK
    assert torch.equal(rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b), want)


# ------------------------------------------------------------------ refusals
def test_helpers_refuse(rtq):
    x = randn(8, 64)
    c, s = rtq.quantize_a8(x)
    w, ws = rtq.quantize_a8(randn(24, 64, seed=1))
    with pytest.raises(TypeError, match="float32"):
        rtq.quantize_a8(x.double())
    with pytest.raises(ValueError, match="2-D"):
        rtq.quantize_a8(x[0])
    with pytest.raises(ValueError, match="contiguous"):
        rtq.quantize_a8(randn(64, 8).t())
    with pytest.raises(ValueError, match="contiguous"):
        rtq.gate_a8(randn(8, 256)[:, :128])
    with pytest.raises(ValueError, match="halves"):
        rtq.gate_a8(randn(8, 33))
    with pytest.raises(ValueError, match="shape"):
        rtq.quantize_a8(x, codes=c[:4].contiguous())
    with pytest.raises(TypeError, match="int8"):
        rtq.quantize_a8(x, codes=c.view(torch.uint8))
    with pytest.raises(TypeError, match="residual"):
        rtq.addnorm_a8(x, residual=x.half())
    with pytest.raises(ValueError, match="gain"):
        rtq.addnorm_a8(x, randn(32))
    with pytest.raises(TypeError, match="CUDA"):
        rtq.addnorm_a8(x, torch.ones(64))
    with pytest.raises(rtq.RtqError, match="unsupported shape"):
        rtq.quantize_a8(randn(4, 24))
    with pytest.raises(rtq.RtqError, match="misaligned"):
        rtq.quantize_a8(randn(8 * 64 + 1)[1:].view(8, 64))
    with pytest.raises(rtq.RtqError, match="invalid"):
        rtq.addnorm_a8(x, eps=0.0)
    with pytest.raises(TypeError, match="scales"):
        rtq.qgemm_a8(Q8, c, s, w)
    with pytest.raises(ValueError, match="Wq has shape"):
        rtq.qgemm_a8(Q8, c, s, w[:, :32].contiguous(), ws)
    with pytest.raises(ValueError, match="x_scales"):
        rtq.qgemm_a8(Q8, c, s[:4], w, ws)
    with pytest.raises(TypeError, match="dtype"):
        rtq.qgemm_a8(Q8, c, s, w, ws, Y=randn(8, 24), dtype=torch.float16)
    with pytest.raises(TypeError, match="int8|uint8"):
        rtq.qgemm_a8(E4M3, c, s, w, ws)
    with pytest.raises(rtq.RtqError, match="invalid"):
        big = torch.empty(8 * 64 * 4, dtype=torch.uint8, device="cuda")
        rtq.dequant_a8(Q8, big[:512].view(torch.int8).view(8, 64), s, out=big.view(torch.float32).view(8, 64))


def test_no_rows(rtq):
    x = randn(0, 64)
    c, s = rtq.quantize_a8(x)
    w, ws = rtq.quantize_a8(randn(24, 64))
    assert rtq.qgemm_a8(Q8, c, s, w, ws).shape == (0, 24)
    assert rtq.addnorm_a8(x, residual=x)[0].shape == (0, 64)
    assert rtq.gate_a8(randn(0, 128))[0].shape == (0, 64)
    assert rtq.dequant_a8(Q8, c, s).shape == (0, 64)
