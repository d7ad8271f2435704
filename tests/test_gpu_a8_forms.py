"""The 8-bit product in each of its forms, at sizes chosen for the form and asked of
the plan (and of the kernels that ran): shared K with wide tiles, CTA pairs of one
tile and of many, kept and streamed activations, results at the edge of every form."""
import re

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

Q8, E4M3 = 8, 3
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


def values(codes):
    """Codes as 64-bit numbers."""
    return codes.double() if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn).double()


def codes_of(rows, K, fmt, seed):
    if fmt == Q8:
        return torch.randint(-128, 128, (rows, K), generator=gen(seed), device="cuda", dtype=torch.int8)
    bits = torch.randint(0, 256, (rows, K), generator=gen(seed), device="cuda", dtype=torch.uint8)
    return torch.where((bits & 0x7F) == 0x7F, bits - 1, bits)          # no NaN codes


def operands(fmt, M, N, K, seed):
    xs = 0.5 + torch.rand(M, generator=gen(seed), device="cuda")
    ws = (0.5 + torch.rand(N, generator=gen(seed + 1), device="cuda")) * (2.0 ** -16)
    b = torch.randn(N, generator=gen(seed + 2), device="cuda")
    return codes_of(M, K, fmt, seed + 3), xs, codes_of(N, K, fmt, seed + 4), ws, b


def check_product(rtq, fmt, M, N, K, seed, dtypes=DTYPES):
    """Against 64 bits: three fp32 roundings (u of the value each) and the output
    type's; an e4m3 sum is off by at most 2^-23 of the running sum of magnitudes an addition."""
    xc, xs, wc, ws, b = operands(fmt, M, N, K, seed)
    xv, wv = values(xc), values(wc)
    scale = xs.double()[:, None] * ws.double()[None]
    y = (xv @ wv.t()) * scale
    slack = 2.5 * U * y.abs()
    if fmt == E4M3:
        slack += K * 2.0 ** -23 * (xv.abs() @ wv.abs().t()) * scale
    y += b.double()
    slack += U * y.abs()
    for dtype in dtypes:
        # guard bands on both sides of Y keep their bits
        buf = torch.full((M * N + 512,), 7.0, dtype=dtype, device="cuda")
        Y = buf[256:256 + M * N].view(M, N)
        rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b, Y=Y)
        info = torch.finfo(dtype)
        edge = slack + (0 if dtype == torch.float32 else info.eps / 2) * (y.abs() + slack) + info.tiny * info.eps
        assert bool(((Y.double() - y).abs() <= edge).all()), dtype
        assert bool((buf[:256] == 7).all()) and bool((buf[256 + M * N:] == 7).all())


def kernels(call):
    """Names of the product's kernels that `call` launches, as the profiler gives them:
    a8_qgemm_kernel<format, type of Y, pair, groups, split, kept>."""
    from torch.profiler import ProfilerActivity, profile
    call()
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [m.group(1) for m in (re.search(r"(a8_\w+_kernel<.*>)\(", e.name) for e in p.events()) if m]


def runs_as(rtq, fmt, M, N, K, dtype, want):
    xc, xs, wc, ws, b = operands(fmt, M, N, K, seed=1)
    Y = torch.empty(M, N, dtype=dtype, device="cuda")
    names = kernels(lambda: rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b, Y=Y))
    if not names:                                # no device profiler here
        return
    assert len(names) == 1 and names[0].endswith(want), names


# K shared by 2, 4 and 8 CTAs with tiles of every width from 32 to 128 rows: where the
# rows a rank adds (rows / split) are no multiple of the 16 that are sent at a time,
# its columns straddle what is sent
SPLITS = [(596, 261, 1696, 32, 2), (296, 130, 1312, 32, 4), (150, 139, 3600, 32, 8), (479, 513, 1984, 48, 2),
          (389, 257, 1424, 48, 4), (295, 130, 2624, 48, 8), (301, 273, 5680, 64, 8), (940, 517, 3312, 80, 2),
          (601, 388, 2320, 80, 4), (408, 261, 5728, 80, 8), (725, 919, 4528, 96, 2), (330, 387, 9024, 96, 8),
          (969, 771, 6320, 112, 2), (700, 554, 3360, 112, 4), (436, 389, 7952, 112, 8), (821, 1190, 9184, 128, 2),
          (792, 532, 5040, 128, 4), (485, 412, 10784, 128, 8)]


@pytest.mark.parametrize("M,N,K,rows,split", SPLITS)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_shared_k(rtq, fmt, M, N, K, rows, split):
    p = rtq.a8_plan(M, N, K, fmt)
    assert (p["rows"], p["split"]) == (rows, split)
    check_product(rtq, fmt, M, N, K, seed=M + N)


# CTA pairs: one tile each, and walks with the activations kept and streamed
PAIRS = [(256, 8192, 8192, False), (512, 4096, 8192, False), (9001, 2003, 640, False), (9000, 2050, 1280, False),
         (7003, 4100, 1040, True), (9000, 4096, 640, True), (9001, 2003, 592, True), (20000, 250, 1040, False)]


@pytest.mark.parametrize("M,N,K,kept", PAIRS)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_pairs(rtq, fmt, M, N, K, kept):
    p = rtq.a8_plan(M, N, K, fmt)
    assert p["pair"] and p["walk"]
    check_product(rtq, fmt, M, N, K, seed=M + N)
    runs_as(rtq, fmt, M, N, K, torch.bfloat16, f"true, 4, false, {str(kept).lower()}>")


@pytest.mark.parametrize("M,N,K,dtype,kept", [
    (65536, 2003, 400, torch.float32, False), (65536, 2003, 400, torch.bfloat16, False),   # ragged rows of Y
    (65536, 2003, 1040, torch.bfloat16, True), (65536, 2048, 400, torch.bfloat16, True),
    (65536, 2003, 512, torch.bfloat16, False), (65536, 4096, 512, torch.bfloat16, True),
    (65536, 4096, 512, torch.float32, False), (65536, 200, 272, torch.float32, False)])    # one weight tile
def test_activations_are_kept_where_that_is_faster(rtq, M, N, K, dtype, kept):
    assert rtq.a8_plan(M, N, K)["pair"]
    runs_as(rtq, Q8, M, N, K, dtype, f"true, 4, false, {str(kept).lower()}>")


# one form each: name, M, N, K
EDGES = [("cores", 3, 130, 512), ("cores", 80, 130, 512), ("narrow", 131, 130, 512), ("split", 150, 130, 2048),
         ("split", 295, 130, 2624), ("walk", 2500, 1000, 512), ("walk", 5001, 1003, 512),
         ("pair", 9001, 2003, 640), ("pair", 9001, 2051, 1280)]


def form(p):
    if p["cores"] or p["pair"]:
        return "cores" if p["cores"] else "pair"
    return "walk" if p["walk"] else "split" if p["split"] > 1 else "narrow"


@pytest.mark.parametrize("name,M,N,K", EDGES)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_only_results_that_exist_are_reported(rtq, fmt, name, M, N, K):
    """A bias beyond fp16 that the sums bring back into range: what a tile computes
    beyond the last row (0 + bias) is not an output.  And an output that is not
    finite is reported wherever it stands: last row, last column, both."""
    assert form(rtq.a8_plan(M, N, K, fmt)) == name
    if fmt == Q8:
        one, other, product = 100, -100, -1e4
        kind = torch.int8
    else:
        one, other, product = 0x58, 0xD8, -256.0     # 16 and -16
        kind = torch.uint8
    xc = torch.full((M, K), one, dtype=kind, device="cuda")
    wc = torch.full((N, K), other, dtype=kind, device="cuda")
    xs, ws = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    b = torch.full((N,), -product * K, device="cuda")
    assert float(b[0]) > 65504
    Y = rtq.qgemm_a8(fmt, xc, xs, wc, ws, bias=b, dtype=torch.float16)
    assert bool((Y == 0).all()) and rtq.device_status() == rtq.OK
    for m, n in ((M - 1, 0), (0, N - 1), (M - 1, N - 1)):
        x2, w2 = torch.zeros_like(xs), torch.zeros_like(ws)
        x2[m], w2[n] = 1, 1                      # one product alone, and no bias
        Y = rtq.qgemm_a8(fmt, xc, x2, wc, w2, dtype=torch.float16)
        assert rtq.device_status() == RANGE
        assert bool(Y[m, n].isinf()) and int(Y.isinf().sum()) == 1
