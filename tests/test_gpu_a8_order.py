"""8-bit rows and the calls around them in stream order: weights made by
quantize_a8 in the launch just before the product that reads them, on every kernel of the
weight-only products, each turn's weights in the buffers of the last.  Results
are the bits of the same product from weights that were complete long before."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

Q8, E4M3 = 8, 3
TURNS = 6


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


def randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.fixture(scope="module")
def busy():
    """Work that keeps the GPU long enough for the launches behind it to queue up."""
    t = torch.zeros(1 << 28, device="cuda")
    return lambda: t.mul_(1.0)


def turns(rtq, fmt, N, K, product, busy, want):
    """product(codes, scales) right behind quantize_a8, against want(codes, scales)."""
    ws = [randn(N, K, seed=i) for i in range(TURNS)]
    done = [rtq.quantize_a8(w, fmt) for w in ws]
    torch.cuda.synchronize()
    expected = []
    for c, s in done:
        expected.append(want(c, s))
        torch.cuda.synchronize()
    c, s = torch.empty_like(done[0][0]), torch.empty_like(done[0][1])
    got = []
    busy()
    for w in ws:
        rtq.quantize_a8(w, fmt, codes=c, scales=s)
        got.append(product(c, s))
    torch.cuda.synchronize()
    for a, b in zip(expected, got):
        assert torch.equal(a, b)


KERNELS = [(1, 4096, 512, "simt"), (80, 4096, 512, "tc_w_stationary"), (300, 4096, 512, "tc_x_resident"),
           (3000, 4096, 512, "tc_x_resident"), (300, 512, 2048, "tc_w_streamed"),
           (16384, 4096, 512, "tc_x_resident_pair")]


@pytest.mark.parametrize("M,N,K,kernel", KERNELS)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_weight_only_products(rtq, busy, M, N, K, kernel, fmt):
    assert rtq.plan(fmt, M, N, K) == kernel
    x = randn(M, K, seed=90)
    Y = [torch.empty(M, N, device="cuda") for _ in range(TURNS)]
    rtq.workspace_reserve(rtq.workspace_bytes(fmt, M, N, K))
    turn = iter(range(TURNS))

    def product(c, s, out=None):
        return rtq.qgemm(fmt, x, c, s if fmt == Q8 else None, Y=out if out is not None else Y[next(turn)])

    turns(rtq, fmt, N, K, product, busy, lambda c, s: product(c, s, torch.empty(M, N, device="cuda")))


@pytest.mark.parametrize("M,N,K,kernel", KERNELS)
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_weight_only_products_captured(rtq, M, N, K, kernel, fmt):
    """The same pair of launches twice in one graph, from two weights into one buffer of
    codes, replayed back to back."""
    assert rtq.plan(fmt, M, N, K) == kernel
    x, ws = randn(M, K, seed=90), [randn(N, K, seed=i) for i in range(2)]
    want = []
    for w in ws:
        c, s = rtq.quantize_a8(w, fmt)
        torch.cuda.synchronize()
        want.append(rtq.qgemm(fmt, x, c, s if fmt == Q8 else None))
    Y = [torch.empty(M, N, device="cuda") for _ in ws]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    rtq.workspace_reserve(rtq.workspace_bytes(fmt, M, N, K), stream=stream)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for w, y in zip(ws, Y):
            rtq.quantize_a8(w, fmt, codes=c, scales=s)
            rtq.qgemm(fmt, x, c, s if fmt == Q8 else None, Y=y)
    for _ in range(5):
        for y in Y:
            y.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for y, v in zip(Y, want):
            assert torch.equal(y, v)


@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_list_launch(rtq, busy, fmt):
    """The first entry's weights are the fresh ones, the others' old."""
    M, N, K = 80, 2048, 512
    x, x2 = randn(M, K, seed=90), randn(M, 2048, seed=91)
    old = rtq.quantize_a8(randn(512, 2048, seed=92), fmt)
    Y = [torch.empty(M, N, device="cuda") for _ in range(TURNS)]
    Y2 = [torch.empty(M, 512, device="cuda") for _ in range(47)]
    turn = iter(range(TURNS))

    def product(c, s, out=None):
        out = out if out is not None else Y[next(turn)]
        q8 = fmt == Q8
        projs = [rtq.Proj(fmt, x, c, s if q8 else None, out)]
        projs += [rtq.Proj(fmt, x2, old[0], old[1] if q8 else None, y) for y in Y2]
        assert rtq.batch_plan(projs) == "tc_list"
        rtq.qgemm_batch(projs)
        return out

    turns(rtq, fmt, N, K, product, busy, lambda c, s: product(c, s, torch.empty(M, N, device="cuda")))


@pytest.mark.parametrize("fmt", [Q8, E4M3])
@pytest.mark.parametrize("M", [80, 300, 2048])
def test_block_driver(rtq, busy, M, fmt):
    """w2 fresh: the grouped launch of few rows, and the launch behind the others' group
    with its activations rounded on a second stream."""
    d, f = 512, 2048
    old = {n: rtq.quantize_a8(randn(*shape, seed=80 + i), fmt)
           for i, (n, shape) in enumerate((("qkvg", (4 * d, d)), ("wo", (d, d)), ("w13", (2 * f, d))))}
    X = [randn(M, k, seed=90 + i) for i, k in enumerate((d, d, d, f))]
    Y = [[torch.empty(M, n, device="cuda") for n in (4 * d, d, 2 * f, d)] for _ in range(TURNS)]
    turn = iter(range(TURNS))

    def weight(c, s):
        return (fmt, c, s if fmt == Q8 else None)

    def product(c, s, out=None):
        out = out if out is not None else Y[next(turn)]
        blk = rtq.QBlockFmt(weight(*old["qkvg"]), weight(*old["wo"]), weight(*old["w13"]), weight(c, s))
        rtq.qblock_project_fmt(blk, *X, *out)
        return out[3]

    turns(rtq, fmt, d, f, product, busy, lambda c, s: product(c, s, [torch.empty_like(y) for y in Y[0]]))


@pytest.mark.parametrize("M", [2, 80, 600, 9000])
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_8bit_product(rtq, busy, M, fmt):
    N, K = 2048, 640
    x = rtq.quantize_a8(randn(M, K, seed=90), fmt)
    turns(rtq, fmt, N, K, lambda c, s: rtq.qgemm_a8(fmt, *x, c, s), busy,
          lambda c, s: rtq.qgemm_a8(fmt, *x, c, s))


def test_outputs_a_helper_allocates_on_another_stream(rtq, busy):
    """Blocks that work pending on the current stream still uses are not given to a
    call on another one, and its results are the current stream's."""
    M, K, N = 700, 512, 300
    x, r = randn(M, K, seed=1), randn(M, K, seed=2)
    w = rtq.quantize_a8(randn(N, K, seed=3), Q8)
    want = [*rtq.quantize_a8(x, Q8), *rtq.addnorm_a8(x, None, Q8, residual=r), *rtq.gate_a8(x, Q8)]
    want += [rtq.dequant_a8(Q8, *want[:2]), rtq.qgemm_a8(Q8, *want[:2], *w), rtq.qgemm_q8(x, *w)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of every output's size, used by work behind `busy` and then free
    busy()
    held = [torch.full_like(t, 5) for t in want]
    kept = [t + 0 for t in held]
    blocks = {t.data_ptr() for t in held}
    del held
    got = [*rtq.quantize_a8(x, Q8, stream=side), *rtq.addnorm_a8(x, None, Q8, residual=r, stream=side),
           *rtq.gate_a8(x, Q8, stream=side)]
    got += [rtq.dequant_a8(Q8, *got[:2], stream=side), rtq.qgemm_a8(Q8, *got[:2], *w, stream=side),
            rtq.qgemm_q8(x, *w, stream=side)]
    assert not blocks & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b, k in zip(want, got, kept):
        assert torch.equal(a, b) and bool((k == 5).all())
