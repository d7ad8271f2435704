"""How many roundings the row operators take, in units of u = 2^-24 (half an ulp of
fp32 at most): bounds counted operation by operation, before their first run."""
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


def uniform(lo, hi, *shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lo + (hi - lo) * torch.rand(*shape, generator=g, device="cuda", dtype=torch.float64)


@pytest.mark.parametrize("lo,hi", [(-1, 1), (-8, -1), (1, 8), (-20, -8), (8, 80), (-80, -20)])
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_gate_roundings(rtq, fmt, lo, hi):
    """One product a row: its scale is that product over the format's largest code.
    exp2 is documented to 4 u of relative error, and takes the argument that a
    rounding of a log2 e (|a| u, put right to first order) and of log2 e's own last
    bit (at most 0.05 u |a|) leave; a factor near 1, the sum with 1 and the
    reciprocal add 1 + 1 + 2 u, two products 2 u, the scale 1 u."""
    M, K = 1 << 16, 16
    a = uniform(lo, hi, M, seed=7).float()
    # a power of two that keeps the products of the far range in fp32's normal range
    b = torch.full_like(a, 2.0 ** 40 if lo < -20 else 1.0)
    u = torch.zeros(M, 2 * K, device="cuda")
    u[:, 3], u[:, K + 3] = a, b
    _, s = rtq.gate_a8(u, fmt)
    x = a.double()
    y = (x * torch.sigmoid(x) * b.double()).abs()
    err = ((s.double() * TOP[fmt] - y).abs() / y / U)
    assert float((err - 0.05 * x.abs()).max()) <= 11


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [16, 528, 1024, 2048, 4096])
@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_gate_of_the_largest_values(rtq, fmt, dtype, K):
    """Finite a up to the type's end give finite rows, in one block with rows that are
    not finite: silu(a) = a from a = 30 on to below u, then a rounding of a / 1, a
    product, and the scale."""
    M = 9
    g = torch.Generator(device="cuda").manual_seed(K)
    a = torch.randn(M, K, generator=g, device="cuda")
    b = torch.randn(M, K, generator=g, device="cuda")
    big = torch.tensor([3.0e38, -3.0e38, 2.4e38, 3.3e38], device="cuda")
    a[::2, 5:9], b[::2, 5:9] = big, 1e-3 * big.sign()
    u = torch.cat([a, b], 1).to(dtype)
    u[4, 0] = float("inf")
    c, s = rtq.gate_a8(u, fmt)
    assert rtq.device_status() == RANGE              # the row with the infinity
    want, ws = rtq.gate_a8(u[1::2].contiguous(), fmt)
    assert torch.equal(c[1::2], want) and torch.equal(s[1::2], ws)
    assert bool(s[4].isnan()) and bool((c[4] == 0).all())
    x, z = u.double().chunk(2, dim=1)
    top = (x * torch.sigmoid(x) * z).abs().amax(1)
    for row in (0, 2, 6, 8):
        assert abs(float(s[row]) * TOP[fmt] / float(top[row]) - 1) <= 4 * U
        values = c[row].double() if fmt == Q8 else c[row].view(torch.float8_e4m3fn).double()
        at = int((x * z)[row].abs().argmax())
        assert abs(float(values[at])) == TOP[fmt] and float(values[6]) == 0


@pytest.mark.parametrize("fmt", [Q8, E4M3])
def test_gate_of_the_smallest_sigmoids(rtq, fmt):
    """Down to a = -87 a factor b of any size brings a row back; sigmoid(a) below
    2^-126 counts as 0, so such a row is one of zeros, and is not reported."""
    a = torch.tensor([-80.0, -85.0, -87.0, -88.0, -89.0, -200.0, -3e38], device="cuda")
    u = torch.zeros(len(a), 32, device="cuda")
    u[:, 2], u[:, 18] = a, 3e30
    c, s = rtq.gate_a8(u, fmt)
    assert rtq.device_status() == rtq.OK
    x = a[:3].double()
    y = (x * torch.sigmoid(x) * u[:3, 18].double()).abs()
    assert float(((s[:3].double() * TOP[fmt] - y).abs() / y / U - 0.05 * x.abs()).max()) <= 11
    assert bool((s[3:] == 0).all()) and bool((c[3:].to(torch.int32) == 0).all())


@pytest.mark.parametrize("K", [16, 80, 208, 512, 528, 1040, 2048, 4112])
def test_norm_roundings(rtq, K):
    """Rows of small integers, whose maximum and sum of squares are exact.  The
    formula's own steps in fp32, rounded once each: the quotient by K and the sum with
    eps (halved by the root), the root, the maximum over 127 and the product, 1 + 1 +
    1 + 1 = 4 u.  The kernel's rounded 1 / K and approximate root are to add nothing
    to that."""
    M, eps = 1 << 15, float(np.float32(1e-5))
    g = torch.Generator(device="cuda").manual_seed(K)
    top = torch.randint(1, 16, (M, 1), generator=g, device="cuda")
    x = torch.randint(-15, 16, (M, K), generator=g, device="cuda").clamp(-top, top)
    x[:, 0] = top[:, 0]
    _, s, _ = rtq.addnorm_a8(x.float(), None, Q8, eps=eps)
    h = x.double()
    ss = h.square().sum(1)
    assert float(ss.max()) < 2 ** 24
    want = h.abs().amax(1) / TOP[Q8] / torch.sqrt(ss / K + eps)
    err = float(((s.double() - want).abs() / want).max() / U)
    assert err <= 4, err
