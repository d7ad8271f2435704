"""8-bit activations: argument checks of the C ABI and of the Python helpers,
before any CUDA call (the pointers below are never dereferenced)."""
import math

import pytest

import int8_dequant_gemm_b200 as rtq
from int8_dequant_gemm_b200 import build as rtq_build

RT_OK, INVALID, ALIGN, SHAPE = 0, 1, 2, 3
Q8, E4M3, Q4 = 8, 3, 4
F32, F16, BF16 = 0, 1, 2
EPS = 1e-6
# fake, well-aligned, non-overlapping device addresses
X, R, G, H, C, S, W, WS, B, Y = (0x10000000 * i for i in range(1, 11))


@pytest.fixture(scope="module", autouse=True)
def built():
    rtq_build.build()
    return rtq.lib()


def quantize(fmt=Q8, dtype=F32, x=X, c=C, s=S, M=4, K=64):
    return rtq.rt_quantize_a8(fmt, dtype, x, c, s, M, K, None)


def gate(fmt=Q8, dtype=F32, x=X, c=C, s=S, M=4, K=64):
    return rtq.rt_gate_a8(fmt, dtype, x, c, s, M, K, None)


def dequant(fmt=Q8, dtype=F32, x=X, c=C, s=S, M=4, K=64):
    return rtq.rt_dequant_a8(fmt, dtype, c, s, x, M, K, None)


def addnorm(fmt=Q8, dtype=F32, x=X, c=C, s=S, M=4, K=64, r=R, g=G, eps=EPS, h=H):
    return rtq.rt_addnorm_a8(fmt, dtype, x, r, g, eps, h, c, s, M, K, None)


@pytest.mark.parametrize("call", [quantize, gate, dequant, addnorm])
def test_row_operators_refuse(call):
    assert call(fmt=Q4) == INVALID and call(fmt=0) == INVALID
    assert call(dtype=3) == INVALID and call(dtype=-1) == INVALID
    assert call(M=-1) == INVALID and call(M=2 ** 31 - 1023) == INVALID
    assert call(K=0) == INVALID and call(K=-16) == INVALID
    assert call(K=24) == SHAPE and call(K=131072) == SHAPE
    if call is not dequant:
        assert call(K=32784) == SHAPE            # longer than a block's registers hold
    assert call(x=None) == INVALID and call(c=None) == INVALID and call(s=None) == INVALID
    assert call(x=X + 8) == ALIGN and call(c=C + 4) == ALIGN and call(s=S + 2) == ALIGN
    assert call(c=X) == INVALID                   # codes over the values
    assert call(s=X + 16) == INVALID              # scales inside the values
    assert call(s=C + 64) == INVALID or call is dequant
    assert call(M=0) == RT_OK and call(M=0, x=None, c=None, s=None) == RT_OK
    assert call(M=0, K=24) == SHAPE               # sizes are checked for no rows too


def test_gate_input_is_twice_as_wide():
    M, F = 4, 64
    end = X + M * 2 * F * 4
    assert gate(c=end - 16) == INVALID            # inside the second half
    assert gate(dtype=BF16, c=X + M * 2 * F * 2 - 16) == INVALID


def test_addnorm_refuses():
    for eps in (0.0, -1e-6, math.inf, math.nan, 1e-40):
        assert addnorm(eps=eps) == INVALID
        assert addnorm(eps=eps, M=0) == INVALID
    assert addnorm(r=R + 8) == ALIGN and addnorm(g=G + 4) == ALIGN and addnorm(h=H + 8) == ALIGN
    assert addnorm(h=X + 64) == INVALID           # shifted against X
    assert addnorm(h=R + 64) == INVALID
    assert addnorm(h=G) == INVALID
    assert addnorm(c=H) == INVALID and addnorm(s=G) == INVALID and addnorm(c=R) == INVALID
    assert addnorm(h=X, r=X + 64) == INVALID      # X itself, but shifted against R


def product(fmt=Q8, dtype=F32, x=X, xs=S, w=W, ws=WS, b=B, y=Y, M=4, N=24, K=64):
    return rtq.rt_qgemm_a8(fmt, dtype, x, xs, w, ws, b, y, M, N, K, None)


def test_product_refuses():
    assert product(fmt=Q4) == INVALID and product(dtype=3) == INVALID
    assert product(M=-1) == INVALID and product(N=0) == INVALID and product(K=0) == INVALID
    assert product(M=2 ** 31) == INVALID and product(N=2 ** 31) == INVALID
    assert product(K=40) == SHAPE and product(K=131072) == SHAPE
    for name in ("x", "xs", "w", "y"):
        assert product(**{name: None}) == INVALID
    assert product(ws=None) == INVALID            # q8 weights have scales
    assert product(x=X + 8) == ALIGN and product(w=W + 8) == ALIGN and product(y=Y + 8) == ALIGN
    assert product(xs=S + 2) == ALIGN and product(ws=WS + 2) == ALIGN and product(b=B + 2) == ALIGN
    assert product(y=X) == INVALID and product(y=W) == INVALID
    assert product(xs=Y + 4) == INVALID and product(ws=Y + 8) == INVALID and product(b=Y) == INVALID
    assert product(M=0) == RT_OK and product(M=0, x=None, xs=None, y=None) == RT_OK
    assert product(M=0, w=None) == INVALID


def test_product_plan():
    assert rtq.a8_plan(4, 24, 40) is None and rtq.a8_plan(4, 0, 64) is None
    assert rtq.a8_plan(-1, 24, 64) is None and rtq.a8_plan(4, 24, 131072) is None
    assert rtq.a8_plan(4, 24, 64, Q4) is None
    for fmt in (Q8, E4M3):
        assert rtq.a8_plan(1, 512, 512, fmt)["cores"] and not rtq.a8_plan(129, 64, 64, fmt)["cores"]
        assert not rtq.a8_plan(8, 8192, 8192, fmt)["cores"]
        for M in (0, 1, 8, 16, 17, 80, 128, 129, 300, 4096, 65536, 2 ** 31 - 1024):
            for N in (1, 128, 512, 4096):
                for K in (16, 512, 2048, 131056):
                    p = rtq.a8_plan(M, N, K, fmt)
                    if p["cores"]:
                        assert 1 <= M <= 128
                        continue
                    assert 1 <= p["split"] <= min(8, -(-K // 128))
                    assert p["rows"] % (32 if p["pair"] else 16) == 0 and 16 <= p["rows"] <= 256
                    assert not (p["pair"] and p["split"] > 1) and not (p["walk"] and p["split"] > 1)
                    assert p["walk"] or (p["rows"] <= 128 and not p["pair"])
                    if p["split"] > 1:            # partial sums fit where the ring was
                        assert p["rows"] * 512 <= 100 * 1024


def test_helpers_refuse_host_tensors_and_formats():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for f in (lambda: rtq.quantize_a8(x), lambda: rtq.addnorm_a8(x), lambda: rtq.gate_a8(x),
              lambda: rtq.dequant_a8(8, c, s), lambda: rtq.qgemm_a8(8, c, s, c, s),
              lambda: rtq.quantize_a8(None), lambda: rtq.qgemm_a8(8, None, s, c, s)):
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            f()
    for f in (lambda: rtq.quantize_a8(x, 4), lambda: rtq.gate_a8(x, 0),
              lambda: rtq.dequant_a8(4, c, s), lambda: rtq.qgemm_a8([], c, s, c, s)):
        with pytest.raises(ValueError, match="fmt must be"):
            f()
