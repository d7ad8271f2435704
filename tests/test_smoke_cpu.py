"""What the smoke run covers, asked of the plans without a GPU (148 SMs)."""
import __graft_entry__ as entry
import int8_dequant_gemm_b200 as rtq
from int8_dequant_gemm_b200 import build as rtq_build


def test_smoke_reaches_every_form_of_the_8bit_product():
    rtq_build.build()
    for form, M, N, K, fmt in entry.A8_FORMS:
        assert entry.a8_form(rtq.a8_plan(M, N, K, fmt)) == form, (form, M, N, K, fmt)
    forms = [f[0] for f in entry.A8_FORMS]
    assert set(forms) == {"cores", "narrow", "split", "walk", "pair"}
    assert {f[4] for f in entry.A8_FORMS} == {8, 3}
    # pairs with the activation tile kept (rows across L2 lines, at most 9 pieces of 128) and streamed
    pairs = [K for form, _, _, K, _ in entry.A8_FORMS if form == "pair"]
    assert any(K % 64 and K <= 9 * 128 for K in pairs) and any(K > 9 * 128 for K in pairs)
