"""The binding's check of the norm's sum (host only, stand-ins for the tensors)."""
import pytest

import bit_quantized_gemm_gb300 as qg
from test_fp8_devices import library  # noqa: F401
from test_more_host import arguments


@pytest.mark.parametrize("int8", [False, True])
def test_a_sum_without_a_residual_is_refused(library, int8):  # noqa: F811
    # (nothing would write it; the C ABI refuses the pair, too)
    a = arguments()
    call = qg.rmsnorm_quantize_act if int8 else qg.rmsnorm_quantize_act_fp8
    out = (a["q8"], a["scale8"], a["bs"], a["q16"]) if int8 else (a["q"], a["scale"])
    with pytest.raises(ValueError):
        call(a["x"], a["weight"], out=out + (a["sum"],))
    assert not library.calls
    assert call(a["x"], a["weight"], out=out + (None,))[-1] is None
    assert len(library.calls) == 1
