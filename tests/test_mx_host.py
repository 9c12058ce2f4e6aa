"""The host side of the microscaled operators (no GPU): sizes, refusals and which
form a call takes."""
import ctypes

import pytest

qb = pytest.importorskip("bit_nf4_quantized_encode_b200")
lib = qb._lib


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_backward_of_few_tokens_reserves_no_dx_in_fp32(fmt):
    """Between a layer of 64 and one of 65536 columns the work buffer grows by
    counters and at most 32 partial tiles of 32 KB, not by [m, cols] floats."""
    wide, narrow = (qb.qlora_mx_linear_workspace_size(4096, c, fmt, 16, 8)[1] for c in (65536, 64))
    assert wide - narrow < 16 * (65536 - 64) * 4 // 2
