"""The largest sizes that the row operators take, on the CPU: past them every call is refused before any device work."""
import pytest

from convolution_implicit_gemm_fwd_amd import abi
from test_row_ops_host import FP32, MX, deq, lin, linb, ln, lnb, lnq, quant

RANGE = abi.CONVIMG_ERR_RANGE
COLS = (1 << 31) - (1 << 14)        # a kernel's column counter steps up to 8192 past the end of a row


@pytest.mark.parametrize("cols", [COLS + 1, COLS + 8192, 0x7FFFFF00, 0x7FFFFFFF])
def test_columns_past_the_counters_are_refused(cols):
    assert ln(rows=1, cols=cols, ldx=cols) == RANGE
    assert lnq(rows=1, cols=cols, ldx=cols) == RANGE
    assert lnb(rows=1, cols=cols, ldx=cols, lddy=cols) == RANGE
    assert abi.layer_norm_bwd_workspace(1, cols)[0] == RANGE
    assert abi.mxfp4_bytes(1, cols)[0] == RANGE
    assert quant(rows=1, cols=cols, ldx=cols) == RANGE
    assert quant(rows=cols, cols=1, ldx=1, transpose=1) == RANGE
    assert deq(rows=1, cols=cols) == RANGE
    assert abi.mxfp4_linear_workspace(1, 1, cols, MX)[0] == RANGE
    assert lin(M=1, N=1, K=cols, ldx=cols) == RANGE
    assert abi.mxfp4_linear_bwd_workspace(cols, 1, 1)[0] == RANGE
    assert abi.mxfp4_linear_bwd_workspace(1, cols, 1)[0] == RANGE
    assert linb(M=1, N=1, K=cols, ldx=cols, ldw=cols) == RANGE


def test_columns_up_to_the_counters_are_taken():
    assert abi.mxfp4_bytes(1, COLS) == (0, COLS // 2, COLS // 32)
    assert abi.layer_norm_bwd_workspace(1, COLS) == (0, 8 * COLS)
    assert abi.mxfp4_linear_workspace(0, 1, COLS, FP32)[0] == 0
    for cols in (COLS, 1):
        assert ln(rows=0, cols=cols, ldx=cols) == 0 and quant(rows=0, cols=cols, ldx=cols) == 0


def test_rows_past_32_bits_are_refused():
    assert abi.layer_norm_bwd_workspace(1 << 31, 1)[0] == RANGE
    assert lnb(rows=1 << 31) == RANGE


@pytest.mark.parametrize("rows,cols", [(1 << 20, 1 << 12), (1 << 27, 1), (1, COLS), (1 << 26, 33)])
def test_codes_of_2_gib_are_refused_by_every_call(rows, cols):
    refused = abi.mxfp4_bytes(rows, cols)[0]
    assert refused == (RANGE if cols != COLS else 0)
    if refused:
        assert lnq(rows=rows, cols=cols, ldx=cols, codes=1 << 45, scales=1 << 46) == RANGE
        assert quant(rows=rows, cols=cols, ldx=cols) == RANGE
        assert deq(rows=rows, cols=cols) == RANGE
        assert lin(x_dtype=MX, x_scales=1 << 45, M=rows, K=cols, ldx=cols) == RANGE
