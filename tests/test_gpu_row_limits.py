"""The row operators at sizes whose single launch would hold 2^32 threads or more, on the GPU."""
import pytest
import torch

import convolution_implicit_gemm_fwd_amd as cim
from gpu_harness import need_gpu
from row_reference import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def test_layer_norm_gradient_sums_of_very_wide_rows():
    """2^26 + 48 sums of five partial sums, 64 threads each."""
    rows, cols = 5, (1 << 25) + 24
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    mean, rstd = torch.full((rows,), 0.125, device="cuda"), torch.full((rows,), 1.5, device="cuda")
    _, dgamma, dbeta = cim.layer_norm_bwd_nhwc(dy, x, None, mean, rstd)
    n = (x.double() - 0.125) * 1.5
    # n is off by 2 u, a product by u, and each of the sums' additions (three levels, five terms) by u
    for got, terms in ((dgamma, dy.double() * n), (dbeta, dy.double())):
        assert bool(((got - terms.sum(0)).abs() <= 8 * U * terms.abs().sum(0) + 1e-40).all())


def test_quantisation_down_a_very_long_column():
    """2^23 + 2 tiles of 512 threads.  The column as a row gives the same codes by another kernel."""
    rows = (1 << 30) + 130
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(rows, 1, generator=g, device="cuda", dtype=torch.bfloat16)
    x[-1] = 77
    down, along = cim.mxfp4_quantize_nhwc(x, transpose=True), cim.mxfp4_quantize_nhwc(x.view(1, rows))
    assert (down.rows, down.cols) == (along.rows, along.cols) == (1, rows)
    assert torch.equal(down.codes, along.codes) and torch.equal(down.scales, along.scales)
    assert down.codes[0, -16] >> 4 == 6      # the last value, second of its block: 77 / 16 rounds to 4
