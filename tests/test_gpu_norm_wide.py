"""Rows wider than one octet a thread, more of them than workgroups (so that every workgroup loops over rows),
and weights that are not finite: the norm's and its gradient's bounds are those of test_gpu_norm."""
import math

import pytest
import torch

import layer_ref as ref
from test_gpu_norm import check_norm, grad_inputs

pytestmark = pytest.mark.gpu

U = ref.U


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


@pytest.mark.parametrize("rows,cols", [(700, 8208), (520, 12304), (600, 16384), (530, 16400), (515, 32768)])
@pytest.mark.parametrize("dt,ht", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32)])
def test_gradient_of_wide_rows(rt, rows, cols, dt, ht):
    """As test_gradient: 80 u of the terms for dx; a workgroup adds at most 3 rows, the shares at most 512 / 16 + 16
    terms in sequence, within dweight's (rows / 256 + 72) u."""
    dy, h, w, rstd, res = grad_inputs(rows, cols, dt, ht, 16, True)
    dx = torch.full((rows, cols), 7.0, dtype=dt).cuda()
    dw = torch.full((cols,), 7.0).cuda()
    rt.fp8_rmsnorm_backward(dy, h, w, rstd, dx, dw, dresidual=res)
    want, wdw, terms, wterms = ref.norm_grad(dy, h, w, rstd, res)  # (in 64 bits, on the device)
    tol = 80 * U * terms + (2.0 ** -8 * want.abs() if dt == torch.bfloat16 else 0)
    assert bool(((dx.double() - want).abs() <= tol).all())
    assert bool(((dw.double() - wdw).abs() <= (rows / 256 + 72) * U * wterms).all())
    rt.fp8_rmsnorm_backward(dy, h, w, rstd, res, None, dresidual=res)  # in place of the residual's gradient
    assert torch.equal(res, dx)


@pytest.mark.parametrize("rows,cols", [(520, 12304), (530, 16400), (515, 32768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_wide_rows(rt, rows, cols, dtype):
    check_norm(rt, rows, cols, dtype=dtype, pad=16)
    check_norm(rt, rows, cols, dtype=dtype, gran=(1, 128), alias="res")
    check_norm(rt, rows, cols, dtype=dtype, gran=(0, 0), mode=rt.GIVEN, residual=False)


@pytest.mark.parametrize("cols", [16, 48, 512, 1024, 1040, 8208, 16400])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_gradient_with_a_weight_that_is_not_finite(rt, cols, value):
    """The formula's infinities and NaN, whether or not a row fills its threads."""
    rows = 3
    dy, h, w, rstd, _ = grad_inputs(rows, cols, torch.float32, torch.float32, 0, False)
    w[0] = value
    dx, dw = torch.empty_like(dy), torch.empty(cols).cuda()
    rt.fp8_rmsnorm_backward(dy, h, w, rstd, dx, dw)
    want, wdw, _, wterms = ref.norm_grad(dy.cpu(), h.cpu(), w.cpu(), rstd.cpu(), None)
    got = dx.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0, 1, -1), want.nan_to_num(0, 1, -1))  # (nothing in such a row is finite)
    assert bool(((dw.cpu().double() - wdw).abs() <= 76 * U * wterms).all())  # the weight has no part in it
