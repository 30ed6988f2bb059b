"""Rows wider than one octet a thread, more of them than workgroups (so that every workgroup loops over rows): the norm's and its gradient's bounds are those of test_gpu_norm."""
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
