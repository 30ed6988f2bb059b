"""Weights of fp8_expert_route below binary32's normal numbers: 1 / (1 + e^-l) of far negative logits is e^l, not 0, as long
as it is a number.  Subnormal results carry their exponential's error (2 u of the last place at 2^-149 each) and the
quotient's rounding: 3 2^-149 beside the relative bound of expert_ref.route."""
import pytest
import torch

import expert_ref as ref
from test_gpu_expert_route import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
def test_far_negative_logits(rt, dtype, biased):
    x = -torch.linspace(80, 104, 64).view(4, 16).to(dtype)
    bias = torch.arange(16.0) if biased else None
    o = run(rt, x.cuda(), 16, score="sigmoid", renorm=False, bias=None if bias is None else bias.cuda())
    ids, want, rel = ref.route(x.float(), 16, score="sigmoid", renorm=False, bias=bias)
    assert torch.equal(o["ids"].cpu(), ids)
    got = o["weights"].cpu().double()
    assert bool(((got - want).abs() <= rel * want + 3 * 2.0 ** -149).all())
    assert bool((got[want > 2.0 ** -140] > 0).all())
