"""More of what the norm, the choice of experts and the adapters refuse before any
launch, without a GPU."""

import pytest

import prefill_q8_mxfp4_amd as q
from test_layer_cpu import BF16, F32, P, norm, norm_grad


@pytest.mark.parametrize("call,bad", [
    (norm, dict(dt=BF16, rt=F32, res=P, x=2 * P, h=4 * P, y=P)), (norm, dict(dt=F32, rt=BF16, res=P, x=2 * P, h=None, y=P)),
    (norm, dict(dt=BF16, rt=F32, x=2 * P, h=2 * P)), (norm, dict(dt=F32, rt=BF16, x=2 * P, h=2 * P)),
    (norm_grad, dict(dt=BF16, rt=F32, dx=2 * P)), (norm_grad, dict(dt=F32, rt=BF16, dx=4 * P)),
    (norm_grad, dict(dt=BF16, rt=F32, dr=P)),
])
def test_outputs_over_inputs_of_another_type(call, bad):
    """A row of one size over rows of another: rows that are not read yet would be written."""
    assert call(**bad) == q.EINVAL and b"type" in q.lib().qgemm_last_error()


def test_codes_with_h_over_x_of_another_type():
    assert q.lib().qgemm_rms_norm_codes(BF16, F32, F32, 4, 64, P, 2 * P, P, 1e-6, P, 3 * P, 64, 4 * P, None) == q.EINVAL
    assert b"type" in q.lib().qgemm_last_error()
