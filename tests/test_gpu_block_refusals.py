"""What the library refuses, it refuses with its own message from the backward
calls as from the forward ones: sizes without a workspace."""
import pytest
import torch

from test_gpu_block import gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [3, 0, -1, 16])
def test_gated_norm_of_groups_that_do_not_divide(ssm, groups):
    x, w = randn(gen(1), 4, 8), torch.ones(8, device="cuda")
    for call in (lambda: ssm.ssm_gated_norm_fwd(x, x, w, groups=groups),
                 lambda: ssm.ssm_gated_norm_bwd(x, x, w, x, groups=groups)):
        with pytest.raises(ssm.SsmError, match=f"groups {groups} does not divide d 8") as e:
            call()
        assert e.value.status == ssm.SSM_ERR_INVALID_ARG


def test_conv1d_of_nine_taps(ssm):
    x, w = randn(gen(1), 1, 6, 8), randn(gen(2), 8, 9)
    for call in (lambda: ssm.ssm_conv1d_fwd(x, w), lambda: ssm.ssm_conv1d_bwd(x, w, x),
                 lambda: ssm.ssm_conv1d_update(randn(gen(3), 6, 8, 9), x[0], w)):
        with pytest.raises(ssm.SsmError, match="d_conv 9") as e:
            call()
        assert e.value.status == ssm.SSM_ERR_UNSUPPORTED
