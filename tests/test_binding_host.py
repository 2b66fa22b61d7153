"""Host-side tests of the binding's calls that the library refuses (tensors on
the CPU, whose data no call reaches)."""
import pytest
import torch

from selective_state_space_25_b200 import ssmscan as S


@pytest.mark.parametrize("saved", [False, True])
def test_scan_bwd_of_an_unsupported_d_state(saved):
    u, A, BC = torch.zeros(1, 8, 4), torch.zeros(4, 3), torch.zeros(1, 8, 3)
    states = torch.zeros(64) if saved else None
    with pytest.raises(S.SsmError, match="d_state") as e:
        S.ssm_scan_bwd(u, u, A, BC, BC, u, states=states, stream=0)
    assert e.value.status == S.SSM_ERR_UNSUPPORTED
