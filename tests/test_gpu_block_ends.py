"""Gradients of the gated recurrence where its gates are saturated or infinite
and its decays 0 and 1, against automatic differentiation in 64 bits.

Limit: 2^-14 of the largest value that the terms can reach, as in
test_gpu_block.test_gated_scan_gates_at_their_ends."""
import pytest
import torch

from _block_ref import close, up
from test_gpu_block import BF, F32, gated_all, gated_case, gated_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", [False, True])
def test_gated_scan_gradients_of_gates_at_their_ends(ssm, gate, dtype):
    b, L, d = 1, 40, 8
    c, dout, dh = gated_case(b, L, d, dtype, seed=4, gate=gate, bias=False)
    c["A"] = torch.tensor([0.0, -1e-6, -0.1, -1.0, -20.0, -200.0, -1e4, -0.01], device="cuda")
    c["gate_a"][:, ::3] = 60.0
    c["gate_a"][:, 1::3] = -60.0
    c["gate_a"][:, 9] = float("inf")
    c["gate_a"][:, 10] = float("-inf")
    c["gate_x"][:, 5] = float("-inf")
    c["gate_x"][:, 6] = float("inf")
    ref = gated_ref(c, dout, dh)
    got = gated_all(ssm, c, dout, dh)
    for k in ("dgate_a", "dgate_x", "du", "dA", "dh0") + (("dz",) if gate else ()):
        r = ref[k]
        top = r.abs().amax(dim=tuple(range(r.dim() - 1)))  # a channel's largest
        if k == "dA":
            # its terms, of either sign, reach lam (|h| + sqrt(1 / (2 |A|)) |g u|): of the channel, some 40 steps
            A = up(c["A"]).abs()
            top = 40 * float(up(dout).abs().max()) * (
                float(ref["y"].abs().max()) + torch.where(A > 0, 1 / torch.sqrt(2 * A.clamp_min(1e-30)), 0.0) *
                float(up(c["u"]).abs().max()))
        close(k, got[k], r, 2.0 ** -14 * top.clamp_min(1.0).expand_as(r).contiguous())
