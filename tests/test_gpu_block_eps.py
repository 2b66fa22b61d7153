"""The norms with eps = 0, over row counts that leave some of a CTA's places
without a row: finite for rows that are not zero, and right in 64 bits.  Limits:
_norm_ref.py."""
import pytest
import torch

from _norm_ref import add_norm_check, gated_norm_check
from test_gpu_block import BF, F32, gen, randn

pytestmark = pytest.mark.gpu

SIZES = [(5, 64), (1, 16), (3, 33), (13, 200), (129, 1001), (149, 512), (2, 5120)]


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("form", ["plain", "scale", "post", "both"])
def test_add_norm_without_eps(ssm, rows, d, form, dtype, res):
    add_norm_check(ssm, rows, d, form, dtype, res, eps=0.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("form", ["after", "before", "none"])
def test_gated_norm_without_eps(ssm, rows, d, form, dtype):
    gated_norm_check(ssm, rows, d, 1, form, dtype, eps=0.0)


def test_add_norm_of_small_rows_without_eps(ssm):
    """Rows of some 1e-12, far below any usual eps, norm as rows of 1 do."""
    g = gen(1)
    x, w, dy = randn(g, 5, 64), 1 + randn(g, 64, scale=0.1), randn(g, 5, 64)
    y, r = ssm.ssm_add_norm_fwd(x, None, w, eps=0.0)
    k = 2.0 ** -40
    ys, rs = ssm.ssm_add_norm_fwd(x * k, None, w, eps=0.0)
    assert torch.equal(rs, r * k) and torch.allclose(ys, y, rtol=2.0 ** -20, atol=0)
    a = ssm.ssm_add_norm_bwd(None, r, w, dy, eps=0.0)
    s = ssm.ssm_add_norm_bwd(None, rs, w, dy, eps=0.0)
    assert torch.allclose(s["dweight"], a["dweight"], rtol=0, atol=2.0 ** -18 * float(dy.abs().sum()))
    assert torch.isfinite(s["dx"]).all()
