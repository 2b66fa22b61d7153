"""The backward kernels whose CTAs walk many rows or segments, over several
rounds with a ragged last one, against the formulas in 64 bits; sums are held
against the magnitudes of their own terms, so that a lost or doubled row shows."""
import pytest
import torch

import _block_ref as R
from _block_ref import F64, close, up
from _norm_ref import add_norm_check, gated_norm_check
from test_gpu_block import BF, F32, U, amax, conv_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF, F32), (BF, BF)])
# a CTA holds several rows; one row; a row is read again (odd width; wider than a CTA holds)
@pytest.mark.parametrize("rows,d", [(9001, 96), (4099, 768), (1801, 2051), (1301, 8200)])
@pytest.mark.parametrize("form", ["plain", "scale", "post", "both"])
def test_add_norm_over_many_rounds(ssm, rows, d, form, dtype, res):
    add_norm_check(ssm, rows, d, form, dtype, res)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,d,groups", [(9001, 96, 1), (4099, 768, 1), (3001, 256, 4), (1801, 2051, 1),
                                           (1301, 8200, 1)])
@pytest.mark.parametrize("form", ["after", "before", "none"])
def test_gated_norm_over_many_rounds(ssm, rows, d, groups, form, dtype):
    gated_norm_check(ssm, rows, d, groups, form, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,L,d,K,silu", [(3001, 9, 33, 4, True), (8003, 9, 64, 4, True),
                                          (4001, 40, 33, 8, True), (5003, 21, 48, 3, False)])
def test_conv1d_over_many_rounds(ssm, b, L, d, K, silu, dtype):
    c, dy = conv_case(b, L, d, K, dtype, seed=b, packed=True)
    got = ssm.ssm_conv1d_bwd(**c, dy=dy, silu=silu)
    x, w, bias, do, win = (up(t) for t in (c["x"], c["weight"], c["bias"], dy, c["conv_state"]))
    xp = torch.cat([win.transpose(1, 2), x], 1)  # step t is row t + K
    t = torch.arange(L)
    age = t - torch.cummax(torch.where(c["seq_start"].cpu() != 0, t, -L - K), 1).values
    live = [(age >= m).unsqueeze(-1).to(F64) for m in range(K)]  # the tap m steps back
    taps = [live[m] * xp[:, K - m:K - m + L] for m in range(K)]
    p = bias + sum(w[:, K - 1 - m] * taps[m] for m in range(K))
    s = R.sig(p)
    dp = do * (s + p * s * (1 - s)) if silu else do
    dx = torch.zeros_like(x)
    for m in range(K):
        dx[:, :L - m] += w[:, K - 1 - m] * (live[m] * dp)[:, m:]
    # limits of one dp and dx as in test_gpu_block.conv_check
    xm, wm, dm = max(1.0, amax(x), amax(win)), amax(w.abs().sum(1)), amax(do)
    e = dm * (2.0 ** -20 * (1 + wm * xm) + 0.5 * (K + 1) * U * (wm * xm + 1.0)) if silu else 0.0
    close("dx", got["dx"], dx, wm * (e + K * U * dm * 1.1))
    # a sum's longest chain: the steps of one segment after another (at least a CTA's 8 places on each
    # SM), 256 places, an eighth of 3 SMs CTAs, 8 lanes
    n, sms = b * L, torch.cuda.get_device_properties(0).multi_processor_count
    links = (n / (8 * sms) + 128 + 256 + sms / 2 + 8) * U
    dw = torch.stack([(dp * taps[K - 1 - j]).sum((0, 1)) for j in range(K)], -1)
    mag = torch.stack([(dp * taps[K - 1 - j]).abs().sum((0, 1)) for j in range(K)], -1)
    off = torch.stack([taps[K - 1 - j].abs().sum((0, 1)) for j in range(K)], -1)
    close("dweight", got["dweight"], dw, links * mag + e * off)
    close("dbias", got["dbias"], dp.sum((0, 1)), links * dp.abs().sum((0, 1)) + e * n)
