"""The gated recurrence where most gates are closed (sigmoids of 2^-86 to 2^-60, as
masked steps have them) beside open ones: the backward's outputs are right each
for itself, however small, against the formulas in 64 bits.

Limits, each of the same expression over magnitudes.  A gate x is off by the
rounding of its scaled argument, |x| 2^-24 of itself and so 2^-18 at most here, and
the SFU's 2^-21; a decay by |A| r times that (|A| <= 8, r open: 2^-18).  At most 8
such factors meet in an output, 2^-15, with (L + 64) u for the recurrences.
Input gates stay above 2^-64, below which the forward's drive is 0."""
import pytest
import torch

import _block_ref as R
from _block_ref import close, up
from test_gpu_block import BF, F32, U, gen, randn

pytestmark = pytest.mark.gpu


def reference(c, dout, dh):
    """{name: (value, the same over magnitudes)}"""
    q = {k: up(v) for k, v in c.items()}
    b, L, d = q["u"].shape
    s = torch.zeros(b, L, 1, dtype=torch.bool)
    if c.get("seq_start") is not None:
        s = (c["seq_start"].cpu() != 0).unsqueeze(-1)
    r, g = R.sig(q["gate_a"] + q["bias_a"]), R.sig(q["gate_x"] + q["bias_x"])
    a, f = torch.exp(q["A"] * r), torch.sqrt(-torch.expm1(2 * q["A"] * r))
    af = a * a / f * g * q["u"]
    a, f = torch.where(s, 0.0, a), torch.where(s, 1.0, f)
    x = f * g * q["u"]
    h, hm, hs, hms = q["h0"], q["h0"].abs(), [], []
    for t in range(L):
        hs.append(h), hms.append(hm)
        h, hm = a[:, t] * h + x[:, t], a[:, t] * hm + x[:, t].abs()
    prev, mprev = torch.stack(hs, 1), torch.stack(hms, 1)
    cur, mcur = torch.stack([*hs[1:], h], 1), torch.stack([*hms[1:], hm], 1)
    z = q["z"]
    sz, go = R.sig(z), up(dout) * z * R.sig(z)
    lam, mlam, m, mm = torch.empty_like(x), torch.empty_like(x), up(dh), up(dh).abs()
    for t in range(L - 1, -1, -1):
        lam[:, t], mlam[:, t] = m + go[:, t], mm + go[:, t].abs()
        m, mm = a[:, t] * lam[:, t], a[:, t] * mlam[:, t]
    dl, ml = torch.where(s, 0.0, lam * (a * prev - af)), torch.where(s, 0.0, mlam * (a * mprev + af.abs()))
    dga, mga = dl * q["A"] * r * (1 - r), ml * q["A"].abs() * r
    dgx, mgx = lam * x * (1 - g), mlam * x.abs()
    total = lambda t: t.sum((0, 1))  # noqa: E731
    return dict(du=(lam * f * g, mlam * f * g), dgate_x=(dgx, mgx), dgate_a=(dga, mga), dh0=(m, mm),
                dz=(up(dout) * cur * (sz + z * sz * (1 - sz)), (up(dout) * mcur).abs() * (1 + z.abs())),
                dA=(total(dl * r), total(ml * r)), dbias_a=(total(dga), total(mga)),
                dbias_x=(total(dgx), total(mgx)))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,L,d,packed", [(1, 700, 16, False), (2, 90, 33, True), (40, 64, 64, False)])
def test_gated_scan_gradients_of_closed_gates(ssm, b, L, d, packed, dtype):
    g = gen(b + L + d)
    c = dict(u=randn(g, b, L, d, dtype=dtype), z=randn(g, b, L, d, dtype=dtype), bias_a=randn(g, d, scale=0.5),
             bias_x=randn(g, d, scale=0.5), h0=randn(g, b, d))
    for k, lo in (("gate_a", -58.0), ("gate_x", -41.0)):
        open_ = torch.rand(b, L, d, generator=g) < 0.1
        shut = lo + 2 * torch.rand(b, L, d, generator=g)
        c[k] = torch.where(open_, torch.randn(b, L, d, generator=g), shut).to(dtype).cuda()
    c["A"] = -(10 ** (-3 + 3.9 * torch.rand(d, generator=g))).cuda()
    if packed:
        c["seq_start"] = (torch.rand(b, L, generator=g) < 0.1).to(torch.uint8).cuda()
    dout, dh = randn(g, b, L, d, dtype=dtype), randn(g, b, d)
    states = torch.empty(ssm.ssm_gated_scan_states_bytes(b, L, d) // 4, device="cuda")
    ssm.ssm_gated_scan_fwd(**c, chunk_states=states)
    got = ssm.ssm_gated_scan_bwd(**{k: v for k, v in c.items() if k != "h0"}, dout=dout, states=states,
                                 dh_last=dh, want_dh0=True)
    rel = 2.0 ** -15 + (L + 64) * U
    n = b * L * U  # a column's sum, in any order
    for k, (ref, mag) in reference(c, dout, dh).items():
        close(k, got[k], ref, (rel + (n if k in ("dA", "dbias_a", "dbias_x") else 0.0)) * mag)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("low", [-1e4, -3.0e38, -float("inf")])
def test_gated_scan_masked_steps_take_and_give_nothing(ssm, low, dtype):
    """Both gates at a mask's value: the state passes (taken up again from its map
    every few steps, a rounding each), and the step's inputs get no gradient."""
    g = gen(9)
    b, L, d = 2, 75, 24
    c = dict(u=randn(g, b, L, d, dtype=dtype), gate_a=randn(g, b, L, d, dtype=dtype),
             gate_x=randn(g, b, L, d, dtype=dtype), A=torch.full((d,), -3.0, device="cuda"))
    mask = (torch.rand(b, L, 1, generator=g) < 0.5).cuda()
    c["gate_a"], c["gate_x"] = (c[k].masked_fill(mask, low) for k in ("gate_a", "gate_x"))
    states = torch.empty(ssm.ssm_gated_scan_states_bytes(b, L, d) // 4, device="cuda")
    y = ssm.ssm_gated_scan_fwd(**c, chunk_states=states)
    got = ssm.ssm_gated_scan_bwd(**c, dout=randn(g, b, L, d, dtype=dtype), states=states)
    front = torch.cat([torch.zeros_like(y[:, :1]), y[:, :-1]], 1)
    close("y", y[mask[..., 0]], up(front[mask[..., 0]]), 2.0 ** -20 * float(y.abs().max()))
    for k in ("du", "dgate_a", "dgate_x"):
        assert (got[k][mask[..., 0]] == 0).all(), k
        assert torch.isfinite(got[k]).all(), k
