"""What a NaN or an infinite state of the gated recurrence does inside a
sequence: a decay is positive however small, so it stays one, over any number of
steps and tiles, until a sequence starts; the adjoint likewise, backwards.
Against the definition taken step by step in 64 bits, with decays whose products
over a tile are below any fp32 number.  Limits as in test_gpu_block.py."""
import pytest
import torch

import _block_ref as R
from _block_ref import F64, close, up
from test_gpu_block import BF, F32, U, gated_all, gen, randn

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# 0.25 and 0.5 a step pass below 2^-149 after 75 and 150 of them, 2^-29 after 6, 2^-288 at once
A_ROWS = torch.tensor([-1.3862944, -0.6931472, -20.0, -200.0])


def case(b, L, d, dtype, starts, seed):
    g = gen(seed)
    k = torch.arange(d)
    c = dict(u=randn(g, b, L, d, dtype=dtype), gate_x=randn(g, b, L, d, dtype=dtype),
             gate_a=torch.full((b, L, d), 60.0, dtype=dtype, device="cuda"), A=A_ROWS[k % 4].cuda())
    kind = (k // 4 % 4).cuda()  # of a channel's start state and last adjoint: NaN, the infinities, a number
    ends = []
    for _ in range(2):
        v = randn(g, b, d)
        ends.append(torch.where(kind == 0, NAN, torch.where(kind == 1, INF, torch.where(kind == 2, -INF, v))))
    c["h0"], dh = ends
    if starts is not None:
        s = torch.zeros(b, L, dtype=torch.uint8)
        for t in starts:
            s[:, t] = 1
        c["seq_start"] = s.cuda()
    return c, randn(g, b, L, d, dtype=dtype), dh


def adjoint(c, dout, dh):
    """du, dgate_x, dh0 in 64 bits; no gradient goes back over a start."""
    a = torch.exp(up(c["A"]) * R.sig(up(c["gate_a"])))
    f = torch.sqrt(-torch.expm1(2 * up(c["A"]) * R.sig(up(c["gate_a"]))))
    g, u, do = R.sig(up(c["gate_x"])), up(c["u"]), up(dout)
    s = torch.zeros(u.shape[:2]) if c.get("seq_start") is None else c["seq_start"].cpu()
    du, dgx, acc = torch.empty_like(u), torch.empty_like(u), up(dh)
    for t in range(u.shape[1] - 1, -1, -1):
        m = s[:, t, None] != 0
        lam = do[:, t] + acc
        ft = torch.where(m, 1.0, f[:, t])
        du[:, t] = lam * ft * g[:, t]
        dgx[:, t] = du[:, t] * u[:, t] * (1 - g[:, t])
        acc = torch.where(m, 0.0, a[:, t] * lam)
    return dict(du=du, dgate_x=dgx, dh0=acc)


# (1, 1100, 16) and (2, 600, 48) take clusters over time, (330, 200, 64) a CTA for each tile
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,L,d", [(1, 1100, 16), (2, 600, 48), (1, 300, 33), (330, 200, 64)])
@pytest.mark.parametrize("starts", [None, (), (97,)])
def test_gated_scan_keeps_nonfinite_states(ssm, b, L, d, starts, dtype):
    c, dout, dh = case(b, L, d, dtype, starts, seed=b + L + d)
    got = gated_all(ssm, c, dout, dh)
    v = {k: up(c[k]) for k in ("u", "gate_a", "gate_x", "A")}
    s = None if starts is None else c["seq_start"].cpu()
    y, h = R.gated(**v, seq_start=s, h0=up(c["h0"]))
    ref = dict(adjoint(c, dout, dh), y=y, h_last=h)
    if starts == (97,):
        assert torch.isfinite(h).all() and torch.isfinite(ref["dh0"]).all()
    else:
        assert (torch.isnan(h) == torch.isnan(up(c["h0"]))).all()
    # |h| <= |h0| + sum of drives over a memory of at most two steps; the adjoint likewise
    rel = 2.0 ** -18 + (min(L, 1000) + 64) * U
    finite = lambda t: float(t[torch.isfinite(t)].abs().max())  # noqa: E731
    top_h = finite(up(c["h0"])) + 2 * finite(up(c["u"]))
    top_l = finite(up(dh)) + 2 * finite(up(dout))
    close("y", got["y"], y, rel * top_h)
    close("h_last", got["h_last"], h, rel * top_h)
    for k, amp in (("du", 1.0), ("dgate_x", finite(up(c["u"]))), ("dh0", 1.0)):
        close(k, got[k], ref[k], rel * top_l * amp)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("packed", [False, True])
def test_gated_scan_keeps_a_nan_that_arises_on_the_way(ssm, packed, dtype):
    """A NaN input spoils its channel from there on, whatever the decays, in the
    chunk states that the backward starts from too."""
    b, L, d = 1, 900, 16
    c, dout, _ = case(b, L, d, dtype, () if packed else None, seed=2)
    c["h0"] = None
    c["u"][:, 130, ::2] = NAN
    states = torch.zeros(ssm.ssm_gated_scan_states_bytes(b, L, d) // 4, device="cuda")
    h = torch.empty(b, d, device="cuda")
    y = ssm.ssm_gated_scan_fwd(**c, h_last=h, chunk_states=states)
    nan = torch.zeros(L, d, dtype=torch.bool)
    nan[130:, ::2] = True
    assert torch.equal(torch.isnan(y[0]).cpu(), nan)
    assert torch.equal(torch.isnan(h[0]).cpu(), nan[-1])
    front = torch.cat([torch.zeros(1, d, dtype=torch.bool), nan[:-1]])  # in front of each step
    assert torch.equal(torch.isnan(states.view(-1, d)).cpu(), front[::32])
    kw = {k: v for k, v in c.items() if k != "h0"}
    g = ssm.ssm_gated_scan_bwd(**kw, dout=dout, states=states)
    # u only enters what its own step and later ones give the gates
    assert torch.isfinite(g["du"]).all() and torch.isfinite(g["dgate_a"][0, :130]).all()
    assert torch.isnan(g["dgate_a"][0, 131:, ::2]).all() and torch.isfinite(g["dgate_a"][..., 1::2]).all()
