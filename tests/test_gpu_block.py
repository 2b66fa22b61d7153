"""GPU tests of the operators around the scan (gated recurrence, causal
convolution, gated norm, residual-add norm) against their definitions in 64
bits.

Limits.  An output is off by half a step of its type (its one rounding) plus
the fp32 arithmetic in front of it.  With u = 2^-24: a sigmoid, exponential or
root costs at most 2^-21 of its value (two-step SFU results and the rounded
argument, |x| < 8), a product or sum u.

gated scan: every step's decay and drive are off by less than 2^-19 of
  themselves -- 1 - a included, since it is formed to full relative accuracy --
  so h, which forgets over 1 / (1 - a) steps what each step adds, by less than
  2^-18 of the largest |h| the channel's inputs can reach, plus a rounding u per
  step over that memory: (min(L, 1000) + 64) u.  The adjoint is the same
  recurrence of dout.
sums over n rows: n u of the sum of the terms' magnitudes (a worst case for
  any order), plus the terms' own error.
"""
import pytest
import torch

import _block_ref as R
from _block_ref import F64, close, up

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def amax(t):
    return float(t.abs().max()) if t.numel() else 1.0


def strided(t):
    """t's values as the second half of wider rows."""
    wide = torch.full((*t.shape[:-1], 2 * t.shape[-1] + 8), 7.0, dtype=t.dtype, device=t.device)
    half = wide[..., t.shape[-1]:2 * t.shape[-1]]
    half.copy_(t)
    return half


# ------------------------------------------------------------- gated scan
def gated_case(b, L, d, dtype, seed=0, gate=True, carry=True, packed=False, bias=True, view=False):
    g = gen(seed)
    v = strided if view else (lambda t: t)
    c = dict(u=v(randn(g, b, L, d, dtype=dtype)), gate_a=v(randn(g, b, L, d, dtype=dtype)),
             gate_x=v(randn(g, b, L, d, dtype=dtype)),
             A=torch.log(0.9 + 0.0995 * torch.rand(d, generator=g)).cuda())
    c["z"] = v(randn(g, b, L, d, dtype=dtype)) if gate else None
    c["bias_a"], c["bias_x"] = (randn(g, d, scale=0.5), randn(g, d, scale=0.5)) if bias else (None, None)
    c["h0"] = randn(g, b, d) if carry else None
    if packed:
        s = (torch.rand(b, L, generator=g) < 0.06).to(torch.uint8)
        if L:
            s[0, 0] = 1
            s[-1, -1] = 1
        c["seq_start"] = s.cuda()
    dout = v(randn(g, b, L, d, dtype=dtype))
    dh = randn(g, b, d) if carry else None
    return c, dout, dh


def gated_all(S, c, dout, dh, out=None, stream=None, y=None):
    """Forward with states and backward; every output by name."""
    b, L, d = c["u"].shape
    states = torch.full((S.ssm_gated_scan_states_bytes(b, L, d) // 4 + 1,), float("nan"), device="cuda")
    h_last = torch.empty(b, d, device="cuda")
    y = S.ssm_gated_scan_fwd(**c, h_last=h_last, chunk_states=states[:-1], y=y, stream=stream)
    kw = {k: v for k, v in c.items() if k != "h0"}
    got = S.ssm_gated_scan_bwd(**kw, dout=dout, states=states[:-1], dh_last=dh, want_dh0=True, out=out,
                               stream=stream)
    return dict(got, y=y, h_last=h_last)


def gated_ref(c, dout, dh):
    names = [k for k in ("u", "gate_a", "gate_x", "A", "bias_a", "bias_x", "z") if c.get(k) is not None]
    v = {k: up(c[k], True) for k in names}
    b, L, d = c["u"].shape
    h0 = torch.zeros(b, d, dtype=F64) if c.get("h0") is None else up(c["h0"])
    h0.requires_grad_(True)
    s = None if c.get("seq_start") is None else c["seq_start"].cpu()
    y, h = R.gated(**v, seq_start=s, h0=h0)
    loss = (y * up(dout)).sum() + ((h * up(dh)).sum() if dh is not None else 0.0 * h.sum())
    gr = torch.autograd.grad(loss, [*v.values(), h0], allow_unused=True)
    ref = {"d" + k: torch.zeros_like(t) if g is None else g
           for (k, t), g in zip([*v.items(), ("h0", h0)], gr)}
    ref.update(y=y, h_last=h)
    return {k: t.detach() for k, t in ref.items()}


def gated_check(got, ref, c, dout, dh):
    b, L, d = c["u"].shape
    if L == 0 or b == 0:
        scale_h = scale_l = 1.0
    else:
        # the recurrence over |inputs|, the largest the states and adjoints can be
        v = {k: up(c[k]) for k in ("gate_a", "gate_x", "A", "bias_a", "bias_x") if c.get(k) is not None}
        s = None if c.get("seq_start") is None else c["seq_start"].cpu()
        h0 = None if c.get("h0") is None else up(c["h0"]).abs()
        scale_h = float(R.gated(up(c["u"]).abs(), **v, seq_start=s, h0=h0)[0].max())
        lam = up(dout).abs()
        if c.get("z") is not None:
            z = up(c["z"])
            lam = lam * (z * R.sig(z)).abs()
        a = torch.exp(v["A"] * R.sig(v["gate_a"] + v.get("bias_a", 0.0)))
        acc = torch.zeros(b, d, dtype=F64) if dh is None else up(dh).abs()
        top = torch.zeros_like(lam)
        for t in range(L - 1, -1, -1):
            top[:, t] = acc + lam[:, t]
            acc = a[:, t] * top[:, t]
        scale_l = float(top.max())
    rel = 2.0 ** -18 + (min(L, 1000) + 64) * U
    zmax = 1.0 if c.get("z") is None else amax(up(c["z"]))
    umax, dmax = max(1.0, amax(up(c["u"]))), max(1.0, amax(up(dout)))
    lim = dict(y=rel * scale_h * max(1.0, zmax), h_last=rel * scale_h, du=rel * scale_l,
               dgate_x=rel * scale_l * umax, dz=rel * scale_h * dmax * 1.1, dh0=rel * scale_l,
               # |A| r a h_{t-1} and A a^2 g u / f <= sqrt(|A|) u: |A| < 0.11
               dgate_a=rel * scale_l * (0.11 * scale_h + 0.34 * umax))
    n = max(1, b * L)
    if L and b:
        one = 1 - R.sig(up(c["gate_a"]) + (0 if c.get("bias_a") is None else up(c["bias_a"])))
        terms = ref["dgate_a"].abs()
        lim["dbias_a"] = n * U * terms.sum((0, 1)) + n ** 0.5 * 8 * lim["dgate_a"]
        lim["dbias_x"] = n * U * ref["dgate_x"].abs().sum((0, 1)) + n ** 0.5 * 8 * lim["dgate_x"]
        inv = 1 / (up(c["A"]).abs() * one)
        lim["dA"] = (n * U * (terms * inv).sum((0, 1))
                     + n ** 0.5 * 8 * rel * scale_l * (scale_h + umax * 0.75 / up(c["A"]).abs().sqrt()))
    else:
        lim["dbias_a"] = lim["dbias_x"] = lim["dA"] = 0.0
    for k, r in ref.items():
        if k in got or k in ("y", "h_last"):
            close(k, got[k], r, lim[k])
    assert set(got) >= {"du", "dgate_a", "dgate_x", "dA", "dh0", "y", "h_last"}


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,L,d,kw", [
    (1, 1, 1, {}), (2, 1, 64, dict(packed=True)), (3, 7, 5, {}), (1, 63, 66, dict(gate=False)),
    (2, 64, 8, dict(packed=True)), (2, 65, 130, dict(carry=False)), (1, 129, 72, dict(view=True)),
    (1, 300, 33, dict(packed=True, gate=False)), (2, 200, 128, dict(bias=False, packed=True)),
    (1, 1100, 64, dict(packed=True)), (5, 129, 200, dict(view=True, packed=True)),
    (0, 5, 8, {}), (2, 0, 8, {}), (2, 513, 24, dict(gate=False, carry=False))])
def test_gated_scan(ssm, b, L, d, kw, dtype):
    c, dout, dh = gated_case(b, L, d, dtype, seed=L + d, **kw)
    got = gated_all(ssm, c, dout, dh)
    gated_check(got, gated_ref(c, dout, dh), c, dout, dh)


def test_gated_scan_long(ssm):
    """Few channels over a long sequence."""
    c, dout, dh = gated_case(1, 4500, 16, BF, seed=5)
    got = gated_all(ssm, c, dout, dh)
    gated_check(got, gated_ref(c, dout, dh), c, dout, dh)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gated_scan_nothing_crosses_a_start(ssm, dtype):
    """NaN and infinities in front of a sequence's start (in u, the gates, z,
    the start state) and in the gradients behind it stay on their side."""
    b, L, d, cut = 1, 200, 64, 133
    c, dout, dh = gated_case(b, L, d, dtype, seed=3)
    c["seq_start"] = torch.zeros(b, L, dtype=torch.uint8, device="cuda")
    c["seq_start"][:, cut] = 1
    clean = gated_all(ssm, c, dout, dh)
    bad = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    bad["u"][:, 100] = float("nan")
    bad["u"][:, 40, ::2] = float("inf")
    bad["gate_a"][:, 60] = float("nan")
    bad["h0"][:, 1] = float("inf")
    got = gated_all(ssm, bad, dout, dh)
    for k in ("y", "du", "dgate_a", "dgate_x", "dz"):
        assert torch.equal(got[k][:, cut:], clean[k][:, cut:]), k
    assert torch.equal(got["h_last"], clean["h_last"])
    assert torch.isnan(got["y"][:, 100:cut]).all()
    d2 = dout.clone()
    d2[:, cut + 20:] = float("nan")
    got = gated_all(ssm, c, d2, dh)
    for k in ("du", "dgate_a", "dgate_x", "dz"):
        assert torch.equal(got[k][:, :cut], clean[k][:, :cut]), k
    assert torch.equal(got["dh0"], clean["dh0"])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gated_scan_gates_at_their_ends(ssm, dtype):
    """Saturated and infinite gates, decays of 0, 1 and below 2^-126."""
    b, L, d = 1, 40, 8
    c, dout, dh = gated_case(b, L, d, dtype, seed=4, gate=False, bias=False)
    c["A"] = torch.tensor([0.0, -1e-6, -0.1, -1.0, -20.0, -200.0, -1e4, -0.01], device="cuda")
    c["gate_a"][:, ::3] = 60.0
    c["gate_a"][:, 1::3] = -60.0
    c["gate_a"][:, 9] = float("inf")
    c["gate_a"][:, 10] = float("-inf")
    c["gate_x"][:, 5] = float("-inf")
    c["gate_x"][:, 6] = float("inf")
    ref = gated_ref(c, dout, dh)
    got = gated_all(ssm, c, dout, dh)
    top = float(ref["y"].abs().max())
    for k in ("y", "h_last"):
        close(k, got[k], ref[k], 2.0 ** -16 * top)
    for k in ("du", "dgate_x", "dh0"):
        close(k, got[k], ref[k], 2.0 ** -14 * max(1.0, float(ref[k].abs().max())))
    for k in ("dgate_a", "dA"):
        assert torch.isfinite(got[k]).all(), k


def test_gated_scan_in_place_and_outside(ssm):
    """h_last in place of h0, dh0 in place of dh_last, outputs in halves of
    wider rows whose other elements stay."""
    c, dout, dh = gated_case(2, 70, 24, BF, seed=6)
    plain = gated_all(ssm, c, dout, dh)
    wide = {k: torch.full((2, 70, 56), 9.0, dtype=BF, device="cuda")
            for k in ("y", "du", "dgate_a", "dgate_x", "dz")}
    h = c["h0"].clone()
    states = torch.empty(ssm.ssm_gated_scan_states_bytes(2, 70, 24) // 4, device="cuda")
    ssm.ssm_gated_scan_fwd(**{**c, "h0": h}, h_last=h, y=wide["y"][..., 24:48], chunk_states=states)
    out = {k: wide[k][..., 24:48] for k in ("du", "dgate_a", "dgate_x", "dz")}
    out["dh0"] = dh.clone()
    kw = {k: v for k, v in c.items() if k != "h0"}
    ssm.ssm_gated_scan_bwd(**kw, dout=dout, states=states, dh_last=out["dh0"], want_dh0=True, out=out)
    assert torch.equal(h, plain["h_last"]) and torch.equal(out["dh0"], plain["dh0"])
    for k, w in wide.items():
        assert torch.equal(w[..., 24:48], plain[k]), k
        assert (w[..., :24] == 9).all() and (w[..., 48:] == 9).all(), k


def test_gated_scan_gradients_against_differences(ssm):
    """<gradient, v> = d/de loss(inputs + e v), the loss in 64 bits."""
    c, dout, dh = gated_case(2, 90, 10, F32, seed=7, packed=True)
    got = gated_all(ssm, c, dout, dh)
    s = c["seq_start"].cpu()
    v = {k: up(t) for k, t in c.items() if k != "seq_start"}

    def loss(w):
        y, h = R.gated(**w, seq_start=s)
        return float((y * up(dout)).sum() + (h * up(dh)).sum())

    for k in v:
        dirn = torch.randn(v[k].shape, generator=gen(11), dtype=F64)
        e = 1e-6
        num = (loss({**v, k: v[k] + e * dirn}) - loss({**v, k: v[k] - e * dirn})) / (2 * e)
        ana = float((up(got["d" + k]) * dirn).sum())
        # the loss is some 1e3 in 64 bits: the quotient is good to 1e-6; the fp32 gradient to 2^-17 of its terms
        lim = 1e-5 * max(1.0, abs(num)) + 2.0 ** -17 * float((up(got["d" + k]) * dirn).abs().sum())
        assert abs(num - ana) <= lim, (k, num, ana)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,d,view", [(1, 1, False), (3, 37, False), (5, 64, True), (2, 130, True),
                                      (64, 2560, False)])
def test_gated_state_update(ssm, b, d, view, dtype):
    """Three tokens through the step equal the scan over them."""
    c, _, _ = gated_case(b, 3, d, dtype, seed=d, view=view)
    ref, h_ref = R.gated(**{k: up(v) for k, v in c.items()})
    st = c["h0"].clone()
    at = lambda k, t: None if c[k] is None else c[k][:, t]  # noqa: E731
    top = float(ref.abs().max())
    for t in range(3):
        y = ssm.ssm_gated_state_update(st, at("u", t), at("gate_a", t), at("gate_x", t), c["A"],
                                       bias_a=c["bias_a"], bias_x=c["bias_x"], z=at("z", t))
        close("y", y, ref[:, t], 2.0 ** -18 * max(1.0, top))
    close("state", st, h_ref, 2.0 ** -18 * float(h_ref.abs().max()))


# ------------------------------------------------------------ convolution
def conv_case(b, L, d, K, dtype, seed=0, carry=True, packed=False, bias=True, view=False):
    g = gen(seed)
    v = strided if view else (lambda t: t)
    c = dict(x=v(randn(g, b, L, d, dtype=dtype)), weight=randn(g, d, K, scale=K ** -0.5),
             bias=randn(g, d, scale=0.3) if bias else None,
             conv_state=randn(g, b, d, K, dtype=dtype) if carry else None)
    if packed:
        s = (torch.rand(b, L, generator=g) < 0.15).to(torch.uint8)
        if L:
            s[0, 0] = 1
            s[-1, -1] = 1
        c["seq_start"] = s.cuda()
    return c, v(randn(g, b, L, d, dtype=dtype))


def conv_check(S, c, dy, silu=True):
    b, L, d = c["x"].shape
    K = c["weight"].shape[1]
    win = torch.full((b, d, K), float("nan"), dtype=c["x"].dtype, device="cuda")
    y = S.ssm_conv1d_fwd(**c, silu=silu, conv_state_out=win)
    got = S.ssm_conv1d_bwd(**c, dy=dy, silu=silu)
    v = {k: up(c[k], True) for k in ("x", "weight", "bias") if c[k] is not None}
    s = None if c.get("seq_start") is None else c["seq_start"].cpu()
    ref, w_ref = R.conv(**v, silu=silu, conv_state=up(c["conv_state"]), seq_start=s)
    loss = (ref * up(dy)).sum()
    if loss.requires_grad:
        gr = torch.autograd.grad(loss, list(v.values()), allow_unused=True)
    else:
        gr = [None] * len(v)
    gr = [torch.zeros_like(t) if g is None else g for g, t in zip(gr, v.values())]
    # K + 1 products and sums of magnitude <= |w| |x|, then silu
    xm = max(1.0, amax(up(c["x"])), 0.0 if c["conv_state"] is None else amax(up(c["conv_state"])))
    wm, dm = amax(up(c["weight"]).abs().sum(1)), amax(up(dy))
    pre = (K + 1) * U * (wm * xm + 1.0)
    close("y", y, ref, 1.1 * pre + 2.0 ** -20 * wm * xm)
    assert torch.equal(win.cpu().to(F64), w_ref.detach()), "window"
    n = max(1, b * L)
    dp = dm * (2.0 ** -20 * (1 + wm * xm) + 0.5 * pre)  # of one dp: |silu''| <= 1/2
    lim = dict(x=wm * (dp + K * U * dm * 1.1), weight=(n * U * 1.1 * dm + n ** 0.5 * 8 * dp) * xm,
               bias=n * U * 1.1 * dm + n ** 0.5 * 8 * dp)
    if n > 1:  # n u of the sum of magnitudes, below the worst one by their mean
        lim["weight"] = n * U * 1.1 * dm * xm * n * 0.7 + n ** 0.5 * 8 * dp * xm
        lim["bias"] = n * U * 1.1 * dm * n * 0.7 + n ** 0.5 * 8 * dp
    for (k, _), g in zip(v.items(), gr):
        close("d" + k, got["d" + k], g, lim[k])
    return y, win, got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,L,d,K,kw", [
    (1, 1, 1, 4, {}), (2, 2, 8, 4, dict(packed=True)), (3, 3, 33, 4, {}), (1, 5, 64, 8, {}),
    (2, 70, 24, 4, dict(packed=True)), (2, 65, 130, 3, dict(carry=False, bias=False)),
    (1, 200, 72, 2, dict(view=True)), (1, 130, 48, 1, dict(packed=True)),
    (2, 300, 264, 5, dict(view=True, packed=True)), (1, 131, 40, 6, dict(packed=True)),
    (2, 40, 16, 7, {}), (1, 600, 520, 4, dict(carry=False)), (1, 37, 256, 8, dict(packed=True)),
    (2, 0, 8, 4, {}), (0, 4, 8, 4, {})])
def test_conv1d(ssm, b, L, d, K, kw, dtype):
    conv_check(ssm, *conv_case(b, L, d, K, dtype, seed=L + d + K, **kw))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_conv1d_without_silu(ssm, dtype):
    conv_check(ssm, *conv_case(2, 50, 40, 4, dtype, seed=8, packed=True), silu=False)


@pytest.mark.parametrize("L", [2, 3, 100])
def test_conv1d_window_in_place(ssm, L):
    c, _ = conv_case(2, L, 40, 4, BF, seed=9)
    win = torch.empty_like(c["conv_state"])
    y = ssm.ssm_conv1d_fwd(**c, conv_state_out=win)
    c["conv_state"] = c["conv_state"].clone()
    y2 = ssm.ssm_conv1d_fwd(**c, conv_state_out=c["conv_state"])
    assert torch.equal(y, y2) and torch.equal(win, c["conv_state"])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_conv1d_nothing_crosses_a_start(ssm, dtype):
    c, dy = conv_case(1, 90, 40, 4, dtype, seed=10)
    cut = 47
    c["seq_start"] = torch.zeros(1, 90, dtype=torch.uint8, device="cuda")
    c["seq_start"][:, cut] = 1
    y = ssm.ssm_conv1d_fwd(**c)
    g = ssm.ssm_conv1d_bwd(**c, dy=dy)
    bad = dict(c, x=c["x"].clone())
    bad["x"][:, cut - 3:cut] = float("nan")
    assert torch.equal(ssm.ssm_conv1d_fwd(**bad)[:, cut:], y[:, cut:])
    gb = ssm.ssm_conv1d_bwd(**bad, dy=dy)
    assert torch.equal(gb["dx"][:, cut:], g["dx"][:, cut:])
    d2 = dy.clone()
    d2[:, cut:] = float("inf")
    gb = ssm.ssm_conv1d_bwd(**c, dy=d2)
    assert torch.equal(gb["dx"][:, :cut], g["dx"][:, :cut])
    # the first sequence's start cuts off the window
    c["seq_start"][:, 0] = 1
    c["conv_state"].fill_(float("nan"))
    assert torch.isfinite(ssm.ssm_conv1d_fwd(**c)).all()
    win = torch.empty_like(c["conv_state"])
    ssm.ssm_conv1d_fwd(**{**c, "x": c["x"][:, :2], "seq_start": c["seq_start"][:, :2].contiguous()},
                       conv_state_out=win)
    assert (win[..., :2] == 0).all() and torch.equal(win[0, :, 2:], c["x"][0, :2].t())


def test_conv1d_gradients_against_differences(ssm):
    c, dy = conv_case(2, 30, 9, 4, F32, seed=12, packed=True)
    got = ssm.ssm_conv1d_bwd(**c, dy=dy)
    s, v = c["seq_start"].cpu(), {k: up(c[k]) for k in ("x", "weight", "bias", "conv_state")}
    loss = lambda w: float((R.conv(**w, seq_start=s)[0] * up(dy)).sum())  # noqa: E731
    for k in ("x", "weight", "bias"):
        dirn = torch.randn(v[k].shape, generator=gen(13), dtype=F64)
        e = 1e-6
        num = (loss({**v, k: v[k] + e * dirn}) - loss({**v, k: v[k] - e * dirn})) / (2 * e)
        ana = float((up(got["d" + k]) * dirn).sum())
        lim = 1e-5 * max(1.0, abs(num)) + 2.0 ** -18 * float((up(got["d" + k]) * dirn).abs().sum())
        assert abs(num - ana) <= lim, (k, num, ana)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("b,d,K", [(1, 1, 4), (3, 37, 4), (2, 64, 3), (5, 130, 8), (2, 9, 1), (64, 2560, 4),
                                   (3, 256, 2)])
def test_conv1d_update(ssm, b, d, K, dtype):
    c, _ = conv_case(b, 3, d, K, dtype, seed=d + K)
    ref, w_ref = R.conv(*(up(c[k]) for k in ("x", "weight", "bias")), conv_state=up(c["conv_state"]))
    win = c["conv_state"].clone()
    lim = (K + 6) * 2.0 ** -21 * float(up(c["weight"]).abs().sum(1).max()) * 5.0
    for t in range(3):
        y = ssm.ssm_conv1d_update(win, c["x"][:, t], c["weight"], bias=c["bias"])
        close("y", y, ref[:, t], lim)
    assert torch.equal(win.cpu().to(F64), w_ref)


# ------------------------------------------------------------------ norms
NORM_SIZES = [(1, 1, 1), (1, 8, 2), (3, 33, 1), (5, 64, 4), (2, 130, 1), (129, 1001, 1), (7, 2048, 8),
              (300, 768, 1), (4, 4096, 2), (3, 5120, 1), (2, 8192, 1), (2, 12345, 1), (1, 40000, 1),
              (700, 24, 3), (0, 16, 1), (64, 512, 64)]


def norm_limits(d, n):
    """fp32 error of a normed value, relative: the mean of d squares in any
    order d u / 2 at most, in pairs of lanes far less; sqrt and divisions 2^-21."""
    return d * U / 2 + 2.0 ** -19


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,d,groups", NORM_SIZES)
@pytest.mark.parametrize("form", ["after", "before", "none"])
def test_gated_norm(ssm, rows, d, groups, form, dtype):
    g = gen(rows + d)
    view = strided if (rows + d) % 2 else (lambda t: t)
    x, z = view(randn(g, rows, d, dtype=dtype)), view(randn(g, rows, d, dtype=dtype))
    w, dy = 1 + randn(g, d, scale=0.1), view(randn(g, rows, d, dtype=dtype))
    z = None if form == "none" else z
    kw = dict(groups=groups, norm_before_gate=form == "before")
    y = ssm.ssm_gated_norm_fwd(x, z, w, **kw)
    got = ssm.ssm_gated_norm_bwd(x, z, w, dy, **kw)
    v = [up(t, True) for t in (x, z, w) if t is not None]
    ref = R.gated_norm(v[0], v[1] if z is not None else None, v[-1], groups, before=form == "before")
    gr = torch.autograd.grad((ref * up(dy)).sum(), v)
    rel = norm_limits(d // groups, rows)
    ym = amax(ref.detach())
    close("y", y, ref, rel * ym)
    close("dx", got["dx"], gr[0], 4 * rel * max(amax(gr[0]), 1e-3) + rel * amax(v[-1].detach()) * amax(up(dy)))
    if z is not None:
        close("dz", got["dz"], gr[1], 4 * rel * max(amax(gr[1]), 1e-3) + rel * ym * amax(up(dy)))
    close("dweight", got["dweight"], gr[-1], (rows * U + rel) * max(rows, 1) * amax(up(dy)) * ym * 1.3)


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("rows,d", [(n, d) for n, d, _ in NORM_SIZES])
@pytest.mark.parametrize("form", ["plain", "scale", "post", "both", "first"])
def test_add_norm(ssm, rows, d, form, dtype, res):
    g = gen(rows + d)
    view = strided if (rows + d) % 2 else (lambda t: t)
    x = view(randn(g, rows, d, dtype=dtype))
    r = None if form == "first" else view(randn(g, rows, d, dtype=res, scale=2.0))
    w = 1 + randn(g, d, scale=0.1)
    scale = 0.5 + randn(g, d, scale=0.1) if form in ("scale", "both") else None
    post = 1 + randn(g, d, scale=0.1) if form in ("post", "both") else None
    dy, dro = view(randn(g, rows, d, dtype=dtype)), view(randn(g, rows, d, dtype=res))
    y, ro = ssm.ssm_add_norm_fwd(x, r, w, scale=scale, post_weight=post, residual_dtype=res)
    got = ssm.ssm_add_norm_bwd(x, ro, w, dy, dresidual_out=dro, scale=scale, post_weight=post)
    rel = norm_limits(d, rows)
    v = {k: up(t, True) for k, t in dict(x=x, residual=r, weight=w, scale=scale, post=post).items()}
    _, r_ref = R.add_norm(**v)
    close("residual_out", ro, r_ref, rel * amax(r_ref.detach()))
    # y and the gradients are those of the rounded residual that the call returned
    ref, r_ref = R.add_norm(**v)
    kept = r_ref + (up(ro) - r_ref.detach())
    ref = R.rms(kept, 1e-5) * v["weight"]
    close("y", y, ref, rel * amax(ref.detach()))
    names = [k for k, t in v.items() if t is not None]
    gr = dict(zip(names, torch.autograd.grad((ref * up(dy)).sum() + (kept * up(dro)).sum(),
                                             [v[k] for k in names])))
    dm, drm = amax(up(dy)), amax(up(dro))
    rs = 1.0 if not rows else float((1 / torch.sqrt((up(ro) ** 2).mean(-1) + 1e-5)).max())
    top = amax(v["weight"].detach()) * dm * rs * (1 + amax(ref.detach())) + drm
    if "residual" in gr:
        close("dresidual", got["dresidual"], gr["residual"], 4 * rel * top)
    amp = 1.0 if not rows or post is None else float((1 / torch.sqrt((up(x) ** 2).mean(-1) + 1e-5)).max())
    xn = amax(R.rms(up(x), 1e-5)) if post is not None else amax(up(x))
    close("dx", got["dx"], gr["x"], 8 * rel * top * amp * 2.0 * (1 + xn ** 2 if post is not None else 1))
    n = max(rows, 1)
    close("dweight", got["dweight"], gr["weight"], (n * U + rel) * n * dm * amax(ref.detach()) * 1.5)
    if scale is not None:
        close("dscale", got["dscale"], gr["scale"], (n * U + 4 * rel) * n * top * xn * 2.0)
    if post is not None:
        close("dpost_weight", got["dpost_weight"], gr["post"], (n * U + 4 * rel) * n * top * xn * 2.0)


def test_add_norm_in_place_and_optional(ssm):
    g = gen(3)
    x, r, w = randn(g, 9, 200, dtype=BF), randn(g, 9, 200), 1 + randn(g, 200, scale=0.1)
    y, ro = ssm.ssm_add_norm_fwd(x, r, w)
    r2 = r.clone()
    y2, ro2 = ssm.ssm_add_norm_fwd(x, r2, w, residual_out=r2)
    assert ro2 is r2 and torch.equal(ro, r2) and torch.equal(y, y2)
    dy, dro = randn(g, 9, 200, dtype=BF), randn(g, 9, 200)
    got = ssm.ssm_add_norm_bwd(None, ro, w, dy, dresidual_out=dro)
    d2 = dro.clone()
    again = ssm.ssm_add_norm_bwd(x, ro, w, dy, dresidual_out=d2, out=dict(dresidual=d2))
    assert again["dresidual"] is d2
    for k in got:
        assert torch.equal(got[k], again[k]), k
    none = ssm.ssm_add_norm_bwd(None, ro, w, dy, want_dresidual=False)
    zero = ssm.ssm_add_norm_bwd(None, ro, w, dy, dresidual_out=torch.zeros_like(dro))
    assert "dresidual" not in none and torch.equal(none["dx"], zero["dx"])


@pytest.mark.parametrize("post", [False, True])
def test_norm_gradients_against_differences(ssm, post):
    g = gen(21)
    x, r, z = randn(g, 6, 40), randn(g, 6, 40), randn(g, 6, 40)
    w, sc, pw = 1 + randn(g, 40, scale=0.1), 0.5 + randn(g, 40, scale=0.1), 1 + randn(g, 40, scale=0.1)
    dy, dro = randn(g, 6, 40), randn(g, 6, 40)
    if post:
        _, ro = ssm.ssm_add_norm_fwd(x, r, w, scale=sc, post_weight=pw)
        got = ssm.ssm_add_norm_bwd(x, ro, w, dy, dresidual_out=dro, scale=sc, post_weight=pw)
        got["dpost"] = got["dpost_weight"]
        v = dict(x=x, residual=r, weight=w, scale=sc, post=pw)

        def loss(q):
            y, o = R.add_norm(**q)
            return float((y * up(dy)).sum() + (o * up(dro)).sum())
    else:
        got = ssm.ssm_gated_norm_bwd(x, z, w, dy, groups=2)
        v = dict(x=x, z=z, weight=w)
        loss = lambda q: float((R.gated_norm(**q, groups=2) * up(dy)).sum())  # noqa: E731
    v = {k: up(t) for k, t in v.items()}
    for k in v:
        dirn = torch.randn(v[k].shape, generator=gen(22), dtype=F64)
        e = 1e-6
        num = (loss({**v, k: v[k] + e * dirn}) - loss({**v, k: v[k] - e * dirn})) / (2 * e)
        gk = up(got["d" + k])
        lim = 1e-6 * max(1.0, abs(num)) + 2.0 ** -18 * float((gk * dirn).abs().sum())
        assert abs(num - float((gk * dirn).sum())) <= lim, k


def test_norm_of_zero_rows_and_bad_rows(ssm):
    """A row of zeros norms to zero (eps), and a row with NaN or infinities
    leaves its neighbours alone."""
    x = torch.randn(6, 300, generator=gen(5)).cuda()
    z, w = torch.randn(6, 300, generator=gen(6)).cuda(), torch.ones(300, device="cuda")
    x[2] = 0
    y = ssm.ssm_gated_norm_fwd(x, z, w)
    assert (y[2] == 0).all()
    g = ssm.ssm_gated_norm_bwd(x, z, w, torch.ones_like(x))
    assert torch.isfinite(g["dx"]).all()
    xb = x.clone()
    xb[3, 7] = float("nan")
    xb[4, 7] = float("inf")
    yb = ssm.ssm_gated_norm_fwd(xb, z, w)
    assert torch.isnan(yb[3]).all()
    for k in (0, 1, 2, 5):
        assert torch.equal(yb[k], y[k])


# ------------------------------------------------ how calls are made
def every_call(S, seed=0, stream=None, keep=None):
    """One call of everything; outputs by name.  keep: tensors of an earlier
    call to write into."""
    k = keep or {}
    c, dout, dh = k.get("gated") or gated_case(2, 300, 96, BF, seed=seed, packed=True)
    cc, dy = k.get("conv") or conv_case(2, 300, 96, 4, BF, seed=seed, packed=True)
    g = gen(seed)
    n = k.get("norm") or dict(x=randn(g, 400, 768, dtype=BF), z=randn(g, 400, 768, dtype=BF),
                              w=1 + randn(g, 768, scale=0.1), s=0.5 + randn(g, 768, scale=0.1),
                              r=randn(g, 400, 768), dy=randn(g, 400, 768, dtype=BF), dr=randn(g, 400, 768))
    st, win = c["h0"].clone(), cc["conv_state"].clone()
    keep = dict(gated=(c, dout, dh), conv=(cc, dy), norm=n)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    out = gated_all(S, c, dout, dh, stream=stream)
    out["step_y"] = S.ssm_gated_state_update(st, c["u"][:, 0], c["gate_a"][:, 0], c["gate_x"][:, 0], c["A"],
                                             stream=stream)
    out["conv_y"] = S.ssm_conv1d_fwd(**cc, stream=stream)
    out.update({"conv_" + q: t for q, t in S.ssm_conv1d_bwd(**cc, dy=dy, stream=stream).items()})
    out["conv_step_y"] = S.ssm_conv1d_update(win, cc["x"][:, 0], cc["weight"], stream=stream)
    out["norm_y"] = S.ssm_gated_norm_fwd(n["x"], n["z"], n["w"], groups=2, stream=stream)
    out.update({"norm_" + q: t for q, t in
                S.ssm_gated_norm_bwd(n["x"], n["z"], n["w"], n["dy"], groups=2, stream=stream).items()})
    kw = dict(scale=n["s"], post_weight=n["w"], stream=stream)
    out["add_y"], ro = S.ssm_add_norm_fwd(n["x"], n["r"], n["w"], **kw)
    out.update({"add_" + q: t for q, t in
                S.ssm_add_norm_bwd(n["x"], ro, n["w"], n["dy"], dresidual_out=n["dr"], **kw).items()})
    out.update(st=st, win=win, ro=ro)
    return out, keep


def test_calls_repeat_bit_for_bit(ssm):
    a, keep = every_call(ssm)
    for _ in range(2):
        b, _ = every_call(ssm, keep=keep)
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k], b[k]), k


def test_calls_on_another_stream(ssm):
    a, keep = every_call(ssm)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b, _ = every_call(ssm, stream=s, keep=keep)
    s.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_calls_in_two_graphs(ssm):
    """Two graphs captured one after the other, replayed in turn and again,
    give what eager calls give (their scratch is each graph's own)."""
    eager, keeps, graphs, outs = [], [], [], []
    for seed in (1, 2):
        o, keep = every_call(ssm, seed=seed)
        eager.append({k: t.clone() for k, t in o.items()})
        keeps.append(keep)
    torch.cuda.synchronize()
    for keep in keeps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, _ = every_call(ssm, keep=keep)
        graphs.append(g)
        outs.append(o)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        for k in e:
            assert torch.equal(e[k], o[k]), k


def test_rows_beyond_2_32_elements(ssm):
    """Row offsets past 32 bits: three rows 1.6e9 elements apart."""
    ld = 1_600_000_000
    big = torch.empty(2 * ld + 64, dtype=BF, device="cuda")
    rows = big.as_strided((1, 3, 64), (3 * ld, ld, 1))
    src = randn(gen(1), 1, 3, 64, dtype=BF)
    rows.copy_(src)
    c, _, _ = gated_case(1, 3, 64, BF, seed=2)
    want = ssm.ssm_gated_scan_fwd(**{**c, "u": src})
    assert torch.equal(ssm.ssm_gated_scan_fwd(**{**c, "u": rows}), want)
    cc, _ = conv_case(1, 3, 64, 4, BF, seed=2)
    want = ssm.ssm_conv1d_fwd(**{**cc, "x": src})
    assert torch.equal(ssm.ssm_conv1d_fwd(**{**cc, "x": rows}), want)
    w = torch.ones(64, device="cuda")
    want = ssm.ssm_gated_norm_fwd(src, None, w)
    assert torch.equal(ssm.ssm_gated_norm_fwd(rows, None, w), want)
    ssm.ssm_gated_norm_fwd(src, None, w, y=rows)
    assert torch.equal(rows.contiguous(), want)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_block_of_them_all(ssm, dtype):
    """A residual block of the recurrence as a model runs it -- add norm, input
    projection, convolution, gate projections, gated scan, gated norm, output
    projection, the next add norm -- forward and backward over a packed batch,
    against the same block in 64 bits; then prefill and decode of the same
    tokens against the whole forward."""
    b, L, dm, d, K = 2, 96, 32, 48, 4
    g = gen(31)
    rn = lambda *s, k=1.0: torch.randn(*s, generator=g) * k  # noqa: E731
    P = dict(w0=1 + rn(dm, k=0.1), win=rn(dm, 2 * d, k=dm ** -0.5), cw=rn(d, K, k=0.5), cb=rn(d, k=0.1),
             wg=rn(d, 2 * d, k=d ** -0.5), A=torch.log(0.9 + 0.099 * torch.rand(d, generator=g)),
             ba=rn(d, k=0.3), bx=rn(d, k=0.3), wn=1 + rn(d, k=0.1), wo=rn(d, dm, k=d ** -0.5),
             sc=0.5 + rn(dm, k=0.1), w1=1 + rn(dm, k=0.1), pw=1 + rn(dm, k=0.1))
    mats = ("win", "wg", "wo")
    P = {k: v.to(dtype) if k in mats else v for k, v in P.items()}
    x, res = rn(b, L, dm).to(dtype), rn(b, L, dm)
    dy, dro = rn(b, L, dm).to(dtype), rn(b, L, dm)
    start = (torch.rand(b, L, generator=g) < 0.05).to(torch.uint8)
    G = {k: v.cuda() for k, v in P.items()}
    S, sg = ssm, start.cuda()

    def forward(x, res, sg, h0=None, cs=None, keep=False):
        n = x.shape[1]
        y0, r0 = S.ssm_add_norm_fwd(x, res, G["w0"])
        xz = y0 @ G["win"]
        xi, z = xz.split(d, -1)
        cs_out = torch.empty(b, d, K, dtype=dtype, device="cuda")
        u = S.ssm_conv1d_fwd(xi, G["cw"], bias=G["cb"], conv_state=cs, conv_state_out=cs_out, seq_start=sg)
        gates = u @ G["wg"]
        ga, gx = gates.split(d, -1)
        st = torch.empty(S.ssm_gated_scan_states_bytes(b, n, d) // 4, device="cuda") if keep else None
        h = torch.empty(b, d, device="cuda")
        hs = S.ssm_gated_scan_fwd(u, ga, gx, G["A"], bias_a=G["ba"], bias_x=G["bx"], seq_start=sg, h0=h0,
                                  h_last=h, chunk_states=st)
        o = S.ssm_gated_norm_fwd(hs, z, G["wn"])
        out = o @ G["wo"]
        y1, r1 = S.ssm_add_norm_fwd(out, r0, G["w1"], scale=G["sc"], post_weight=G["pw"])
        return y1, r1, h, cs_out, (y0, r0, xi, z, u, gates, ga, gx, st, hs, o, out)

    y1, r1, h, cs, (y0, r0, xi, z, u, gates, ga, gx, st, hs, o, out) = \
        forward(x.cuda(), res.cuda(), sg, keep=True)
    # backward
    kw = dict(scale=G["sc"], post_weight=G["pw"])
    g1 = S.ssm_add_norm_bwd(out, r1, G["w1"], dy.cuda(), dresidual_out=dro.cuda(), **kw)
    do = g1["dx"] @ G["wo"].t()
    got = dict(w1=g1["dweight"], sc=g1["dscale"], pw=g1["dpost_weight"],
               wo=o.flatten(0, 1).t() @ g1["dx"].flatten(0, 1))
    dxz, dg = torch.empty(b, L, 2 * d, dtype=dtype, device="cuda"), torch.empty_like(gates)
    g2 = S.ssm_gated_norm_bwd(hs, z, G["wn"], do, out=dict(dz=dxz[..., d:]))
    got["wn"] = g2["dweight"]
    g3 = S.ssm_gated_scan_bwd(u, ga, gx, G["A"], g2["dx"], st, bias_a=G["ba"], bias_x=G["bx"], seq_start=sg,
                              out=dict(dgate_a=dg[..., :d], dgate_x=dg[..., d:]))
    got.update(A=g3["dA"], ba=g3["dbias_a"], bx=g3["dbias_x"], wg=u.flatten(0, 1).t() @ dg.flatten(0, 1))
    g4 = S.ssm_conv1d_bwd(xi, G["cw"], g3["du"] + dg @ G["wg"].t(), bias=G["cb"], seq_start=sg,
                          out=dict(dx=dxz[..., :d]))
    got.update(cw=g4["dweight"], cb=g4["dbias"], win=y0.flatten(0, 1).t() @ dxz.flatten(0, 1))
    g5 = S.ssm_add_norm_bwd(None, r0, G["w0"], dxz @ G["win"].t(), dresidual_out=g1["dresidual"])
    got.update(w0=g5["dweight"], x=g5["dx"], res=g5["dresidual"])
    # the same block in 64 bits
    v = {k: up(t, True) for k, t in dict(P, x=x, res=res).items()}
    q0, t0 = R.add_norm(v["x"], v["res"], v["w0"])
    qx, qz = (q0 @ v["win"]).split(d, -1)
    qu, _ = R.conv(qx, v["cw"], v["cb"], seq_start=start)
    qa, qg = (qu @ v["wg"]).split(d, -1)
    qh, qlast = R.gated(qu, qa, qg, v["A"], v["ba"], v["bx"], seq_start=start)
    q1, t1 = R.add_norm(R.gated_norm(qh, qz, v["wn"]) @ v["wo"], t0, v["w1"], v["sc"], v["pw"])
    gr = torch.autograd.grad((q1 * up(dy)).sum() + (t1 * up(dro)).sum(), list(v.values()))
    # fp32: some 2^-18 an operator, 10 of them, products of up to 96 terms; bf16: 12 roundings of 2^-8, each
    # amplified by the operators behind it up to 4 times, in the 2-norm
    tol = 2.0 ** -14 if dtype == F32 else 12 * 4 * 2.0 ** -8
    for k, (t, ref) in {**{k: (got[k], r) for k, r in zip(v, gr)}, "y1": (y1, q1), "r1": (r1, t1),
                        "h": (h, qlast)}.items():
        t, ref = up(t), ref.detach()
        assert float((t - ref).norm() / ref.norm()) <= tol, k
    # prefill of all but the last three tokens, then decode (no starts among those)
    sg[:, L - 3:] = 0
    whole = forward(x.cuda(), res.cuda(), sg)
    cut = L - 3
    _, _, h, cs, _ = forward(x[:, :cut].cuda(), res[:, :cut].cuda(), sg[:, :cut].contiguous())
    for t in range(cut, L):
        a0, b0 = S.ssm_add_norm_fwd(x[:, t].cuda(), res[:, t].cuda(), G["w0"])
        xi, z = (a0 @ G["win"]).split(d, -1)
        u = S.ssm_conv1d_update(cs, xi, G["cw"], bias=G["cb"])
        ga, gx = (u @ G["wg"]).split(d, -1)
        hs = S.ssm_gated_state_update(h, u, ga, gx, G["A"], bias_a=G["ba"], bias_x=G["bx"])
        o = S.ssm_gated_norm_fwd(hs, z, G["wn"])
        y, _ = S.ssm_add_norm_fwd(o @ G["wo"], b0, G["w1"], scale=G["sc"], post_weight=G["pw"])
        ref = up(whole[0][:, t])
        assert float((up(y) - ref).norm() / ref.norm()) <= tol
    assert float((up(h) - up(whole[2])).norm() / up(whole[2]).norm()) <= tol
