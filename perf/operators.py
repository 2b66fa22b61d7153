"""Workloads of the recurrent-block operators: the gated linear recurrence, the
causal depthwise convolution over a sequence, the gated RMS norm and the
residual-add norm, each in the directions a training step, a prefill and a
decode loop call them in.

``run`` computes a case in plain fp32 torch operations, or with ``own`` through
selective_state_space_25_b200.ssmscan.  ``exact`` is the definition in 64 bits,
its gradients by automatic differentiation.

Formulas (r, i gates in (0, 1); A <= 0 the log decay of a fully open gate):
  gated scan   r = sigmoid(gate_a + bias_a), i = sigmoid(gate_x + bias_x),
               a = exp(A r), h_t = a h_{t-1} + sqrt(1 - a^2) i u,
               y = h silu(z); where seq_start is set a sequence begins:
               h_t = i u, whatever came before
  conv1d       y_t = silu(sum_j weight[j] x_{t-K+1+j} + bias), taps before the
               first step read the window, taps before a sequence's start are 0
  gated norm   y = rms(x silu(z)) weight per group of channels, or with the
               norm before the gate rms(x) weight silu(z); rms(v) = v /
               sqrt(mean v^2 + eps)
  add norm     r' = residual + scale (post_weight ? rms(x) post_weight : x)
               rounded to the residual's type, y = rms(r') weight
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64


def listed():
    return [
        # one token of a small decode batch, channels of a 2560-wide model: latency
        dict(name="gated-step-b4", op="gated_step", dtype="bf16", b=4, d=2560, gate=True),
        # a training step of the 130M block's shape (b=8, L=2048, d_in=1536)
        dict(name="gated-train-130m", op="gated_train", dtype="bf16", b=8, L=2048, d=1536, gate=True,
             carry=False, packed=False),
        # one long prompt prefilled into a decode state, few channels
        dict(name="gated-prefill-long", op="gated_fwd", dtype="bf16", b=1, L=16384, d=2560, gate=False,
             carry=True, packed=False),
        # fp32 training of packed documents, odd sizes, a carried state
        dict(name="gated-train-odd", op="gated_train", dtype="fp32", b=3, L=1001, d=509, gate=True,
             carry=True, packed=True),
        # the conv step of a full decode batch (b=256, d_in=5120, d_conv=4)
        dict(name="conv-step-b256", op="conv_step", dtype="bf16", b=256, d=5120, K=4),
        # the conv of a training step over packed documents
        dict(name="conv-train-130m", op="conv_train", dtype="bf16", b=8, L=2048, d=1536, K=4,
             halves=False, carry=False, packed=True),
        # the conv of a long prefill, read out of the input projection's (x, z) rows
        dict(name="conv-prefill-long", op="conv_fwd", dtype="bf16", b=1, L=16384, d=4096, K=4,
             halves=True, carry=True, packed=False),
        # the norm and gate in front of the output projection, training
        dict(name="gated-norm-train", op="gated_norm_train", dtype="bf16", rows=16384, d=1536, groups=1,
             before=False, halves=False),
        # the same for one decode step of 256 sequences, 8 groups, norm before gate
        dict(name="gated-norm-b256", op="gated_norm_fwd", dtype="bf16", rows=256, d=5120, groups=8,
             before=True, halves=True),
        # residual + scale * post norm, then the next block's norm: training, fp32 residual
        dict(name="add-norm-train", op="add_norm_train", dtype="bf16", res="fp32", rows=16384, d=768,
             scaled=True, post=True, first=False),
        # the plain pre-norm of a large prefill batch, bf16 residual
        dict(name="add-norm-prefill", op="add_norm_fwd", dtype="bf16", res="bf16", rows=32768, d=2048,
             scaled=False, post=False, first=False),
        # a small fp32 training step of odd sizes
        dict(name="add-norm-odd", op="add_norm_train", dtype="fp32", res="fp32", rows=129, d=1001,
             scaled=True, post=False, first=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.35 else max(lo, d // 64 * 64 or d)  # odd widths among multiples of 64


def draw(rng):
    op = rng.choice(["gated_step", "gated_fwd", "gated_train", "gated_train", "conv_step", "conv_fwd",
                     "conv_train", "gated_norm_fwd", "gated_norm_train", "add_norm_fwd",
                     "add_norm_train"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op.endswith("_step"):
        c.update(b=_log(rng, 1, 256), d=_width(rng, 64, 8192))
    elif "norm" in op:
        d = _width(rng, 16, 8192)
        c.update(rows=_log(rng, 1, max(2, min(32768, (1 << 25) // d))), d=d)
    else:
        d = _width(rng, 16, 4096)
        L = _log(rng, 1, 16384)
        c.update(b=_log(rng, 1, max(1, min(16, (1 << 24) // (d * L)))), L=L, d=d)
        c.update(carry=rng.random() < 0.5, packed=rng.random() < 0.4)
    if op.startswith("gated_norm"):
        groups = [g for g in (1, 2, 4, 8) if c["d"] % g == 0]
        c.update(groups=rng.choice(groups), before=rng.random() < 0.5, halves=rng.random() < 0.4)
    elif op.startswith("gated"):
        c.update(gate=rng.random() < 0.6)
    elif op.startswith("conv"):
        c.update(K=rng.choice([2, 3, 4, 4, 5, 8]))
        if op != "conv_step":
            c.update(halves=rng.random() < 0.4)
    else:
        # in training a bf16 residual's rounding would stand between the two directions
        c.update(res="fp32" if op == "add_norm_train" else rng.choice(["fp32", c["dtype"]]),
                 scaled=rng.random() < 0.5, post=rng.random() < 0.5, first=rng.random() < 0.15)
    return c


# ------------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else F32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    act = _dt(case["dtype"])
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    op, d = case["op"], case["d"]
    s = dict(case=case)
    if "norm" in op:
        lead = (case["rows"],)
    elif op.endswith("_step"):
        lead = (case["b"],)
    else:
        lead = (case["b"], case["L"])

    def pair():  # two activations, as halves of one projection's rows or apart
        if case.get("halves"):
            return n(*lead, 2 * d).to(act).split(d, -1)
        return n(*lead, d).to(act), n(*lead, d).to(act)

    if op.startswith("gated_norm"):
        s["x"], s["z"] = pair()
        s["weight"] = 1 + 0.1 * n(d)
        s["dy"] = n(*lead, d).to(act) if op.endswith("train") else None
        return s
    if op.startswith("add_norm"):
        res = _dt(case["res"])
        s["x"] = n(*lead, d).to(act)
        s["residual"] = None if case["first"] else (2 * n(*lead, d)).to(res)
        s["weight"] = 1 + 0.1 * n(d)
        s["scale"] = 0.5 + 0.1 * n(d) if case["scaled"] else None
        s["post"] = 1 + 0.1 * n(d) if case["post"] else None
        if op.endswith("train"):
            s["dy"], s["dres"] = n(*lead, d).to(act), n(*lead, d).to(res)
        return s
    start = None
    if case.get("packed"):  # documents of some 300 tokens, one starting at step 0 in half of the rows
        start = (uni(*lead) < 1 / 300).to(torch.uint8)
        start[:, 0] = (uni(lead[0]) < 0.5).to(torch.uint8)
    if op.startswith("conv"):
        K = case["K"]
        s["x"] = pair()[0] if case.get("halves") else n(*lead, d).to(act)
        s["weight"] = (2 * uni(d, K) - 1) / math.sqrt(K)
        s["bias"] = (2 * uni(d) - 1) / math.sqrt(K)
        s["window"] = n(case["b"], d, K).to(act) if case.get("carry") or op == "conv_step" else None
        s["start"] = start
        s["dy"] = n(*lead, d).to(act) if op == "conv_train" else None
        return s
    s["u"], s["ga"], s["gx"] = n(*lead, d).to(act), n(*lead, d).to(act), n(*lead, d).to(act)
    s["z"] = n(*lead, d).to(act) if case["gate"] else None
    s["A"] = torch.log(0.9 + 0.099 * uni(d))  # decays of 0.9 to 0.999 a step
    s["ba"], s["bx"] = 0.5 * n(d), 0.5 * n(d)
    s["h"] = n(case["b"], d) if case.get("carry") or op == "gated_step" else None
    s["start"] = start
    if op == "gated_train":
        s["dout"] = n(*lead, d).to(act)
        s["dh"] = n(case["b"], d) if case["carry"] else None
    return s


# -------------------------------------------------------------- plain forms
def _silu(z):
    return z * torch.sigmoid(z)


def _dsilu(z):
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _decay(s, ga, gx):
    """Gates, decay and input factor of the recurrence."""
    r, i = torch.sigmoid(ga.float() + s["ba"]), torch.sigmoid(gx.float() + s["bx"])
    la = s["A"] * r
    a, beta = torch.exp(la), torch.sqrt(torch.clamp(-torch.expm1(2 * la), min=0))
    if s["start"] is not None:
        m = s["start"].bool().unsqueeze(-1)
        a, beta = a.masked_fill(m, 0.0), beta.masked_fill(m, 1.0)
    return r, i, a, beta


def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t along dim 1 from h = 0, by doubling spans; a
    decay of 0 cuts off what is before it, infinities and NaN too."""
    L, span = x.shape[1], 1
    while span < L:
        p = a[:, span:]
        x = torch.cat([x[:, :span], x[:, span:] + torch.where(p == 0, 0.0, p * x[:, :-span])], 1)
        a = torch.cat([a[:, :span], p * a[:, :-span]], 1)
        span *= 2
    return x


def _plain_gated(s):
    c, act = s["case"], s["u"].dtype
    u = s["u"].float()
    r, i, a, beta = _decay(s, s["ga"], s["gx"])
    x = beta * i * u
    if c["op"] == "gated_step":
        h = a * s["h"] + x
        s["h"].copy_(h)
        return dict(y=(h * _silu(s["z"].float()) if c["gate"] else h).to(act), h=s["h"])
    if s["h"] is not None:
        x[:, 0] += torch.where(a[:, 0] == 0, 0.0, a[:, 0] * s["h"])
    h = _scan(a, x)
    out = dict(y=(h * _silu(s["z"].float()) if c["gate"] else h).to(act))
    if s["h"] is not None:
        out["h_last"] = h[:, -1].contiguous()
    if c["op"] == "gated_fwd":
        return out
    do = s["dout"].float()
    g = do * _silu(s["z"].float()) if c["gate"] else do.clone()
    if s["dh"] is not None:
        g[:, -1] += s["dh"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _scan(later.flip(1), g.flip(1)).flip(1)
    h0 = torch.zeros_like(h[:, :1]) if s["h"] is None else s["h"].unsqueeze(1)
    prev = torch.cat([h0, h[:, :-1]], 1)
    da = torch.where(a == 0, 0.0, lam * (prev * a - i * u * (a * a / torch.where(beta > 0, beta, math.inf))))
    dga = da * s["A"] * r * (1 - r)
    dgx = lam * beta * u * i * (1 - i)
    out.update(du=(lam * beta * i).to(act), dgate_a=dga.to(act), dgate_x=dgx.to(act),
               dA=(da * r).sum((0, 1)), dbias_a=dga.sum((0, 1)), dbias_x=dgx.sum((0, 1)))
    if c["gate"]:
        out["dz"] = (do * h * _dsilu(s["z"].float())).to(act)
    if s["h"] is not None:
        out["dh0"] = torch.where(a[:, 0] == 0, 0.0, a[:, 0] * lam[:, 0])
    return out


def _plain_conv(s):
    c, act = s["case"], s["x"].dtype
    K, w = c["K"], s["weight"]
    if c["op"] == "conv_step":
        s["window"].copy_(torch.cat([s["window"][:, :, 1:], s["x"].unsqueeze(-1)], -1))
        return dict(y=_silu((s["window"].float() * w).sum(-1) + s["bias"]).to(act), window=s["window"])
    x = s["x"].float()
    b, L, d = x.shape
    before = x.new_zeros(b, K, d) if s["window"] is None else s["window"].float().transpose(1, 2)
    xp = torch.cat([before, x], 1)  # step t is row t + K
    t = torch.arange(L, device=x.device)
    if s["start"] is None:
        age = torch.full((b, L), L + K, device=x.device)
    else:
        first = torch.where(s["start"] != 0, t, -L - K)
        age = t - torch.cummax(first, 1).values  # steps since the sequence's start
    taps = [torch.where((age >= m).unsqueeze(-1), xp[:, K - m:K - m + L], 0.0) for m in range(K)]
    pre = sum(taps[m] * w[:, K - 1 - m] for m in range(K)) + s["bias"]
    out = dict(y=_silu(pre).to(act))
    if c["carry"]:
        back = torch.arange(K - 1, -1, -1, device=x.device)  # how far behind the last step
        alive = age[:, -1:] >= back
        out["window"] = torch.where(alive.unsqueeze(-1), xp[:, L:], 0.0).transpose(1, 2).contiguous().to(act)
    if c["op"] == "conv_fwd":
        return out
    dp = s["dy"].float() * _dsilu(pre)
    dpp = torch.cat([dp, dp.new_zeros(b, K, d)], 1)
    agep = torch.cat([age, age.new_zeros(b, K)], 1)
    dx = sum(torch.where((agep[:, m:m + L] >= m).unsqueeze(-1), dpp[:, m:m + L], 0.0) * w[:, K - 1 - m]
             for m in range(K))
    dw = torch.stack([(dp * taps[K - 1 - j]).sum((0, 1)) for j in range(K)], -1)
    out.update(dx=dx.to(act), dweight=dw, dbias=dp.sum((0, 1)))
    return out


EPS = 1e-5


def _plain_gated_norm(s):
    c, act = s["case"], s["x"].dtype
    R, d, G = c["rows"], c["d"], c["groups"]
    x, z = s["x"].float().reshape(R, G, -1), s["z"].float().reshape(R, G, -1)
    w, gate = s["weight"].reshape(G, -1), _silu(z)
    v = x if c["before"] else x * gate
    rs = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    n = v * rs
    y = n * w * gate if c["before"] else n * w
    out = dict(y=y.reshape(R, d).to(act))
    if c["op"] == "gated_norm_fwd":
        return out
    dy = s["dy"].float().reshape(R, G, -1)
    dn = dy * w * gate if c["before"] else dy * w
    dv = rs * (dn - n * (dn * n).mean(-1, keepdim=True))
    dx = dv if c["before"] else dv * gate
    dz = (dy * n * w if c["before"] else dv * x) * _dsilu(z)
    dw = (dy * n * gate if c["before"] else dy * n).sum(0)
    out.update(dx=dx.reshape(R, d).to(act), dz=dz.reshape(R, d).to(act), dweight=dw.reshape(d))
    return out


def _plain_add_norm(s):
    c, act = s["case"], s["x"].dtype
    res = _dt(c["res"])
    x, w = s["x"].float(), s["weight"]
    if c["post"]:
        rx = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xn = x * rx
        v = xn * s["post"]
    else:
        v = x
    r = v * s["scale"] if c["scaled"] else v
    r = r if c["first"] else r + s["residual"].float()
    ro = r.to(res)
    r = ro.float()
    rs = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n = r * rs
    out = dict(y=(n * w).to(act), residual=ro)
    if c["op"] == "add_norm_fwd":
        return out
    dn = s["dy"].float() * w
    dr = rs * (dn - n * (dn * n).mean(-1, keepdim=True)) + s["dres"].float()
    dv = dr * s["scale"] if c["scaled"] else dr
    out["dweight"] = (s["dy"].float() * n).sum(0)
    if c["scaled"]:
        out["dscale"] = (dr * v).sum(0)
    if not c["first"]:
        out["dresidual"] = dr.to(res)
    if c["post"]:
        out["dpost_weight"] = (dv * xn).sum(0)
        dxn = dv * s["post"]
        dv = rx * (dxn - xn * (dxn * xn).mean(-1, keepdim=True))
    out["dx"] = dv.to(act)
    return out


# ------------------------------------------------------ the framework's calls
def _own_gated(S, s):
    c = s["case"]
    kw = dict(bias_a=s["ba"], bias_x=s["bx"], z=s["z"])
    if c["op"] == "gated_step":
        y = S.ssm_gated_state_update(s["h"], s["u"], s["ga"], s["gx"], s["A"], **kw)
        return dict(y=y, h=s["h"])
    kw["seq_start"] = s["start"]
    last = None if s["h"] is None else torch.empty_like(s["h"])
    if c["op"] == "gated_fwd":
        y = S.ssm_gated_scan_fwd(s["u"], s["ga"], s["gx"], s["A"], h0=s["h"], h_last=last, **kw)
        return dict(y=y) if last is None else dict(y=y, h_last=last)
    b, L, d = s["u"].shape
    states = torch.empty(S.ssm_gated_scan_states_bytes(b, L, d) // 4, device=s["u"].device)
    y = S.ssm_gated_scan_fwd(s["u"], s["ga"], s["gx"], s["A"], h0=s["h"], h_last=last,
                             chunk_states=states, **kw)
    out = S.ssm_gated_scan_bwd(s["u"], s["ga"], s["gx"], s["A"], s["dout"], states, dh_last=s["dh"],
                               want_dh0=s["h"] is not None, **kw)
    out["y"] = y
    if last is not None:
        out["h_last"] = last
    return out


def _own_conv(S, s):
    c = s["case"]
    if c["op"] == "conv_step":
        y = S.ssm_conv1d_update(s["window"], s["x"], s["weight"], bias=s["bias"])
        return dict(y=y, window=s["window"])
    last = torch.empty_like(s["window"]) if s["window"] is not None else None
    kw = dict(bias=s["bias"], conv_state=s["window"], seq_start=s["start"])
    y = S.ssm_conv1d_fwd(s["x"], s["weight"], conv_state_out=last, **kw)
    out = S.ssm_conv1d_bwd(s["x"], s["weight"], s["dy"], **kw) if c["op"] == "conv_train" else {}
    out["y"] = y
    if last is not None:
        out["window"] = last
    return out


def _own_gated_norm(S, s):
    c = s["case"]
    kw = dict(groups=c["groups"], eps=EPS, norm_before_gate=c["before"])
    y = S.ssm_gated_norm_fwd(s["x"], s["z"], s["weight"], **kw)
    if c["op"] == "gated_norm_fwd":
        return dict(y=y)
    return dict(S.ssm_gated_norm_bwd(s["x"], s["z"], s["weight"], s["dy"], **kw), y=y)


def _own_add_norm(S, s):
    c = s["case"]
    kw = dict(scale=s["scale"], post_weight=s["post"], eps=EPS)
    y, ro = S.ssm_add_norm_fwd(s["x"], s["residual"], s["weight"], residual_dtype=_dt(c["res"]), **kw)
    if c["op"] == "add_norm_fwd":
        return dict(y=y, residual=ro)
    out = S.ssm_add_norm_bwd(s["x"], ro, s["weight"], s["dy"], dresidual_out=s["dres"],
                             want_dresidual=not c["first"], **kw)
    return dict(out, y=y, residual=ro)


def run(state):
    op = state["case"]["op"]
    kind = "_gated_norm" if op.startswith("gated_norm") else "_add_norm" if op.startswith("add") else \
        "_conv" if op.startswith("conv") else "_gated"
    if own:
        from selective_state_space_25_b200 import ssmscan
        return globals()["_own" + kind](ssmscan, state)
    return globals()["_plain" + kind](state)


# ------------------------------------------------------------------ counting
def work(case):
    """Each input read once, each output written once; flops with one for each
    multiply, add and function."""
    op, d = case["op"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    train = op.endswith("train")
    if "norm" in op:
        n = case["rows"] * d
        if op.startswith("gated_norm"):  # x, z, y; and x, z, dy, dx, dz
            return dict(bytes=n * e * (3 + (3 if train else 0)) + 4 * d * (2 if train else 1),
                        flops=n * (9 + (25 if train else 0)))
        r = 2 if case["res"] == "bf16" else 4
        params = 4 * d * (1 + case["scaled"] + case["post"])
        # x, residual, y, residual out; dy, dresidual in and out, dx
        by = n * (2 * e + r * (2 - case["first"])) + params
        by += n * (2 * e + r * (2 - case["first"])) + params if train else 0
        return dict(bytes=by, flops=n * (6 + 4 * case["post"]) * (3 if train else 1))
    n = case["b"] * d * case.get("L", 1)
    if op.startswith("conv"):
        K = case["K"]
        by = n * e * (4 if train else 2) + 4 * d * (K + 1) * (2 if train else 1)
        if op == "conv_step" or case["carry"]:
            by += 2 * case["b"] * d * K * e
        return dict(bytes=by, flops=n * (2 * K + 5) * (3 if train else 1))
    # u, gates, y (and z); dout, du, dgates (and dz)
    by = n * e * (4 + case["gate"] + ((4 + case["gate"]) if train else 0)) + 12 * d * (2 if train else 1)
    if op == "gated_step" or case["carry"]:
        by += 8 * case["b"] * d * (2 if train else 1)
    return dict(bytes=by, flops=n * (18 + (45 if train else 0)))


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definition in 64 bits, step by step in time; gradients by automatic
    differentiation of it."""
    s = prepare(case, seed)
    op = case["op"]
    train = op.endswith("train")
    leaf = {}

    def val(key):
        if s.get(key) is None:
            return None
        if key not in leaf:
            leaf[key] = s[key].to(F64).detach().requires_grad_(train)
        return leaf[key]

    def rms(v):
        return v / ((v ** 2).mean(-1, keepdim=True) + EPS).sqrt()

    def grads(loss, names):
        keys = [k for k in names if s.get(k) is not None]
        got = torch.autograd.grad(loss, [val(k) for k in keys])
        return {names[k]: g for k, g in zip(keys, got)}

    if op.startswith("gated_norm"):
        shape = (case["rows"], case["groups"], -1)
        x, z, w = val("x").reshape(shape), val("z").reshape(shape), val("weight").reshape(shape[1:])
        gate = z / (1 + torch.exp(-z))
        y = (rms(x) * w * gate if case["before"] else rms(x * gate) * w).reshape(case["rows"], -1)
        out = dict(y=y.detach())
        if train:
            out.update(grads((y * s["dy"].to(F64)).sum(), dict(x="dx", z="dz", weight="dweight")))
        return out
    if op.startswith("add_norm"):
        r = val("x") if val("post") is None else rms(val("x")) * val("post")
        r = r if val("scale") is None else r * val("scale")
        r = r if val("residual") is None else r + val("residual")
        kept = r.detach().to(_dt(case["res"]))
        if case["res"] == "bf16":
            r = r + (kept.to(F64) - r.detach())
        y = rms(r) * val("weight")
        out = dict(y=y.detach(), residual=kept.to(F64) if case["res"] == "bf16" else r.detach())
        if train:
            loss = (y * s["dy"].to(F64)).sum() + (r * s["dres"].to(F64)).sum()
            out.update(grads(loss, dict(x="dx", residual="dresidual", weight="dweight", scale="dscale",
                                        post="dpost_weight")))
        return out
    if op.startswith("conv"):
        K, b = case["K"], case["b"]
        x = val("x") if op != "conv_step" else val("x").unsqueeze(1)
        win = val("window")
        hist = [torch.zeros_like(x[:, 0])] * K if win is None else [win[:, :, j] for j in range(K)]
        w, bias, ys = val("weight"), val("bias"), []
        for t in range(x.shape[1]):
            if s["start"] is not None:
                m = s["start"][:, t].bool().view(b, 1)
                hist = [torch.where(m, 0.0, v) for v in hist]
            hist = hist[1:] + [x[:, t]]
            pre = bias
            for j in range(K):
                pre = pre + w[:, j] * hist[j]
            ys.append(pre / (1 + torch.exp(-pre)))
        y = torch.stack(ys, 1)
        out = dict(y=(y if op != "conv_step" else y[:, 0]).detach())
        if win is not None:
            out["window"] = torch.stack(hist, -1).detach()
        if train:
            out.update(grads((y * s["dy"].to(F64)).sum(), dict(x="dx", weight="dweight", bias="dbias")))
        return out
    step = op == "gated_step"
    seq = (lambda v: v.unsqueeze(1)) if step else (lambda v: v)
    u, ga, gx = seq(val("u")), seq(val("ga")), seq(val("gx"))
    r = 1 / (1 + torch.exp(-(ga + val("ba"))))
    i = 1 / (1 + torch.exp(-(gx + val("bx"))))
    a = torch.exp(val("A") * r)
    drive = torch.sqrt(-torch.expm1(2 * val("A") * r)) * (i * u)
    if s["start"] is not None:
        m = s["start"].bool().unsqueeze(-1)
        a, drive = torch.where(m, 0.0, a), torch.where(m, i * u, drive)
    h = torch.zeros_like(u[:, 0]) if s["h"] is None else val("h")
    hs = []
    for at, xt in zip(a.unbind(1), drive.unbind(1)):
        h = at * h + xt
        hs.append(h)
    y = torch.stack(hs, 1)
    if case["gate"]:
        z = seq(val("z"))
        y = y * (z / (1 + torch.exp(-z)))
    out = dict(y=(y[:, 0] if step else y).detach())
    if step:
        out["h"] = h.detach()
    elif s["h"] is not None:
        out["h_last"] = h.detach()
    if train:
        loss = (y * s["dout"].to(F64)).sum()
        if s["dh"] is not None:
            loss = loss + (h * s["dh"].to(F64)).sum()
        out.update(grads(loss, dict(u="du", ga="dgate_a", gx="dgate_x", A="dA", ba="dbias_a", bx="dbias_x",
                                    z="dz", h="dh0")))
    return out
