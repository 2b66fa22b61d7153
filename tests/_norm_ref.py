"""Checks of the two norms, forward and backward, against their formulas in 64
bits, element by element.

Limits.  With u = 2^-24 a normed value is off by rel = d u / 2 + 2^-19 of itself
(the mean of d squares in any order, the root, the products); a gate or its
derivative by 2^-20 (1 + |z|).  A gradient has at most 8 such factors, so it is
off by 8 rel of the same expression over magnitudes.  A column's sum adds 8 rel
of the sum of its terms' magnitudes, and u for each link of the longest chain of
additions: the rows of one place (at most rows groups / SMs, one CTA an SM at
least), a CTA's 32 places at most, an eighth of 4 SMs partial rows, 8 lanes."""
import torch

import _block_ref as R
from _block_ref import close, up
from test_gpu_block import U, gen, randn, strided


def chain(rows, groups=1):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-rows * groups // sms) + 32 + sms // 2 + 8


def rel_of(n):
    return n * U / 2 + 2.0 ** -19


def add_norm_check(S, rows, d, form, dtype, res, eps=1e-5):
    g = gen(rows + d)
    view = strided if (rows + d) % 2 else (lambda t: t)
    x, r = view(randn(g, rows, d, dtype=dtype)), view(randn(g, rows, d, dtype=res, scale=2.0))
    w = 1 + randn(g, d, scale=0.1)
    scale = 0.5 + randn(g, d, scale=0.1) if form in ("scale", "both") else None
    post = 1 + randn(g, d, scale=0.1) if form in ("post", "both") else None
    dy, dro = view(randn(g, rows, d, dtype=dtype)), view(randn(g, rows, d, dtype=res))
    kw = dict(scale=scale, post_weight=post, eps=eps)
    y, ro = S.ssm_add_norm_fwd(x, r, w, **kw)
    got = S.ssm_add_norm_bwd(x, ro, w, dy, dresidual_out=dro, **kw)

    rel = rel_of(d)
    x, r, w, dy, dro = up(x), up(r), up(w), up(dy), up(dro)
    one = torch.ones(d, dtype=torch.float64)
    sc, pw = one if scale is None else up(scale), one if post is None else up(post)
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    rx = 1.0 if post is None else 1 / torch.sqrt(mean(x * x) + eps)
    xn = x * rx
    close("residual_out", ro, r + sc * xn * pw, 8 * rel * (r.abs() + (sc * xn * pw).abs()))
    q = up(ro)  # y and the gradients are those of the rounded residual
    rs = 1 / torch.sqrt(mean(q * q) + eps)
    n, dn = q * rs, dy * w
    close("y", y, n * w, 8 * rel * (n * w).abs())
    dr = rs * (dn - n * mean(dn * n)) + dro
    mr = rs * (dn.abs() + n.abs() * mean((dn * n).abs())) + dro.abs()
    close("dresidual", got["dresidual"], dr, 8 * rel * mr)
    dv, mv = dr * sc, mr * sc.abs()
    links = chain(rows) * U + 8 * rel
    close("dweight", got["dweight"], (dy * n).sum(0), links * (dy * n).abs().sum(0))
    if scale is not None:
        close("dscale", got["dscale"], (dr * xn * pw).sum(0), links * (mr * (xn * pw).abs()).sum(0))
    if post is not None:
        close("dpost_weight", got["dpost_weight"], (dv * xn).sum(0), links * (mv * xn.abs()).sum(0))
        dv, mv = dv * pw, mv * pw.abs()
        dv, mv = rx * (dv - xn * mean(dv * xn)), rx * (mv + xn.abs() * mean(mv * xn.abs()))
    close("dx", got["dx"], dv, 8 * rel * mv)


def gated_norm_check(S, rows, d, groups, form, dtype, eps=1e-5):
    g = gen(rows + d)
    view = strided if (rows + d) % 2 else (lambda t: t)
    x, z = view(randn(g, rows, d, dtype=dtype)), view(randn(g, rows, d, dtype=dtype))
    w, dy = 1 + randn(g, d, scale=0.1), view(randn(g, rows, d, dtype=dtype))
    z = None if form == "none" else z
    kw = dict(groups=groups, norm_before_gate=form == "before", eps=eps)
    y = S.ssm_gated_norm_fwd(x, z, w, **kw)
    got = S.ssm_gated_norm_bwd(x, z, w, dy, **kw)

    rel = rel_of(d // groups)
    shape = (rows, groups, d // groups)
    x, dy, w = up(x).reshape(shape), up(dy).reshape(shape), up(w).reshape(shape[1:])
    zz = torch.zeros_like(x) if z is None else up(z).reshape(shape)
    s = R.sig(zz)
    gate, ds, mds = (torch.ones_like(x), s, s) if z is None else (zz * s, s + zz * s * (1 - s), 1 + zz.abs())
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    before = form == "before"
    v, dn = (x, dy * w * gate) if before else (x * gate, dy * w)
    rs = 1 / torch.sqrt(mean(v * v) + eps)
    n = v * rs
    flat = lambda t: t.reshape(rows, d)  # noqa: E731
    ref = n * w * gate if before else n * w
    close("y", y, flat(ref), flat(8 * rel * ref.abs()))
    dv = rs * (dn - n * mean(dn * n))
    mv = rs * (dn.abs() + n.abs() * mean((dn * n).abs()))
    dx, mx = (dv, mv) if before else (dv * gate, mv * gate.abs())
    close("dx", got["dx"], flat(dx), flat(8 * rel * mx))
    if z is not None:
        dz = (dy * n * w if before else dv * x) * ds
        mz = ((dy * n * w).abs() if before else mv * x.abs()) * mds
        close("dz", got["dz"], flat(dz), flat(8 * rel * mz))
    terms = dy * n * gate if before else dy * n
    close("dweight", got["dweight"], terms.sum(0).reshape(d),
          (chain(rows, groups) * U + 8 * rel) * terms.abs().sum(0).reshape(d))
