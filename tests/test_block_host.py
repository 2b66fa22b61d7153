"""Host-side tests of the operators around the scan: the C ABI's refusals
before anything touches CUDA (pointers are fake and never dereferenced), the
size queries, and the binding's checks of tensors."""
import ctypes

import pytest
import torch

from selective_state_space_25_b200 import ssmscan as S

L = S.lib()
MB = 1 << 20
NONE = ctypes.c_size_t(-1).value
INV, UNS, WSP, OK = S.SSM_ERR_INVALID_ARG, S.SSM_ERR_UNSUPPORTED, S.SSM_ERR_WORKSPACE, S.SSM_OK


def at(k):
    return (k + 1) * MB  # far apart, aligned


def caller(fn, names, defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(names), set(kw) - set(names)
        a.update(kw)
        return fn(*(a[n] for n in names))
    return call


SIZES = dict(b=2, L=8, d=16, dtype=S.SSM_BF16, stream=None)
gated_fwd = caller(
    L.ssm_gated_scan_fwd,
    "u u_ld ga ga_ld gx gx_ld A ba bx z z_ld start h0 h_last y y_ld st st_b b L d dtype stream".split(),
    dict(u=at(0), u_ld=16, ga=at(1), ga_ld=16, gx=at(2), gx_ld=16, A=at(3), ba=at(4), bx=at(5), z=at(6),
         z_ld=16, start=at(7), h0=at(8), h_last=at(9), y=at(10), y_ld=16, st=at(11), st_b=128, **SIZES))
gated_bwd = caller(
    L.ssm_gated_scan_bwd,
    ("u u_ld ga ga_ld gx gx_ld A ba bx z z_ld start dout dout_ld dh du du_ld dga dga_ld dgx dgx_ld dz dz_ld "
     "dA dba dbx dh0 b L d dtype st st_b ws ws_b stream").split(),
    dict(u=at(0), u_ld=16, ga=at(1), ga_ld=16, gx=at(2), gx_ld=16, A=at(3), ba=at(4), bx=at(5), z=at(6),
         z_ld=16, start=at(7), dout=at(8), dout_ld=16, dh=at(9), du=at(10), du_ld=16, dga=at(11), dga_ld=16,
         dgx=at(12), dgx_ld=16, dz=at(13), dz_ld=16, dA=at(14), dba=at(15), dbx=at(16), dh0=at(17),
         st=at(18), st_b=128, ws=at(19), ws_b=MB, **SIZES))
gated_step = caller(
    L.ssm_gated_state_update,
    "state u u_ld ga ga_ld gx gx_ld A ba bx z z_ld y y_ld b d dtype stream".split(),
    dict(state=at(0), u=at(1), u_ld=16, ga=at(2), ga_ld=16, gx=at(3), gx_ld=16, A=at(4), ba=at(5), bx=at(6),
         z=at(7), z_ld=16, y=at(8), y_ld=16, b=2, d=16, dtype=S.SSM_BF16, stream=None))
conv_fwd = caller(
    L.ssm_conv1d_fwd, "x x_ld w bias silu cs cso start y y_ld b L d K dtype stream".split(),
    dict(x=at(0), x_ld=16, w=at(1), bias=at(2), silu=1, cs=at(3), cso=at(4), start=at(5), y=at(6), y_ld=16,
         K=4, **SIZES))
conv_bwd = caller(
    L.ssm_conv1d_bwd,
    "x x_ld w bias silu cs start dy dy_ld dx dx_ld dw db b L d K dtype ws ws_b stream".split(),
    dict(x=at(0), x_ld=16, w=at(1), bias=at(2), silu=1, cs=at(3), start=at(4), dy=at(5), dy_ld=16, dx=at(6),
         dx_ld=16, dw=at(7), db=at(8), K=4, ws=at(9), ws_b=MB, **SIZES))
conv_step = caller(
    L.ssm_conv1d_update, "cs x x_ld w bias silu y y_ld b d K dtype stream".split(),
    dict(cs=at(0), x=at(1), x_ld=16, w=at(2), bias=at(3), silu=1, y=at(4), y_ld=16, b=2, d=16, K=4,
         dtype=S.SSM_BF16, stream=None))
gnorm_fwd = caller(
    L.ssm_gated_norm_fwd, "x x_ld z z_ld w groups eps before y y_ld rows d dtype stream".split(),
    dict(x=at(0), x_ld=16, z=at(1), z_ld=16, w=at(2), groups=2, eps=1e-5, before=0, y=at(3), y_ld=16, rows=8,
         d=16, dtype=S.SSM_BF16, stream=None))
gnorm_bwd = caller(
    L.ssm_gated_norm_bwd,
    "x x_ld z z_ld w groups eps before dy dy_ld dx dx_ld dz dz_ld dw rows d dtype ws ws_b stream".split(),
    dict(x=at(0), x_ld=16, z=at(1), z_ld=16, w=at(2), groups=2, eps=1e-5, before=0, dy=at(3), dy_ld=16,
         dx=at(4), dx_ld=16, dz=at(5), dz_ld=16, dw=at(6), rows=8, d=16, dtype=S.SSM_BF16, ws=at(7),
         ws_b=MB, stream=None))
anorm_fwd = caller(
    L.ssm_add_norm_fwd,
    "x x_ld r r_ld w post scale eps y y_ld ro ro_ld rows d dtype rdtype stream".split(),
    dict(x=at(0), x_ld=16, r=at(1), r_ld=16, w=at(2), post=at(3), scale=at(4), eps=1e-5, y=at(5), y_ld=16,
         ro=at(6), ro_ld=16, rows=8, d=16, dtype=S.SSM_BF16, rdtype=S.SSM_F32, stream=None))
anorm_bwd = caller(
    L.ssm_add_norm_bwd,
    ("x x_ld ro ro_ld w post scale eps dy dy_ld dro dro_ld dx dx_ld dr dr_ld dw dpost dscale rows d dtype "
     "rdtype ws ws_b stream").split(),
    dict(x=at(0), x_ld=16, ro=at(1), ro_ld=16, w=at(2), post=at(3), scale=at(4), eps=1e-5, dy=at(5),
         dy_ld=16, dro=at(6), dro_ld=16, dx=at(7), dx_ld=16, dr=at(8), dr_ld=16, dw=at(9), dpost=at(10),
         dscale=at(11), rows=8, d=16, dtype=S.SSM_BF16, rdtype=S.SSM_F32, ws=at(12), ws_b=MB, stream=None))

NAN, INF = float("nan"), float("inf")
REFUSED = [
    # sizes, types, presence
    (gated_fwd, dict(b=-1), INV), (gated_fwd, dict(L=-1), INV), (gated_fwd, dict(d=-1), INV),
    (gated_fwd, dict(b=2 ** 40, L=2 ** 40), INV), (gated_fwd, dict(dtype=7), UNS),
    (gated_fwd, dict(u=None), INV), (gated_fwd, dict(A=None), INV), (gated_fwd, dict(gx=None), INV),
    (gated_fwd, dict(y=None), INV), (gated_fwd, dict(st_b=127), WSP),
    (gated_bwd, dict(dout=None), INV), (gated_bwd, dict(dz=None), INV), (gated_bwd, dict(dA=None), INV),
    (gated_bwd, dict(st=None), INV), (gated_bwd, dict(st_b=64), WSP), (gated_bwd, dict(ws=None), WSP),
    (gated_bwd, dict(ws_b=16), WSP), (gated_bwd, dict(d=-1), INV),
    (gated_step, dict(state=None), INV), (gated_step, dict(y=None), INV), (gated_step, dict(b=-1), INV),
    (conv_fwd, dict(K=0), UNS), (conv_fwd, dict(K=9), UNS), (conv_fwd, dict(x=None), INV),
    (conv_fwd, dict(w=None), INV), (conv_fwd, dict(L=-2), INV), (conv_fwd, dict(dtype=2), UNS),
    (conv_bwd, dict(dx=None), INV), (conv_bwd, dict(dw=None), INV), (conv_bwd, dict(ws=None), WSP),
    (conv_bwd, dict(K=9), UNS), (conv_step, dict(cs=None), INV), (conv_step, dict(K=0), UNS),
    (gnorm_fwd, dict(groups=3), INV), (gnorm_fwd, dict(groups=0), INV), (gnorm_fwd, dict(groups=-2), INV),
    (gnorm_fwd, dict(eps=-1.0), INV), (gnorm_fwd, dict(eps=NAN), INV), (gnorm_fwd, dict(eps=INF), INV),
    (gnorm_fwd, dict(w=None), INV), (gnorm_fwd, dict(rows=-1), INV), (gnorm_fwd, dict(y=None), INV),
    (gnorm_bwd, dict(dz=None), INV), (gnorm_bwd, dict(dw=None), INV), (gnorm_bwd, dict(ws=None), WSP),
    (anorm_fwd, dict(w=None), INV), (anorm_fwd, dict(ro=None), INV), (anorm_fwd, dict(x=None), INV),
    (anorm_fwd, dict(rdtype=5), UNS), (anorm_fwd, dict(dtype=S.SSM_F32, rdtype=S.SSM_BF16), UNS),
    (anorm_fwd, dict(eps=-1e-9), INV),
    (anorm_bwd, dict(x=None), INV), (anorm_bwd, dict(dpost=None), INV), (anorm_bwd, dict(dscale=None), INV),
    (anorm_bwd, dict(dw=None), INV), (anorm_bwd, dict(ws_b=0), WSP), (anorm_bwd, dict(ro=None), INV),
    # strides and alignment
    (gated_fwd, dict(u_ld=15), INV), (gated_fwd, dict(y_ld=0), INV), (gated_fwd, dict(u=at(0) + 1), INV),
    (gated_fwd, dict(A=at(3) + 2), INV), (gated_fwd, dict(u_ld=2 ** 62), INV),
    (conv_fwd, dict(x_ld=8), INV), (conv_bwd, dict(ws=at(9) + 4), INV), (gnorm_fwd, dict(z_ld=1), INV),
    (anorm_fwd, dict(r=at(1) + 2), INV), (gated_bwd, dict(ws=at(19) + 8), INV),
    # outputs over other arguments
    (gated_fwd, dict(y=at(0)), INV), (gated_fwd, dict(y=at(0) + 510), INV), (gated_fwd, dict(h_last=at(3)), INV),
    (gated_fwd, dict(h_last=at(8) + 4), INV), (gated_fwd, dict(st=at(10)), INV),
    (gated_bwd, dict(du=at(8)), INV), (gated_bwd, dict(dga=at(10)), INV), (gated_bwd, dict(ws=at(18)), INV),
    (gated_bwd, dict(dh0=at(9) + 4), INV), (gated_step, dict(y=at(1)), INV), (gated_step, dict(y=at(0)), INV),
    (conv_fwd, dict(y=at(0)), INV), (conv_fwd, dict(cso=at(3) + 2), INV), (conv_bwd, dict(dx=at(5)), INV),
    (conv_step, dict(y=at(1)), INV), (gnorm_fwd, dict(y=at(1)), INV), (gnorm_bwd, dict(dx=at(5)), INV),
    (anorm_fwd, dict(ro=at(1) + 4), INV), (anorm_fwd, dict(y=at(6)), INV), (anorm_bwd, dict(dr=at(6) + 8), INV),
    # halves of one buffer: the rows interleave only if they are as wide as they say
    (gnorm_bwd, dict(dx=at(4), dx_ld=31, dz=at(4) + 32, dz_ld=31), INV),
    (gnorm_bwd, dict(dx=at(4), dx_ld=32, dz=at(4) + 30, dz_ld=32), INV),
    (gnorm_bwd, dict(dx=at(4), dx_ld=32, dz=at(4) + 32, dz_ld=33), INV),
    # in place with another stride
    (anorm_fwd, dict(ro=at(1), ro_ld=17), INV),
    # empty problems
    (gated_fwd, dict(b=0), OK), (gated_fwd, dict(d=0), OK), (gated_bwd, dict(d=0), OK),
    (gated_step, dict(b=0), OK), (conv_fwd, dict(b=0), OK), (conv_fwd, dict(L=0, cso=None), OK),
    (conv_bwd, dict(d=0), OK), (conv_step, dict(d=0), OK), (gnorm_fwd, dict(rows=0), OK),
    (gnorm_fwd, dict(d=0), OK), (gnorm_bwd, dict(d=0), OK), (anorm_fwd, dict(rows=0), OK),
    (anorm_bwd, dict(d=0), OK),
]


@pytest.mark.parametrize("k", range(len(REFUSED)))
def test_refusals(k):
    fn, kw, status = REFUSED[k]
    assert fn(**kw) == status, (kw, S.last_error())
    assert (S.last_error() != "") == (status != OK)


def test_size_queries():
    assert S.ssm_gated_scan_states_bytes(2, 32, 8) == 2 * 8 * 4
    assert S.ssm_gated_scan_states_bytes(2, 33, 8) == 2 * 2 * 8 * 4
    assert S.ssm_gated_scan_states_bytes(2, 0, 8) == 0
    for q in (L.ssm_gated_scan_states_bytes(-1, 2, 3), L.ssm_gated_scan_bwd_workspace_bytes(1, -2, 3),
              L.ssm_conv1d_bwd_workspace_bytes(1, 2, 3, 9), L.ssm_conv1d_bwd_workspace_bytes(1, 2, 3, 0),
              L.ssm_gated_norm_bwd_workspace_bytes(2, 8, 3), L.ssm_gated_norm_bwd_workspace_bytes(2, 8, 0),
              L.ssm_add_norm_bwd_workspace_bytes(-1, 8), L.ssm_add_norm_bwd_workspace_bytes(2 ** 40, 2 ** 40)):
        assert q == NONE
    for s in [(0, 5, 8), (2, 0, 8), (2, 5, 0), (0, 0, 0)]:  # empty problems have a size too
        assert S.ssm_gated_scan_bwd_workspace_bytes(*s) >= 0 and S.ssm_conv1d_bwd_workspace_bytes(*s, 4) >= 0
        assert S.ssm_gated_norm_bwd_workspace_bytes(s[0], s[2]) >= 0
        assert S.ssm_add_norm_bwd_workspace_bytes(s[0], s[2]) >= 0
    # whole partial rows of the parameters' gradients
    assert S.ssm_gated_scan_bwd_workspace_bytes(2, 100, 24) % (3 * 24 * 4) == 0
    assert S.ssm_conv1d_bwd_workspace_bytes(2, 100, 24, 4) % (5 * 24 * 4) == 0
    assert S.ssm_gated_norm_bwd_workspace_bytes(1, 24) >= 24 * 4
    assert S.ssm_add_norm_bwd_workspace_bytes(1, 24) >= 3 * 24 * 4


def cpu(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype)


def test_binding_refuses_cpu_tensors():
    x, A = cpu(2, 3, 8), cpu(8)
    for call in (lambda: S.ssm_gated_scan_fwd(x, x, x, A), lambda: S.ssm_conv1d_fwd(x, cpu(8, 4)),
                 lambda: S.ssm_gated_scan_bwd(x, x, x, A, x, cpu(2, 1, 8)),
                 lambda: S.ssm_gated_state_update(cpu(2, 8), x[:, 0], x[:, 0], x[:, 0], A),
                 lambda: S.ssm_conv1d_bwd(x, cpu(8, 4), x), lambda: S.ssm_gated_norm_fwd(x, x, A),
                 lambda: S.ssm_conv1d_update(cpu(2, 8, 4), x[:, 0], cpu(8, 4)),
                 lambda: S.ssm_gated_norm_bwd(x, x, A, x), lambda: S.ssm_add_norm_fwd(x, x, A),
                 lambda: S.ssm_add_norm_bwd(x, x, A, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        S.ssm_gated_scan_fwd([1.0], x, x, A)


def test_row_strides():
    f = torch.float32
    rows = lambda t, shape=None: S._rows(t, "t", t.shape if shape is None else torch.Size(shape),  # noqa: E731
                                         f, t.device)[1]
    wide = cpu(4, 5, 20)
    assert rows(cpu(4, 5, 8)) == 8 and rows(wide[..., 2:10]) == 20
    assert rows(wide[:1, :, :8]) == 20 and rows(wide[:, :1, :8]) == 100 and rows(wide[:1, :1, :8]) == 8
    assert rows(wide[:, 0, :8]) == 100 and rows(cpu(3, 1).expand(3, 1)) == 1
    assert S._rows(None, "t", (1,), f, wide.device) == (None, 0)
    for t, why in ((wide[..., ::2], "adjacent"), (wide[:, :3, :8], "fixed stride"),
                   (cpu(4, 5, 8).transpose(0, 1), "fixed stride"), (cpu(1, 8).expand(4, 8), "overlap"),
                   (cpu(20).as_strided((3, 8), (4, 1)), "overlap")):
        with pytest.raises(ValueError, match=why):
            rows(t)
    with pytest.raises(ValueError, match="shape"):
        rows(cpu(4, 8), (4, 9))
    with pytest.raises(TypeError, match="dtype"):
        S._rows(cpu(4, 8, dtype=torch.bfloat16), "t", torch.Size((4, 8)), f, wide.device)
    with pytest.raises(TypeError, match="Tensor"):
        S._rows(3, "t", torch.Size((4, 8)), f, wide.device)
