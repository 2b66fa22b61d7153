"""64-bit definitions of the operators around the scan, on the CPU, one step at
a time; gradients by automatic differentiation.  Inputs are the tensors a call
gets (rounded already); every result is float64."""
import torch

F64 = torch.float64


def up(t, grad=False):
    return None if t is None else t.detach().cpu().to(F64).requires_grad_(grad)


sig = torch.sigmoid  # its derivative s (1 - s) holds at infinite arguments too


def gated(u, gate_a, gate_x, A, bias_a=None, bias_x=None, z=None, seq_start=None, h0=None):
    """(y, h_last) of float64 tensors."""
    r = sig(gate_a if bias_a is None else gate_a + bias_a)
    g = sig(gate_x if bias_x is None else gate_x + bias_x)
    la = A * r
    a, w = torch.exp(la), -torch.expm1(2 * la)
    f = torch.where(w > 0, torch.sqrt(torch.where(w > 0, w, 1.0)), 0.0)
    h = u.new_zeros(u.shape[0], u.shape[2]) if h0 is None else h0
    ys = []
    for t in range(u.shape[1]):
        new = a[:, t] * h + f[:, t] * g[:, t] * u[:, t]
        if seq_start is not None:
            new = torch.where(seq_start[:, t, None] != 0, g[:, t] * u[:, t], new)
        h = new
        ys.append(h)
    y = torch.stack(ys, 1) if ys else u.clone()
    return (y if z is None else y * z * sig(z)), h


def conv(x, weight, bias=None, silu=True, conv_state=None, seq_start=None):
    """(y, window after) of float64 tensors."""
    b, L, d = x.shape
    K = weight.shape[1]
    hist = [x.new_zeros(b, d)] * K if conv_state is None else list(conv_state.unbind(-1))
    ys = []
    for t in range(L):
        if seq_start is not None:
            s = seq_start[:, t, None] != 0
            hist = [torch.where(s, 0.0, v) for v in hist]
        hist = hist[1:] + [x[:, t]]
        p = sum(hist[j] * weight[:, j] for j in range(K))
        p = p if bias is None else p + bias
        ys.append(p * sig(p) if silu else p)
    return (torch.stack(ys, 1) if ys else x.clone()), torch.stack(hist, -1)


def rms(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def gated_norm(x, z, weight, groups=1, eps=1e-5, before=False):
    split = x.shape[:-1] + (groups, x.shape[-1] // groups)
    v, w = x.reshape(split), weight.reshape(split[-2:])
    gate = None if z is None else (z * sig(z)).reshape(split)
    if z is None:
        y = rms(v, eps) * w
    else:
        y = rms(v, eps) * w * gate if before else rms(v * gate, eps) * w
    return y.reshape(x.shape)


def add_norm(x, residual, weight, scale=None, post=None, eps=1e-5, round_to=None):
    """(y, residual_out); round_to: the type residual_out is rounded to, its
    gradient passed through."""
    v = x if post is None else rms(x, eps) * post
    v = v if scale is None else v * scale
    r = v if residual is None else v + residual
    if round_to is not None:
        r = r + (r.detach().to(torch.float32).to(round_to).to(F64) - r.detach())
    return rms(r, eps) * weight, r


def close(name, got, ref, atol, steps=1):
    """Every |got - ref| within `steps` half steps of got's type relative to
    |ref|, plus atol (a number, or a tensor like ref): the rest of the error
    budget, in absolute terms."""
    got = got.detach().cpu()
    half = torch.finfo(got.dtype).eps / 2
    ref = ref.detach().cpu().to(F64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    bad = torch.isnan(ref) | torch.isinf(ref)
    g = got.to(F64)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{name}: NaN at other places"
    assert torch.equal(g[torch.isinf(ref)], ref[torch.isinf(ref)]), f"{name}: infinities differ"
    lim = steps * half * ref.abs() + (atol if isinstance(atol, float) else atol.cpu().to(F64))
    off = torch.where(bad, 0.0, (g - ref).abs() / lim.clamp_min(1e-30))
    k = int(off.argmax())
    assert float(off.max()) <= 1.0, (f"{name}: {float(g.flatten()[k])} for {float(ref.flatten()[k])} "
                                     f"({float(off.max()):.3g} times the limit)")
