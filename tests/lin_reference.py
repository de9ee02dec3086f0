"""64-bit references of the decayed linear attention and the block norms, with
the magnitudes that rounding bounds are multiplied by.

The recurrence runs token by token in numpy; every function also runs on the
absolute values of its inputs, which gives the sum of the absolute values of
the terms of each output.  A sum of n fp32 products is off by at most about
n 2^-24 times that sum; an operand rounded to bf16 adds 2^-8 times it.
"""
import numpy as np
import torch

U32 = 2.0 ** -24    # half a step of fp32, relative
U16 = 2.0 ** -8     # half a step of bf16, relative


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def bounds_of(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))])


def lin_forward(q, k, v, log_decay, lens, S0=None, scale=1.0):
    """o [T, H, dv], S [N, H, dk, dv] of S = a S + k v^T, o = scale S^T q."""
    T, H, dk = q.shape
    dv = v.shape[2]
    with np.errstate(over="ignore"):
        a = np.exp(log_decay)[:, None, None]
    o = np.zeros((T, H, dv))
    S_out = np.zeros((len(lens), H, dk, dv))
    cu = bounds_of(lens)
    for n in range(len(lens)):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = a * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hij,hi->hj", S, q[t])
        S_out[n] = S
    return o, S_out


def lin_backward(q, k, v, log_decay, lens, dO, S0=None, dS=None, scale=1.0):
    """dq, dk, dv, dS0 by the reverse recurrence G = scale q dO^T + a G."""
    T, H, dk = q.shape
    dv = v.shape[2]
    a = np.exp(log_decay)[:, None, None]
    dq, dkk, dvv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dS0 = np.zeros((len(lens), H, dk, dv))
    cu = bounds_of(lens)
    for n in range(len(lens)):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = a * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hij,hj->hi", S, dO[t])
        G = np.zeros((H, dk, dv)) if dS is None else dS[n].copy()
        for t in reversed(range(cu[n], cu[n + 1])):
            G = G + scale * q[t][:, :, None] * dO[t][:, None, :]
            dkk[t] = np.einsum("hij,hj->hi", G, v[t])
            dvv[t] = np.einsum("hij,hi->hj", G, k[t])
            G = a * G
        dS0[n] = G
    return dict(dq=dq, dk=dkk, dv=dvv, dS0=dS0)


def absolute(*arrays):
    return [None if x is None else np.abs(x) for x in arrays]


def fp32_terms(lens, d):
    """Roundings an output's terms pass through in fp32: a product over d, the
    sums over at most a sequence's tokens, a power of the decay (a few units)."""
    return 2 * d + max(lens) + 16


def check(name, got, want, mag, terms, out_bf16=False, operand_roundings=0):
    """|got - want| elementwise within the roundings counted: fp32 sums of
    `terms` terms and `operand_roundings` operands rounded to bf16, each against
    the absolute sum `mag`, and the rounding of a bf16 output."""
    got = f64(got)
    bound = (terms * U32 + operand_roundings * U16) * mag + 1e-37
    if out_bf16:
        bound = bound + U16 * (np.abs(want) + bound)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} outside, worst ratio "
                           f"{np.nanmax(np.abs(got - want) / bound)}")


def rel_fro(got, want):
    n = np.linalg.norm(want)
    d = np.linalg.norm(f64(got) - want)
    return d / n if n else d


def make(lens, H, dk, dv, dtype, seed=0, state=False, g=None):
    """Inputs on the host: unit-length q and k, normal v and dO, states N(0, 0.3)."""
    gen = torch.Generator().manual_seed(seed)
    T = int(sum(lens))

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    q, k = (normal(T, H, dk) / dk ** 0.5 for _ in range(2))
    v, dO = normal(T, H, dv), normal(T, H, dv)
    decay = -torch.rand(H, generator=gen) * 0.3 if g is None else torch.as_tensor(
        [float(x) for x in g], dtype=torch.float32)
    S0 = 0.3 * normal(len(lens), H, dk, dv) if state else None
    dS = 0.3 * normal(len(lens), H, dk, dv) if state else None
    cu = torch.tensor(bounds_of(lens), dtype=torch.int32)
    return dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), dO=dO.to(dtype),
                log_decay=decay.float(), S0=S0, dS=dS, cu=cu, lens=list(lens))


def dev(x):
    return {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}


# ---------------------------------------------------------------- block norms
def rms(x, w, group, eps):
    b = x.unflatten(-1, (-1, group))
    return (b / (b.pow(2).mean(-1, keepdim=True) + eps).sqrt()).flatten(-2) * w


def branch(y, w_post, gate, res_scale, act, eps):
    group = w_post.numel()
    u = rms(y, w_post.repeat(y.shape[-1] // group), group, eps)
    if gate is not None:
        u = u * (torch.sigmoid(gate) if act == "sigmoid" else gate * torch.sigmoid(gate))
    return u if res_scale is None else u * res_scale


def norm_forward(y, w_post, gate=None, x=None, res_scale=None, w_pre=None, act="sigmoid",
                 eps=1e-6):
    """(x_out, h) in 64 bits."""
    y, w_post, gate, x, res_scale, w_pre = (None if t is None else t.double().cpu() for t in (
        y, w_post, gate, x, res_scale, w_pre))
    u = branch(y, w_post, gate, res_scale, act, eps)
    out = u if x is None else x + u
    return out, None if w_pre is None else rms(out, w_pre, out.shape[-1], eps)


def norm_backward(y, w_post, dx_out, gate=None, x_out=None, res_scale=None, w_pre=None, dh=None,
                  act="sigmoid", eps=1e-6):
    """Gradients in 64 bits by autograd of the two formulas, joined at x_out."""
    f = {n: t.double().cpu().requires_grad_(True) for n, t in dict(
        y=y, w_post=w_post, gate=gate, x_out=x_out, res_scale=res_scale, w_pre=w_pre).items()
        if t is not None}
    total = torch.zeros(y.shape, dtype=torch.float64) if dx_out is None else dx_out.double().cpu()
    out = {}
    if w_pre is not None:
        h = rms(f["x_out"], f["w_pre"], y.shape[-1], eps)
        through, out["dw_pre"] = torch.autograd.grad(h, (f["x_out"], f["w_pre"]),
                                                     dh.double().cpu())
        total = total + through
    out["dx"] = total
    names = [n for n in ("y", "w_post", "gate", "res_scale") if n in f]
    u = branch(f["y"], f["w_post"], f.get("gate"), f.get("res_scale"), act, eps)
    grads = torch.autograd.grad(u, [f[n] for n in names], total)
    out.update({"d" + n: t for n, t in zip(names, grads)})
    return out
