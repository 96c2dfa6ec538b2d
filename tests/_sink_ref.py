"""Plain 64-bit forms of the sink-window attention and its backward, with
the error bounds that the kernels' roundings allow (test infrastructure).

u = eps / 2 is the rounding of the storage type.  Beside it every weight
carries a relative error E = 2^-12 from 32-bit work: a score is a sum of d
products whose 32-bit accumulation is off by at most d 2^-23 scale sum|q k|
(for d = 128 and normal inputs about 128 2^-23 7 = 2^-13), the exponential
and the sums add a few 2^-22."""
import math

import torch

E = 2.0 ** -12
TINY = 1e-6


def visible(n_q, n_k, pos0, window, sinks, dev="cuda"):
    p = pos0 + torch.arange(n_q, device=dev)[:, None]
    j = torch.arange(n_k, device=dev)[None, :]
    return (j <= p) & ((p - j < window) | (j < sinks))


def fwd(q, k, v, pos0, window, sinks, scale=None):
    """One sequence: q [t,Hq,d], k/v [n,Hkv,d] -> out, lse, bound of |out error| (all fp64)."""
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    scale = 1 / math.sqrt(d) if scale is None else scale
    see = visible(q.shape[0], k.shape[0], pos0, window, sinks, q.device)
    kd, vd = (x.double().repeat_interleave(G, 1) for x in (k, v))
    z = torch.einsum("thd,jhd->htj", q.double(), kd) * scale
    z = z.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(z, -1)
    P = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    vz = torch.where(torch.isfinite(vd), vd, 0.0)
    out = torch.einsum("htj,jhd->thd", P, vz)
    A = torch.einsum("htj,jhd->thd", P, vz.abs())
    return out, lse.T, A * (u + E) + u * out.abs() + TINY


def bwd(q, k, v, dout, pos0, window, sinks, scale=None):
    """-> (dq, dk, dv) and their bounds."""
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse, bout = fwd(q, k, v, pos0, window, sinks, scale)
    see = visible(q.shape[0], k.shape[0], pos0, window, sinks, q.device)
    qd, gd = q.double(), dout.double()
    kd, vd = (x.double().repeat_interleave(G, 1) for x in (k, v))
    z = torch.einsum("thd,jhd->htj", qd, kd) * scale
    L = torch.where(lse == -math.inf, 0.0, lse).T[..., None]
    P = torch.where(see, torch.exp(z - L), 0.0)
    dP = torch.einsum("thd,jhd->htj", gd, vd)
    dPa = torch.einsum("thd,jhd->htj", gd.abs(), vd.abs())
    D = torch.einsum("thd,thd->ht", gd, out)[..., None]
    eD = torch.einsum("thd,thd->ht", gd.abs(), bout)[..., None] + E * dPa
    dS = P * (dP - D)
    eS = (u + 2 * E) * dS.abs() + P * eD
    eP = (u + 2 * E) * P

    def heads(x):
        return x.unflatten(1, (-1, G)).sum(2)

    dq = torch.einsum("htj,jhd->thd", dS, kd) * scale
    dk = heads(torch.einsum("htj,thd->jhd", dS, qd)) * scale
    dv = heads(torch.einsum("htj,thd->jhd", P, gd))
    bq = torch.einsum("htj,jhd->thd", eS, kd.abs()) * scale + u * dq.abs() + TINY
    bk = heads(torch.einsum("htj,thd->jhd", eS, qd.abs())) * scale + u * dk.abs() + TINY
    bv = heads(torch.einsum("htj,thd->jhd", eP, gd.abs())) + u * dv.abs() + TINY
    return (dq, dk, dv), (bq, bk, bv)


def close(got, ref, bound, what):
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    over = ((g - ref).abs() - bound).max().item() if g.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} above its bound (largest value {ref.abs().max().item():.3g})"


def close_lse(got, ref, what):
    none = ref == -math.inf
    assert torch.equal(got == -math.inf, none), f"{what}: rows without a key differ"
    err = (got.double() - ref)[~none].abs()
    assert err.numel() == 0 or err.max().item() <= 2 * E, f"{what}: {err.max().item():.3e}"
