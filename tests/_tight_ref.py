"""Error bounds of the paths that take their weights in two parts of the
storage type, or that keep D of the backward in 32 bits (test infrastructure;
the values are those of _sink_ref).

A weight in two parts is off by at most R = 2^-16 of itself in bf16 (8 bits
each, the first rounded towards zero at worst) and by less in fp16, where what
lies below 2^-24 is lost as well: with the largest weight of a row at 1 or
more, 2^-24 a key.  So the storage type's u enters once, for the output's own
rounding, and beside it stands the 32-bit work E of _sink_ref."""
import math

import torch

from _sink_ref import E, TINY, fwd as _fwd, visible

R = 2.0 ** -16


def fwd(q, k, v, pos0, window, sinks, scale=None, parts=2):
    """One sequence: out, lse, bound of |out error| with the weights in `parts` parts."""
    out, lse, loose = _fwd(q, k, v, pos0, window, sinks, scale)
    if parts == 1:
        return out, lse, loose
    u = torch.finfo(q.dtype).eps / 2
    A = (loose - u * out.abs() - TINY) / (u + E)                  # sum of weight times |v|
    floor = 0.0
    if q.dtype == torch.float16 and v.numel():
        floor = k.shape[0] * 2.0 ** -24 * torch.where(torch.isfinite(v), v, 0).abs().max().item()
    return out, lse, A * (E + R) + u * out.abs() + floor + TINY


def bwd(q, k, v, dout, pos0, window, sinks, scale=None, parts=2):
    """-> (dq, dk, dv) and their bounds: P is off by 2 E (its score's and its lse's), dP by E of its terms' sizes,
    D = sum P dP by what these two make, and with one part P and dS are rounded to the storage type."""
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    w = R if parts == 2 else u
    scale = 1 / math.sqrt(d) if scale is None else scale
    see = visible(q.shape[0], k.shape[0], pos0, window, sinks, q.device)
    qd, gd = q.double(), dout.double()
    kd, vd = (x.double().repeat_interleave(G, 1) for x in (k, v))
    z = torch.einsum("thd,jhd->htj", qd, kd) * scale
    z = z.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(z, -1, keepdim=True)
    P = torch.where(see, torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)), 0.0)
    dP = torch.einsum("thd,jhd->htj", gd, vd)
    size = torch.einsum("thd,jhd->htj", gd.abs(), vd.abs())
    D = (P * dP).sum(-1, keepdim=True)
    eD = (P * (2 * E * dP.abs() + E * size)).sum(-1, keepdim=True)
    dS = P * (dP - D)
    eS = (w + 2 * E) * dS.abs() + P * (E * size + eD)
    eP = (w + 2 * E) * P

    def heads(x):
        return x.unflatten(1, (-1, G)).sum(2)

    dq = torch.einsum("htj,jhd->thd", dS, kd) * scale
    dk = heads(torch.einsum("htj,thd->jhd", dS, qd)) * scale
    dv = heads(torch.einsum("htj,thd->jhd", P, gd))
    bq = torch.einsum("htj,jhd->thd", eS, kd.abs()) * scale + u * dq.abs() + TINY
    bk = heads(torch.einsum("htj,thd->jhd", eS, qd.abs())) * scale + u * dk.abs() + TINY
    bv = heads(torch.einsum("htj,thd->jhd", eP, gd.abs())) + u * dv.abs() + TINY
    return (dq, dk, dv), (bq, bk, bv)
