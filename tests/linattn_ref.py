"""Linear attention with one decay per head in float64 on the CPU, token by token, with its gradients,
and the size of the sums behind each value (the same sums over magnitudes), which tolerances scale with."""
from types import SimpleNamespace

import torch


def spans(T, B, cu):
    """(batch row, first token, last token + 1) of each sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = cu.tolist()
    return [(0, x, y) for x, y in zip(c, c[1:])]


def forward(q, k, v, g, cu=None, s0=None):
    """float64 tensors shaped as the operator's: o, final state, and the state after every token."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    seqs = spans(T, B, cu)
    q, k = (x.repeat_interleave(H // Hk, dim=2) for x in (q, k))
    a = g.expand(B, T, H).exp()
    o = torch.zeros(B, T, H, dv, dtype=torch.float64)
    S_all = torch.zeros(B, T, H, dk, dv, dtype=torch.float64)
    sf = []
    for n, (b, lo, hi) in enumerate(seqs):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if s0 is None else s0[n]
        for t in range(lo, hi):
            S = a[b, t, :, None, None] * S + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = torch.einsum("hij,hi->hj", S, q[b, t])
            S_all[b, t] = S
        sf.append(S)
    return o, torch.stack(sf), S_all


def backward(q, k, v, g, do, dsf=None, cu=None, s0=None):
    """Adjoint of each step: G += q do^T; dq = S do, dk = G v, dv = G^T k, da = <S_{t-1}, G>; G <- a G."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    group = H // Hk
    _, sf, S_all = forward(q, k, v, g, cu, s0)
    qr, kr = (x.repeat_interleave(group, dim=2) for x in (q, k))
    a = g.expand(B, T, H).exp()
    out = SimpleNamespace(dq=torch.zeros_like(qr), dk=torch.zeros_like(kr), dv=torch.zeros_like(v),
                          dg=torch.zeros(B, T, H, dtype=torch.float64), ds0=torch.zeros_like(sf))
    for n, (b, lo, hi) in enumerate(spans(T, B, cu)):
        G = torch.zeros(H, dk, dv, dtype=torch.float64) if dsf is None else dsf[n].clone()
        for t in reversed(range(lo, hi)):
            before = S_all[b, t - 1] if t > lo else (torch.zeros_like(G) if s0 is None else s0[n])
            G = G + qr[b, t, :, :, None] * do[b, t, :, None, :]
            out.dq[b, t] = torch.einsum("hij,hj->hi", S_all[b, t], do[b, t])
            out.dk[b, t] = torch.einsum("hij,hj->hi", G, v[b, t])
            out.dv[b, t] = torch.einsum("hij,hi->hj", G, kr[b, t])
            out.dg[b, t] = a[b, t] * (before * G).sum((-1, -2))
            G = a[b, t, :, None, None] * G
        out.ds0[n] = G
    out.dq = out.dq.reshape(B, T, Hk, group, dk).sum(3)
    out.dk = out.dk.reshape(B, T, Hk, group, dk).sum(3)
    if g.dim() == 1:
        out.dg = out.dg.sum((0, 1))
    return out


def gate_sum_size(q, k, g, mag, dsf_size, cu):
    """Size of the sums that the gate gradient is formed from: sum over r >= t of |q| |dq| + |k| |dk| (plus the
    final state's inner product), `mag` the backward over magnitudes."""
    B, T, Hk, _ = q.shape
    H = mag.dg.shape[-1]
    per = ((q * mag.dq).sum(-1) + (k * mag.dk).sum(-1)).repeat_interleave(H // Hk, dim=2)
    out = torch.zeros(B, T, H, dtype=torch.float64)
    for n, (b, lo, hi) in enumerate(spans(T, B, cu)):
        out[b, lo:hi] = per[b, lo:hi].flip(0).cumsum(0).flip(0)
        if dsf_size is not None:
            out[b, lo:hi] += dsf_size[n]
    return out.sum((0, 1)) if g.dim() == 1 else out


def pair_size(q, k, z, g, cu=None, back=False):
    """Sum over the pairs of tokens s <= r of a sequence of |e^{c_r - c_s} (q_r . k_s)| |z|: at r over z_s, or with
    `back` at s over z_r.  What rounding each pair's weight once can cost o (z = v) or dv (z = d_o)."""
    B, T, Hk, _ = q.shape
    H = z.shape[2]
    out = torch.zeros_like(z)
    c = g.expand(B, T, H).clamp(min=-1e4)
    for b, lo, hi in spans(T, B, cu):
        for h in range(H):
            cc = c[b, lo:hi, h].cumsum(0)
            w = torch.exp((cc[:, None] - cc[None, :]).tril()).tril()
            w = (w * (q[b, lo:hi, h // (H // Hk)] @ k[b, lo:hi, h // (H // Hk)].T)).abs()
            out[b, lo:hi, h] = (w.T if back else w) @ z[b, lo:hi, h].abs()
    return out
