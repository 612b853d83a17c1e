"""Plain 64-bit implementation of linear attention with a decay for each head,
straight from the token recurrence, for the tests: the forward in torch, its
gradients by torch's own differentiation of that forward."""
import torch


def lengths(B, T, cu):
    return [T] * B if cu is None else [int(b) - int(a) for a, b in zip(cu[:-1], cu[1:])]


def forward(q, k, v, g, S0=None, cu=None):
    """q, k [B,T,Hk,dk], v [B,T,H,dv], g [B,T,H] or [H], all float64; returns
    (out [B,T,H,dv], S_final [N,H,dv,dk]).  Rows of no sequence are NaN."""
    B, T, H, dv = v.shape
    r = H // q.shape[2]
    rows = [x.reshape(B * T, *x.shape[2:]) for x in (q, k, v)]
    q, k, v = rows[0].repeat_interleave(r, 1), rows[1].repeat_interleave(r, 1), rows[2]
    a = (g.expand(B * T, H) if g.dim() == 1 else g.reshape(B * T, H)).exp()
    starts = [s * T for s in range(B)] if cu is None else [int(x) for x in cu[:-1]]
    outs, finals = [None] * (B * T), []
    for s, (t0, n) in enumerate(zip(starts, lengths(B, T, cu))):
        S = v.new_zeros(H, dv, k.shape[-1]) if S0 is None else S0[s]
        for t in range(t0, t0 + n):
            S = a[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            outs[t] = (S @ q[t][:, :, None])[..., 0]
        finals.append(S)
    gap = torch.full_like(v[0], float("nan")) if B * T else None
    out = torch.stack([gap if o is None else o for o in outs]) if B * T else v
    return out.view(B, T, H, dv), torch.stack(finals)


def gradients(q, k, v, g, dout, S0=None, dS=None, cu=None):
    """(dq, dk, dv, dg, dS0) of <out, dout> + <S_final, dS>."""
    B, T, H, dv = v.shape
    n = len(lengths(B, T, cu))
    S0 = v.new_zeros(n, H, dv, q.shape[-1]) if S0 is None else S0
    x = [t.detach().clone().requires_grad_(True) for t in (q, k, v, g, S0)]
    out, S = forward(*x, cu=cu)
    loss = (out.nan_to_num(0.0) * dout).sum()
    if dS is not None:
        loss = loss + (S * dS).sum()
    got = torch.autograd.grad(loss, x, allow_unused=True)
    return [torch.zeros_like(t) if y is None else y for t, y in zip(x, got)]
