"""The gated delta rule in 64 bits, token by token, with bounds on what fp32 arithmetic may leave.

Bounds.  Errors of a state's column (value channel) are measured by the 2-norm E over key channels.  A step
multiplies an error by exp(g) (I - beta k k^T), whose norm is at most exp(g) for |k| <= 1 and beta in [0, 2], and
adds its own roundings (eps = 2^-24, s the old column's norm): the sum over key channels (d_k + 2) eps s, exp(g)
4 eps s, the sums and products of u 4 eps (s + |v|) times beta |k| <= 2, the update 2 eps (s + |u|) with |u| <= 2 (s + |v|):
in all no more than eps ((2 d_k + 24) s + 16 |v|).
"""
import torch

EPS = 2.0 ** -24


def recurrence(q, k, v, g, beta, lengths, init=None, scale=1.0):
    """(out, state, state bound, out bound) in 64 bits.  The bounds are for exact operands and fp32 arithmetic: of
    a state's column [N, H, d_v], and of an output before it is rounded to its type."""
    t, h, dv = v.shape
    share, dk, n = h // q.shape[1], q.shape[2], len(lengths)
    dev = v.device
    q, k = (x.double().repeat_interleave(share, 1) for x in (q, k))
    v, beta = v.double(), beta.double()
    a = g.double().exp().expand(t, h)
    state = torch.zeros(n, h, dk, dv, dtype=torch.float64, device=dev) if init is None else init.double().clone()
    err = torch.zeros(n, h, dv, dtype=torch.float64, device=dev)
    out = torch.zeros(t, h, dv, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    at = 0
    for s, length in enumerate(lengths):
        for i in range(at, at + length):
            norm = state[s].norm(dim=-2)
            x = state[s] * a[i][:, None, None]
            u = beta[i][:, None] * (v[i] - (k[i][:, :, None] * x).sum(-2))
            state[s] = x + k[i][:, :, None] * u[:, None, :]
            out[i] = scale * (q[i][:, :, None] * state[s]).sum(-2)
            err[s] = a[i][:, None] * err[s] + EPS * ((2 * dk + 24) * norm + 16 * v[i].abs())
            bound[i] = abs(scale) * q[i].norm(dim=-1)[:, None] * (err[s] + (dk + 4) * EPS * state[s].norm(dim=-2))
        at += length
    return out, state, err, bound


def inputs(lengths, heads, keys, dk, dv, dtype, seed, per_token=True, init=False, tail=0, device="cuda"):
    """Operands of one call; `tail` rows more than the sequences have."""
    gen = torch.Generator().manual_seed(seed)
    t = sum(lengths) + tail
    normal = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    # unit keys, shrunk by their rounding so that |k| <= 1 holds for the rounded ones
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True) * (1 - 2.0 ** -8)).to(dtype)  # noqa: E731
    common = 0.5 * normal(keys, dk)
    x = dict(q=unit(normal(t, keys, dk)), k=unit(normal(t, keys, dk) + common), v=normal(t, heads, dv).to(dtype),
             g=-torch.nn.functional.softplus(normal(t, heads) - 2) if per_token else -torch.rand(heads, generator=gen),
             beta=torch.sigmoid(normal(t, heads)))
    ends = torch.tensor([0] + lengths).cumsum(0).int()
    x["cu"] = ends
    x["init"] = 0.3 * normal(len(lengths), heads, dk, dv) if init else None
    return {n: y if y is None else y.to(device) for n, y in x.items()}


def chunked_bounds(q, k, v, g, beta, lengths, init=None, scale=1.0, chunk=64):
    """(out, state, state bound, out bound) as of recurrence(), for the evaluation in chunks on tensor cores:
        A_ij = beta_i w_ij (k_i . k_j),  T = (I + A)^-1,  R = beta v - beta e^G S^T k,  U = T R
    with w = exp of a difference x of sums of log decays.  What it may leave of U, given the chunk's start state:
      - R and T in three bf16 parts (8 bits each, all of fp32's), of whose nine products the three smallest, each at
        most 2^-24 |T| |R|, are left out
      - w off by 2^-22 (1 + |x|) of itself, A by that and its sums' roundings, T by |T| dA |T| and by the block
        inverse's: three joins of two products each, whose operands' parts leave out 2^-21 of |a| |b| thrice at most and
        whose sums of up to 32 terms round twice eps: 6 (24 + 64) eps |T| (I + |A|) |T|
      - sums in fp32 of 3 d_k, or 6 x 64, terms, each rounding twice eps (the accumulator may cut off)
    An error of the start state only shrinks (see recurrence), so a chunk adds sum_j e^(G_C - G_j) |du_j| to it, and
    the roundings of its own sum.  Outputs take one bf16 rounding (2^-8) of the state, of P = w (q . k) and of u each."""
    t, h, dv = v.shape
    share, dk = h // q.shape[1], q.shape[2]
    want = recurrence(q, k, v, g, beta, lengths, init, scale)[:2]
    gg = (g if g.dim() == 2 else g.expand(t, h)).double()
    err = torch.zeros(len(lengths), h, dv, dtype=torch.float64, device=v.device)
    bound = torch.zeros(t, h, dv, dtype=torch.float64, device=v.device)
    at = 0
    for s, length in enumerate(lengths):
        state = None if init is None else init[s:s + 1]
        for b in range(at, at + length, chunk):
            e = min(b + chunk, at + length)
            part = [x[b:e] for x in (q, k, v)] + [gg[b:e], beta[b:e]]
            start = torch.zeros(1, h, dk, dv, dtype=torch.float64, device=v.device) if state is None else state.double()
            _, state, _, _ = recurrence(*part, [e - b], start, 1.0)
            qq, kk = (x.double().repeat_interleave(share, 1).transpose(0, 1) for x in part[:2])     # [h, c, dk]
            vv, bb = part[2].double().transpose(0, 1), part[4].double().t()                          # [h, c, dv], [h, c]
            cum = part[3].clamp(min=-128).cumsum(0).t()                                              # [h, c]
            low = torch.ones(e - b, e - b, dtype=torch.bool, device=v.device).tril()
            x = torch.where(low, cum[:, :, None] - cum[:, None, :], 0.0)
            w = torch.where(low, x.exp(), 0.0)
            dw = w * 2.0 ** -22 * (1 + x.abs())
            gram = kk @ kk.transpose(1, 2)
            a = (bb[:, :, None] * w * gram).tril(-1)
            da = (bb[:, :, None] * (dw + 2 * dk * EPS * w)).tril(-1)                                # |k| <= 1
            eye = torch.eye(e - b, dtype=torch.float64, device=v.device)
            inv = torch.linalg.inv(eye + a)
            ti = inv.abs()
            dt = ti @ da @ ti + 528 * EPS * ti @ (eye + a.abs()) @ ti
            gam, dgam = cum.exp()[..., None], (cum.exp() * 2.0 ** -22 * (1 + cum.abs()))[..., None]
            norm = start[0].norm(dim=-2)[:, None, :]                                                 # [h, 1, dv]
            r = bb[..., None] * (vv - gam * (kk @ start[0]))
            dr = bb[..., None] * ((gam * (6 * dk + 16) * EPS + dgam) * norm + 8 * EPS * vv.abs())
            u = inv @ r
            tr = ti @ r.abs()
            du = dt @ r.abs() + ti @ dr + (3 + 800) * EPS * tr
            late = (cum[:, -1:] - cum)
            lat, dlat = late.exp()[..., None], (late.exp() * 2.0 ** -22 * (1 + late.abs()))[..., None]
            total = cum[:, -1].exp()[:, None]
            dtot = total * 2.0 ** -22 * (1 + cum[:, -1].abs()[:, None])
            p, dp = w * (qq @ kk.transpose(1, 2)), dw + 2 * dk * EPS * w
            o = (gam * ((2.0 ** -8 + 8 * dk * EPS) * (qq.abs() @ start[0].abs()) + err[s][:, None, :] + dgam * norm)
                 + (p.abs() + dp) @ du + dp @ u.abs() + (2 * 2.0 ** -8 + 2.0 ** -14) * (p.abs() @ u.abs()))
            bound[b:e] = abs(scale) * o.transpose(0, 1)
            err[s] = (1 + 2.0 ** -20) * total * err[s] + ((lat * du).sum(1) + (dlat * u.abs()).sum(1)
                                                          + 400 * EPS * (lat * u.abs()).sum(1)
                                                          + (dtot + 4 * EPS * total) * norm[:, 0] + 4 * EPS * state[0].norm(dim=-2))
        at += length
    return *want, err, bound
