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
