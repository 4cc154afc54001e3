"""What the tensor-core prefill of the gated delta rule may leave of its outputs, and its roundings in 64 bits.

    o = scale (e^G S^T q + sum_j P_j u_j),   P = w (q . k)
An output takes two bf16 parts of the state S before its chunk and of u, and one of P.  A rounding to bf16 is off by 2^-8
of the value at most, so two parts leave 2^-16 and one 2^-8: 2^-16 of sum |q| |S| and 2^-8 + 2^-14 of sum |P| |u| (2^-14
for u's parts, products of the two and the sums in fp32, as in chunked_bounds, whose other terms stay).
"""
import torch

from delta_plain import chunked_bounds, recurrence


def parts(x, n, sign=1.0):
    """x held in n bf16 parts, those behind the first times `sign`."""
    held, left = torch.zeros_like(x), x
    for i in range(n):
        part = left.float().bfloat16().double()
        held, left = held + (part if i == 0 else sign * part), left - part
    return held


def outputs(x, lengths, scale=1.0, hold_s=None, hold_u=None, hold_p=None, chunk=64):
    """(out, state term, score term): the outputs in 64 bits from S, u and P of each chunk as `hold_*` keep them, and
    the sums of magnitudes |scale| e^G sum |q| |S| and |scale| sum |P| |u|."""
    same = lambda y: y  # noqa: E731
    hold_s, hold_u, hold_p = (h or same for h in (hold_s, hold_u, hold_p))
    t, h, dv = x["v"].shape
    share, dk = h // x["q"].shape[1], x["q"].shape[2]
    g = (x["g"] if x["g"].dim() == 2 else x["g"].expand(t, h)).double()
    out = torch.zeros(t, h, dv, dtype=torch.float64, device=x["v"].device)
    of_s, of_p = torch.zeros_like(out), torch.zeros_like(out)
    at = 0
    for s, length in enumerate(lengths):
        start = x["init"][s:s + 1].double() if x["init"] is not None else out.new_zeros(1, h, dk, dv)
        for b in range(at, at + length, chunk):
            e = min(b + chunk, at + length)
            q, k = (x[n][b:e].double().repeat_interleave(share, 1).transpose(0, 1) for n in ("q", "k"))   # [h, c, dk]
            v, beta = x["v"][b:e].double().transpose(0, 1), x["beta"][b:e].double().t()
            cum = g[b:e].clamp(min=-128).cumsum(0).t()
            low = torch.ones(e - b, e - b, dtype=torch.bool, device=out.device).tril()
            w = torch.where(low, (cum[:, :, None] - cum[:, None, :]).masked_fill(~low, 0.0).exp(), 0.0)
            a = (beta[:, :, None] * w * (k @ k.transpose(1, 2))).tril(-1)
            gam = cum.exp()[..., None]
            r = beta[..., None] * (v - gam * (k @ start[0]))
            u = torch.linalg.solve_triangular(torch.eye(e - b, dtype=torch.float64, device=out.device) + a, r, upper=False)
            p = scale * w * (q @ k.transpose(1, 2))
            out[b:e] = (scale * gam * (q @ hold_s(start[0])) + hold_p(p) @ hold_u(u)).transpose(0, 1)
            of_s[b:e] = (abs(scale) * gam * (q.abs() @ start[0].abs())).transpose(0, 1)
            of_p[b:e] = (p.abs() @ u.abs()).transpose(0, 1)
            part = [x[n][b:e] for n in ("q", "k", "v")] + [g[b:e], x["beta"][b:e]]
            start = recurrence(*part, [e - b], start)[1]
        at += length
    return out, of_s, of_p


def output_bounds(x, lengths, scale=1.0, exact_scores=False):
    """(out, bound of an output before it is rounded to its type); exact_scores: those that P is rounded in none of."""
    want, _, _, loose = chunked_bounds(*(x[n] for n in ("q", "k", "v", "g", "beta")), lengths, x["init"], scale)
    _, of_s, of_p = outputs(x, lengths, scale)
    # chunked_bounds counts 2^-8 of S, and 2^-8 of P and of u each
    return want, loose - (2.0 ** -8 - 2.0 ** -16) * of_s - (2 if exact_scores else 1) * 2.0 ** -8 * of_p


def within(out, want, bound, slack=1e-30):
    """Every output within its bound and its type's rounding; a NaN is not."""
    half = torch.finfo(out.dtype).eps / 2 if out.dtype is not torch.float64 else 0.0
    ok = (out.double() - want).abs() <= bound + half * (want.abs() + bound) + slack
    return bool(ok.all())


def unit_keys(x, tokens):
    """The operands with keys that are one channel each, another for every token of a chunk, queries that are 2^-4 in all
    channels (of norm at most 1, as chunked_bounds has them), and no decay: P is then 2^-4 throughout."""
    dk = x["k"].shape[2]
    assert dk >= 64
    x["k"].zero_()
    x["k"].scatter_(2, (torch.arange(tokens, device=x["k"].device) % 64)[:, None, None].expand(-1, x["k"].shape[1], 1), 1.0)
    x["q"].fill_(2.0 ** -4)
    x["g"].zero_()
    return x
