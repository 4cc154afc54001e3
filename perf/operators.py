"""The linear-attention layer's operators as they are measured: cases, inputs, plain forms, exact values.

Four operators make the layer around a mixer whose heads each have one decay:
  prefill   kda.linear_prefill   S_t = exp(g_t) S_(t-1) + k_t v_t^T,  o_t = scale S_t^T q_t over packed prompts
  decode    kda.linear_decode    the same for one token per sequence, state updated in place
  gate      kda.norm_gate        o * rsqrt(mean(o^2) + eps) * w * sigmoid(z) per (token, head)
  residual  kda.residual_norm    r = x + scale sigmoid(z) norm(y) w_post,  n = norm(r) w
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one long prompt through every head of the layer
        dict(name="prefill-prompt", op="prefill", lengths="8192", heads=96, kv=96, dk=128, dv=128,
             dtype="bf16", decay="token", init=False),
        # a batch of ragged prompts continuing cached prefixes, keys and values shared by 4 heads
        dict(name="prefill-ragged", op="prefill", lengths="5000,129,1,8191,2750,640,127,4100", heads=32,
             kv=8, dk=128, dv=128, dtype="bf16", decay="head", init=True),
        # a long document on few heads (the share of one rank)
        dict(name="prefill-long", op="prefill", lengths="65536", heads=8, kv=8, dk=128, dv=128,
             dtype="bf16", decay="token", init=True),
        # short chat turns, where latency counts, narrow heads
        dict(name="prefill-short", op="prefill", lengths="1,17,64,3,200,31,90,128,5,77,11,45,2,150,33,8",
             heads=16, kv=16, dk=64, dv=64, dtype="bf16", decay="token", init=True),
        # single-precision evaluation of a middling prompt, keys narrower than values
        dict(name="prefill-f32", op="prefill", lengths="2047,513", heads=16, kv=16, dk=64, dv=128,
             dtype="f32", decay="token", init=True),
        # a full decode batch
        dict(name="decode-batch", op="decode", batch=256, heads=96, kv=96, dk=128, dv=128, dtype="bf16",
             decay="token"),
        # one stream being generated
        dict(name="decode-single", op="decode", batch=1, heads=32, kv=32, dk=128, dv=128, dtype="bf16",
             decay="head"),
        # a middling batch with narrow shared heads in single precision
        dict(name="decode-f32", op="decode", batch=37, heads=16, kv=4, dk=64, dv=64, dtype="f32",
             decay="token"),
        # the head norm and gate after the mixer: the long prompt, and a decode step
        dict(name="gate-prompt", op="gate", tokens=8192, heads=96, d=128, dtype="bf16"),
        dict(name="gate-step", op="gate", tokens=5, heads=32, d=128, dtype="bf16"),
        # the residual add between two blocks: the long prompt with post-norm and gate, and a decode batch
        dict(name="residual-prompt", op="residual", tokens=8192, width=12288, dtype="bf16", post=True,
             gated=True),
        dict(name="residual-step", op="residual", tokens=33, width=4096, dtype="bf16", post=True, gated=False),
    ]


def _log(rng, lo, hi):
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return n - (n % 1024 == 0)   # the round sizes are listed


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "gate", "residual"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "prefill":
        heads, share = rng.choice([(8, 1), (16, 1), (16, 4), (32, 1), (32, 4), (96, 1)])
        dk = rng.choice([64, 128, 128])
        dv = rng.choice([dk, dk, 64, 128])
        budget = (8192 * 96 if dtype == "bf16" else 2560 * 16) // heads
        total, lengths = _log(rng, 64, budget), []
        for i in range(rng.choice([1, 1, 2, 5, 12])):
            left = total - sum(lengths)
            if left < 1:
                break
            lengths.append(_log(rng, 1, left))
        return dict(op=op, lengths=",".join(map(str, lengths)), heads=heads, kv=heads // share, dk=dk, dv=dv,
                    dtype=dtype, decay=rng.choice(["token", "head"]), init=rng.random() < 0.5)
    if op == "decode":
        heads, share = rng.choice([(8, 1), (16, 4), (32, 1), (32, 8), (96, 1)])
        d = rng.choice([64, 128, 128])
        return dict(op=op, batch=_log(rng, 1, 256), heads=heads, kv=heads // share, dk=d, dv=d, dtype=dtype,
                    decay=rng.choice(["token", "head"]))
    if op == "gate":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.choice([8, 16, 32, 64, 96]),
                    d=rng.choice([64, 128, 128]), dtype=dtype)
    return dict(op=op, tokens=_log(rng, 1, 8192), width=rng.choice([1024, 1536, 2048, 2560, 4096, 5120, 8192]),
                dtype=dtype, post=rng.random() < 0.7, gated=rng.random() < 0.5)


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


# ---------------------------------------------------------------------------------------------
# inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _decay(gen, case, rows):
    """Log decays: per token as a gate gives them (memory of some 4 to 200 tokens), or one slope per head."""
    h = case["heads"]
    if case["decay"] == "head":
        return -torch.exp2(-8.0 * (torch.arange(h, device=DEV) + torch.rand(h, generator=gen, device=DEV)) / h)
    return -torch.nn.functional.softplus(_normal(gen, rows, h) - 3.0)


def _heads(gen, case, rows, dt):
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    return dict(q=unit(_normal(gen, rows, case["heads"], case["dk"])),
                k=unit(_normal(gen, rows, case["kv"], case["dk"])),
                v=_normal(gen, rows, case["kv"], case["dv"]).to(dt), g=_decay(gen, case, rows),
                scale=case["dk"] ** -0.5)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt, op = TYPES[case["dtype"]], case["op"]
    s = dict(op=op)
    if op == "prefill":
        lengths = _lengths(case)
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        s.update(_heads(gen, case, ends[-1], dt), lengths=lengths)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        s["init"] = None
        if case["init"]:
            s["init"] = 0.05 * _normal(gen, len(lengths), case["heads"], case["dk"], case["dv"])
    elif op == "decode":
        s.update(_heads(gen, case, case["batch"], dt))
        s["state"] = 0.3 * _normal(gen, case["batch"], case["heads"], case["dk"], case["dv"])
    elif op == "gate":
        shape = (case["tokens"], case["heads"], case["d"])
        s.update(o=_normal(gen, *shape).mul_(0.2).to(dt), z=_normal(gen, *shape).to(dt),
                 w=1 + 0.1 * _normal(gen, case["d"]))
    else:
        shape, width = (case["tokens"], case["width"]), case["width"]
        s.update(x=_normal(gen, *shape).to(dt), y=_normal(gen, *shape).mul_(0.3).to(dt),
                 w=1 + 0.1 * _normal(gen, width), scale=0.5,
                 w_post=1 + 0.1 * _normal(gen, width) if case["post"] else None,
                 z=_normal(gen, *shape).to(dt) if case["gated"] else None)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        import kimi_delta_attention_13_gb300 as kda

        if s["op"] == "prefill":
            return kda.linear_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"], s["init"], scale=s["scale"])
        if s["op"] == "decode":
            return kda.linear_decode(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"]), s["state"]
        if s["op"] == "gate":
            return kda.norm_gate(s["o"], s["z"], s["w"], eps=EPS)
        return kda.residual_norm(s["x"], s["y"], s["w"], w_post=s["w_post"], z=s["z"], scale=s["scale"], eps=EPS)
    return {"prefill": _prefill, "decode": _decode, "gate": _gate, "residual": _residual}[s["op"]](s)


def _prefill(s):
    """Chunks of 64 tokens at once: products within a chunk, and the chunks' states joined by one product with
    the matrix of decays between chunks.  Sums of log decays are in 64 bits."""
    q, k, v, g, cu, lengths = s["q"], s["k"], s["v"], s["g"], s["cu"].long(), s["lengths"]
    c, (t, h, dk), dv, n = 64, q.shape, v.shape[-1], len(lengths)
    counts = (cu[1:] - cu[:-1] + c - 1) // c
    chunks = sum(-(-x // c) for x in lengths)
    first = torch.cumsum(counts, 0) - counts
    seq = torch.repeat_interleave(torch.arange(n, device=q.device), counts, output_size=chunks)
    tok = (cu[seq] + (torch.arange(chunks, device=q.device) - first[seq]) * c)[:, None] \
        + torch.arange(c, device=q.device)
    live = tok < cu[seq + 1][:, None]
    at = tok.clamp(max=t - 1)

    def packed(x):  # [T, heads, d] -> [H, chunks, c, d] in 32 bits, nothing past a sequence's end
        x = x.repeat_interleave(h // x.shape[1], 1).float()
        return (x[at] * live[..., None, None]).permute(2, 0, 1, 3).contiguous()

    q32, k32, v32 = packed(q), packed(k), packed(v)
    g64 = (g if g.dim() == 2 else g.expand(t, h)).double()
    b = torch.cumsum((g64[at] * live[..., None]).permute(2, 0, 1), -1)                    # [H, chunks, c]
    lower = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    w = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~lower, -math.inf)).float()
    o = (q32 @ k32.transpose(-1, -2) * w) @ v32
    d = k32.transpose(-1, -2) @ (v32 * torch.exp(b[..., -1:] - b).float()[..., None])     # [H, chunks, dk, dv]
    total = b[..., -1]
    before = torch.cumsum(total, -1) - total
    i = torch.arange(chunks, device=q.device)
    joined = (seq[:, None] == seq) & (i[:, None] > i)
    m = torch.exp((before[:, :, None] - (before + total)[:, None, :]).masked_fill(~joined, -math.inf)).float()
    start = (m @ d.view(h, chunks, dk * dv)).view(h, chunks, dk, dv)
    init = s["init"] if s["init"] is not None else torch.zeros(n, h, dk, dv, device=q.device)
    start += torch.exp(before - before[:, first.clamp(max=chunks - 1)][:, seq]).float()[..., None, None] \
        * init[seq].transpose(0, 1)
    o += (q32 * torch.exp(b).float()[..., None]) @ start
    out = (o.permute(1, 2, 0, 3)[live] * s["scale"]).to(q.dtype)
    last = first + counts - 1
    final = (start[:, last] * torch.exp(total[:, last]).float()[..., None, None] + d[:, last]).transpose(0, 1)
    return out, torch.where((counts > 0)[:, None, None, None], final, init)


def _decode(s):
    h = s["q"].shape[1]
    wide = lambda x: x.repeat_interleave(h // x.shape[1], 1).float()  # noqa: E731
    k, v, state = wide(s["k"]), wide(s["v"]), s["state"]
    state.mul_(torch.exp(s["g"])[..., None, None]).add_(k[..., :, None] * v[..., None, :])
    out = (s["q"].float()[..., None, :] @ state)[..., 0, :] * s["scale"]
    return out.to(s["q"].dtype), state


def _gate(s):
    o, z = s["o"].float(), s["z"].float()
    out = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["w"] / (1 + torch.exp(-z))
    return out.to(s["z"].dtype)


def _residual(s):
    u = s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["w_post"]
    if s["z"] is not None:
        u = u / (1 + torch.exp(-s["z"].float()))
    r = s["x"].float() + s["scale"] * u
    n = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["w"]
    return r.to(s["x"].dtype), n.to(s["x"].dtype)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("prefill", "decode"):
        rows = sum(_lengths(case)) if case["op"] == "prefill" else case["batch"]
        seqs = len(_lengths(case)) if case["op"] == "prefill" else case["batch"]
        h, kv, dk, dv = case["heads"], case["kv"], case["dk"], case["dv"]
        state = 4 * seqs * h * dk * dv
        move = e * rows * (h * (dk + dv) + kv * (dk + dv)) + 4 * h * (rows if case["decay"] == "token" else 1)
        move += state * (2 if case["op"] == "decode" or case["init"] else 1)
        return {"bytes": move, "flops": 4 * rows * h * dk * dv}
    if case["op"] == "gate":
        n = case["tokens"] * case["heads"] * case["d"]
        return {"bytes": 3 * e * n + 4 * case["d"], "flops": 8 * n}
    n = case["tokens"] * case["width"]
    return {"bytes": (4 + case["gated"]) * e * n + 4 * case["width"] * (1 + case["post"]), "flops": 12 * n}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    wide = {n: x.double() for n, x in s.items() if isinstance(x, torch.Tensor) and x.is_floating_point()}
    if case["op"] in ("prefill", "decode"):
        return _exact_recurrence(case, s, wide)
    if case["op"] == "gate":
        o = wide["o"]
        return o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * wide["w"] * torch.sigmoid(wide["z"])
    u = wide["y"]
    if "w_post" in wide:
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * wide["w_post"]
    if "z" in wide:
        u = u * torch.sigmoid(wide["z"])
    r = wide["x"] + s["scale"] * u
    return r, r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * wide["w"]


def _exact_recurrence(case, s, wide):
    """Token by token, all sequences side by side."""
    h, share = case["heads"], case["heads"] // case["kv"]
    lengths = _lengths(case) if case["op"] == "prefill" else [1] * case["batch"]
    n, rows = len(lengths), sum(lengths)
    decay = wide["g"].exp().expand(rows, h)
    if "state" in wide:
        state = wide["state"]
    else:
        state = wide["init"] if "init" in wide else torch.zeros(n, h, case["dk"], case["dv"], device=DEV).double()
    state = state.clone()
    out = torch.empty(rows, h, case["dv"], device=DEV, dtype=torch.float64)
    order = sorted(range(n), key=lambda i: -lengths[i])
    start = [sum(lengths[:i]) for i in range(n)]
    state = state[order]
    begin = torch.tensor([start[i] for i in order], device=DEV)
    live = n
    for t in range(max(lengths)):
        while lengths[order[live - 1]] <= t:
            live -= 1
        at, cur = begin[:live] + t, state[:live]
        k = wide["k"][at].repeat_interleave(share, 1)
        v = wide["v"][at].repeat_interleave(share, 1)
        cur.mul_(decay[at][..., None, None])
        cur.addcmul_(k[..., :, None], v[..., None, :])
        out[at] = torch.matmul(wide["q"][at][..., None, :], cur)[..., 0, :]
    final = torch.empty_like(state)
    final[order] = state
    return out * s["scale"], final
