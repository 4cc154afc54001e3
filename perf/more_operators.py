"""The gated delta rule's operators as they are measured: cases, inputs, plain forms, exact values.

Heads whose state has one decay and a delta-rule write, for prompts and for single tokens, and their
states kept in fewer bits for prefix reuse:
  prefill   kda.delta_prefill   S' = exp(g_t) S_(t-1),  S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,
                                o_t = scale S_t^T q_t over packed prompts; q and k shared by value heads
  decode    kda.delta_decode    the same for one token per sequence, state updated in place
  store     kda.state_pack      states into slots of a pool, 8 bits with a scale a row, or bf16; what the
                                pool then holds is read back by kda.state_unpack
  restore   kda.state_unpack    states from the slots of such a pool
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8}


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one long prompt through every head of the layer
        dict(name="prefill-prompt", op="prefill", lengths="8192", heads=96, keys=96, dk=128, dv=128, dtype="bf16",
             decay="token", init=False),
        # a batch of ragged prompts continuing cached prefixes, queries and keys shared by two value heads
        dict(name="prefill-ragged", op="prefill", lengths="5000,129,1,8191,2750,640,127,4100", heads=32, keys=16,
             dk=128, dv=128, dtype="bf16", decay="token", init=True),
        # short chat turns, where latency counts, narrow heads
        dict(name="prefill-short", op="prefill", lengths="1,17,64,3,200,31,90,128,5,77,11,45,2,150,33,8", heads=16,
             keys=16, dk=64, dv=64, dtype="bf16", decay="head", init=True),
        # single-precision evaluation of a middling prompt, keys narrower than values
        dict(name="prefill-f32", op="prefill", lengths="2047,513", heads=16, keys=8, dk=64, dv=128, dtype="f32",
             decay="token", init=True),
        # a full decode batch
        dict(name="decode-batch", op="decode", batch=256, heads=96, keys=96, dk=128, dv=128, dtype="bf16",
             decay="token"),
        # one stream being generated
        dict(name="decode-single", op="decode", batch=1, heads=32, keys=16, dk=128, dv=128, dtype="bf16",
             decay="token"),
        # a middling batch with narrow heads in single precision
        dict(name="decode-f32", op="decode", batch=37, heads=16, keys=4, dk=64, dv=64, dtype="f32", decay="head"),
        # a long prompt's checkpoints of one layer into the pool, scattered over its slots
        dict(name="store-checkpoints", op="store", states=64, slots=80, heads=96, dk=128, dv=128, dtype="int8"),
        # a few states of short requests
        dict(name="store-few", op="store", states=3, slots=7, heads=16, dk=64, dv=64, dtype="bf16"),
        # a batch of requests that continue cached prefixes
        dict(name="restore-batch", op="restore", states=64, slots=80, heads=96, dk=128, dv=128, dtype="int8"),
        # one request
        dict(name="restore-one", op="restore", states=1, slots=9, heads=32, dk=128, dv=128, dtype="int8"),
        # two requests from a pool in half precision, widths of an odd size
        dict(name="restore-bf16", op="restore", states=2, slots=5, heads=96, dk=96, dv=72, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return n - (n % 1024 == 0)   # the round sizes are listed


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "store", "restore"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "prefill":
        heads, share = rng.choice([(8, 1), (16, 1), (16, 2), (32, 1), (32, 2), (32, 4), (96, 1)])
        dk = rng.choice([64, 96, 128, 128])
        dv = rng.choice([dk, dk, 64, 128])
        longest = 8192 if dtype == "bf16" else 2560
        total, lengths = _log(rng, 64, longest * (96 if dtype == "bf16" else 16) // heads), []
        for i in range(rng.choice([1, 1, 2, 5, 12])):
            left = min(total - sum(lengths), longest - 1)
            if left < 1:
                break
            lengths.append(_log(rng, 1, left))
        return dict(op=op, lengths=",".join(map(str, lengths)), heads=heads, keys=heads // share, dk=dk, dv=dv,
                    dtype=dtype, decay=rng.choice(["token", "token", "head"]), init=rng.random() < 0.5)
    if op == "decode":
        heads, share = rng.choice([(8, 1), (16, 4), (32, 1), (32, 2), (96, 1)])
        dk = rng.choice([64, 128, 128])
        return dict(op=op, batch=_log(rng, 1, 255), heads=heads, keys=heads // share, dk=dk,
                    dv=rng.choice([dk, dk, 64, 128]), dtype=dtype, decay=rng.choice(["token", "head"]))
    states = _log(rng, 1, 63)
    return dict(op=op, states=states, slots=states + rng.choice([0, 1, 5, 16]), heads=rng.choice([8, 16, 32, 96]),
                dk=rng.choice([64, 96, 128, 128]), dv=rng.choice([64, 72, 128, 128]),
                dtype=rng.choice(["int8", "int8", "bf16"]))


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
    common = 0.4 * _normal(gen, case["keys"], case["dk"])   # a head's keys have a direction in common
    return dict(q=unit(_normal(gen, rows, case["keys"], case["dk"])),
                k=unit(_normal(gen, rows, case["keys"], case["dk"]) + common),
                v=_normal(gen, rows, case["heads"], case["dv"]).to(dt), g=_decay(gen, case, rows),
                beta=torch.sigmoid(_normal(gen, rows, case["heads"])), scale=case["dk"] ** -0.5)


def _states(gen, n, case):
    """States as a mixer leaves them: rows (key channels) of unlike magnitude, some never written."""
    s = _normal(gen, n, case["heads"], case["dk"], case["dv"]).mul_(0.1)
    s.mul_(torch.exp(_normal(gen, n, case["heads"], case["dk"], 1)))
    return s.mul_((torch.rand(n, case["heads"], case["dk"], 1, generator=gen, device=DEV) > 0.01).float())


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
            s["init"] = 0.1 * _normal(gen, len(lengths), case["heads"], case["dk"], case["dv"])
        return s
    if op == "decode":
        s.update(_heads(gen, case, case["batch"], dt))
        s["state"] = 0.1 * _normal(gen, case["batch"], case["heads"], case["dk"], case["dv"])
        return s
    n, slots = case["states"], case["slots"]
    s["idx"] = torch.randperm(slots, generator=gen, device=DEV)[:n].contiguous()
    shape = (slots, case["heads"], case["dk"], case["dv"])
    s["states"] = _states(gen, n, case)     # restore: where the states go
    s["pool"] = torch.zeros(shape, device=DEV, dtype=dt)
    s["scales"] = torch.zeros(shape[:3], device=DEV) if case["dtype"] == "int8" else None
    if op == "restore":
        if case["dtype"] == "int8":
            s["pool"] = torch.randint(-127, 128, shape, generator=gen, device=DEV, dtype=torch.int8)
            s["scales"] = torch.rand(shape[:3], generator=gen, device=DEV).mul_(0.02)
        else:
            s["pool"] = (0.1 * _normal(gen, *shape)).to(dt)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        import kimi_delta_attention_13_gb300 as kda

        if s["op"] == "prefill":
            return kda.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], s["init"], scale=s["scale"])
        if s["op"] == "decode":
            return kda.delta_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"]), s["state"]
        if s["op"] == "store":
            kda.state_pack(s["pool"], s["states"], dst_idx=s["idx"], scales=s["scales"])
            return kda.state_unpack(torch.empty_like(s["states"]), s["pool"], src_idx=s["idx"], scales=s["scales"])
        return kda.state_unpack(s["states"], s["pool"], src_idx=s["idx"], scales=s["scales"])
    return {"prefill": _prefill, "decode": _decode, "store": _store, "restore": _restore}[s["op"]](s)


def _inverse(a):
    """(I + a)^-1 for strictly lower triangular a [..., c, c]: blocks of 1, 2, 4, ... joined in pairs."""
    c = a.shape[-1]
    t = torch.eye(c, device=a.device).expand(a.shape).clone()
    s = 1
    while s < c:
        blocks = lambda x, i, j: x.view(*x.shape[:-2], c // (2 * s), 2, s, c // (2 * s), 2, s) \
            .diagonal(dim1=-6, dim2=-3)[..., i, :, j, :, :].movedim(-1, -3)  # noqa: E731
        low = -(blocks(t, 1, 1) @ blocks(a, 1, 0) @ blocks(t, 0, 0))
        t.view(*t.shape[:-2], c // (2 * s), 2, s, c // (2 * s), 2, s).diagonal(dim1=-6, dim2=-3)[..., 1, :, 0, :, :] \
            .copy_(low.movedim(-3, -1))
        s *= 2
    return t


def _prefill(s):
    """Chunks of 64 tokens: products within a chunk at once, then chunk after chunk, all sequences side by side.
    Sums of log decays are in 64 bits."""
    q, k, v, g, cu, lengths = s["q"], s["k"], s["v"], s["g"], s["cu"].long(), s["lengths"]
    c, (t, h, dv), n = 64, v.shape, len(lengths)
    chunks = max(-(-x // c) for x in lengths)
    tok = cu[:-1, None] + torch.arange(chunks * c, device=q.device)
    live = tok < cu[1:, None]
    at = tok.clamp(max=t - 1)

    def packed(x):   # [T, heads, ...] -> [chunks, N, H, c, ...], nothing past a sequence's end
        x = x.repeat_interleave(h // x.shape[1], 1)
        x = torch.where(live.view(n, -1, *[1] * (x.dim() - 1)), x[at], torch.zeros((), dtype=x.dtype, device=x.device))
        return x.view(n, chunks, c, *x.shape[2:]).transpose(2, 3).transpose(0, 1)

    q, k, v, beta = packed(q).float(), packed(k).float(), packed(v).float(), packed(s["beta"])
    b = torch.cumsum(packed(g if g.dim() == 2 else g.expand(t, h)).double(), -1)          # [chunks, N, H, c]
    lower = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    w = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~lower, -math.inf)).float()
    inv = _inverse((k @ k.transpose(-1, -2) * w * beta[..., None]).tril(-1))
    p = q @ k.transpose(-1, -2) * w
    gamma, later, total = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None], \
        torch.exp(b[..., -1]).float()[..., None, None]
    state = s["init"].clone() if s["init"] is not None else torch.zeros(n, h, k.shape[-1], dv, device=q.device)
    out = []
    for i in range(chunks):   # the recurrence
        u = inv[i] @ (beta[i][..., None] * (v[i] - gamma[i] * (k[i] @ state)))
        out.append(gamma[i] * (q[i] @ state) + p[i] @ u)
        state = total[i] * state + k[i].transpose(-1, -2) @ (later[i] * u)
    out = torch.stack(out).transpose(0, 1).transpose(2, 3).reshape(n, chunks * c, h, dv)[live]
    return (out * s["scale"]).to(s["q"].dtype), state


def _decode(s):
    h = s["v"].shape[1]
    wide = lambda x: x.repeat_interleave(h // x.shape[1], 1).float()  # noqa: E731
    q, k, v, state = wide(s["q"]), wide(s["k"]), s["v"].float(), s["state"]
    state.mul_(torch.exp(s["g"])[..., None, None])
    u = s["beta"][..., None] * (v - (k[..., None, :] @ state)[..., 0, :])
    state.add_(k[..., :, None] * u[..., None, :])
    out = (q[..., None, :] @ state)[..., 0, :] * s["scale"]
    return out.to(s["q"].dtype), state


def _store(s):
    x, idx = s["states"], s["idx"]
    if s["scales"] is None:
        s["pool"][idx] = x.to(s["pool"].dtype)
    else:
        # quotients in 64 bits: in 32 one can fall on a border between two codes
        scale = (x.abs().amax(-1).double() / 127).float()
        code = torch.where(scale[..., None] > 0, x.double() / scale[..., None].double(), 0.0).round()
        s["pool"][idx], s["scales"][idx] = code.to(torch.int8), scale
    return _values(s)


def _values(s):
    x = s["pool"][s["idx"]].float()
    return x if s["scales"] is None else x * s["scales"][s["idx"]][..., None]


def _restore(s):
    return s["states"].copy_(_values(s))


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    h, dk, dv = case["heads"], case["dk"], case["dv"]
    if case["op"] in ("prefill", "decode"):
        rows = sum(_lengths(case)) if case["op"] == "prefill" else case["batch"]
        seqs = len(_lengths(case)) if case["op"] == "prefill" else case["batch"]
        move = e * rows * (2 * case["keys"] * dk + 2 * h * dv)
        move += 4 * h * (rows + (rows if case["decay"] == "token" else 1))
        move += 4 * seqs * h * dk * dv * (2 if case["op"] == "decode" or case["init"] else 1)
        return {"bytes": move, "flops": 6 * rows * h * dk * dv}
    n = case["states"] * h * dk * dv
    held = n * 2 if case["dtype"] == "bf16" else n + n // dv * 4
    # a store is written and read back
    return {"bytes": (4 * n + held) * (2 if case["op"] == "store" else 1), "flops": 4 * n}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prefill", "decode"):
        return _exact_recurrence(case, {n: x.double() for n, x in s.items()
                                        if isinstance(x, torch.Tensor) and x.is_floating_point()}, s["scale"])
    if case["op"] == "restore":
        held = s["pool"].double()
        return (held if s["scales"] is None else held * s["scales"].double()[..., None])[s["idx"]]
    x = s["states"].double()
    if case["dtype"] == "bf16":   # the value held: nearest of 8 significant bits, ties to even
        m, e = torch.frexp(x)
        return torch.ldexp(torch.round(m * 256), e - 8)
    scale = (x.abs().amax(-1, keepdim=True) / 127).float().double()   # held in 32 bits
    return torch.where(scale > 0, torch.round(x / scale), 0.0) * scale


def _exact_recurrence(case, wide, scale):
    """Token by token, all sequences side by side."""
    h, share = case["heads"], case["heads"] // case["keys"]
    lengths = _lengths(case) if case["op"] == "prefill" else [1] * case["batch"]
    n, rows = len(lengths), sum(lengths)
    decay = wide["g"].exp().expand(rows, h)
    if "state" in wide:
        state = wide["state"]
    else:
        state = wide["init"] if "init" in wide else torch.zeros(n, h, case["dk"], case["dv"], device=DEV).double()
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
        q = wide["q"][at].repeat_interleave(share, 1)
        k = wide["k"][at].repeat_interleave(share, 1)
        cur.mul_(decay[at][..., None, None])
        miss = wide["v"][at] - torch.matmul(k[..., None, :], cur)[..., 0, :]
        cur.addcmul_(k[..., :, None], (wide["beta"][at][..., None] * miss)[..., None, :])
        out[at] = torch.matmul(q[..., None, :], cur)[..., 0, :]
    final = torch.empty_like(state)
    final[order] = state
    return out * scale, final
