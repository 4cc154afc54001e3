"""state_pack and state_unpack against their definitions in 64 bits: equal codes, scales and values."""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda

pytestmark = pytest.mark.gpu
INT8, BF16 = torch.int8, torch.bfloat16


def states(n, h, dk, dv, seed):
    gen = torch.Generator().manual_seed(seed)
    s = torch.randn(n, h, dk, dv, generator=gen) * torch.exp(2 * torch.randn(n, h, dk, 1, generator=gen))
    return s.cuda()


def quantised(x):
    """(codes, scales): the quotient in 64 bits is exact enough to round (a tie is a tie there too)."""
    scale = (x.abs().amax(-1).double() / 127).float()
    code = torch.where(scale[..., None] > 0, x.double() / scale[..., None].double(), 0.0).round().clamp(-127, 127)
    return code.to(INT8), scale


def pool(slots, like, dtype):
    held = torch.zeros(slots, *like.shape[1:], dtype=dtype, device="cuda")
    return held, torch.zeros(held.shape[:3], device="cuda") if dtype is INT8 else None


SHAPES = [(1, 8, 8), (3, 128, 128), (2, 64, 64), (5, 72, 96), (2, 40, 32), (1, 256, 256), (2, 9, 132), (1, 3, 4), (96, 128, 128)]


@pytest.mark.parametrize("dtype", [INT8, BF16])
@pytest.mark.parametrize("h,dk,dv", SHAPES)
def test_values(dtype, h, dk, dv):
    x = states(4, h, dk, dv, seed=dk + dv)
    x[0, 0, 0] = 0.0
    held, scales = pool(6, x, dtype)
    held.fill_(3)
    dst = torch.tensor([5, 0, 2], device="cuda")
    src = torch.tensor([1, 0, 3], device="cuda")
    assert kda.state_pack(held, x, dst, src, scales=scales) is held
    if dtype is INT8:
        code, scale = quantised(x)
        assert torch.equal(held[dst], code[src]) and torch.equal(scales[dst], scale[src])
        assert bool((scales[[1, 3, 4]] == 0).all())
        want = (code[src].float() * scale[src][..., None])
    else:
        assert torch.equal(held[dst], x[src].to(BF16))
        want = x[src].to(BF16).float()
    assert bool((held[[1, 3, 4]] == 3).all())        # slots that no index names
    back = torch.full((5, h, dk, dv), 9.0, device="cuda")
    to = torch.tensor([4, 1, 0], device="cuda")
    assert kda.state_unpack(back, held, to, dst, scales=scales) is back
    assert torch.equal(back[to], want) and bool((back[[2, 3]] == 9).all())
    assert kda.device_status() == 0


def test_borders():
    """Ties, values next to one, the largest and the smallest magnitudes, infinities and NaN."""
    h, dk, dv = 1, 64, 128
    x = torch.zeros(1, h, dk, dv, device="cuda")
    gen = torch.Generator().manual_seed(2)
    for r in range(16):                               # scale 1: half numbers are ties, their neighbours are not
        x[0, 0, r] = (torch.randint(-126, 126, (dv,), generator=gen) + 0.5).cuda()
        x[0, 0, r, 0] = 127
    up = torch.full_like(x, float("inf"))
    x[0, 0, 4:8] = torch.nextafter(x[0, 0, 4:8], up[0, 0, 4:8])
    x[0, 0, 8:12] = torch.nextafter(x[0, 0, 8:12], -up[0, 0, 8:12])
    x[0, 0, 4:12, 0] = 127
    for r in range(16, 40):                           # scales that are no round number
        x[0, 0, r] = ((torch.randint(-126, 126, (dv,), generator=gen) + 0.5) * (0.37 + r)).cuda()
        x[0, 0, r, 0] = 127 * (0.37 + r)
    x[0, 0, 40] = torch.randn(dv, generator=gen).cuda() * 1e38
    x[0, 0, 41] = torch.randn(dv, generator=gen).cuda() * 1e-36
    x[0, 0, 42] = torch.randn(dv, generator=gen).cuda() * 1e-42      # subnormal
    x[0, 0, 43] = 1e-45
    x[0, 0, 44, 5] = -3.4e38
    x[0, 0, 45, 7] = -1.0
    held, scales = pool(1, x, INT8)
    kda.state_pack(held, x, scales=scales)
    code, scale = quantised(x)
    assert torch.equal(scales, scale) and torch.equal(held, code)
    x[0, 0, 0, 3], x[0, 0, 1, 127], x[0, 0, 2, 0] = float("nan"), float("inf"), -float("inf")
    kda.state_pack(held, x, scales=scales)
    assert bool(scales[0, 0, :3].isnan().all()) and torch.equal(held[0, 0, 3:], code[0, 0, 3:])
    back = kda.state_unpack(torch.zeros_like(x), held, scales=scales)
    assert bool(back[0, 0, :3].isnan().all()) and bool(back[0, 0, 3:].isfinite().all())
    half, _ = pool(1, x, BF16)
    kda.state_pack(half, x)
    want = x.to(BF16)
    assert torch.equal(half.isnan(), want.isnan()) and torch.equal(half.nan_to_num(0.0), want.nan_to_num(0.0))


def test_quotients_next_to_a_border():
    """Rows whose quotients in 32 bits would often round to a half: the code is the exact quotient's."""
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(1, 16, 256, 128, generator=gen).cuda()
    _, scale = quantised(x)
    half = torch.randint(-126, 126, x.shape, generator=gen).cuda() + 0.5
    near = (half.double() * scale[..., None].double()).float()         # the fp32 value nearest a border
    near[..., 0] = x.abs().amax(-1)                                    # keeps the row's scale
    held, scales = pool(1, near, INT8)
    kda.state_pack(held, near, scales=scales)
    code, want = quantised(near)
    assert torch.equal(want, scale) and torch.equal(scales, want) and torch.equal(held, code)


@pytest.mark.parametrize("dtype", [INT8, BF16])
def test_index_out_of_range(dtype):
    x = states(3, 2, 64, 64, seed=1)
    held, scales = pool(4, x, dtype)
    for bad in (4, -1):
        kda.state_pack(held, x, torch.tensor([0, bad, 2], device="cuda"), scales=scales)
        assert kda.device_status() == 6 and kda.device_status() == 0
    assert bool((held[[1, 3]] == 0).all()) and not bool((held[[0, 2]] == 0).all())
    back = torch.full_like(x, 5.0)
    kda.state_unpack(back, held, torch.tensor([0, 3], device="cuda"), torch.tensor([0, 2], device="cuda"), scales=scales)
    assert kda.device_status() == 6
    want = held[0].float() if scales is None else held[0].float() * scales[0][..., None]
    assert bool((back[1:] == 5).all()) and torch.equal(back[0], want)


def test_large_pool():
    """Slots past 2^31 bytes and elements from the pool's start."""
    h, dk, dv = 96, 128, 128
    slots = 1500                                      # 2.4e9 elements
    held = torch.zeros(slots, h, dk, dv, dtype=INT8, device="cuda")
    scales = torch.zeros(slots, h, dk, device="cuda")
    x = states(2, h, dk, dv, seed=4)
    to = torch.tensor([1499, 1400], device="cuda")
    kda.state_pack(held, x, to, scales=scales)
    code, scale = quantised(x)
    assert torch.equal(held[to], code) and torch.equal(scales[to], scale)
    back = kda.state_unpack(torch.empty_like(x), held, None, to, scales=scales)
    assert torch.equal(back, code.float() * scale[..., None])


def test_refusals():
    x = states(2, 2, 8, 8, seed=1)
    held, scales = pool(2, x, INT8)
    half, _ = pool(2, x, BF16)
    for args, kw in (((held, x), {}), ((half, x), dict(scales=scales)), ((x, x), {}), ((held, half), dict(scales=scales)),
                     ((held, x[:, :1].contiguous()), dict(scales=scales)), ((held, x), dict(scales=scales[:1].contiguous())),
                     ((held, x, torch.tensor([0], device="cuda"), torch.tensor([0, 1], device="cuda")), dict(scales=scales)),
                     ((held, x, torch.tensor([0], device="cuda")), dict(scales=scales, n=2)),
                     ((held, x, torch.tensor([0], device="cuda", dtype=torch.int32)), dict(scales=scales)),
                     ((held.cpu(), x), dict(scales=scales))):
        with pytest.raises(ValueError):
            kda.state_pack(*args, **kw)
    with pytest.raises(kda.KDAError):
        kda.state_pack(held, x, n=3, scales=scales)
    wide = states(1, 1, 8, 260, seed=1)
    with pytest.raises(kda.KDAError):
        kda.state_pack(pool(1, wide, BF16)[0], wide)
    memory = torch.zeros(2, 2, 8, 8, device="cuda")
    with pytest.raises(kda.KDAError):                 # the pool lies in the states' own memory
        kda.state_pack(memory.view(BF16).view(-1)[:256].view(2, 2, 8, 8), memory)
    assert kda.device_status() == 0


def test_graph():
    x = states(3, 4, 64, 64, seed=1)
    held, scales = pool(5, x, INT8)
    back, idx = torch.empty_like(x), torch.tensor([4, 1, 2], device="cuda")

    def both():
        kda.state_pack(held, x, idx, scales=scales)
        kda.state_unpack(back, held, None, idx, scales=scales)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    x.copy_(states(3, 4, 64, 64, seed=7))
    graph.replay()
    torch.cuda.synchronize()
    code, scale = quantised(x)
    assert torch.equal(back, code.float() * scale[..., None])


@pytest.mark.parametrize("dtype", [INT8, BF16])
def test_store_of_packed_checkpoints(dtype):
    """A prompt's checkpoints in a packed store, and requests that resume from them."""
    from kimi_delta_attention_13_gb300 import synth
    from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore, resume_prefill

    lengths = [96, 64]
    s = synth.make_inputs(lengths, heads=2, dtype="bf16", seed=5, device="cuda")
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu_seqlens"])
    _, _, ckpts = kda.prefill(*args, ckpt_stride=32, lengths=lengths)
    store = CheckpointStore(8, 2, device="cuda", dtype=dtype)
    kept = store.add_checkpoints(["a", "b"], ckpts, 32, lengths)
    assert [(k, n) for k, n, _ in kept] == [("a", 32), ("a", 64), ("a", 96), ("b", 32), ("b", 64)]
    if dtype is INT8:
        code, scale = quantised(ckpts)
        want = code.float() * scale[..., None]
    else:
        want = ckpts.to(BF16).float()
    slot, covered = store.lookup("a", 70)
    assert covered == 64
    n = [32, 64]                                      # the rest of "a" after 64 tokens; "b" anew
    part = [torch.cat([t[64:96], t[96:160]]).contiguous() for t in args[:5]]
    cu = torch.tensor([0, 32, 96], dtype=torch.int32, device="cuda")
    out, final, init = resume_prefill(store, [slot, None], *part, cu, n)
    assert torch.equal(init[0], want[1]) and bool((init[1] == 0).all())
    ref, ref_final, _ = kda.prefill(*part, cu, torch.stack([want[1], torch.zeros_like(want[1])]), lengths=n)
    assert torch.equal(out, ref) and torch.equal(final, ref_final)
    with pytest.raises(ValueError):
        CheckpointStore(8, 2, device="cuda", dtype=torch.float16)
