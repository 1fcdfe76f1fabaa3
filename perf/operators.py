"""The operators around the block-scaled linear layers of a diffusion
transformer, as they are timed and checked: each in its plain form
(elementary torch operations) and as a user of the library calls it.

* ``mxfp4``: a linear layer with MXFP4 operands (E2M1 elements, one
  power-of-two scale per 32 of them): the activations quantized at run time,
  times a weight that was quantized once.
* ``rope``: rotary positions with several axes (time, height, width) on the
  query and key heads, optionally after the RMS norm of each head.
* ``attention``: attention of a sequence over states of another length, each
  batch entry with its own number of valid states.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one conditioning vector through a hidden x hidden projection: the smallest call
        {"name": "mxfp4_vector", "op": "mxfp4", "M": 1, "K": 3072, "N": 3072, "bias": True},
        # the text stream of an image model (512 tokens) through the same projection
        {"name": "mxfp4_text", "op": "mxfp4", "M": 512, "K": 3072, "N": 3072, "bias": True},
        # a ragged patch count; K ends in the middle of a scale word, N in the middle of a tile
        {"name": "mxfp4_ragged", "op": "mxfp4", "M": 777, "K": 1088, "N": 2056, "bias": False},
        # the MLP-up layer over image and text tokens
        {"name": "mxfp4_mlp_up", "op": "mxfp4", "M": 4608, "K": 3072, "N": 12288, "bias": True},
        # one new token per request against a grouped-query cache: latency
        {"name": "rope_token", "op": "rope", "B": 4, "L": 1, "Hq": 32, "Hk": 8, "D": 64, "axes": "16,24,24",
         "type": "bf16", "interleaved": False, "shared": True, "norm": False, "far": 100000, "fractional": False},
        # a joint image-and-text block: the Q and K columns of the fused QKV projection, with the heads' norms
        {"name": "rope_joint", "op": "rope", "B": 1, "L": 4608, "Hq": 24, "Hk": 24, "D": 128, "axes": "16,56,56",
         "type": "bf16", "interleaved": True, "shared": False, "norm": True, "far": 64, "fractional": False},
        # a video (17 x 26 x 35 patches, two guidance branches), time on a scaled, fractional axis
        {"name": "rope_video", "op": "rope", "B": 2, "L": 15470, "Hq": 12, "Hk": 12, "D": 128, "axes": "44,42,42",
         "type": "fp16", "interleaved": False, "shared": False, "norm": False, "far": 2000, "fractional": True},
        # short captions with an empty one (an unconditional branch), heads narrower than a tile
        {"name": "attention_caption", "op": "attention", "B": 3, "Lq": 333, "Lk": 77, "Hq": 16, "Hk": 16, "D": 72,
         "type": "fp16", "empty": True},
        # one query token per request over long encoder states, grouped heads
        {"name": "attention_query", "op": "attention", "B": 4, "Lq": 1, "Lk": 16384, "Hq": 32, "Hk": 8, "D": 128,
         "type": "bf16", "empty": False},
        # image tokens over padded text states
        {"name": "attention_text", "op": "attention", "B": 2, "Lq": 4096, "Lk": 512, "Hq": 24, "Hk": 24, "D": 128,
         "type": "bf16", "empty": False},
        # joint attention over image and text tokens: the largest
        {"name": "attention_joint", "op": "attention", "B": 1, "Lq": 4608, "Lk": 4608, "Hq": 24, "Hk": 24, "D": 128,
         "type": "bf16", "empty": False},
    ]


def spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["mxfp4", "rope", "attention"])
    if op == "mxfp4":
        return {"op": op, "M": spread(rng, 1, 4608), "K": 64 * spread(rng, 1, 64), "N": 8 * spread(rng, 1, 1024),
                "bias": rng.random() < 0.5}
    if op == "rope":
        D = rng.choice([48, 64, 72, 80, 96, 128])
        axes = rng.choice([[D // 2, D // 2], [D - 2 * (D // 3 // 2 * 2), D // 3 // 2 * 2, D // 3 // 2 * 2],
                           [D // 16 * 2, D // 16 * 2, D // 4]])
        Hk = spread(rng, 1, 24)
        B = rng.choice([1, 1, 2, 3])
        return {"op": op, "B": B, "L": spread(rng, 1, 15470 // B), "Hq": Hk * rng.choice([1, 1, 2, 4]), "Hk": Hk,
                "D": D, "axes": ",".join(str(a) for a in rotated(axes)), "type": rng.choice(["bf16", "fp16"]),
                "interleaved": rng.random() < 0.5, "shared": rng.random() < 0.3, "norm": rng.random() < 0.5,
                "far": spread(rng, 16, 1000000), "fractional": rng.random() < 0.3}
    D = 8 * rng.randint(5, 16)
    group = rng.choice([1, 1, 1, 2, 3, 4, 8])
    B = rng.choice([1, 1, 2, 3, 4])
    Hk = spread(rng, 1, max(1, 24 // group))
    Lk = spread(rng, 1, 16384)
    most = 24 * 4608 * 4608 // (B * Hk * group * Lk)  # scores of the largest listed case
    return {"op": op, "B": B, "Lq": spread(rng, 1, max(1, min(4608, most))), "Lk": Lk, "Hq": Hk * group, "Hk": Hk,
            "D": D, "type": rng.choice(["bf16", "fp16"]), "empty": rng.random() < 0.2}


def rotated(axes):
    """The axes with the first one cut so that a multiple of 8 elements is rotated (the rest pass through)."""
    return [axes[0] - sum(axes) % 8] + axes[1:]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def valid_states(case):
    """Valid states of each batch entry: the first has all, the others fewer; the last none where one is empty."""
    B, Lk = case["B"], case["Lk"]
    lens = [max(1, Lk - b * Lk // (2 * B) - (b * 7) % 5) for b in range(B)]
    if case["empty"]:
        lens[-1] = 0
    return lens


def pack_mxfp4(w):
    """``w`` [rows, K] as a checkpoint holds it: E2M1 codes, two to a byte, and
    E8M0 scales in the tensor cores' layout (512-byte atoms of 128 rows x 4
    scale columns)."""
    rows, K = w.shape
    blocks = w.float().view(rows, K // 32, 32)
    amax = blocks.abs().amax(2)
    exponent = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)  # floor(log2) - 2
    scaled = torch.ldexp(blocks, -exponent[:, :, None])
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    size = scaled.abs()
    up, down = torch.bucketize(size, borders, right=True), torch.bucketize(size, borders)
    code = torch.where(up % 2 == 0, up, down)  # a border goes to the even code of its two
    code = (code | torch.signbit(scaled).long() << 3).view(rows, K).to(torch.uint8)
    codes = code[:, 0::2] | code[:, 1::2] << 4
    blocks_m, atoms = (rows + 127) // 128, (K // 32 + 3) // 4
    sf = torch.zeros(blocks_m * 128, atoms * 4, dtype=torch.uint8, device=w.device)
    sf[:rows, :K // 32] = (exponent + 127).to(torch.uint8)
    sf = sf.view(blocks_m, 4, 32, atoms, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes.contiguous(), sf


def inputs(case, seed):
    g = generator(seed)
    if case["op"] == "mxfp4":
        M, K, N = case["M"], case["K"], case["N"]
        x = torch.randn(M, K, generator=g, device="cuda")
        loud = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]
        x[:, loud] *= 20.0  # a hundredth of the channels are outliers, as in trained models
        w = torch.randn(N, K, generator=g, device="cuda") * 0.02
        bias = (torch.randn(N, generator=g, device="cuda") * 0.01).bfloat16() if case["bias"] else None
        return {"x": x.bfloat16(), "w": w.bfloat16(), "bias": bias}
    dtype, B, D, Hq, Hk = TYPES[case["type"]], case["B"], case["D"], case["Hq"], case["Hk"]
    if case["op"] == "rope":
        L, axes = case["L"], [int(a) for a in case["axes"].split(",")]
        qkv = torch.randn(B, L, (Hq + 2 * Hk) * D, generator=g, device="cuda").to(dtype)
        positions = torch.randint(0, case["far"], (L, len(axes)), generator=g, device="cuda", dtype=torch.int32)
        if case["fractional"]:
            positions = positions.float() + torch.randint(0, 8, (L, len(axes)), generator=g, device="cuda") / 8
        weights = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) if case["norm"] else None
                   for _ in range(2)]
        q = qkv[:, :, :Hq * D].unflatten(2, (Hq, D))
        k = qkv[:, :, Hq * D:(Hq + Hk) * D].unflatten(2, (Hk, D))
        return {"q": q, "k": k, "positions": positions, "axes": axes, "q_weight": weights[0], "k_weight": weights[1]}
    q = torch.randn(B, case["Lq"], Hq, D, generator=g, device="cuda").to(dtype)
    kv = torch.randn(B, case["Lk"], 2, Hk, D, generator=g, device="cuda").to(dtype)  # one fused K and V projection
    lens = torch.tensor(valid_states(case), device="cuda", dtype=torch.int32)
    return {"q": q, "k": kv[:, :, 0], "v": kv[:, :, 1], "lens": lens}


def prepare(case, seed):
    state = inputs(case, seed)
    state["case"] = case
    if case["op"] == "mxfp4":
        state["codes"], state["sf"] = pack_mxfp4(state.pop("w"))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return run_own(case, state)
    if case["op"] == "mxfp4":
        return plain_mxfp4(case, state)
    if case["op"] == "rope":
        return [plain_rope(case, state["q"], state["positions"], state["axes"], state["q_weight"]),
                plain_rope(case, state["k"], state["positions"], state["axes"], state["k_weight"])]
    return plain_attention(state["q"], state["k"], state["v"], state["lens"])


def run_own(case, state):
    import nvfp4_block_scaled_12_b200 as F
    if case["op"] == "mxfp4":
        weight = F.MXFP4Tensor(state["codes"], state["sf"], case["N"], case["K"])
        return F.gemm_mxfp4(F.quantize_mxfp4(state["x"]), weight, bias=state["bias"])
    if case["op"] == "rope":
        return list(F.rope(state["q"], state["positions"], state["axes"], k=state["k"], theta=10000.0,
                           q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS,
                           interleaved=case["interleaved"], shared=case["shared"]))
    return F.cross_attention(state["q"], state["k"], state["v"], kv_lens=state["lens"])


def plain_mxfp4(case, state):
    M, K, N = case["M"], case["K"], case["N"]
    # the activations: block exponent floor(log2 max) - 2, elements to the nearest of 0, 1/2, .. 6, ties to even
    blocks = state["x"].float().view(M, K // 32, 32)
    amax = blocks.abs().amax(2, keepdim=True)
    exponent = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    scaled = torch.ldexp(blocks, -exponent)
    step = torch.where(scaled.abs() < 2, 0.5, torch.where(scaled.abs() < 4, 1.0, 2.0))
    a = torch.ldexp((torch.round(scaled / step) * step).clamp(-6, 6), exponent).view(M, K)
    # the weight, from its codes and scales
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    codes = torch.stack([state["codes"] & 15, state["codes"] >> 4], 2).view(N, K // 32, 32)
    blocks_m, atoms = (N + 127) // 128, (K // 32 + 3) // 4
    sf = state["sf"].view(blocks_m, atoms, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(blocks_m * 128, atoms * 4)
    b = torch.ldexp(values[codes.long()], sf[:N, :K // 32, None].int() - 127).view(N, K)
    y = a @ b.T
    return (y if state["bias"] is None else y + state["bias"].float()).bfloat16()


def angles(case, positions, axes):
    """Angle of every position and pair, [L, pairs], in 64 bits (far positions lose theirs in 32)."""
    total = sum(axes)
    step = torch.cat([torch.arange(0, a, 2, device="cuda", dtype=torch.float64) / a for a in axes])
    if case["shared"]:
        step = torch.arange(0, total, 2, device="cuda", dtype=torch.float64) / total
    axis = torch.repeat_interleave(torch.tensor([a // 2 for a in axes], device="cuda"), output_size=total // 2)
    return positions.double()[:, axis] * 10000.0 ** -step


def plain_rope(case, x, positions, axes, weight):
    y, total = x.float(), sum(axes)
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = angles(case, positions, axes)[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()
    rotary, rest = y[..., :total], y[..., total:]
    if case["interleaved"]:
        a, b = rotary[..., 0::2], rotary[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = rotary[..., :total // 2], rotary[..., total // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1).to(x.dtype)


def plain_attention(q, k, v, lens):
    B, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1], k.shape[2]
    valid = torch.arange(Lk, device="cuda") < lens[:, None]
    qh = q.float().view(B, Lq, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    kh, vh = k.float().permute(0, 2, 3, 1), (v.float() * valid[:, :, None, None]).permute(0, 2, 1, 3)
    s = (qh @ kh) * D ** -0.5
    s = s.masked_fill(~valid[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38))
    o = (p @ vh) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(B, Hk, Hq // Hk, Lq, D).permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, D).to(q.dtype)


# ---------------------------------------------------------------------------
# cost and definition
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "mxfp4":
        M, K, N = case["M"], case["K"], case["N"]
        # activations in 16 bits, the weight's codes and scales, the result
        return {"bytes": 2 * M * K + N * K / 2 + N * K / 32 + 2 * M * N, "flops": 2 * M * N * K}
    B, D, Hq, Hk = case["B"], case["D"], case["Hq"], case["Hk"]
    if case["op"] == "rope":
        n, axes = B * case["L"] * (Hq + Hk) * D, case["axes"].split(",")
        return {"bytes": 4 * n + 4 * case["L"] * len(axes), "flops": (7 if case["norm"] else 3) * n}
    states = sum(valid_states(case))
    return {"bytes": 4 * B * case["Lq"] * Hq * D + 4 * states * Hk * D, "flops": 4 * case["Lq"] * states * Hq * D}


def exact(case, seed):
    data = inputs(case, seed)
    if case["op"] == "mxfp4":
        a, b = (exact_mxfp4(data[n]) for n in "xw")
        y = torch.einsum("mk,nk->mn", a, b)
        return y if data["bias"] is None else y + data["bias"].double()
    if case["op"] == "rope":
        return [exact_rope(case, data[n], data["positions"], data["axes"], data[n + "_weight"]) for n in "qk"]
    return exact_attention(data["q"], data["k"], data["v"], data["lens"])


def exact_mxfp4(x):
    """The values that MXFP4 keeps of ``x``: the nearest grid point by distance, the even one of two as near."""
    blocks = x.double().unflatten(1, (-1, 32))
    amax = blocks.abs().amax(2, keepdim=True)
    power = torch.floor(torch.log2(amax.clamp(min=1e-300)))
    power = power + (2.0 ** (power + 1) <= amax).double() - (2.0 ** power > amax).double()
    scale = 2.0 ** (power - 2).clamp(-127, 127)
    size, kept = blocks.abs() / scale, torch.zeros_like(blocks)
    near = size.clone()
    for point in (1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0):  # the even codes first: a tie stays with them
        closer = (size - point).abs() < near
        if point == 6.0:
            closer |= size > 6
        kept, near = torch.where(closer, point, kept), torch.where(closer, (size - point).abs(), near)
    return (kept * blocks.sign() * scale).flatten(1)


def exact_rope(case, x, positions, axes, weight):
    y, total = x.double(), sum(axes)
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    turns, at = [], 0
    for axis, width in enumerate(axes):
        for i in range(width // 2):
            power = 2 * (at + i) / total if case["shared"] else 2 * i / width
            turns.append(positions[:, axis].double() / 10000.0 ** power)
        at += width // 2
    phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.stack(turns, 1))[:, None]
    if case["interleaved"]:
        pairs = torch.view_as_complex(y[..., :total].unflatten(-1, (-1, 2)).contiguous()) * phase
        turned = torch.view_as_real(pairs).flatten(-2)
    else:
        pairs = torch.complex(y[..., :total // 2], y[..., total // 2:total]) * phase
        turned = torch.cat([pairs.real, pairs.imag], -1)
    return torch.cat([turned, y[..., total:]], -1)


def exact_attention(q, k, v, lens):
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    group = q.shape[2] // k.shape[2]
    for b, n in enumerate(lens.tolist()):
        for h in range(k.shape[2] if n else 0):
            heads = slice(h * group, (h + 1) * group)
            s = torch.einsum("qgd,kd->gqk", q[b, :, heads].double(), k[b, :n, h].double()) / math.sqrt(q.shape[3])
            out[b, :, heads] = torch.einsum("gqk,kd->qgd", torch.softmax(s, -1), v[b, :n, h].double())
    return out
