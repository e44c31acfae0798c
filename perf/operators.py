"""The block-scaled FP8 products and the rotary positions, case by case: inputs, plain forms in
elementary torch operations, the library's calls, and the same results in 64 bits.

Three operators of a diffusion transformer that keeps some projections in 8 bits:

  linear   Y = GELU?(q(X) q(W) + b), q() the 8-bit format of the library: e4m3 codes under one
           power-of-two scale per row (of X) or column (of W) and 128 elements along K
  experts  the same product by expert: rows [offsets[e], offsets[e+1]) of X meet weight e; rows
           behind the last offset of Y stay as they were
  rope     rotary positions over several axes (time, height, width) of the query and key heads,
           after an optional RMS norm of each head

`own` chooses between the plain forms and the library's layers.
"""
import math

import torch

own = False

BLOCK = 128          # elements along K under one scale
E4M3_MAX = 448.0
EPILOGUES = {"none": 0, "gelu": 1, "gelu_tanh": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the timestep embedding's first projection, one row: a call that is all latency
        dict(name="linear 1x256 2560 gelu", op="linear", m=1, k=256, n=2560, epilogue="gelu", bias=True),
        # the six modulation vectors of a block for two conditioning rows: one pass over the weight
        dict(name="linear 2x2560 15360", op="linear", m=2, k=2560, n=15360, epilogue="none", bias=True),
        # a short prompt's tokens into the model's width: an odd row count, still bound by the weight
        dict(name="linear 77x4096 2560 tanh", op="linear", m=77, k=4096, n=2560, epilogue="gelu_tanh", bias=True),
        # query, key and value of the text stream
        dict(name="linear 512x2560 7680", op="linear", m=512, k=2560, n=7680, epilogue="none", bias=True),
        # the MLP's first product over image and text tokens together
        dict(name="linear 4608x2560 10240 gelu", op="linear", m=4608, k=2560, n=10240, epilogue="gelu", bias=True),
        # two images through a wide MLP: the largest product
        dict(name="linear 9216x4096 16384", op="linear", m=9216, k=4096, n=16384, epilogue="none", bias=False),
        # eight tokens of two experts each: most experts have no row, the others one or two
        dict(name="experts 16 of 32", op="experts", t=16, e=32, k=1024, n=2816, skew=0.5, empty=4, tail=0,
             epilogue="gelu_tanh", bias=False),
        # many small experts, ragged: a few rows each, a width that ends inside a tile
        dict(name="experts 1001 of 64", op="experts", t=1001, e=64, k=2048, n=1416, skew=0.7, empty=3, tail=7,
             epilogue="gelu", bias=True),
        # an image's tokens, two experts each, the experts unevenly liked
        dict(name="experts 9216 of 8", op="experts", t=9216, e=8, k=2560, n=10240, skew=0.6, empty=1, tail=0,
             epilogue="gelu", bias=True),
        # a prompt's positions for grouped heads in the half-split pairing, turned back
        dict(name="rope 77 half", op="rope", m=77, hq=8, hk=2, d=64, axes="16,24,24", half=True, norm=False,
             inverse=True, frames=1),
        # image and text tokens: normed query and key heads out of the fused projection's output
        dict(name="rope 4608 norm", op="rope", m=4608, hq=20, hk=20, d=128, axes="16,56,56", half=False, norm=True,
             inverse=False, frames=1),
        # a video's tokens, 21 latent frames
        dict(name="rope 32761 video", op="rope", m=32761, hq=20, hk=20, d=128, axes="44,42,42", half=False,
             norm=False, inverse=False, frames=21),
    ]


def _log_int(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "experts", "rope"])
    if op == "linear":
        return dict(op=op, m=_log_int(rng, 1, 6000), k=_log_int(rng, 256, 4096, 8), n=_log_int(rng, 256, 12288, 8),
                    epilogue=rng.choice(sorted(EPILOGUES)), bias=rng.random() < 0.7)
    if op == "experts":
        e = _log_int(rng, 2, 64)
        return dict(op=op, t=_log_int(rng, 4, 6000), e=e, k=_log_int(rng, 256, 2560, 8),
                    n=_log_int(rng, 256, 2816, 8), skew=round(rng.uniform(0.0, 1.2), 3), empty=rng.randrange(0, e // 2 + 1),
                    tail=rng.choice([0, 0, 1, 3]), epilogue=rng.choice(sorted(EPILOGUES)), bias=rng.random() < 0.7)
    d, axes = rng.choice([(64, "16,24,24"), (64, "32,32"), (128, "16,56,56"), (128, "44,42,42"), (256, "64,96,96"),
                          (80, "80")])
    hq = rng.choice([3, 8, 12, 16, 20])
    norm = rng.random() < 0.5
    return dict(op=op, m=_log_int(rng, 1, 12000), hq=hq, hk=rng.choice([1, hq]), d=d, axes=axes,
                half=rng.random() < 0.4, norm=norm, inverse=not norm and rng.random() < 0.3,
                frames=rng.choice([1, 5, 13]))


def _expert_counts(case):
    """Rows of each expert, most liked first: shares (rank)^-skew of the rows before the tail, the last
    `empty` experts without any."""
    live, rows = case["e"] - case["empty"], case["t"] - case["tail"]
    p = [(i + 1.0) ** -case["skew"] for i in range(live)]
    edges = [0] + [int(round(rows * sum(p[:i + 1]) / sum(p))) for i in range(live)]
    return [b - a for a, b in zip(edges, edges[1:])] + [0] * case["empty"]


def work(case):
    if case["op"] == "linear":
        m, k, n, e, rows = case["m"], case["k"], case["n"], 1, case["m"]
    elif case["op"] == "experts":
        counts = _expert_counts(case)
        m, k, n, e, rows = case["t"], case["k"], case["n"], sum(c > 0 for c in counts), sum(counts)
    else:
        elems = case["m"] * (case["hq"] + case["hk"]) * case["d"]
        axes = len(case["axes"].split(","))
        return {"bytes": 4 * elems + 4 * case["m"] * axes, "flops": elems * (3 + (4 if case["norm"] else 0))}
    blocks = -(-k // BLOCK)
    return {"bytes": 2 * rows * k + e * n * (k + blocks) + 2 * rows * n + (2 * n * e if case["bias"] else 0),
            "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs

def _activations(g, rows, k):
    """Normal activations with one channel in a hundred twenty times as large."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    loud = torch.rand(k, generator=g, device="cuda") < 0.01
    return torch.where(loud, x * 20, x).to(torch.bfloat16)


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        m, hq, hk, d = case["m"], case["hq"], case["hk"], case["d"]
        # query, key and value heads side by side, as a fused projection leaves them
        qkv = torch.randn(m, (hq + 2 * hk) * d, generator=g, device="cuda").to(torch.bfloat16)
        q = qkv[:, :hq * d].unflatten(1, (hq, d))
        k = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        axes = [int(a) for a in case["axes"].split(",")]
        # token -> (frame, row, column) of a grid that starts at a place of its own
        side = max(1, math.isqrt(max(1, m // case["frames"])))
        t = torch.arange(m, device="cuda")
        start = torch.randint(0, 1000, (3,), generator=g, device="cuda")
        grid = torch.stack([t // (side * side), t // side % side, t % side], 1) + start
        s = dict(q=q, k=k, pos=grid[:, 3 - len(axes):].to(torch.int32).contiguous(), axes=axes)
        if case["norm"]:
            s["q_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        return s
    k, n = case["k"], case["n"]
    lead = (case["e"],) if case["op"] == "experts" else ()
    s = dict(x=_activations(g, case["t"] if lead else case["m"], k))
    s["w"] = (0.02 * torch.randn(*lead, k, n, generator=g, device="cuda")).to(torch.bfloat16)
    s["bias"] = (0.1 * torch.randn(*lead, n, generator=g, device="cuda")).to(torch.bfloat16) if case["bias"] else None
    if lead:
        counts = torch.tensor(_expert_counts(case), device="cuda")
        counts = counts[torch.randperm(case["e"], generator=g, device="cuda")]
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["rows"], s["most"] = sum(_expert_counts(case)), max(_expert_counts(case))
        s["y"] = torch.zeros(case["t"], n, dtype=torch.bfloat16, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "rope":
        if own:
            from bit_w4a4_diffusion_smooth_b200 import layer
            s["rope"] = layer.RotaryND(s["axes"], interleaved=not case["half"], q_norm=s.get("q_norm"),
                                       k_norm=s.get("k_norm"))
        else:
            # per pair of a head: its axis and its frequency theta^(-2i/d_a)
            pairs = [(a, 10000.0 ** (-2.0 * i / d)) for a, d in enumerate(s["axes"]) for i in range(d // 2)]
            s["axis"] = torch.tensor([p[0] for p in pairs], device="cuda")
            s["freq"] = torch.tensor([p[1] for p in pairs], dtype=torch.float64, device="cuda")
        return s
    w = s.pop("w")
    if own:
        from bit_w4a4_diffusion_smooth_b200 import layer
        make = layer.FP8Experts if case["op"] == "experts" else layer.FP8Linear
        s["layer"] = make(w, s.pop("bias"), epilogue=EPILOGUES[case["epilogue"]])
    else:
        s["codes"], s["scales"] = _quantize(w.transpose(-1, -2))
    return s


# ------------------------------------------------------------------ plain forms

def _quantize(x):
    """x [..., K] -> e4m3 codes [..., B, 128] (zero past K) and scales [..., B, 1]: per block the smallest power
    of two under which the largest magnitude is at most 448."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))
    mantissa, exponent = torch.frexp(x.abs().amax(-1, keepdim=True))
    scale = torch.ldexp(torch.ones_like(mantissa), exponent - 9 + (mantissa > E4M3_MAX / 512).int())
    return (x / scale).to(torch.float8_e4m3fn), scale


def _values(codes, scales):
    return (codes.float() * scales).flatten(-2)


def _gelu(y, kind):
    if kind == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _plain_linear(s):
    y = _values(*_quantize(s["x"])) @ _values(s["codes"], s["scales"]).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return _gelu(y, s["case"]["epilogue"]).to(torch.bfloat16)


def _plain_experts(s):
    x = _values(*_quantize(s["x"][:s["rows"]]))
    row = torch.arange(s["rows"], device=x.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    slot = row - s["offsets"].long()[expert]
    padded = x.new_zeros(s["case"]["e"], s["most"], x.shape[1])
    padded[expert, slot] = x
    y = torch.bmm(padded, _values(s["codes"], s["scales"]).transpose(1, 2))[expert, slot]
    if s["bias"] is not None:
        y = y + s["bias"].float()[expert]
    s["y"][:s["rows"]] = _gelu(y, s["case"]["epilogue"]).to(torch.bfloat16)
    return s["y"]


def _turn(x, cos, sin, half):
    """The pairs of each head turned by their angles; cos, sin [M, 1, D / 2]."""
    a, b = (x.chunk(2, -1) if half else (x[..., 0::2], x[..., 1::2]))
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def _plain_rope(s):
    case = s["case"]
    angle = (s["pos"].double()[:, s["axis"]] * s["freq"]).unsqueeze(1)
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = s["q"].float(), s["k"].float()
    if case["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_norm"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_norm"].float()
    if case["inverse"]:
        sin = -sin
    return [_turn(t, cos, sin, case["half"]).to(torch.bfloat16) for t in (q, k)]


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "linear":
            return s["layer"](s["x"])
        if op == "experts":
            return s["layer"](s["x"], s["offsets"], s["y"])
        return list(s["rope"](s["q"], s["k"], s["pos"], inverse=s["case"]["inverse"]))
    return {"linear": _plain_linear, "experts": _plain_experts, "rope": _plain_rope}[op](s)


# ------------------------------------------------------------------ 64 bits

def _nearest8(x):
    """The 8-bit values of x [R, K] in float64: per row and block of 128 a scale 2^ceil(log2(amax / 448)), each
    element the nearest multiple of an eighth of its own power of two (of 2^-9 below 2^-6), ties to even."""
    out = x.double().clone()
    for k0 in range(0, x.shape[1], BLOCK):
        v = out[:, k0:k0 + BLOCK]
        top = v.abs().max(1, keepdim=True).values
        scale = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX))), torch.ones_like(top))
        u = v / scale
        power = torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6)))
        step = torch.exp2(power - 3)
        out[:, k0:k0 + BLOCK] = torch.round(u / step) * step * scale
    return out


def _act64(y, kind):
    if kind == "gelu":
        return y * torch.special.ndtr(y)
    if kind == "gelu_tanh":
        z = 2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
        return y * torch.sigmoid(z)
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        freq = []
        for a, d in enumerate(s["axes"]):
            i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
            freq.append(s["pos"][:, a:a + 1].double() * torch.exp(-2 * i / d * math.log(10000.0)))
        angle = torch.cat(freq, 1) * (-1.0 if case["inverse"] else 1.0)
        turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
        out = []
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt() * s[name + "_norm"].double()
            n = case["d"] // 2
            pairs = (x.unflatten(-1, (2, n)).transpose(-1, -2) if case["half"] else x.unflatten(-1, (n, 2))).contiguous()
            y = torch.view_as_real(torch.view_as_complex(pairs) * turn)
            out.append((y.transpose(-1, -2) if case["half"] else y).flatten(-2))
        return out
    x = _nearest8(s["x"])
    if case["op"] == "linear":
        y = x @ _nearest8(s["w"].t()).t()
        return _act64(y if s["bias"] is None else y + s["bias"].double(), case["epilogue"])
    out = s["y"].double()
    ends = s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if b > a:
            y = x[a:b] @ _nearest8(s["w"][e].t()).t()
            out[a:b] = _act64(y if s["bias"] is None else y + s["bias"][e].double(), case["epilogue"])
    return out
