"""What a decoder layer does around its projections and its attention, at the sizes it meets, for timing and comparison.

Three operators:

  norm    h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, as bf16 or in 8 bits with scales: int8 or E4M3 codes
          with one scale a token (the values turned by a Walsh-Hadamard transform in blocks of 128 first, where the
          projection behind it wants that), or E4M3 codes with one scale for each 128 columns;
  rope    queries and keys turned by their positions: pairs of neighbours or of the two halves, the whole head or its
          first part, frequencies scaled for long contexts;
  block   y = x W^T + b in E4M3 with a scale for each 128 columns of a token and each 128 x 128 block of the weight,
          x quantized on the way.

``run`` computes them from elementary torch operations in 32 bits (positions times frequencies in 64), or, where ``own``
is true, with the calls that a program makes of the library.  Both take the same state: weights laid out once, at load
time, frequencies as the library's 64-bit fractions of a turn.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
EPS = 1e-6


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # before the MLP of a single-token step: latency counts
        dict(name="norm_1x5120_bf16", op="norm", tokens=1, width=5120, residual=True, out="bf16", rotated=False),
        # a decode batch into a rotated int8 projection
        dict(name="norm_61x4096_int8_rot", op="norm", tokens=61, width=4096, residual=True, out="int8", rotated=True),
        # an odd prompt, the first norm of a layer, into an E4M3 projection with one scale a token
        dict(name="norm_2270x5120_fp8", op="norm", tokens=2270, width=5120, residual=False, out="fp8", rotated=False),
        # eight records of 1,502 tokens into a block-scaled projection
        dict(name="norm_12016x5120_block", op="norm", tokens=12016, width=5120, residual=True, out="block", rotated=False),
        # one token of a short sequence: latency counts
        dict(name="rope_1x1of298", op="rope", seqs=1, tokens=1, longest=298, q_heads=16, kv_heads=16, dim=64, rotary=64,
             pairs="halves", scaling="none", factor=1),
        # a decode batch of long sequences, half of the head turned, neighbours in pairs
        dict(name="rope_32x1of131072", op="rope", seqs=32, tokens=1, longest=131072, q_heads=40, kv_heads=8, dim=128, rotary=64,
             pairs="neighbours", scaling="yarn", factor=32),
        # whole prompts
        dict(name="rope_8x1502", op="rope", seqs=8, tokens=1502, longest=1502, q_heads=40, kv_heads=8, dim=128, rotary=128,
             pairs="halves", scaling="none", factor=1),
        # the smallest projection of a decode step: latency counts
        dict(name="block_1x1024x1024", op="block", tokens=1, k=1024, n=1024, bias=True),
        # a down projection for a few sequences
        dict(name="block_5x17408x5120", op="block", tokens=5, k=17408, n=5120, bias=False),
        # gate and up in one matrix, a full decode batch
        dict(name="block_64x5120x34816", op="block", tokens=64, k=5120, n=34816, bias=False),
        # a square projection of one record
        dict(name="block_1502x4096x4096", op="block", tokens=1502, k=4096, n=4096, bias=True),
        # gate and up for a long prompt
        dict(name="block_2270x5120x34816", op="block", tokens=2270, k=5120, n=34816, bias=False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(("norm", "norm", "rope", "block", "block"))
    if op == "norm":
        out = rng.choice(("bf16", "int8", "fp8", "block"))
        rotated = out in ("int8", "fp8") and rng.random() < 0.5
        unit = 8 if out == "bf16" else BLOCK if out == "block" or rotated else 32
        width = unit * _spread(rng, 256 // unit, 17408 // unit)
        return dict(op="norm", tokens=_spread(rng, 1, min(12016, 12016 * 5120 // width)), width=width,
                    residual=rng.random() < 0.6, out=out, rotated=rotated)
    if op == "rope":
        dim, kv_heads = rng.choice((64, 128)), rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 3, 4, 5, 8))
        tokens = rng.choice((1, 1, _spread(rng, 2, 1502)))
        most = max(1, min(64, 8 * 1502 * 48 * 128 // (tokens * (heads + kv_heads) * dim)))
        scaling = rng.choice(("none", "linear", "ntk", "yarn", "wavelength"))
        return dict(op="rope", seqs=_spread(rng, 1, most), tokens=tokens, longest=tokens + _spread(rng, 1, 1 << 18),
                    q_heads=heads, kv_heads=kv_heads, dim=dim, rotary=16 * rng.randint(1, dim // 16),
                    pairs=rng.choice(("halves", "neighbours")), scaling=scaling,
                    factor=1 if scaling == "none" else rng.choice((2, 4, 8, 32)))
    while True:
        k, n = BLOCK * _spread(rng, 8, 136), 8 * _spread(rng, 128, 4352)
        if k * n <= 5120 * 34816:
            return dict(op="block", tokens=_spread(rng, 1, 2270), k=k, n=n, bias=rng.random() < 0.5)


def _lens(case):
    """How many tokens each sequence holds, the new ones counted: the first holds the longest, the others are ragged, some
    shorter than the call's tokens (those rows have no position), and of six or more sequences one is empty."""
    longest, tokens, seqs = case["longest"], case["tokens"], case["seqs"]
    rng = random.Random(longest * 7919 + tokens * 31 + seqs)
    lens = [longest] + [rng.randint(max(1, tokens - tokens // 8), longest) for _ in range(seqs - 1)]
    if seqs >= 6 and tokens == 1:
        lens[seqs // 2] = 0
    return lens


def _frequencies(case, base=10000.0, original=4096):
    """(frequencies [rotary / 2] in radians a position, what cosines and sines are multiplied by)."""
    r, s, kind = case["rotary"], float(case["factor"]), case["scaling"]
    if kind == "ntk":                                      # a larger base: the slowest frequency divided by the factor
        base = base * s ** (r / (r - 2)) if r > 2 else base
    f = [base ** (-2 * i / r) for i in range(r // 2)]
    if kind == "linear":
        return [v / s for v in f], 1.0
    if kind == "wavelength":                               # short waves as they are, long ones divided, a ramp between
        turns = [original * v / (2 * math.pi) for v in f]
        keep = [min(1.0, max(0.0, (t - 1.0) / (4.0 - 1.0))) for t in turns]
        return [v / s * (1 - g) + v * g for v, g in zip(f, keep)], 1.0
    if kind == "yarn":                                     # the ramp over the index, between 32 turns and one
        at = [r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32, 1)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        gone = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(r // 2)]
        return [v / s * g + v * (1 - g) for v, g in zip(f, gone)], 0.1 * math.log(s) + 1.0
    return f, 1.0


def work(case):
    if case["op"] == "norm":
        m, k = case["tokens"], case["width"]
        out = {"bf16": 2 * m * k, "int8": m * k + 4 * m, "fp8": m * k + 4 * m, "block": m * k + m * k // BLOCK * 4}[case["out"]]
        return {"bytes": (6 if case["residual"] else 2) * m * k + 2 * k + out,
                "flops": m * k * (4 + (7 if case["rotated"] else 0) + (1 if case["residual"] else 0))}
    if case["op"] == "rope":
        rows = case["seqs"] * case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 4 * rows * case["dim"], "flops": 3 * rows * case["rotary"]}
    m, n, k = case["tokens"], case["n"], case["k"]
    return {"bytes": n * k + 4 * -(-n // BLOCK) * (k // BLOCK) + 2 * m * (n + k) + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ inputs ----

def _normal(gen, *shape, by=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * by


def _outliers(gen, x):
    """One channel in a hundred is twenty times the others, as activations are."""
    x[:, torch.randperm(x.shape[1], generator=gen, device="cuda")[: max(1, x.shape[1] // 100)]] *= 20
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "norm":
        m, k = case["tokens"], case["width"]
        x = _outliers(gen, _normal(gen, m, k, by=0.5)).to(torch.bfloat16)
        residual = _outliers(gen, _normal(gen, m, k, by=2.0)).to(torch.bfloat16) if case["residual"] else None
        weight = (1.0 + 0.2 * _normal(gen, k)).to(torch.bfloat16)
        return dict(op="norm", x=x, residual=residual, weight=weight, out=case["out"], rotated=case["rotated"])
    if case["op"] == "rope":
        b, t, hq, hk, d = (case[f] for f in ("seqs", "tokens", "q_heads", "kv_heads", "dim"))
        qkv = _normal(gen, b, t, hq + 2 * hk, d).to(torch.bfloat16)        # as one projection leaves them
        f, amplitude = _frequencies(case)
        turns = [round(v / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for v in f]
        turns = [v - (1 << 64) if v >> 63 else v for v in turns]
        return dict(op="rope", q=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hk], lens=torch.tensor(_lens(case), dtype=torch.int32).cuda(),
                    frequencies=torch.tensor(f, dtype=torch.float64).cuda(), turns=torch.tensor(turns, dtype=torch.int64).cuda(),
                    amplitude=amplitude, pairs=case["pairs"])
    m, n, k = case["tokens"], case["n"], case["k"]
    x = _outliers(gen, _normal(gen, m, k)).to(torch.bfloat16)
    rows = -(-n // 32) * 32
    scale = torch.empty(-(-n // BLOCK), k // BLOCK, device="cuda")
    packed = torch.empty(rows * k, dtype=torch.uint8, device="cuda")
    for a in range(0, rows, 4096):                          # 128 x 128 blocks of the weight, each with its own scale
        z = min(rows, a + 4096)
        w = torch.zeros(-(-(z - a) // BLOCK) * BLOCK, k, device="cuda")
        w[: min(z, n) - a] = _normal(gen, min(z, n) - a, k, by=0.02)
        w = w.view(-1, BLOCK, k // BLOCK, BLOCK)
        s = w.abs().amax((1, 3)) / torch.full((), 448.0, device="cuda")
        scale[a // BLOCK:a // BLOCK + s.shape[0]] = s
        codes = (w / torch.where(s > 0, s, 1.0)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, k)[: z - a]
        # the packed layout: blocks of 32 rows x 64 bytes
        packed[a * k:z * k] = codes.view(-1, 32, k // 64, 64).permute(0, 2, 1, 3).reshape(-1)
    bias = _normal(gen, n, by=0.01).to(torch.bfloat16) if case["bias"] else None
    return dict(op="block", x=x, w=packed, scale=scale, n=n, bias=bias)


# --------------------------------------------------------------------- run ----

def run(state):
    if own:
        import w8a8_quantized_linear_amd as w8
        if state["op"] == "rope":
            rope = w8.Rope(state["turns"], state["pairs"] == "neighbours", state["amplitude"])
            q, k = w8.w8a8_rope(state["q"], state["k"], state["lens"], rope)
            return {"q": q, "k": k}
        if state["op"] == "block":
            return w8.w8a8_fp8_block_linear_packed(state["x"], state["w"], state["n"], state["scale"], state["bias"])
        x, weight, residual, out, rotate = state["x"], state["weight"], state["residual"], state["out"], BLOCK if state["rotated"] else 0
        if out == "bf16":
            y, h = w8.w8a8_rmsnorm(x, weight, residual, EPS)
            return y if h is None else (y, h)
        if out == "int8":
            q, s, h = w8.w8a8_rmsnorm_quantize(x, weight, residual, EPS, rot_block=rotate)
            return _answer(torch.mul(q, s[:, None], out=torch.empty_like(x)), s, h)
        if out == "fp8":
            q, s, h = w8.w8a8_rmsnorm_quantize_fp8(x, weight, residual, EPS, rot_block=rotate)
        else:
            q, s, h = w8.w8a8_rmsnorm_quantize_block(x, weight, residual, EPS)
        return _answer(q.view(torch.float8_e4m3fn), s, h)
    return {"norm": _plain_norm, "rope": _plain_rope, "block": _plain_block}[state["op"]](state)


def _answer(values, scales, h):
    """int8 codes as the bf16 values that they stand for, E4M3 codes as they are (they are values, in steps of the scale)."""
    return {"values": values, "scales": scales} | ({} if h is None else {"h": h})


def _over(x, s):
    return x / torch.where(s > 0, s, 1.0)


def _hadamard(like):
    """The normalized transform of 128 values: the sign of (i, j) is the parity of i & j."""
    i = torch.arange(BLOCK, device=like.device)
    both = i[:, None] & i
    odd = sum((both >> b) & 1 for b in range(7)) % 2
    return (1 - 2 * odd).to(like.dtype) / math.sqrt(BLOCK)


def _plain_norm(state):
    x, residual, out = state["x"].float(), state["residual"], state["out"]
    m, k = x.shape
    h = None
    if residual is not None:
        h = (x + residual.float()).to(torch.bfloat16)       # the sum that the layer hands on is what is normed
        x = h.float()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * state["weight"].float()
    if out == "bf16":
        y = y.to(torch.bfloat16)
        return y if h is None else (y, h)
    if state["rotated"]:
        y = (y.view(-1, BLOCK) @ _hadamard(y)).view(m, k)
    if out == "int8":
        s = y.abs().amax(-1) / torch.full((), 127.0, device=y.device)
        q = _over(y, s[:, None]).round().clamp(-127, 127)
        return _answer((q * s[:, None]).to(torch.bfloat16), s, h)
    y = y.view(m, 1, k) if out == "fp8" else y.view(m, -1, BLOCK)
    s = y.abs().amax(-1) / torch.full((), 448.0, device=y.device)
    q = _over(y, s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(m, k)
    return _answer(q, s[:, 0] if out == "fp8" else s, h)


def _plain_rope(state):
    f, lens = state["frequencies"], state["lens"].long()
    t = state["q"].shape[1]
    at = lens[:, None] - t + torch.arange(t, device=f.device)
    angle = (at[:, :, None].double() * f)[:, :, None]       # 64 bits: far positions
    still = (at < 0)[:, :, None, None]                      # rows before the sequence's first token
    c, s = (angle.cos() * state["amplitude"]).float(), (angle.sin() * state["amplitude"]).float()

    def turned(x):
        x, r = x.float(), 2 * f.numel()
        if state["pairs"] == "neighbours":
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat((a * c - b * s, b * c + a * s), -1)
        return torch.where(still, x, torch.cat((y, x[..., r:]), -1)).to(torch.bfloat16)
    return {"q": turned(state["q"]), "k": turned(state["k"])}


def _plain_block(state):
    x, n = state["x"].float(), state["n"]
    m, k = x.shape
    x = x.view(m, -1, BLOCK)
    s = (x.abs().amax(-1) / torch.full((), 448.0, device=x.device))[..., None]
    x = (_over(x, s).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s).view(m, k)
    w = state["w"].view(torch.float8_e4m3fn).view(-1, k // 64, 32, 64).permute(0, 2, 1, 3).reshape(-1, k)[:n].float()
    w = w.view(n, -1, BLOCK) * state["scale"].repeat_interleave(BLOCK, 0)[:n, :, None]
    y = x @ w.view(n, k).t()
    if state["bias"] is not None:
        y = y + state["bias"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    return {"norm": _exact_norm, "rope": _exact_rope, "block": _exact_block}[case["op"]](prepare(case, seed))


def _e4m3(v):
    """The nearest E4M3 value of each, ties to the even code: steps of 2^-3 of the power of two below, 2^-9 at least."""
    v = v.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_norm(state):
    h = state["x"].double()
    m, k = h.shape
    keep = None
    if state["residual"] is not None:
        keep = (h + state["residual"].double()).to(torch.bfloat16).double()
        h = keep
    norm = torch.linalg.vector_norm(h, dim=1) / math.sqrt(k)
    y = h * state["weight"].double() / torch.sqrt(norm * norm + EPS)[:, None]
    if state["out"] == "bf16":
        return y if keep is None else (y, keep)
    if state["rotated"]:                                    # butterflies
        y = y.view(-1, BLOCK).clone()
        step = 1
        while step < BLOCK:
            a, b = y.view(-1, BLOCK // (2 * step), 2, step).unbind(2)
            y = torch.stack((a + b, a - b), 2).reshape(-1, BLOCK)
            step *= 2
        y = (y / 2 ** 3.5).view(m, k)
    of = k if state["out"] != "block" else BLOCK
    g = y.view(m, k // of, of)
    s = g.abs().max(-1).values / (127 if state["out"] == "int8" else 448)
    q = g / s.clamp(min=1e-300)[..., None]
    q = q.round() * s[..., None] if state["out"] == "int8" else _e4m3(q)
    return _answer(q.reshape(m, k), s if state["out"] == "block" else s[:, 0], keep)


def _exact_rope(state):
    f, lens = state["frequencies"].cpu().numpy(), state["lens"].tolist()
    r, a = 2 * f.size, state["amplitude"]
    first, second = (np.arange(0, r, 2), np.arange(1, r, 2)) if state["pairs"] == "neighbours" else (np.arange(r // 2), np.arange(r // 2, r))
    out = {}
    for name in ("q", "k"):
        x = state[name].double().cpu().numpy()
        y = x.copy()
        for i, held in enumerate(lens):
            at = np.arange(held - x.shape[1], held)
            on = at >= 0
            turn = a * np.exp(1j * (at[on, None] * f[None, :]))
            z = (x[i, on][..., first] + 1j * x[i, on][..., second]) * turn[:, None, :]
            row = y[i, on]
            row[..., first], row[..., second] = z.real, z.imag
            y[i, on] = row
        out[name] = y
    return out


def _exact_block(state):
    """Each code by its address in the packed layout, a panel of rows at a time."""
    x, n, bias = state["x"].double(), state["n"], state["bias"]
    m, k = x.shape
    g = x.view(m, k // BLOCK, BLOCK)
    s = (g.abs().max(-1).values / 448).float().double()     # scales are held in 32 bits
    x = (_e4m3(g / s.clamp(min=1e-300)[..., None]) * s[..., None]).view(m, k)
    value = torch.tensor([(-1) ** (c >> 7) * (2.0 ** ((c >> 3 & 15) - 7) * (1 + (c & 7) / 8) if c >> 3 & 15 else 2.0 ** -9 * (c & 7))
                          for c in range(256)], dtype=torch.float64, device=x.device)
    value[[127, 255]] = torch.nan
    col = torch.arange(k, device=x.device)
    y = torch.empty(m, n, dtype=torch.float64, device=x.device)
    for a in range(0, n, 2048):
        row = torch.arange(a, min(n, a + 2048), device=x.device)[:, None]
        w = value[state["w"][(row // 32 * (k // 64) + col // 64) * 2048 + row % 32 * 64 + col % 64].long()]
        y[:, a:a + 2048] = x @ (w * state["scale"][row // BLOCK, col // BLOCK].double()).t()
    return y if bias is None else y + bias.double()
