"""The decode-side operators at the sizes they meet, for timing and comparison.

Three operators of single-token and short-chunk serving:

  w4      y = x W^T + b with 4-bit weights in groups that share a bf16 scale, for a few tokens;
  append  new keys and values into a paged cache of 8-bit codes with one fp32 scale for each
          page and head, then the sequences read back as bf16;
  attend  attention of each sequence's newest tokens over that cache, causal among themselves.

``run`` computes them from elementary torch operations in 32 bits, or, where ``own`` is true, with
the calls that a program makes of the library.  Both take the same state: weights in the packed
4-bit layout (laid out once, at load time) and a cache with its page table.
"""
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # the smallest projection of a decode step: one token, latency counts
        dict(name="w4_1x1024x1024", op="w4", tokens=1, k=1024, n=1024, group=128, bias=True),
        # gate and up in one matrix, one token: the largest weight read for one token
        dict(name="w4_1x5120x34816", op="w4", tokens=1, k=5120, n=34816, group=128, bias=False),
        # a down projection for a few sequences, small groups
        dict(name="w4_5x17408x5120", op="w4", tokens=5, k=17408, n=5120, group=32, bias=True),
        # gate and up for a full decode batch
        dict(name="w4_64x5120x34816", op="w4", tokens=64, k=5120, n=34816, group=64, bias=False),
        # one new token for each sequence of a decode batch
        dict(name="append_61x1", op="append", seqs=61, tokens=1, longest=299, q_heads=16, kv_heads=8, dim=64, page=32),
        # eight records of 1,502 tokens enter the cache behind a short prefix
        dict(name="append_8x1502", op="append", seqs=8, tokens=1502, longest=1531, q_heads=40, kv_heads=8, dim=128, page=64),
        # one short sequence: latency counts
        dict(name="attend_1x1of298", op="attend", seqs=1, tokens=1, longest=298, q_heads=16, kv_heads=16, dim=64, page=16),
        # a decode batch of ragged lengths, one slot empty
        dict(name="attend_32x1of2270", op="attend", seqs=32, tokens=1, longest=2270, q_heads=40, kv_heads=8, dim=128, page=64),
        # one token of one very long sequence
        dict(name="attend_1x1of131072", op="attend", seqs=1, tokens=1, longest=131072, q_heads=32, kv_heads=8, dim=128, page=128),
        # four proposed tokens for each of a few sequences
        dict(name="attend_7x4of1502", op="attend", seqs=7, tokens=4, longest=1502, q_heads=32, kv_heads=4, dim=64, page=32),
        # whole prompts attend to themselves
        dict(name="attend_4x1502of1502", op="attend", seqs=4, tokens=1502, longest=1502, q_heads=40, kv_heads=8, dim=128, page=64),
        # a piece of a long prompt behind what is already in the cache
        dict(name="attend_1x500of12016", op="attend", seqs=1, tokens=500, longest=12016, q_heads=32, kv_heads=8, dim=128, page=64),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(("w4", "w4", "append", "attend", "attend", "chunk"))
    if op == "w4":
        while True:
            k, n = 128 * _spread(rng, 8, 136), 8 * _spread(rng, 128, 4352)
            if k * n <= 5120 * 34816:
                return dict(op="w4", tokens=_spread(rng, 1, 64), k=k, n=n, group=rng.choice((32, 64, 128)),
                            bias=rng.random() < 0.5)
    dim, page, kv_heads = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 4, 8))
    heads = dict(q_heads=kv_heads * rng.choice((1, 3, 4, 5, 8)), kv_heads=kv_heads, dim=dim, page=page)
    if op == "append":
        tokens = _spread(rng, 1, 1502)
        return dict(op="append", seqs=_spread(rng, 1, max(1, min(61, 8 * 1502 // tokens))), tokens=tokens,
                    longest=tokens + rng.randrange(0, 300 if tokens < 100 else 30), **heads)
    if op == "attend":
        tokens = rng.choice((1, 1, 1, 2, 4, 5))
        longest = _spread(rng, 16, 65536)
        seqs = _spread(rng, 1, max(1, min(64, 131072 // longest)))
        return dict(op="attend", seqs=seqs, tokens=tokens, longest=longest, **heads)
    most = 4 * _visible([1502], 1502) * 40 * 128
    while True:
        tokens = _spread(rng, 17, 1502)
        longest = tokens + rng.choice((0, rng.randrange(0, 4000)))
        one = _visible([longest], tokens) * heads["q_heads"] * dim
        if one <= most:
            return dict(op="attend", seqs=rng.randint(1, min(4, most // one)), tokens=tokens, longest=longest, **heads)


def _lens(case):
    """How many tokens each sequence holds in the cache, the new ones counted: the first holds the
    longest, the others are ragged, and where attention has six or more one slot is empty."""
    longest, tokens, seqs = case["longest"], case["tokens"], case["seqs"]
    rng = random.Random(longest * 7919 + tokens * 31 + seqs)
    low = tokens if case["op"] == "append" else min(longest, max(tokens, longest // 4))
    lens = [longest] + [rng.randint(low, longest) for _ in range(seqs - 1)]
    if case["op"] == "attend" and seqs >= 6:
        lens[seqs // 2] = 0
    return lens


def _visible(lens, tokens):
    """(query, key) pairs of one head: query i of a sequence of L tokens sees L - tokens + 1 + i keys."""
    total = 0
    for held in lens:
        first = max(0, tokens - held)                      # queries before the sequence's start see none
        total += sum(held - tokens + 1 + i for i in range(first, tokens))
    return total


def work(case):
    if case["op"] == "w4":
        m, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": n * k // 2 + 2 * n * k // case["group"] + 2 * m * (n + k) + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    lens, row = _lens(case), case["kv_heads"] * case["dim"]
    scales = 8 * case["kv_heads"] * sum(-(-held // case["page"]) for held in lens)
    if case["op"] == "append":
        new = case["seqs"] * case["tokens"]
        held = sum(lens) - new
        # new rows read (bf16) and written (codes), held codes read, all of it read back as bf16
        return {"bytes": 2 * row * (new * 3 + held + 2 * case["seqs"] * case["longest"]) + 2 * scales,
                "flops": 2 * row * (6 * new + sum(lens))}
    q = case["seqs"] * case["tokens"] * case["q_heads"] * case["dim"]
    return {"bytes": 2 * row * sum(lens) + scales + 4 * q,
            "flops": 4 * case["dim"] * case["q_heads"] * _visible(lens, case["tokens"])}


# ------------------------------------------------------------------ inputs ----

def _normal(gen, *shape, by=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * by


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "w4":
        m, n, k, group = case["tokens"], case["n"], case["k"], case["group"]
        rows = -(-n // 16) * 16
        x = _normal(gen, m, k)
        x[:, torch.randperm(k, generator=gen, device="cuda")[: k // 100]] *= 20      # outlier channels
        codes = torch.full((rows, k), 8, dtype=torch.uint8, device="cuda")
        for a in range(0, n, 4096):
            b = min(n, a + 4096)
            codes[a:b] = (_normal(gen, b - a, k, by=2.6).round_().clamp_(-7, 7) + 8).to(torch.uint8)
        scale = torch.zeros(rows, k // group, dtype=torch.bfloat16, device="cuda")
        scale[:n] = (0.006 + 0.005 * torch.rand(n, k // group, generator=gen, device="cuda")).to(torch.bfloat16)
        # the packed layout: blocks of 16 rows and 128 columns; 16 bytes for each (quarter h, row r),
        # four words of 8 nibbles, the even elements in a word's low half, the odd ones in its high half
        e = codes.view(rows // 16, 16, k // 128, 4, 4, 8).permute(0, 2, 4, 1, 3, 5)
        e = e[..., [0, 4, 1, 5]] | (e[..., [2, 6, 3, 7]] << 4)
        s = scale.view(rows // 16, 16, k // 128, 128 // group).permute(0, 2, 3, 1)
        bias = _normal(gen, n, by=0.01).to(torch.bfloat16) if case["bias"] else None
        return dict(op="w4", x=x.to(torch.bfloat16), w=e.reshape(-1).contiguous(), s=s.reshape(-1).contiguous(), n=n,
                    group=group, bias=bias)
    b, t, hq, hk, d, page = (case[f] for f in ("seqs", "tokens", "q_heads", "kv_heads", "dim", "page"))
    lens = _lens(case)
    width = -(-case["longest"] // page)
    used = [-(-held // page) for held in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).cpu()
    table, at = torch.full((b, width), -1, dtype=torch.int32), 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    codes, scale = [], []
    for _ in range(2):
        codes.append(torch.empty(pages, hk, page, d, dtype=torch.int8, device="cuda"))
        for a in range(0, pages, 1024):
            z = min(pages, a + 1024)
            codes[-1][a:z] = _normal(gen, z - a, hk, page, d, by=36).round_().clamp_(-127, 127).to(torch.int8)
        scale.append(0.02 + 0.015 * torch.rand(pages, hk, generator=gen, device="cuda"))
    # queries, keys and values of the new tokens as one projection leaves them
    qkv = _normal(gen, b, t, hq + 2 * hk, d)
    qkv[:, :, :hq] *= 2
    qkv = qkv.to(torch.bfloat16)
    return dict(op=case["op"], q=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hk], v=qkv[:, :, hq + hk:], k_codes=codes[0], v_codes=codes[1],
                k_scale=scale[0], v_scale=scale[1], table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                longest=case["longest"])


# --------------------------------------------------------------------- run ----

def run(state):
    if own:
        import w8a8_quantized_linear_amd as w8
        if state["op"] == "w4":
            return w8.w8a8_w4_linear(state["x"], state["w"], state["s"], state["n"], state["group"], state["bias"])
        cache = w8.KVCache(state["k_codes"], state["v_codes"], state["k_scale"], state["v_scale"])
        if state["op"] == "attend":
            return w8.w8a8_kv_attention(state["q"], cache, state["table"], state["lens"])
        w8.w8a8_kv_append(state["k"], state["v"], cache, state["table"], state["lens"])
        k, v = w8.w8a8_kv_read(cache, state["table"], state["lens"], state["longest"])
        return {"k": k, "v": v, "k_scale": state["k_scale"], "v_scale": state["v_scale"]}
    if state["op"] == "w4":
        return _plain_w4(state)
    if state["op"] == "attend":
        return _plain_attend(state)
    return {"k": _plain_append(state, "k"), "v": _plain_append(state, "v"), "k_scale": state["k_scale"],
            "v_scale": state["v_scale"]}


def _plain_w4(state):
    x, n, group = state["x"], state["n"], state["group"]
    k = x.shape[1]
    e = state["w"].view(-1, k // 128, 4, 16, 4, 4)
    e = torch.cat((e & 15, e >> 4), -1)[..., [0, 2, 4, 6, 1, 3, 5, 7]]     # read as elements 0 4 1 5, 2 6 3 7
    codes = e.permute(0, 3, 1, 4, 2, 5).reshape(-1, k)[:n].float() - 8
    scale = state["s"].view(-1, k // 128, 128 // group, 16).permute(0, 3, 1, 2).reshape(-1, k // group)[:n].float()
    w = (codes.view(n, -1, group) * scale[:, :, None]).view(n, k)
    y = x.float() @ w.t()
    if state["bias"] is not None:
        y = y + state["bias"].float()
    return y.to(torch.bfloat16)


def _gathered(state, which):
    """The sequences' keys or values as the codes stand for them: fp32 [seqs, kv_heads, width * page, dim]."""
    codes, scale, table = state[which + "_codes"], state[which + "_scale"], state["table"].clamp(min=0).long()
    x = codes[table].float() * scale[table][:, :, :, None, None]
    b, w, h, p, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, w * p, d)


def _plain_attend(state):
    q, lens = state["q"].float(), state["lens"].long()
    b, t, hq, d = q.shape
    k, v = _gathered(state, "k"), _gathered(state, "v")
    h, n = k.shape[1], k.shape[2]
    q = q.view(b, t, h, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, h, t * (hq // h), d)
    s = (q @ k.transpose(2, 3).contiguous()) * d ** -0.5
    last = lens[:, None] - t + torch.arange(t, device=q.device)           # the last key each query sees
    seen = torch.arange(n, device=q.device) <= last[:, :, None]            # [seqs, tokens, keys]
    seen = seen[:, None, :, None].expand(b, h, t, hq // h, n).reshape(b, h, t * (hq // h), n)
    s = s.masked_fill(~seen, -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    y = (p @ v) / torch.where(total == 0, 1.0, total)                      # a query that sees nothing gives 0
    return y.view(b, h, t, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(torch.bfloat16)


def _plain_append(state, which):
    new, lens, table = state[which].float(), state["lens"].long(), state["table"].long()
    codes, scale = state[which + "_codes"], state[which + "_scale"]
    b, t, h, d = new.shape
    page = codes.shape[2]
    touched = (t + page - 2) // page + 1
    at = lens - t                                                          # where the new tokens begin
    block = (at // page)[:, None] + torch.arange(touched, device=new.device)
    valid = block * page < lens[:, None]
    where = torch.gather(table, 1, block.clamp(max=table.shape[1] - 1))
    pos = block[:, :, None] * page + torch.arange(page, device=new.device)
    is_new = ((pos >= at[:, None, None]) & (pos < lens[:, None, None]))[:, :, None, :, None]
    is_old = (pos < at[:, None, None])[:, :, None, :, None]
    src = (pos - at[:, None, None]).clamp(0, t - 1).view(b, -1, 1, 1).expand(b, touched * page, h, d)
    x = torch.gather(new, 1, src).view(b, touched, page, h, d).transpose(2, 3) * is_new
    where = where.clamp(min=0)
    old, old_scale = codes[where], scale[where] * is_old.any(3)[..., 0]
    s = torch.maximum(old_scale, x.abs().amax((3, 4)) / torch.full_like(old_scale, 127))
    by = torch.where(s > 0, s, 1.0)
    kept = (old.float() * (old_scale / by)[..., None, None]).round()
    put = (x / by[..., None, None]).round().clamp(-127, 127)
    put = torch.where(is_new, put, torch.where(is_old, kept, old.float())).to(torch.int8)
    codes[where[valid]] = put[valid]
    scale[where[valid]] = s[valid]
    n = state["longest"]
    inside = torch.arange(n, device=new.device) < lens[:, None]
    return (_gathered(state, which)[:, :, :n].transpose(1, 2) * inside[:, :, None, None]).to(torch.bfloat16)


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    state = prepare(case, seed)
    return {"w4": _exact_w4, "append": _exact_append, "attend": _exact_attend}[case["op"]](state)


def _exact_w4(state):
    """Each weight fetched by its address in the packed layout."""
    x, n, group = state["x"].double(), state["n"], state["group"]
    m, k = x.shape
    col = torch.arange(k, device=x.device)
    j, h, st, kb = col % 8, col // 8 % 4, col // 32 % 4, col // 128
    y = torch.empty(m, n, dtype=torch.float64, device=x.device)
    for a in range(0, n, 1024):
        row = torch.arange(a, min(n, a + 1024), device=x.device)[:, None]
        byte = ((row // 16) * (k // 128) + kb) * 1024 + (16 * h + row % 16) * 16 + 4 * st + 2 * (j % 2) + j // 4
        code = (state["w"][byte].long() >> (4 * (j // 2 % 2))) % 16 - 8
        at = (((row // 16) * (k // 128) + kb) * (128 // group) + col % 128 // group) * 16 + row % 16
        y[:, a:a + 1024] = x @ (code.double() * state["s"][at].double()).t()
    return y if state["bias"] is None else y + state["bias"].double()


def _exact_attend(state):
    q, page = state["q"].double(), state["k_codes"].shape[2]
    b, t, hq, d = q.shape
    h = state["k_codes"].shape[1]
    y = torch.zeros(b, t, hq, d, dtype=torch.float64, device=q.device)
    for i, held in enumerate(state["lens"].tolist()):
        if not held:
            continue
        rows = state["table"][i, : -(-held // page)].long()
        for c in range(h):
            k, v = ((state[w + "_codes"][rows, c].double() * state[w + "_scale"][rows, c].double()[:, None, None])
                    .reshape(-1, d)[:held] for w in "kv")
            for a in range(0, t, 256):
                z = min(t, a + 256)
                for g in range(c * (hq // h), (c + 1) * (hq // h)):
                    s = q[i, a:z, g] @ k.t() / d ** 0.5
                    last = held - t + torch.arange(a, z, device=q.device)
                    s[torch.arange(held, device=q.device)[None, :] > last[:, None]] = -torch.inf
                    blind = last < 0
                    s[blind] = 0.0
                    p = torch.softmax(s, -1)
                    p[blind] = 0.0
                    y[i, a:z, g] = p @ v
    return y


def _exact_append(state):
    out = {}
    lens, table, longest = state["lens"].tolist(), state["table"].cpu().numpy(), state["longest"]
    for which in "kv":
        new = state[which].double().cpu().numpy()
        codes = state[which + "_codes"].cpu().numpy().astype(np.float64)
        scale = state[which + "_scale"].double().cpu().numpy()
        b, t, h, d = new.shape
        page = codes.shape[2]
        for i, held in enumerate(lens):
            at = held - t
            while at < held:                               # the part of one page that is new
                to, p = min(held, (at // page + 1) * page), table[i, at // page]
                x, first = new[i, at - held + t:to - held + t].transpose(1, 0, 2), at % page
                s = np.abs(x).max((1, 2)) / 127
                if first:
                    s = np.maximum(s, scale[p])
                    codes[p, :, :first] = np.rint(codes[p, :, :first] * (scale[p] / s)[:, None, None])
                codes[p, :, first:first + to - at] = np.rint(x / np.where(s > 0, s, 1)[:, None, None])
                scale[p] = s
                at = to
        back = np.zeros((b, longest, h, d))
        for i, held in enumerate(lens):
            rows = table[i, : -(-held // page)]
            x = (codes[rows] * scale[rows][:, :, None, None]).transpose(0, 2, 1, 3).reshape(-1, h, d)
            back[i, :held] = x[:held]
        out[which], out[which + "_scale"] = back, scale
    return out
