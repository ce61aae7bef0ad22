"""Measured cases of what stands around attention: queries and keys normalised
and rotated, the same written straight into the paged 8-bit cache, and
attention of a batch whose requests share long prefixes.

``qk_norm_rope`` divides each head of q and k by its root mean square, times a
weight, and rotates it by its token's position; ``qk_norm_rope_backward`` is
its gradient. ``qk_norm_rope_append`` does the same to new tokens and stores
their keys and values in the cache of ``cache_append``. ``forward_paged_prefix``
attends over a prefix that a group of requests shares and over each request's
own tokens. A ``step`` case is the last two in a row, as one layer of a serving
step calls them.

``run`` computes plain torch forms in 32 bits where ``own`` is false, and makes
the package's calls where it is true.
"""

import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
E4M3_MAX = 448.0
EXP_MIN = -126  # exponent of the smallest scale of a cache block
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _norm(name, op, layout, B, new, Hq, Hkv, d, rot, ends=0, inter=False, norms="qk", dtype="bf16", theta=1e4, seed=1):
    return dict(name=name, op=op, layout=layout, B=B, new_lo=new[0], new_hi=new[1], ends=ends, Hq=Hq, Hkv=Hkv, d=d,
                rot=rot, inter=inter, norms=norms, dtype=dtype, theta=theta, sizes=seed)


def _cached(name, op, B, lens, new, Hq, Hkv, d, bs, groups=1, prefix=(0, 0), rot=None, theta=1e6, causal=True, seed=1):
    return dict(name=name, op=op, B=B, len_lo=lens[0], len_hi=lens[1], new_lo=new[0], new_hi=new[1], Hq=Hq, Hkv=Hkv,
                d=d, bs=bs, groups=groups, pre_lo=prefix[0], pre_hi=prefix[1], rot=d if rot is None else rot,
                inter=False, theta=theta, causal=causal, sizes=seed)


def listed():
    return [
        # one token for each of 16 requests, far positions: nothing but latency
        _norm("norm_decode", "norm", "serve", 16, (1, 1), 32, 8, 128, 128, ends=131072, theta=1e6),
        # a training step's packed projection to the [B, H, N, d] tensors that attention reads: [2, 16, 16384, 128]
        _norm("norm_train16k", "norm", "dense", 2, (16384, 16384), 16, 16, 128, 128),
        # the gradient for eight packed sequences, d = 64, half of each head rotated in neighbouring pairs
        _norm("grad_packed64", "grad", "packed", 8, (256, 512), 16, 16, 64, 32, inter=True),
        # the gradient of norm_train16k, back into the projection's gradient
        _norm("grad_train16k", "grad", "dense", 2, (16384, 16384), 16, 16, 128, 128),
        # one new token for each of 128 requests into the cache, grouped heads
        _cached("append_decode", "append", 128, (1, 8192), (1, 1), 32, 8, 128, 64),
        # whole prompts into the cache, every head with keys of its own
        _cached("append_prompts", "append", 4, (0, 0), (512, 8191), 32, 32, 128, 64),
        # a few requests behind one short instruction: the smallest call that attends
        _cached("prefix_short", "prefix", 4, (1, 40), (1, 1), 32, 8, 128, 64, prefix=(1000, 1000)),
        # 64 conversations that start with the same documents
        _cached("prefix_decode", "prefix", 64, (1, 4096), (1, 1), 32, 8, 128, 64, prefix=(32768, 32768)),
        # 16 answers sampled from one very long document
        _cached("prefix_long", "prefix", 16, (1, 512), (1, 1), 32, 8, 128, 64, prefix=(262001, 262001)),
        # six groups with prefixes of very different lengths, several drafted tokens each, d = 64
        _cached("prefix_groups64", "prefix", 48, (1, 600), (2, 5), 24, 6, 64, 32, groups=6, prefix=(500, 12000)),
        # questions of a prompt's length about one document, d = 64
        _cached("prefix_prompts64", "prefix", 8, (0, 0), (256, 1999), 16, 16, 64, 64, prefix=(8192, 8192)),
        # one layer of a serving step: norm, rotation and append, then attention
        _cached("step_prefix", "step", 32, (1, 1024), (1, 1), 32, 8, 128, 64, prefix=(4096, 4096)),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "grad", "grad", "append", "append", "prefix", "prefix", "prefix", "step"])
    sizes = rng.randrange(1 << 20)
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 1, 3, 4, 7, 8]) if Hkv <= 8 else 1
    d = rng.choice([64, 128, 128])
    rot = rng.choice([d, d, d, d // 2, 16])
    theta = rng.choice([1e4, 5e5, 1e6])
    if op in ("norm", "grad"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        layout = rng.choice(["dense", "packed", "serve"])
        most = 100_000_000 // (Hkv * (group + 1) * d * (2 if dtype == "fp32" else 1))
        tokens = _log_int(rng, 1, min(most, 65536))
        B = _log_int(rng, 1, min(tokens, 4 if layout == "dense" else 256))
        hi = tokens // B
        lo = hi if layout == "dense" else rng.choice([0, hi // 2, hi])
        if layout != "dense":
            hi = min(2 * hi - lo, most // B)  # the same number of tokens on average
        norms = rng.choice(["qk", "qk", "qk", "q", ""])
        return dict(op=op, layout=layout, B=B, new_lo=min(lo, hi), new_hi=max(hi, 1),
                    ends=_log_int(rng, 1, 1 << 20) if layout == "serve" else 0,
                    Hq=Hkv * group, Hkv=Hkv, d=d, rot=rot, inter=rng.random() < 0.4, norms=norms, dtype=dtype,
                    theta=theta, sizes=sizes)
    bs = rng.choice([16, 32, 64, 128])
    case = dict(op=op, Hq=Hkv * group, Hkv=Hkv, d=d, bs=bs, groups=1, pre_lo=0, pre_hi=0, rot=rot,
                inter=rng.random() < 0.3, theta=theta, causal=True, sizes=sizes)
    if op == "append":
        if rng.random() < 0.5:
            B = _log_int(rng, 1, 512)
            return case | dict(B=B, len_lo=0, len_hi=_log_int(rng, 1, max(2, 300_000_000 // (B * Hkv * d))),
                               new_lo=1, new_hi=rng.choice([1, 1, 4]))
        B = _log_int(rng, 1, 8)
        hi = _log_int(rng, 9, min(8192, 60_000_000 // (B * Hkv * (group + 2) * d)))
        return case | dict(B=B, len_lo=0, len_hi=rng.choice([0, 100]), new_lo=rng.choice([1, hi]), new_hi=hi)
    kind = "decode" if op == "step" else rng.choice(["decode", "decode", "draft", "prompt"])
    if kind == "prompt":
        B = _log_int(rng, 1, 6)
        new_hi = _log_int(rng, 9, 1500)
        new = (rng.choice([1, new_hi // 2 + 1, new_hi]), new_hi)
        len_hi = rng.choice([0, 0, 500])
        most = max(16, 1_000_000_000 // (B * Hkv * group * new_hi))
    else:
        B = _log_int(rng, 1, 128)
        new = (1, 1) if kind == "decode" else (1, _log_int(rng, 2, 8))
        len_hi = _log_int(rng, 1, max(2, min(4096, 300_000_000 // (B * Hkv * d))))
        most = max(16, min(250_000_000 // (Hkv * d), 2_000_000_000 // (B * Hkv * group * new[1])))
    groups = rng.choice([1, 1, 1, min(B, 2), min(B, 5)])
    pre_hi = _log_int(rng, 8, min(200_000, most // groups + 8))
    return case | dict(B=B, len_lo=rng.choice([0, len_hi]), len_hi=len_hi, new_lo=new[0], new_hi=new[1],
                       groups=groups, pre_lo=rng.choice([0, pre_hi // 2, pre_hi]), pre_hi=pre_hi,
                       causal=rng.random() < 0.8 or op == "step")


def _ceil(a, b):
    return -(-a // b)


def _sizes(case):
    """The same for every seed of a case: cached and new tokens of each
    request, first request of each group and the groups' prefix lengths."""
    r = random.Random(case["sizes"])
    B = case["B"]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    if sum(new) == 0:
        new[0] = 1
    if "bs" not in case:
        return [r.randint(0, case["ends"]) for _ in range(B)], new, [0, B], [0]
    cached = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(B)]
    first = sorted(r.randint(1, B - 1) for _ in range(case["groups"] - 1)) if B > 1 else [B] * (case["groups"] - 1)
    prefix = [r.randint(case["pre_lo"], case["pre_hi"]) for _ in range(case["groups"])]
    return cached, new, [0, *first, B], prefix


def work(case):
    cached, new, first, prefix = _sizes(case)
    total, Hq, Hkv, d = sum(new), case["Hq"], case["Hkv"], case["d"]
    if case["op"] in ("norm", "grad"):
        if case["layout"] == "dense":
            total = case["B"] * case["new_hi"]
        size = 4 if case["dtype"] == "fp32" else 2
        n = {c: total * h * d for c, h in (("q", Hq), ("k", Hkv))}
        weights = d * sum(c in case["norms"] for c in "qk")
        elems = n["q"] + n["k"]
        if case["op"] == "norm":  # in and out; squares, products and rotation
            return {"bytes": 2 * size * elems + size * weights, "flops": 8 * elems}
        # the upstream gradient in and the gradient out; the input where it is normalised
        moved = 2 * elems + sum(n[c] for c in case["norms"])
        return {"bytes": size * moved + (size + 4) * weights, "flops": 14 * elems}
    bs = case["bs"]
    bytes_ = flops = 0
    if case["op"] in ("append", "step"):
        touched = sum(_ceil(c + n, bs) - c // bs for c, n in zip(cached, new) if n > 0)
        # q in and out, new rows in (bf16) and out (8 bits), slots and positions, scales in and out
        bytes_ += 4 * total * Hq * d + 6 * total * Hkv * d + 8 * total + 16 * touched * Hkv
        flops += 8 * total * (Hq + Hkv) * d
    if case["op"] in ("prefix", "step"):
        bytes_ += total * Hq * (4 * d + 4)
        for c, n in zip(cached, new):
            bytes_ += 2 * (c + n) * Hkv * d + _ceil(c + n, bs) * (8 * Hkv + 4)
            flops += 4 * (n * c + (n * (n + 1) // 2 if case["causal"] else n * n)) * Hq * d
        for p, a, z in zip(prefix, first[:-1], first[1:]):
            rows = sum(new[a:z])
            if rows:  # each row of a prefix once for all that share it
                bytes_ += 2 * p * Hkv * d + _ceil(p, bs) * (8 * Hkv + 4)
                flops += 4 * rows * p * Hq * d
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEVICE).to(dtype)


def _weight(g, d, dtype):
    return (1 + 0.2 * torch.randn(d, generator=g, device=DEVICE)).to(dtype)


def _inv_freq(case):
    """theta^(-2 i / rot), i = 0 .. rot / 2 - 1, in 64 bits as the calls take it."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEVICE)
    return torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=DEVICE), -i / case["rot"])


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return _prepare_norm(case, g) if case["op"] in ("norm", "grad") else _prepare_cached(case, g)


def _prepare_norm(case, g):
    ends, new, _, _ = _sizes(case)
    B, Hq, Hkv, d, dtype = case["B"], case["Hq"], case["Hkv"], case["d"], TYPES[case["dtype"]]
    s = {"op": case["op"], "inter": case["inter"], "inv_freq": _inv_freq(case), "cu": None, "ends": None}
    # the projection's output: queries, keys and values of a token side by side
    lead = (B, case["new_hi"]) if case["layout"] == "dense" else (sum(new),)
    qkv = _randn(g, (*lead, Hq + 2 * Hkv, d), dtype) * 3
    dense = case["layout"] == "dense"
    s["q"], s["k"], _ = (x.transpose(1, 2) if dense else x for x in qkv.split([Hq, Hkv, Hkv], -2))
    if not dense:
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEVICE)
    if case["layout"] == "serve":  # a request's tokens are the last ones of so many
        s["ends"] = torch.tensor([e + n for e, n in zip(ends, new)], dtype=torch.int32, device=DEVICE)
    s["q_weight"], s["k_weight"] = (_weight(g, d, dtype) if c in case["norms"] else None for c in "qk")
    if case["op"] == "norm":
        s["q_out"], s["k_out"] = (torch.empty(s[c].shape, dtype=dtype, device=DEVICE) for c in "qk")
        return s
    s["dq_out"], s["dk_out"] = (_randn(g, s[c].shape, dtype) for c in "qk")
    dqkv = torch.zeros_like(qkv)
    s["dq"], s["dk"], _ = (x.transpose(1, 2) if dense else x for x in dqkv.split([Hq, Hkv, Hkv], -2))
    for c in "qk":
        s[f"d{c}_weight"] = torch.empty(d, device=DEVICE) if c in case["norms"] else None
    return s


def _prepare_cached(case, g):
    cached, new, first, prefix = _sizes(case)
    B, bs, Hq, Hkv, d, P = case["B"], case["bs"], case["Hq"], case["Hkv"], case["d"], case["groups"]
    total = sum(new)
    i32 = dict(dtype=torch.int32, device=DEVICE)
    lens = [c + n for c, n in zip(cached, new)]
    s = {"op": case["op"], "bs": bs, "total": total, "max_new": max(new), "max_pre": max(sum(new[a:z]) for a, z in
         zip(first[:-1], first[1:])), "causal": case["causal"], "inter": case["inter"], "scale": 1.0 / math.sqrt(d)}
    # blocks of all requests and prefixes in an arbitrary order, a few left over
    tables = []
    counts = [[_ceil(x, bs) for x in lens], [_ceil(x, bs) for x in prefix]]
    num_blocks = sum(map(sum, counts)) + 2
    perm = torch.randperm(num_blocks, generator=g, device=DEVICE).to(torch.int32)
    at = 0
    for c in counts:
        t = torch.full((len(c), max(1, max(c))), -1, **i32)
        t[torch.arange(t.shape[1], device=DEVICE) < torch.tensor(c, device=DEVICE)[:, None]] = perm[at: at + sum(c)]
        tables.append(t)
        at += sum(c)
    s["table"], s["prefix_table"] = tables
    s["cache_len"], s["prefix_len"] = torch.tensor(lens, **i32), torch.tensor(prefix, **i32)
    s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
    s["prefix_cu"] = torch.tensor(first, **i32)
    # the prefix counts as the request's first tokens
    before = np.repeat(prefix, np.diff(first)) if case["op"] != "append" else np.zeros(B, np.int64)
    s["ends"] = torch.tensor(np.asarray(lens) + before, **i32)
    request = torch.repeat_interleave(torch.arange(B, device=DEVICE), torch.tensor(new, device=DEVICE))
    pos = torch.arange(total, device=DEVICE) + (s["cache_len"] - s["cu"][1:])[request]
    s["slots"] = (s["table"][request, pos // bs] * bs + pos % bs).to(torch.int32)
    if case["op"] in ("append", "step"):
        qkv = _randn(g, (total, Hq + 2 * Hkv, d), torch.bfloat16) * 3
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        s["q_weight"], s["k_weight"] = (_weight(g, d, torch.bfloat16) for _ in "qk")
        s["inv_freq"] = _inv_freq(case)
        s["q_out"] = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=DEVICE)
    else:
        s["q"] = _randn(g, (total, Hq, d), torch.bfloat16)
    if case["op"] in ("prefix", "step"):
        s["o"] = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=DEVICE)
        s["lse"] = torch.empty((Hq, total), device=DEVICE)
    # rows that hold tokens: normal values at a scale that uses the E4M3 range. All others: zero where the caches are
    # compared, and otherwise whatever was there, NaN bytes among it
    known = [cached if case["op"] in ("append", "step") else lens, prefix]
    used = torch.zeros(num_blocks * bs, dtype=torch.bool, device=DEVICE)
    for t, n in zip(tables, known):
        pos = torch.arange(t.shape[1] * bs, device=DEVICE)
        rows = t.long()[:, pos // bs] * bs + pos % bs
        used[rows[pos[None] < torch.tensor(n, device=DEVICE)[:, None]]] = True
    junk = torch.randint(0, 256, (bs, d), generator=g, device=DEVICE, dtype=torch.uint8)
    if case["op"] != "prefix":
        junk.zero_()
    for c in ("k", "v"):
        x = torch.empty((num_blocks, Hkv, bs, d), dtype=torch.uint8, device=DEVICE)
        for part in range(0, num_blocks, 1 << 12):
            n = min(1 << 12, num_blocks - part)
            y = (torch.randn((n, Hkv, bs, d), generator=g, device=DEVICE) * 80).clamp(-E4M3_MAX, E4M3_MAX)
            there = used[part * bs: (part + n) * bs].view(n, 1, bs, 1)
            x[part: part + n] = torch.where(there, y.to(torch.float8_e4m3fn).view(torch.uint8), junk)
        s[c + "_cache"] = x.view(torch.float8_e4m3fn)
        e = torch.randint(-7, -4, (num_blocks, Hkv), generator=g, device=DEVICE)
        s[c + "_scale"] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _positions(s, x):
    """Position of each token of x, [total] or [1, N]."""
    if s["cu"] is None:
        return torch.arange(x.shape[2], device=x.device)[None]
    cu = s["cu"].long()
    t = torch.arange(x.shape[0], device=x.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    start = 0 if s["ends"] is None else (s["ends"].long() - (cu[1:] - cu[:-1]))[b]
    return t - cu[b] + start


def _cos_sin(s, x):
    # whole turns are dropped in 64 bits: a far position's angle has no fraction left in 32
    angle = torch.remainder(_positions(s, x).double()[..., None] * s["inv_freq"], 2 * math.pi)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return (cos[:, None], sin[:, None])  # one for all heads


def _rotate(s, x, cos, sin):
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["inter"] else (x[..., : rot // 2], x[..., rot // 2: rot])
    y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1 if s["inter"] else -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_norm(s, c):
    x = s[c].float()
    if s[c + "_weight"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[c + "_weight"].float()
    return _rotate(s, x, *_cos_sin(s, x)).to(s[c].dtype)


def _plain_grad(s, c):
    x, up = s[c].float(), s[f"d{c}_out"].float()
    cos, sin = _cos_sin(s, x)
    up = _rotate(s, up, cos, -sin)
    if s[c + "_weight"] is None:
        return {f"d{c}": up.to(s[c].dtype)}
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * r
    dw = (up * x).flatten(0, -2).sum(0)
    up = up * s[c + "_weight"].float()
    return {f"d{c}": (r * (up - x * (up * x).mean(-1, keepdim=True))).to(s[c].dtype), f"d{c}_weight": dw}


def _plain_append(s):
    bs, slots = s["bs"], s["slots"].long()
    blocks, run = torch.unique(slots // bs, return_inverse=True)
    first = torch.full((blocks.numel(),), bs, device=slots.device).scatter_reduce(0, run, slots % bs, "amin")
    out = {"q": _plain_norm(s, "q")}
    for c in ("k", "v"):
        cache, scale = s[c + "_cache"], s[c + "_scale"]
        # the cache's input is the 16-bit key
        x = (_plain_norm(s, "k") if c == "k" else s["v"]).float()
        top = torch.zeros((blocks.numel(), x.shape[1]), device=x.device)
        top = top.index_reduce(0, run, x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)
        e = torch.where(top > 0, e - 9 + (m > 0.875), EXP_MIN).clamp(min=EXP_MIN)
        old = torch.where(first[:, None] > 0, scale[blocks], 0.0)
        now = torch.maximum(old, torch.ldexp(torch.ones_like(top), e))
        rows = cache[blocks].float()
        there = torch.arange(bs, device=x.device)[None, :] < first[:, None]
        moved = there[:, None, :, None] & (now > old)[:, :, None, None]
        cache[blocks] = torch.where(moved, rows * (old / now)[:, :, None, None], rows).to(torch.float8_e4m3fn)
        cache.view(torch.uint8)[slots // bs, :, slots % bs] = (x / now[run][:, :, None]).to(
            torch.float8_e4m3fn).view(torch.uint8)
        scale[blocks] = now
        out |= {c + "_cache": cache, c + "_scale": scale}
    return out


def _plain_part(s, q, start, n, most, table, length, causal):
    """Rows [start, start + n) of q against the first `length` tokens of each
    table: maximum, sum and product of every row, back in the order of q."""
    bs = s["bs"]
    total, Hq, d = q.shape
    B, L = table.shape[0], table.shape[1] * bs
    Hkv = s["k_scale"].shape[1]
    G = Hq // Hkv
    i = torch.arange(most, device=q.device)
    token = (start[:, None] + i).clamp(max=total - 1)
    x = q[token].float().view(B, most, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * most, d)
    at = table.long().clamp(min=0)
    j = torch.arange(L, device=q.device)
    valid = j < length[:, None]

    def values(c):
        y = s[c + "_cache"][at].float() * s[c + "_scale"][at][..., None, None]
        return torch.where(valid[:, None, :, None], y.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, d), 0.0)

    p = (x @ values("k").transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, most, L)
    last = length[:, None] - n[:, None] + i if causal else (length - 1)[:, None].expand(B, most)
    p.masked_fill_((j > last[:, :, None])[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * most, L) @ values("v")).view(B, Hkv, G, most, d)
    here = i < n[:, None]
    return [y.permute(0, 3, 1, 2, 4).reshape(B, most, Hq, -1)[here] for y in (m, l, o)]


def _plain_prefix(s, q):
    cu, first = s["cu"].long(), s["prefix_cu"].long()
    m1, l1, o1 = _plain_part(s, q, cu[:-1], cu[1:] - cu[:-1], s["max_new"], s["table"], s["cache_len"].long(),
                             s["causal"])
    m2, l2, o2 = _plain_part(s, q, cu[first[:-1]], cu[first[1:]] - cu[first[:-1]], s["max_pre"], s["prefix_table"],
                             s["prefix_len"].long(), False)
    m = torch.maximum(m1, m2)
    ref = torch.where(m == -math.inf, 0.0, m)
    a1, a2 = torch.exp(m1 - ref), torch.exp(m2 - ref)
    l = l1 * a1 + l2 * a2
    o = (o1 * a1 + o2 * a2) / torch.where(l > 0, l, 1.0)
    return {"o": o.to(torch.bfloat16), "lse": (m + l.log()).squeeze(-1).t().contiguous()}


def _run_plain(s):
    if s["op"] == "norm":
        return {c: _plain_norm(s, c) for c in ("q", "k")}
    if s["op"] == "grad":
        return _plain_grad(s, "q") | _plain_grad(s, "k")
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "prefix":
        return _plain_prefix(s, s["q"])
    out = _plain_append(s)
    return out | _plain_prefix(s, out["q"])


# --------------------------------------------------------------------------
# the package's calls
# --------------------------------------------------------------------------

def _run_own(s):
    import io_aware_exact_tiled_gb300 as fa

    out = {}
    if s["op"] != "prefix":
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, inv_freq=s["inv_freq"],
                   interleaved=s["inter"], cu_seqlens=s["cu"], ends=s["ends"])
    if s["op"] == "norm":
        q, k = fa.qk_norm_rope(s["q"], s["k"], **how, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if "ws" not in s:  # kept from the first pass on, as a program keeps it
        if s["op"] == "grad":
            n = fa.fa_qk_norm_rope_bwd_workspace_size(s["q"].shape[-1])
        else:
            total, Hq, d = s["q"].shape
            n = fa.fa_fwd_paged_prefix_workspace_size(s["table"].shape[0], s["prefix_table"].shape[0], Hq,
                                                      s["k_scale"].shape[1], total, s["max_new"], d)
        s["ws"] = fa.workspace(n, DEVICE)
    if s["op"] == "grad":
        dq, dk, dqw, dkw = fa.qk_norm_rope_backward(
            s["q"], s["k"], s["dq_out"], s["dk_out"], **how, dq=s["dq"], dk=s["dk"], dq_weight=s["dq_weight"],
            dk_weight=s["dk_weight"], ws=s["ws"])
        out = {"dq": dq, "dq_weight": dqw, "dk": dk, "dk_weight": dkw}
        return {c: x for c, x in out.items() if x is not None}
    q = s["q"]
    if s["op"] in ("append", "step"):
        q = fa.qk_norm_rope_append(q, s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                   s["slots"], **how, q_out=s["q_out"])
        out = {"q": q} | {c: s[c] for c in ("k_cache", "k_scale", "v_cache", "v_scale")}
    if s["op"] in ("prefix", "step"):
        o, lse = fa.forward_paged_prefix(
            q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["cu"], s["cache_len"], s["table"],
            s["prefix_cu"], s["prefix_len"], s["prefix_table"], s["max_new"], scale=s["scale"], causal=s["causal"],
            out=s["o"], lse=s["lse"], ws=s["ws"])
        out |= {"o": o, "lse": lse}
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _exact_turn(s, c, pos):
    """Complex factors exp(i pos f) as [tokens, rot / 2], by the reduction of
    each angle to [-pi, pi]."""
    a = pos.double()[:, None] * s["inv_freq"][None, :]
    a = a - torch.round(a / (2 * math.pi)) * (2 * math.pi)
    return torch.complex(torch.cos(a), torch.sin(a))


def _exact_pairs(s, x):
    """The rotated part of heads x [.., d] as complex numbers [.., rot / 2]."""
    h = s["inv_freq"].numel()
    if s["inter"]:
        return torch.view_as_complex(x[..., : 2 * h].unflatten(-1, (h, 2)).contiguous())
    return torch.complex(x[..., :h].contiguous(), x[..., h: 2 * h].contiguous())


def _exact_unpair(s, z, x):
    y = x.clone()
    h = z.shape[-1]
    if s["inter"]:
        y[..., : 2 * h] = torch.view_as_real(z).flatten(-2)
    else:
        y[..., :h], y[..., h: 2 * h] = z.real, z.imag
    return y


def _exact_tokens(s, x):
    """x as [tokens, heads, d] in 64 bits, and each token's position."""
    if s["cu"] is None:
        B, H, N, d = x.shape
        return x.double().transpose(1, 2).reshape(B * N, H, d), torch.arange(N, device=x.device).repeat(B)
    cu = s["cu"].tolist()
    ends = [z - a for a, z in zip(cu[:-1], cu[1:])] if s["ends"] is None else s["ends"].tolist()
    pos = [torch.arange(e - (z - a), e, device=x.device) for a, z, e in zip(cu[:-1], cu[1:], ends)]
    return x.double(), torch.cat(pos)


def _exact_back(y, like):
    """[tokens, heads, d] in the layout of `like`."""
    if like.dim() == 3:
        return y
    B, H, N, d = like.shape
    return y.view(B, N, H, d).transpose(1, 2)


def _exact_norm(s, c):
    x, pos = _exact_tokens(s, s[c])
    if s[c + "_weight"] is not None:
        rms = torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS)
        x = x / rms * s[c + "_weight"].double()
    z = _exact_pairs(s, x) * _exact_turn(s, c, pos)[:, None]
    return _exact_back(_exact_unpair(s, z, x), s[c])


def _exact_grad(s, c):
    x, pos = _exact_tokens(s, s[c])
    up, _ = _exact_tokens(s, s[f"d{c}_out"])
    up = _exact_unpair(s, _exact_pairs(s, up) * _exact_turn(s, c, pos)[:, None].conj(), up)
    if s[c + "_weight"] is None:
        return {f"d{c}": _exact_back(up, s[c])}
    d = x.shape[-1]
    rms = torch.sqrt(torch.sum(x * x, -1, keepdim=True) / d + EPS)
    g = up * s[c + "_weight"].double()
    dx = g / rms - x * torch.sum(g * x, -1, keepdim=True) / (d * rms ** 3)
    return {f"d{c}": _exact_back(dx, s[c]), f"d{c}_weight": torch.sum(up * x / rms, (0, 1))}


def _round_e4m3(x):
    """The nearest E4M3 numbers, ties to even, of float64 values up to 448."""
    a = np.abs(x)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, E4M3_MAX), x)


def _exact_append(s):
    bs = s["bs"]
    q = _exact_norm(s, "q")
    slots = s["slots"].cpu().numpy()
    out = {"q": q}
    for c in ("k", "v"):
        x = (_exact_norm(s, "k").to(torch.bfloat16) if c == "k" else s["v"]).double().cpu().numpy()
        cache = s[c + "_cache"].float().cpu().numpy().astype(np.float64)
        scale = s[c + "_scale"].double().cpu().numpy()
        t = 0
        while t < len(slots):
            u = t + 1
            while u < len(slots) and slots[u] // bs == slots[t] // bs:
                u += 1
            b, r = slots[t] // bs, slots[t] % bs
            top = np.abs(x[t:u]).max(axis=(0, 2))
            e = np.ceil(np.log2(np.where(top > 0, top, 1.0) / E4M3_MAX))
            s_new = np.exp2(np.where(top > 0, np.maximum(e, EXP_MIN), EXP_MIN))
            if r > 0:
                s_new = np.maximum(s_new, scale[b])
                for h in np.nonzero(s_new > scale[b])[0]:
                    cache[b, h, :r] = _round_e4m3(cache[b, h, :r] * (scale[b, h] / s_new[h]))
            cache[b][:, slots[t:u] % bs] = _round_e4m3(x[t:u] / s_new[None, :, None]).transpose(1, 0, 2)
            scale[b] = s_new
            t = u
        out |= {c + "_cache": torch.from_numpy(cache), c + "_scale": torch.from_numpy(scale)}
    return out


def _exact_prefix(s, q, kc, ks, vc, vs):
    q, bs = q.double(), s["bs"]
    total, Hq, d = q.shape
    Hkv = ks.shape[1]
    G = Hq // Hkv
    o = torch.zeros((total, Hq, d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((Hq, total), -math.inf, dtype=torch.float64, device=DEVICE)

    def rows(table, length, h):
        at = table[: _ceil(length, bs)].long()
        return [(c[at, h].double() * f[at, h].double()[:, None, None]).reshape(-1, d)[:length]
                for c, f in ((kc, ks), (vc, vs))]

    lens, cu, first, pre = (s[c].tolist() for c in ("cache_len", "cu", "prefix_cu", "prefix_len"))
    for p, (a, z) in enumerate(zip(first[:-1], first[1:])):
        for h in range(Hkv):
            k0, v0 = rows(s["prefix_table"][p], pre[p], h)
            for b in range(a, z):
                t0, t1 = cu[b], cu[b + 1]
                n, length = t1 - t0, lens[b]
                if n == 0 or length + pre[p] == 0:
                    continue
                k1, v1 = rows(s["table"][b], length, h)
                j = torch.arange(length, device=DEVICE)[None, :]
                end = length - n + torch.arange(n, device=DEVICE) if s["causal"] else torch.full((n,), length,
                                                                                                 device=DEVICE)
                for y in range(h * G, (h + 1) * G):
                    x1 = torch.where(j <= end[:, None], (q[t0:t1, y] @ k1.T) * s["scale"], -math.inf)
                    x = torch.cat([(q[t0:t1, y] @ k0.T) * s["scale"], x1], 1)
                    l = torch.logsumexp(x, -1)
                    w = torch.exp(x - torch.where(l == -math.inf, 0.0, l)[:, None])
                    o[t0:t1, y] = w[:, : pre[p]] @ v0 + w[:, pre[p]:] @ v1
                    lse[y, t0:t1] = l
    return {"o": o, "lse": lse}


def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12 or (case["op"] in ("append", "step") and w["bytes"] > 6e8):
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        return {c: _exact_norm(s, c) for c in ("q", "k")}
    if case["op"] == "grad":
        return _exact_grad(s, "q") | _exact_grad(s, "k")
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "prefix":
        return _exact_prefix(s, s["q"], s["k_cache"].float(), s["k_scale"], s["v_cache"].float(), s["v_scale"])
    a = _exact_append(s)
    on = {c: x.to(DEVICE) for c, x in a.items()}
    return a | _exact_prefix(s, on["q"].to(torch.bfloat16), on["k_cache"], on["k_scale"], on["v_cache"], on["v_scale"])
