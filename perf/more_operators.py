"""Measured cases of the operators that serve long streams.

Four operators of the paged cache:

* ``prompt``  attention of whole prompts or chunks of them over a 16-bit cache: a ragged batch of new tokens, each seeing
  the rows up to its own, optionally only a window of the newest ones and the sequence's first rows (sinks);
* ``sinks``   decode attention over a 16-bit cache of such a stream: the newest rows and the sinks, for one or several
  new tokens per sequence;
* ``cache4``  append into a four-bit cache (e2m1 codes, one e4m3 scale for each 16 elements of a row), and the rows that
  were written read back in 16 bits, as a chunk of a prompt needs them that attends to what is cached;
* ``decode4`` decode attention over the four-bit cache, optionally with a window and sinks.

A case gives an operator's sizes. ``prepare`` makes what a serving loop has in hand before the call, ``run`` is one call:
in elementary torch operations (``own`` false) or through the library (``own`` true). ``exact`` gives the results in 64
bits from the operators' definitions.
"""

import math
import random

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the e2m1 codes 0 .. 7
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # halfway between neighbours


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short user turns behind short histories: latency
        {"name": "prompt short", "op": "prompt", "dtype": "bf16", "batch": 3, "new_lo": 5, "new_hi": 40, "past_lo": 0,
         "past_hi": 100, "heads": 16, "kv_heads": 4, "dim": 64, "block": 16, "window": 0, "sinks": 0},
        # a batch of fresh prompts of different lengths, every earlier row visible
        {"name": "prompt batch", "op": "prompt", "dtype": "bf16", "batch": 8, "new_lo": 500, "new_hi": 4000,
         "past_lo": 0, "past_hi": 0, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 0, "sinks": 0},
        # a long document through a window, the first rows kept
        {"name": "prompt stream", "op": "prompt", "dtype": "f16", "batch": 1, "new_lo": 16384, "new_hi": 16384,
         "past_lo": 0, "past_hi": 0, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 4096, "sinks": 4},
        # chunked prefill: the next chunk of two long prompts, few new tokens against many cached rows
        {"name": "prompt chunk", "op": "prompt", "dtype": "bf16", "batch": 2, "new_lo": 200, "new_hi": 256,
         "past_lo": 9000, "past_hi": 30000, "heads": 64, "kv_heads": 8, "dim": 128, "block": 32, "window": 0,
         "sinks": 0},
        # one chat stream that has outgrown its window: latency
        {"name": "sinks short", "op": "sinks", "dtype": "bf16", "out": "bf16", "batch": 1, "tokens": 1, "lo": 700,
         "hi": 700, "heads": 16, "kv_heads": 4, "dim": 64, "block": 16, "window": 255, "sinks": 4},
        # a serving batch of long streams
        {"name": "sinks batch", "op": "sinks", "dtype": "bf16", "out": "f32", "batch": 32, "tokens": 1, "lo": 4096,
         "hi": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 4096, "sinks": 4},
        # verification of speculated tokens; sinks that end inside a block, a window that begins inside one
        {"name": "sinks tokens", "op": "sinks", "dtype": "f16", "out": "f16", "batch": 16, "tokens": 4, "lo": 300,
         "hi": 5000, "heads": 28, "kv_heads": 4, "dim": 128, "block": 32, "window": 1000, "sinks": 21},
        # one decode step of a serving batch
        {"name": "cache4 step", "op": "cache4", "dtype": "bf16", "batch": 64, "tokens": 1, "lo": 40, "hi": 4000,
         "kv_heads": 8, "dim": 128, "block": 16, "pad": 0},
        # a long prompt in one call
        {"name": "cache4 prompt", "op": "cache4", "dtype": "f16", "batch": 1, "tokens": 16384, "lo": 16384,
         "hi": 16384, "kv_heads": 8, "dim": 128, "block": 64, "pad": 0},
        # one short conversation: latency
        {"name": "decode4 short", "op": "decode4", "dtype": "bf16", "out": "bf16", "batch": 1, "tokens": 1, "lo": 131,
         "hi": 131, "heads": 16, "kv_heads": 4, "dim": 64, "block": 16, "window": 0, "sinks": 0},
        # the serving batch of the library's benchmark
        {"name": "decode4 batch", "op": "decode4", "dtype": "bf16", "out": "f32", "batch": 32, "tokens": 1, "lo": 512,
         "hi": 4096, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 0, "sinks": 0},
        # one very long document
        {"name": "decode4 long", "op": "decode4", "dtype": "bf16", "out": "bf16", "batch": 1, "tokens": 1,
         "lo": 131071, "hi": 131071, "heads": 64, "kv_heads": 8, "dim": 128, "block": 32, "window": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "sinks", "cache4", "decode4"])
    kv = rng.choice([1, 2, 4, 8])
    block = rng.choice([16, 16, 32, 48, 64])
    if op == "cache4":
        tokens = _log(rng, 1, 4000)
        lo = tokens + _log(rng, 1, 500)
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "batch": _log(rng, 1, max(1, min(64, 16000 // tokens))), "tokens": tokens, "lo": lo,
                "hi": lo + _log(rng, 1, 1000), "kv_heads": kv, "dim": rng.choice([64, 128, 128, 256]), "block": block,
                "pad": rng.choice([0, tokens // 3])}
    group = rng.choice([1, 2, 3, 4, 7, 8])
    window = rng.choice([0, _log(rng, 1, 5000)])
    sinks = rng.choice([0, 4, rng.randint(1, 200)]) if window else 0
    if op == "prompt":
        new = _log(rng, 1, 4000)
        past = rng.choice([0, _log(rng, 1, 20000)])
        # pairs of a token and a row, over heads: far below the long document's
        most = 4 * 10 ** 9 // (new * (new + past) * kv * group)
        batch = min(rng.choice([1, 2, 3, 5, 8, 17]), max(1, most))
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "batch": batch, "new_lo": max(1, new // 3),
                "new_hi": new, "past_lo": past // 2, "past_hi": past, "heads": kv * group, "kv_heads": kv,
                "dim": rng.choice([64, 128, 128]), "block": block, "window": window, "sinks": sinks}
    dim = rng.choice([64, 128, 128, 256])
    batch = _log(rng, 1, 48)
    rows = 1200000 // (kv * dim // 64)  # cached rows over the batch at most
    hi = max(40, min(_log(rng, 40, 40000), rows // batch))
    tokens = rng.choice([1, 1, 1, rng.randint(2, max(2, 32 // group))])
    return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "out": rng.choice(["f32", "bf16", "f16"]), "batch": batch,
            "tokens": tokens, "lo": max(tokens, rng.choice([1, hi // 3, hi])), "hi": hi, "heads": kv * group,
            "kv_heads": kv, "dim": dim, "block": block, "window": window or (0 if op == "decode4" else 1000),
            "sinks": sinks}


def _rng(case):
    """Lengths are part of the case, as a serving loop's bookkeeping is, and the same for every seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case):
    """Rows of each sequence, the new ones included."""
    r = _rng(case)
    if case["op"] == "prompt":
        return [r.randint(case["past_lo"], case["past_hi"]) + m for m in _new_tokens(case)]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _new_tokens(case):
    """New tokens of each sequence (cache4: those whose slots are not skipped)."""
    if case["op"] == "prompt":
        r = random.Random(repr(_rng(case).random()))
        return [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    if case["op"] == "cache4":
        return [case["tokens"] - (case["pad"] * i) // max(1, case["batch"] - 1) for i in range(case["batch"])]
    return [case["tokens"]] * case["batch"]


def _visible(case, m, n):
    """(rows that some of the m newest of n tokens sees, pairs of a token and a row it sees)."""
    window, sinks = case["window"] or n, case["sinks"]
    first = max(0, n - m + 1 - window)  # the oldest row in the first new token's window
    pairs = 0
    full = n - m + 1 > window  # every new token's window is full
    if full:
        pairs = m * window
    else:
        grow = max(0, min(m, window - (n - m)))  # tokens whose window still grows
        pairs = grow * (n - m) + grow * (grow + 1) // 2 + (m - grow) * window
    # sinks outside a token's window
    for t in range(m) if sinks else ():
        pairs += min(sinks, max(0, n - m + t + 1 - window))
    return n - first + min(sinks, first), pairs


def work(case):
    n, m = _lens(case), _new_tokens(case)
    H, D, bs = case["kv_heads"], case["dim"], case["block"]
    if case["op"] == "cache4":
        # each new row read, its codes and scales written, those read back and its values written
        new = sum(m)
        return {"bytes": 2 * new * H * (2 * D * SIZE[case["dtype"]] + 2 * (D // 2 + D // 16)) +
                8 * case["batch"] * case["tokens"], "flops": 6 * new * H * D}
    seen = [_visible(case, a, b) for a, b in zip(m, n)]
    rows, pairs = sum(s[0] for s in seen), sum(s[1] for s in seen)
    row_bytes = D // 2 + D // 16 if case["op"] == "decode4" else D * SIZE[case["dtype"]]
    q = sum(m) * case["heads"] * D
    out = SIZE[case.get("out", case["dtype"])]
    return {"bytes": 2 * rows * H * row_bytes + 4 * (rows // bs) + q * (SIZE[case["dtype"]] + out),
            "flops": 4 * pairs * case["heads"] * D}


# ----------------------------------------------------------------- inputs

def _values(shape, gen):
    """N(0, 1) with a loud channel in sixteen, as keys and values have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = torch.rand(shape[-1], generator=gen, device="cuda") < 1 / 16
    return x * torch.where(loud, 3.0, 1.0)


def _tables(lens, block, gen):
    """Block tables over a shuffled pool."""
    need = [-(-a // block) for a in lens]
    ids = torch.randperm(sum(need), generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(max(need), device="cuda")[None]
    count = torch.tensor(need, device="cuda")[:, None]
    start = torch.cumsum(count, 0) - count
    table = torch.where(at < count, ids[torch.clamp(start + at, max=len(ids) - 1)], 0)
    return table.to(torch.int32).contiguous(), len(ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, H, D, bs = _lens(case), case["kv_heads"], case["dim"], case["block"]
    s = dict(case)
    s["n"], s["m"] = n, _new_tokens(case)
    s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    s["tables"], nb = _tables(n, bs, gen)
    shape = (nb, H, bs, D)
    s["workspace"] = None  # the serving loop's scratch buffer: made at its first step, kept for the others
    if case["op"] in ("cache4", "decode4"):
        # pools of codes with their scales; most of a row's groups are of one size, a few are loud or quiet
        for name in ("k", "v"):
            x = _values(shape, gen) * torch.exp(0.5 * torch.randn(shape[:3], generator=gen, device="cuda"))[..., None]
            s[name], s[name + "s"] = _quantise(x)
    else:
        s["k"], s["v"] = (_values(shape, gen).to(DTYPE[case["dtype"]]) for _ in range(2))
    if case["op"] == "cache4":
        # the newest rows of each sequence are new; the last ones of a padded sequence are skipped
        B, T = case["batch"], case["tokens"]
        new = torch.tensor(s["m"], device="cuda")[:, None]
        t = torch.arange(T, device="cuda")[None]
        pos = torch.where(t < new, s["lens"][:, None].long() - new + t, -1)
        block = torch.gather(s["tables"].long(), 1, torch.clamp(pos // bs, min=0))
        s["slots"] = torch.where(pos >= 0, block * bs + pos % bs, -1).reshape(-1)
        loud = torch.exp(0.4 * torch.randn((B * T, 1, 1), generator=gen, device="cuda"))
        s["kn"], s["vn"] = ((_values((B * T, H, D), gen) * loud).to(DTYPE[case["dtype"]]) for _ in range(2))
        s["at"] = torch.nonzero(s["slots"] >= 0).reshape(-1)  # the tokens that are not skipped, as the host knows them
        s["kr"], s["vr"] = (torch.zeros((B * T, H, D), dtype=DTYPE[case["dtype"]], device="cuda") for _ in range(2))
        return s
    if case["op"] == "prompt":
        starts = [0]
        for a in s["m"]:
            starts.append(starts[-1] + a)
        s["first"] = starts
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        shape = (starts[-1], case["heads"], D)
    else:
        shape = (case["batch"], case["tokens"], case["heads"], D)
    s["q"] = (1.5 * torch.randn(shape, generator=gen, device="cuda")).to(DTYPE[case["dtype"]])
    s["result"] = torch.zeros(shape, dtype=DTYPE[case.get("out", case["dtype"])], device="cuda")
    return s


# ------------------------------------------------------------- plain forms

def _quantise(x):
    """x [..., D] as packed e2m1 codes [..., D/2] (the even element in the low half) and e4m3 scales [..., D/16]."""
    wide = torch.float64  # a quotient next to a border has to fall on its own side
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    top = g.abs().amax(-1).to(wide) / 6.0
    # nearest e4m3: whole multiples of 2^(e - 3), e of the value's own binade, not below 2^-6
    e = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    scale = torch.clamp(torch.round(top / step) * step, max=448.0).float()
    y = g.to(wide) / torch.where(scale > 0, scale, 1.0)[..., None].to(wide)
    code = torch.zeros(g.shape, dtype=torch.uint8, device=x.device)
    for i, mid in enumerate(MIDS):  # ties go to the even code
        code += (y.abs() > mid) if i % 2 == 0 else (y.abs() >= mid)
    code = torch.where(scale[..., None] > 0, code | ((y < 0).to(torch.uint8) << 3), 0).reshape(*x.shape[:-1], -1, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), scale.to(torch.float8_e4m3fn).view(torch.uint8)


def _levels(packed):
    """Packed codes as the e2m1 values they stand for, fp32."""
    table = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=packed.device)
    return table[torch.stack((packed & 15, packed >> 4), -1).long()].flatten(-2)


def _dequantised(packed, scale):
    x = _levels(packed)
    return (x.view(*scale.shape, 16) * scale.view(torch.float8_e4m3fn).float()[..., None]).view(x.shape)


def _cache4_plain(s):
    slots, bs = s["slots"][s["at"]], s["block"]
    b, r = slots // bs, slots % bs
    for new, name, back in ((s["kn"], "k", "kr"), (s["vn"], "v", "vr")):
        codes, scale = _quantise(new[s["at"]].float())
        s[name][b, :, r] = codes
        s[name + "s"][b, :, r] = scale
        s[back][s["at"]] = _dequantised(s[name][b, :, r], s[name + "s"][b, :, r]).to(s[back].dtype)


def _weights(x):
    """Softmax over the last axis, in place."""
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    return x.div_(x.sum(-1, keepdim=True))


def _decode_plain(s):
    B, T, Hq, D = s["q"].shape
    H, t = s["kv_heads"], s["tables"].long()
    rows = []
    for name in ("k", "v"):
        x = s[name][t]  # [B, W, H, bs, ...]
        x = _dequantised(x, s[name + "s"][t]) if s["op"] == "decode4" else x.float()
        rows.append(x.permute(0, 2, 1, 3, 4).reshape(B, H, -1, D))
    q = s["q"].float().view(B, T, H, Hq // H, D).permute(0, 2, 3, 1, 4)  # [B, H, G, T, D]
    x = torch.matmul(q.reshape(B, H, -1, D), rows[0].transpose(2, 3)) * (1.0 / math.sqrt(D))
    at = torch.arange(x.shape[-1], device="cuda")
    pos = s["lens"].long()[:, None] - T + torch.arange(T, device="cuda")[None]
    seen = at <= pos[..., None]  # [B, T, R]
    if s["window"]:
        seen &= (at > pos[..., None] - s["window"]) | (at < s["sinks"])
    x = _weights(torch.where(seen[:, None, None], x.view(B, H, Hq // H, T, -1), -math.inf))
    o = torch.matmul(x.view(B, H, -1, x.shape[-1]), rows[1]).view(B, H, Hq // H, T, D)
    s["result"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D))


def _prompt_plain(s):
    H, G, D, bs = s["kv_heads"], s["heads"] // s["kv_heads"], s["dim"], s["block"]
    for i, (m, n) in enumerate(zip(s["m"], s["n"])):
        t = s["tables"][i, :-(-n // bs)].long()
        k, v = (s[name][t].float().transpose(0, 1).reshape(H, -1, D)[:, :n] for name in ("k", "v"))
        new = slice(s["first"][i], s["first"][i] + m)
        q = s["q"][new].float().view(m, H, G, D).permute(1, 2, 0, 3)  # [H, G, m, D]
        x = torch.matmul(q.reshape(H, G * m, D), k.transpose(1, 2)).view(H, G, m, n).mul_(1.0 / math.sqrt(D))
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        at = torch.arange(n, device="cuda")[None]
        hidden = at > pos
        if s["window"]:
            hidden |= (at <= pos - s["window"]) & (at >= s["sinks"])
        x = _weights(x.masked_fill_(hidden, -math.inf))
        o = torch.matmul(x.view(H, G * m, n), v).view(H, G, m, D)
        s["result"][new] = o.permute(2, 0, 1, 3).reshape(m, H * G, D).to(s["result"].dtype)


def _outputs(s):
    if s["op"] != "cache4":
        return {"out": s["result"]}
    # the codes as the values they stand for, and all scales
    return {"k": s["kr"], "v": s["vr"], "ks": s["ks"].view(torch.float8_e4m3fn), "vs": s["vs"].view(torch.float8_e4m3fn)}


def run(state):
    s = state
    if own:
        import paged_kv_cache_157_gb300 as kvc
        scale, window = 1.0 / math.sqrt(s["dim"]), s.get("window") or None
        if s["op"] == "cache4":
            kvc.append_fp4(s["kn"], s["vn"], s["slots"], s["k"], s["v"], s["ks"], s["vs"])
            kvc.read_fp4(s["slots"], s["k"], s["v"], s["ks"], s["vs"], s["kr"], s["vr"])
        elif s["op"] == "prompt":
            if s["workspace"] is None:
                s["workspace"] = kvc.new_prompt_workspace(s["batch"], len(s["q"]), s["heads"], s["kv_heads"], s["dim"],
                                                          s["block"], s["tables"].shape[1])
            kvc.prompt_attention(s["q"], s["k"], s["v"], s["tables"], s["starts"], s["lens"], scale, s["result"],
                                 s["workspace"], window=window, sinks=s["sinks"])
        else:
            if s["workspace"] is None:
                s["workspace"] = kvc.new_scored_workspace(s["batch"], s["tokens"], s["heads"], s["kv_heads"], s["dim"],
                                                          s["block"], s["tables"].shape[1], scored=False)
            if s["op"] == "sinks":
                kvc.decode_attention_sinks(s["q"], s["k"], s["v"], s["tables"], s["lens"], scale, window, s["sinks"],
                                           s["result"], s["workspace"])
            else:
                kvc.decode_attention_fp4(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["tables"], s["lens"], scale,
                                         s["result"], s["workspace"], window=window, sinks=s["sinks"])
    elif s["op"] == "cache4":
        _cache4_plain(s)
    elif s["op"] == "prompt":
        _prompt_plain(s)
    else:
        _decode_plain(s)
    return _outputs(s)


# ------------------------------------------------------- results in 64 bits

def _nearest(x, table):
    """The entry of the ascending table nearest to each x >= 0; ties to the even index; the last one above it."""
    i = torch.clamp(torch.searchsorted(table, x.contiguous(), right=True) - 1, max=len(table) - 2)
    low, high = table[i], table[i + 1]
    up = (x - low > high - x) | ((x - low == high - x) & (i % 2 == 1))
    return torch.where(up, high, low)


def _exact_cache4(s):
    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    e2m1 = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    res = {}
    for new, name in ((s["kn"], "k"), (s["vn"], "v")):
        scales = s[name + "s"].view(torch.float8_e4m3fn).double()
        x = new.double().unflatten(-1, (-1, 16))
        scale = _nearest(x.abs().amax(-1) / 6, e4m3)
        value = torch.sign(x) * _nearest(x.abs() / torch.where(scale > 0, scale, math.inf)[..., None], e2m1)
        value = (value * scale[..., None]).flatten(-2)
        keep = s["slots"] >= 0
        at = s["slots"][keep]
        scales[at // s["block"], :, at % s["block"]] = scale[keep]
        res[name] = torch.where(keep[:, None, None], value, 0.0)
        res[name + "s"] = scales
    return res


def _exact_rows(s, name, i, n):
    """Sequence i's first n rows of every kv head in 64 bits, [H, n, D]."""
    t = s["tables"][i, :-(-n // s["block"])].long()
    if s["op"] == "decode4":
        c = s[name][t].int()
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)
        # sign, two exponent bits, one mantissa bit
        sign, e, f = 1 - 2 * (c // 8), c % 8 // 2, c % 2
        x = sign * torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * 2.0 ** (e - 1)).double()
        scale = s[name + "s"][t].view(torch.float8_e4m3fn).double()
        x = x * scale.repeat_interleave(16, -1)
    else:
        x = s[name][t].double()
    return x.transpose(0, 1).reshape(s["kv_heads"], -1, s["dim"])[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cache4":
        return _exact_cache4(s)
    H, G, D = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (m, n) in enumerate(zip(s["m"], s["n"])):
        q = s["q"][s["first"][i]:s["first"][i] + m] if case["op"] == "prompt" else s["q"][i]
        o = out[s["first"][i]:s["first"][i] + m] if case["op"] == "prompt" else out[i]
        k, v = _exact_rows(s, "k", i, n), _exact_rows(s, "v", i, n)
        for t0 in range(0, m, 1024):  # the tokens of a stretch see sinks and one range of rows
            t1 = min(m, t0 + 1024)
            last = n - m + t1
            low = max(0, n - m + t0 + 1 - case["window"]) if case["window"] else 0
            rows = torch.cat((torch.arange(min(low, case["sinks"])), torch.arange(low, last))).cuda()
            pos = torch.arange(n - m + t0, last).cuda()[:, None]
            hidden = rows > pos
            if case["window"]:
                hidden = hidden | ((rows <= pos - case["window"]) & (rows >= case["sinks"]))
            for h in range(H):
                kk, vv = k[h, rows], v[h, rows]
                for g in range(G):
                    x = q[t0:t1, h * G + g].double() @ kk.T / math.sqrt(D)
                    o[t0:t1, h * G + g] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ vv
    return {"out": out}
