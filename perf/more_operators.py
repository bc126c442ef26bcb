"""What the serving operators of an attention layer are measured on.

Operators: appending keys and values to a paged 8-bit cache with the position
rotation on the way (and reading them back), attention over that cache, the
linear on 4-bit weights, and the attention layer that runs them all together.

Each has a plain form (elementary torch operations), the calls a user makes
of this package (`own`), and a definition in 64 bits (`exact`). Sizes are
those of the layer workloads here (GPT-7B, GPT-13B, GPT-175B and Llama-2-70B
style layers) or generic, with ragged lengths as served batches have them.

The cache: E4M3 codes, a power-of-two scale for each block of 16 consecutive
tokens and each head, for keys and for values; pages of `page` tokens, named
by a table of each sequence. Tokens of a call are packed; sequence i's end at
position lengths[i] - 1."""
import math

import torch

own = False

TOK = 16                     # tokens of a cache block
E4M3_MAX = 448.0             # 1.75 * 2^8


def listed():
    return [
        # one decoded token of one sequence: the smallest call, launch latency
        {"name": "append-token", "op": "append", "b": 1, "lo": 1000, "hi": 1000, "new": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "rot": 128, "inter": False},
        # a decode batch of ragged lengths on the smallest pages; half of each head is rotated, neighbours paired
        {"name": "append-batch173", "op": "append", "b": 173, "lo": 1, "hi": 9001, "new": 1, "hq": 64, "hkv": 8, "d": 128,
         "page": 16, "rot": 64, "inter": True},
        # ragged prompts through a GPT-13B-style layer: 40 heads, each with its own keys
        {"name": "append-prompts", "op": "append", "b": 5, "lo": 301, "hi": 4097, "new": 4096, "hq": 40, "hkv": 40, "d": 128,
         "page": 128, "rot": 128, "inter": False},
        # one decoded token over a short context: latency
        {"name": "attend-token", "op": "attend", "b": 1, "lo": 777, "hi": 777, "new": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "cap": 0.0, "window": 0},
        # a decode batch of a Llama-2-70B-style layer, lengths spread over a factor of 300
        {"name": "attend-ragged64", "op": "attend", "b": 64, "lo": 100, "hi": 32768, "new": 1, "hq": 64, "hkv": 8, "d": 128,
         "page": 64, "cap": 0.0, "window": 0},
        # two long documents: few rows, a long axis
        {"name": "attend-long", "op": "attend", "b": 2, "lo": 100003, "hi": 131101, "new": 1, "hq": 32, "hkv": 8, "d": 128,
         "page": 256, "cap": 0.0, "window": 0},
        # a few drafted tokens a sequence are verified; capped scores, a sliding window, heads of 64
        {"name": "attend-draft-window", "op": "attend", "b": 16, "lo": 500, "hi": 20011, "new": 5, "hq": 16, "hkv": 16, "d": 64,
         "page": 32, "cap": 50.0, "window": 4096},
        # prompts of a Llama-2-70B-style layer, the longest continuing an earlier part: the largest
        {"name": "attend-prompts", "op": "attend", "b": 3, "lo": 1501, "hi": 6007, "new": 4096, "hq": 64, "hkv": 8, "d": 128,
         "page": 64, "cap": 0.0, "window": 0},
        # one token through the qkv projection of a GPT-7B-style layer: weight-bandwidth bound
        {"name": "fp4-token", "op": "fp4", "m": 1, "k": 4096, "n": 12288},
        # a small decode batch through the qkv projection of a Llama-2-70B-style layer
        {"name": "fp4-batch13", "op": "fp4", "m": 13, "k": 8192, "n": 10240},
        # a short prompt through the qkv projection of a GPT-13B-style layer
        {"name": "fp4-prompt333", "op": "fp4", "m": 333, "k": 5120, "n": 15360},
        # a decode step of a GPT-7B-style attention layer: every operator in its place
        {"name": "layer-decode32", "op": "layer", "b": 32, "lo": 50, "hi": 8192, "new": 1, "hq": 32, "hkv": 32, "d": 128,
         "page": 64, "rot": 128, "inter": False, "k": 4096},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over [lo, hi] by its logarithm: as drawn, or rounded to 16 or to 128."""
    v, step = _log(rng, lo, hi), rng.choice((1, 16, 128, 128))
    return max(lo, v - v % step)


HEADS = ((32, 32), (64, 8), (40, 40), (32, 4), (10, 10), (28, 4), (16, 1), (20, 4))     # query heads, key heads


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "fp4", "layer"))
    if op == "fp4":
        return {"op": op, "m": _log(rng, 1, 512), "k": _size(rng, 256, 12288), "n": _size(rng, 256, 16384)}
    hq, hkv = rng.choice(HEADS)
    d = rng.choice((64, 128, 128, 256))
    c = {"op": op, "b": _log(rng, 1, 200), "hi": _log(rng, 16, 131072), "hq": hq, "hkv": hkv, "d": d,
         "page": rng.choice((16, 32, 64, 128, 256))}
    c["lo"] = max(1, int(c["hi"] * 10.0 ** -rng.uniform(0.0, 2.0)))
    c["new"] = rng.choice((1, rng.randint(2, 9), 4096)) if op != "layer" else rng.choice((1, 1, 3))
    if op == "attend":
        c["cap"], c["window"] = rng.choice((0.0, 0.0, 30.0)), rng.choice((0, 0, 1024, 777))
    else:
        c["rot"], c["inter"] = rng.choice((d, d, d // 2)), rng.random() < 0.5
    if op == "layer":
        c["k"] = 128 * _log(rng, 2, 48)
    while _cost(c) > 1.0:          # no more than the largest listed ones
        if c["b"] > 8:
            c["b"] //= 2
        else:
            c["hi"], c["lo"] = max(16, c["hi"] // 2), max(1, c["lo"] // 2)
    return c


def _cost(c):
    lens = _lens(c)
    new = [min(c["new"], n) for n in lens]
    held = sum(lens) * c["hkv"] * c["d"] / 3.6e8
    rows = sum(new) * (c["hq"] + 2 * c["hkv"]) * c["d"] / 1.1e8
    pairs = sum(n * (t - n / 2) for t, n in zip(lens, new)) * 4 * c["hq"] * c["d"] / 7e11 if c["op"] != "append" else 0
    return max(held, rows, pairs)


def _lens(c):
    """The sequences' lengths after the call: spread over [lo, hi] by their logarithm, in no order."""
    b = c["b"]
    at = sorted(range(b), key=lambda i: (i * 2654435761 + 97) % 4294967296)
    return [int(round(c["lo"] * (c["hi"] / c["lo"]) ** (a / max(1, b - 1)))) for a in at]


def work(case):
    if case["op"] == "fp4":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k // 2 + n * math.ceil(k / 32) + 2 * m * n, "flops": 2 * m * n * k}
    lens, hq, hkv, d = _lens(case), case["hq"], case["hkv"], case["d"]
    new = [min(case["new"], n) for n in lens]
    t = sum(new)
    held = sum(n + (l - n) % TOK for l, n in zip(lens, new))      # tokens that are read back
    # q in and out, k and v in, their codes out and in again, k and v out
    append = {"bytes": t * d * (4 * hq + 4 * hkv + 2 * hkv) + held * 6 * hkv * d, "flops": t * d * (4 * hq + 10 * hkv)}
    if case["op"] == "append":
        return append
    window = case.get("window", 0)
    pairs = seen = 0
    for l, n in zip(lens, new):
        if window:
            pairs += sum(min(window, p + 1) for p in range(l - n, l))
            seen += min(l, window + n - 1)
        else:
            pairs += n * (l - n) + n * (n + 1) // 2
            seen += l
    attend = {"bytes": seen * hkv * 2 * d + seen * hkv // 8 + 4 * t * hq * d, "flops": 4 * pairs * hq * d}
    if case["op"] == "attend":
        return attend
    k, wide = case["k"], (hq + 2 * hkv) * d
    weights = (k * wide + hq * d * k) * 17 // 32
    # x in, y out, both weights, the cache, what is read back of it
    return {"bytes": 4 * t * k + weights + seen * hkv * 2 * d + held * 6 * hkv * d,
            "flops": attend["flops"] + 2 * t * (k * wide + hq * d * k)}


# ---- inputs -------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def _keys(g, tokens, heads, d):
    """Keys: a few channels are far larger than the others, and tokens differ in size."""
    x = torch.randn((tokens, heads, d), generator=g, device="cuda")
    x[:, :, torch.randint(0, d, (max(1, d // 40),), generator=g, device="cuda")] *= 6.0
    x *= torch.exp2(torch.rand((tokens, 1, 1), generator=g, device="cuda") * 2.0 - 1.0)
    return x.to(torch.bfloat16)


def _freqs(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float() if rot else None


def _cum(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _inputs(case, seed):
    """A case's tensors, from the seed alone."""
    g = _gen(seed)
    if case["op"] == "fp4":
        m, k, n = case["m"], case["k"], case["n"]
        return {"x": _normal(g, (m, k)), "w": _normal(g, (k, n), 0.02)}
    lens, hq, hkv, d = _lens(case), case["hq"], case["hkv"], case["d"]
    new = [min(case["new"], n) for n in lens]
    t = sum(new)
    s = {"lens": lens, "new": new}
    if case["op"] == "append":
        # what the touched blocks hold already
        s["off"] = [(l - n) % TOK for l, n in zip(lens, new)]
        s["ko"], s["vo"] = _keys(g, sum(s["off"]), hkv, d), _normal(g, (sum(s["off"]), hkv, d))
        # views of one projection's output
        qkv = _normal(g, (t, (hq + 2 * hkv) * d))
        qkv[:, hq * d:(hq + hkv) * d] = _keys(g, t, hkv, d).reshape(t, -1)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split((hq * d, hkv * d, hkv * d), 1))
    elif case["op"] == "attend":
        s["q"] = _normal(g, (t, hq, d), 1.5)
        s["k"], s["v"] = _keys(g, sum(lens), hkv, d), _normal(g, (sum(lens), hkv, d))
    else:
        k, before = case["k"], sum(lens) - t
        s["x"] = _normal(g, (t, k))
        s["wqkv"], s["wo"] = _normal(g, (k, (hq + 2 * hkv) * d), k ** -0.5), _normal(g, (hq * d, k), (hq * d) ** -0.5)
        s["k"], s["v"] = _keys(g, before, hkv, d), _normal(g, (before, hkv, d))
    pages = [-(-l // case["page"]) for l in lens]
    order = torch.randperm(sum(pages) + 3, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(pages) + 1), -1, dtype=torch.int32, device="cuda")
    for i, (n, at) in enumerate(zip(pages, _cum(pages))):
        table[i, :n] = order[at:at + n]
    s["table"], s["pages"] = table, sum(pages) + 3
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    op = s["op"] = case["op"]
    if op == "fp4":
        w = s.pop("w")           # a serving program holds its weight in 4 bits, made once
        if own:
            import tensor_scaled_fp8_amd as fp8
            s["w"] = fp8.prepare_fp4_weight(w)
        else:
            s["w"] = _fp4(w.t().float())
        return s
    lens, new, hkv, d, page = s["lens"], s["new"], case["hkv"], case["d"], case["page"]
    s["case"] = case
    s["freqs"] = _freqs(case.get("rot", 0))
    before = [l - n for l, n in zip(lens, new)]
    held = s["off"] if op == "append" else lens if op == "attend" else before      # tokens stored beforehand
    until = lens if op == "attend" else before
    k0, v0 = (s.pop("ko"), s.pop("vo")) if op == "append" else (s.pop("k"), s.pop("v"))
    back = [n + b % TOK for n, b in zip(new, before)]                               # tokens read back
    if own:
        import tensor_scaled_fp8_amd as fp8
        s["cache"] = fp8.BlockKVCache(s["pages"], page, hkv, d, device="cuda")
        fp8.fp8_cache_append(s["cache"], k0, v0, s["table"], _ints(until), _ints(_cum(held)))
        s["lengths"], s["starts"] = _ints(lens), None if case["new"] == 1 else _ints(_cum(new))
        s["back"], s["tokens"] = _ints(_cum(back)), sum(back)
        if op == "layer":
            s["layer"] = fp8.InferenceAttention(s.pop("wqkv"), s.pop("wo"), case["hq"], hkv, d, freqs=s["freqs"],
                                                interleaved=case["inter"], bits=4)
        return s
    s["cache"] = [(torch.zeros((s["pages"] * page // TOK, hkv, TOK, d), device="cuda").to(torch.float8_e4m3fn),
                   torch.zeros((s["pages"] * page // TOK, hkv), dtype=torch.int32, device="cuda")) for _ in range(2)]
    plan = _plan(s["table"], page, until, held)
    for part, x in zip(s["cache"], (k0, v0)):
        _store(part, x, plan)
    del k0, v0
    if op != "attend":
        s["plan"] = _plan(s["table"], page, lens, new)
        s["positions"] = torch.cat([torch.arange(b, l, device="cuda") for b, l in zip(before, lens)])
        s["back"] = _plan(s["table"], page, lens, back)
    if op == "layer":
        s["wqkv"], s["wo"] = _fp4(s.pop("wqkv").t().float()), _fp4(s.pop("wo").t().float())
    return s


# ---- plain form ---------------------------------------------------------------------------

def _pow2(e):
    """2^e for whole e in [-126, 127], from the exponent field."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plan(table, page, lens, new):
    """The blocks that tokens lens[i] - new[i] .. lens[i] - 1 lie in: their places in the cache, the packed row of each of
    their 16 slots (the number of rows: none), which slots hold tokens already, and each row's place among the slots."""
    ids, rows, old, where, at = [], [], [], [], 0
    total = sum(new)
    for i, (l, n) in enumerate(zip(lens, new)):
        if n == 0:
            continue
        first, last = (l - n) // TOK, (l - 1) // TOK
        b = torch.arange(first, last + 1, device="cuda")
        pos = (b * TOK)[:, None] + torch.arange(TOK, device="cuda")
        ids.append(table[i, b * TOK // page].long() * (page // TOK) + b % (page // TOK))
        rows.append(torch.where((pos >= l - n) & (pos < l), pos - (l - n) + at, total))
        old.append(pos < l - n)
        at += n
    if not ids:
        return None
    rows = torch.cat(rows)
    return torch.cat(ids), rows, torch.cat(old), torch.nonzero(rows.reshape(-1) < total)[:, 0]


def _e4m3(x):
    """The nearest values of the format to those of x (64 bits), ties to even; |x| <= 448."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4
    return (torch.round(x * _pow2(-e)) * _pow2(e)).to(torch.float8_e4m3fn)


def _bias(amax):
    """floor(log2(448 / amax)) within +-126, 126 for 0."""
    m, e = torch.frexp(amax)
    return torch.where(amax == 0, 126, (8 - (e.int() - 1) - (m > 0.875).int()).clamp(-126, 126))


def _store(part, x, plan, step=1 << 14):
    """Rows x [tokens, heads, d] into their blocks of one part (codes, biases) of the cache."""
    if plan is None:
        return
    codes, biases = part
    for at in range(0, len(plan[0]), step):
        ids, rows, old = (p[at:at + step] for p in plan[:3])
        fresh = (rows < len(x))[:, None, :, None]
        v = torch.where(fresh, x[rows.clamp(max=len(x) - 1)].transpose(1, 2).double(), 0.0)      # [blocks, heads, 16, d]
        held = old.any(1)[:, None]
        before = biases[ids]
        bias = _bias(v.abs().amax((2, 3)))
        bias = torch.where(held, torch.minimum(before, bias), bias)
        kept = codes[ids]
        shift = torch.where(held, bias - before, 0)[:, :, None, None]
        again = _e4m3(kept.double() * _pow2(shift))
        made = _e4m3((v * _pow2(bias)[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX))
        codes.view(torch.uint8)[ids] = torch.where(fresh, made.view(torch.uint8), torch.where(
            old[:, None, :, None], again.view(torch.uint8), kept.view(torch.uint8)))
        biases[ids] = bias


def _load(part, plan):
    """The values of a plan's rows, [tokens, heads, d] in 32 bits."""
    ids, where = plan[0], plan[3]
    v = part[0][ids].float() * _pow2(-part[1][ids])[:, :, None, None]
    return v.transpose(1, 2).reshape(-1, v.shape[1], v.shape[3])[where]


def _rotate(x, positions, freqs, inter):
    """The rotation of x [tokens, heads, d] in 64 bits: far positions, and values next to a border of the 8-bit format."""
    x = x.double()
    if freqs is None:
        return x
    r = 2 * len(freqs)
    angle = (positions.double()[:, None] * freqs.double())[:, None]
    c, s = torch.cos(angle), torch.sin(angle)
    if inter:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_append(s, q, k, v):
    """Stores k and v; the rotated q."""
    rot = (s["positions"], s["freqs"], s["case"]["inter"])
    _store(s["cache"][0], _rotate(k, *rot), s["plan"])
    _store(s["cache"][1], v, s["plan"])
    return _rotate(q, *rot).to(torch.bfloat16)


def _plain_back(s):
    return tuple(_load(part, s["back"]).to(torch.bfloat16) for part in s["cache"])


def _plain_attend(s, q):
    case = s["case"]
    hq, hkv, d, page, cap, window = (case.get(n, 0) for n in ("hq", "hkv", "d", "page", "cap", "window"))
    g, per = hq // hkv, page // TOK
    out = torch.empty_like(q)
    at = 0
    for i, (l, n) in enumerate(zip(s["lens"], s["new"])):
        low = max(0, l - n - window + 1) // TOK if window else 0          # the first block that is seen
        blocks = torch.arange(low, -(-l // TOK), device="cuda")
        ids = s["table"][i, blocks // per].long() * per + blocks % per
        j = torch.arange(low * TOK, l, device="cuda")
        pos = torch.arange(l - n, l, device="cuda")[:, None]
        hidden = (j > pos) | (j <= pos - window) if window else j > pos
        x = q[at:at + n].float().reshape(n, hkv, g, d)
        step = max(1, (1 << 28) // (n * g * len(j)))                       # heads at a time
        for h in range(0, hkv, step):
            k, v = ((codes[ids, h:h + step].float() * _pow2(-bias[ids, h:h + step])[:, :, None, None]).transpose(0, 1)
                    .reshape(-1, len(blocks) * TOK, d)[:, :len(j)] for codes, bias in s["cache"])
            p = x[:, h:h + step].permute(1, 2, 0, 3).reshape(-1, g * n, d) @ k.transpose(1, 2).contiguous() * d ** -0.5
            p = p.view(-1, g, n, len(j))
            if cap:
                p = cap * torch.tanh(p / cap)
            p = p.masked_fill(hidden, -math.inf)
            p = torch.exp(p - p.amax(-1, keepdim=True))
            o = (p / p.sum(-1, keepdim=True)).view(-1, g * n, len(j)) @ v
            out[at:at + n, h * g:(h + step) * g] = o.view(-1, g, n, d).permute(2, 0, 1, 3).reshape(n, -1, d).to(q.dtype)
        at += n
    return out


def _blocks8(x):
    """x [r, c] as its 8-bit form with a scale for each 128 of a row holds it, in 32 bits."""
    r, c = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -c % 128)).reshape(r, -1, 128)
    bias = _bias(b.abs().amax(-1, keepdim=True))
    return ((b * _pow2(bias)).to(torch.float8_e4m3fn).float() * _pow2(-bias)).reshape(r, -1)[:, :c]


def _fp4(x):
    """x [r, c] in 4 bits: values 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (ties to an even mantissa), and the bias of each 32
    elements of a row, floor(log2(6 / amax))."""
    r, c = x.shape
    b = torch.nn.functional.pad(x, (0, -c % 32)).reshape(r, -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    bias = torch.where(amax == 0, 0, (2 - (e.int() - 1) - (m > 0.75).int()).clamp(-126, 126))
    a = b.abs() * _pow2(bias)
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5).float() + 2.0 * (a > 5.0)
    return (q * torch.sign(b)).to(torch.float8_e4m3fn), bias


def _plain_fp4(x, w):
    codes, bias = w
    return _blocks8(x) @ (codes.float() * _pow2(-bias)).reshape(len(codes), -1)[:, :x.shape[1]].t()


def _plain(s):
    if s["op"] == "fp4":
        return _plain_fp4(s["x"], s["w"]).to(torch.bfloat16)
    if s["op"] == "append":
        q = _plain_append(s, s["q"], s["k"], s["v"])
        return (q, *_plain_back(s))
    if s["op"] == "attend":
        return _plain_attend(s, s["q"])
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    qkv = _plain_fp4(s["x"], s["wqkv"]).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split((hq * d, hkv * d, hkv * d), 1))
    o = _plain_attend(s, _plain_append(s, q, k, v))
    return (_plain_fp4(o.reshape(len(o), -1), s["wo"]).to(torch.bfloat16), *_plain_back(s))


# ---- this package's operators -------------------------------------------------------------

def _own(s):
    import tensor_scaled_fp8_amd as fp8
    op = s["op"]
    if op == "fp4":
        return fp8.fp4_linear_fwd_cached(s["x"], s["w"])
    case, cache, table, lengths, starts = (s[n] for n in ("case", "cache", "table", "lengths", "starts"))
    if op == "attend":
        return fp8.fp8_cache_attention(s["q"], cache, table, lengths, starts, softcap=case["cap"], window=case["window"])
    if op == "append":
        y = fp8.fp8_cache_append(cache, s["k"], s["v"], table, lengths, starts, q=s["q"], freqs=s["freqs"],
                                 interleaved=case["inter"])
    else:
        y = s["layer"](s["x"], cache, table, lengths, starts)
    return (y, *fp8.fp8_cache_read(cache, table, lengths, s["back"], s["tokens"]))


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ------------------------------------------------------------

def _exponent(v):
    """floor(log2 |v|) of doubles, for v != 0."""
    return torch.frexp(v)[1].to(torch.int64) - 1


def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _near(t, bits, low):
    """The nearest values with `bits` mantissa bits, normal from 2^low on; ties to even."""
    gap = _two_to(_exponent(torch.where(t == 0, 1.0, t)).clamp(min=low) - bits)
    return torch.round(t / gap) * gap


def _largest(a, top, most, zero):
    """The largest e in +-126 with a 2^e <= most, where top is most's exponent; `zero` for a = 0."""
    safe = torch.where(a > 0, a, 1.0)
    e = top - _exponent(safe)
    e = torch.where(safe * _two_to(e) > most, e - 1, e).clamp(-126, 126)
    return torch.where(a > 0, e, zero)


def _held_after(x, o):
    """A sequence's tokens from a block's first one on, [tokens, heads, d] in 64 bits, as the cache holds them after the call
    that stores all but the first o of them; those were stored by an earlier call and lie in the first block."""
    b = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -len(x) % TOK)).view(-1, TOK, *x.shape[1:])
    old = torch.zeros_like(b)
    old[:1, :o] = b[:1, :o]
    b = b - old
    e = _largest(b.abs().amax((1, 3), keepdim=True), 8, E4M3_MAX, 126)
    if o:
        e0 = _largest(old[:1].abs().amax((1, 3), keepdim=True), 8, E4M3_MAX, 126)
        e[:1] = torch.minimum(e[:1], e0)
        b[:1] += _near(old[:1] * _two_to(e0), 3, -6) * _two_to(-e0)
    return (_near(b * _two_to(e), 3, -6) * _two_to(-e)).view(-1, *x.shape[1:])[:len(x)]


def _turned(x, first, freqs, inter):
    """Rotation by complex numbers: x [tokens, heads, d] of positions first, first + 1, ..."""
    x = x.double()
    if freqs is None:
        return x
    r = 2 * len(freqs)
    pos = torch.arange(first, first + len(x), device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos[:, None, None] * freqs.double())
    z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) if inter else torch.complex(x[..., :r // 2], x[..., r // 2:r])
    z = torch.view_as_real(z * turn)
    y = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
    return torch.cat((y, x[..., r:]), -1)


def _attended(q, k, v, first, cap, window):
    """One sequence: q [n, hq, d] at positions first ..; k, v [tokens, hkv, d]. Head by head."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out = torch.empty((n, hq, d), dtype=torch.float64, device=q.device)
    pos = torch.arange(first, first + n, device=q.device)[:, None]
    j = torch.arange(len(k), device=q.device)
    seen = j <= pos
    if window:
        seen &= pos - j < window
    for h in range(hq):
        s = torch.mm(q[:, h].double(), k[:, h // g].t()) / math.sqrt(d)
        if cap:
            s = torch.tanh(s / cap) * cap
        out[:, h] = torch.mm(torch.softmax(torch.where(seen, s, -math.inf), 1), v[:, h // g])
    return out


def _coded(x, block, top, most, bits, low):
    """Every row of x, block by block, at the nearest values of a format with a scale a block."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[1], block):
        v = x[:, at:at + block].double()
        e = _largest(v.abs().amax(1, keepdim=True), top, most, 0)
        out[:, at:at + block] = _near(v * _two_to(e), bits, low) * _two_to(-e)
    return out


def _product(x, w):
    """x [m, k] in 8 bits by the 4-bit form of w [k, n]."""
    return torch.matmul(_coded(x, 128, 8, E4M3_MAX, 3, -6), _coded(w.t(), 32, 2, 6.0, 1, 0).t())


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "fp4":
        return _product(s["x"], s["w"])
    lens, new, hq, hkv, d = s["lens"], s["new"], case["hq"], case["hkv"], case["d"]
    freqs, inter = _freqs(case.get("rot", 0)), case.get("inter", False)
    cap, window = case.get("cap", 0.0), case.get("window", 0)
    at = _cum(new)
    if op == "append":
        q, ks, vs = [], [], []
        for i, (l, n, o) in enumerate(zip(lens, new, s["off"])):
            before = slice(sum(s["off"][:i]), sum(s["off"][:i + 1]))
            rows = slice(at[i], at[i + 1])
            q.append(_turned(s["q"][rows], l - n, freqs, inter))
            ks.append(_held_after(torch.cat((s["ko"][before].double(), _turned(s["k"][rows], l - n, freqs, inter))), o))
            vs.append(_held_after(torch.cat((s["vo"][before], s["v"][rows])).double(), o))
        return torch.cat(q), torch.cat(ks), torch.cat(vs)
    if op == "attend":
        out = []
        for l, n, a, b in zip(lens, new, _cum(lens), at):
            k, v = (_held_after(x[a:a + l].double(), 0) for x in (s["k"], s["v"]))
            out.append(_attended(s["q"][b:b + n], k, v, l - n, cap, window))
        return torch.cat(out)
    # the path's own roundings (bf16 where it stores bf16) are part of its definition
    qkv = _product(s["x"], s["wqkv"]).to(torch.bfloat16).double().unflatten(1, (-1, d))
    outs, ks, vs = [], [], []
    for i, (l, n, a) in enumerate(zip(lens, new, _cum([l - n for l, n in zip(lens, new)]))):
        p = l - n
        rows = qkv[at[i]:at[i + 1]]
        q = _turned(rows[:, :hq], p, freqs, inter).to(torch.bfloat16)
        o = p % TOK
        kv = []
        for x, y in ((s["k"], _turned(rows[:, hq:hq + hkv], p, freqs, inter)), (s["v"], rows[:, hq + hkv:])):
            x = x[a:a + p].double()
            kv.append((_held_after(x[:p - o], 0), _held_after(torch.cat((x[p - o:], y)), o)))
        outs.append(_attended(q, torch.cat(kv[0]), torch.cat(kv[1]), p, 0.0, 0))
        ks.append(kv[0][1])
        vs.append(kv[1][1])
    o = torch.cat(outs).to(torch.bfloat16).reshape(at[-1], -1)
    return _product(o, s["wo"]), torch.cat(ks), torch.cat(vs)
