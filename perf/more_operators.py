"""Cases of rotation on the way into the 8-bit cache, of attention over prompts and of attention behind a shared prefix.

Each case is one operator at one size: `run` computes it in elementary torch operations, or, with `own` set, through the
package's entry points. `exact` computes it in 64 bits from the definitions.

Sizes are TinyLlama-1.1B's (32 query and 4 key/value heads of 64) where a case is small, and generic ones of larger
decoders (32 query and 8 key/value heads of 128, and other shapes that the cache takes) beyond.
"""
import random

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one sequence's decoding step, early in a conversation
        {"name": "rotary 1x1 bf16", "op": "rotary", "dtype": "bf16", "seqs": 1, "longest": 1, "held": 41, "kv": 4, "group": 8,
         "dim": 64, "rotary": 64, "interleaved": False, "page": 16, "theta": 10000.0},
        # a served batch's decoding step, some of its contexts long
        {"name": "rotary 96x1 f16", "op": "rotary", "dtype": "f16", "seqs": 96, "longest": 1, "held": 120_000, "kv": 8,
         "group": 4, "dim": 128, "rotary": 128, "interleaved": False, "page": 64, "theta": 500000.0},
        # prompts of ragged lengths, some of them continued; the rotated keys go on to the prompts' attention
        {"name": "rotary 9x2000 bf16", "op": "rotary", "dtype": "bf16", "seqs": 9, "longest": 2000, "held": 150, "kv": 8,
         "group": 4, "dim": 128, "rotary": 128, "interleaved": False, "page": 64, "theta": 500000.0},
        # prompts of a decoder that rotates part of a head's channels, in neighbouring pairs
        {"name": "rotary 5x1100 f32", "op": "rotary", "dtype": "f32", "seqs": 5, "longest": 1100, "held": 0, "kv": 4,
         "group": 3, "dim": 96, "rotary": 48, "interleaved": True, "page": 32, "theta": 10000.0},
        # a short question
        {"name": "prompt 1x77 f16", "op": "prompt", "dtype": "f16", "seqs": 1, "longest": 77, "window": 0, "kv": 4, "group": 8,
         "dim": 64},
        # a batch of prompts packed one behind another
        {"name": "prompt 21x900 bf16", "op": "prompt", "dtype": "bf16", "seqs": 21, "longest": 900, "window": 0, "kv": 8,
         "group": 4, "dim": 128},
        # one long document
        {"name": "prompt 1x12000 bf16", "op": "prompt", "dtype": "bf16", "seqs": 1, "longest": 12000, "window": 0, "kv": 8,
         "group": 4, "dim": 128},
        # prompts in full precision, through layers with a sliding window
        {"name": "prompt 3x2500 f32", "op": "prompt", "dtype": "f32", "seqs": 3, "longest": 2500, "window": 1000, "kv": 4,
         "group": 8, "dim": 64},
        # a few answers sampled from one short prompt
        {"name": "shared 6x300+17 f16", "op": "shared", "dtype": "f16", "seqs": 6, "prefix": 300, "longest": 17, "queries": 1,
         "kv": 4, "group": 8, "dim": 64, "page": 16},
        # a served batch behind one long document
        {"name": "shared 64x32000+500 bf16", "op": "shared", "dtype": "bf16", "seqs": 64, "prefix": 32000, "longest": 500,
         "queries": 1, "kv": 8, "group": 4, "dim": 128, "page": 64},
        # many conversations behind one set of instructions
        {"name": "shared 250x1900+1200 f16", "op": "shared", "dtype": "f16", "seqs": 250, "prefix": 1900, "longest": 1200,
         "queries": 1, "kv": 8, "group": 4, "dim": 128, "page": 64},
        # three tokens checked at once in full precision
        {"name": "shared 17x9001+700x3 f32", "op": "shared", "dtype": "f32", "seqs": 17, "prefix": 9001, "longest": 700,
         "queries": 3, "kv": 4, "group": 3, "dim": 192, "page": 32},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["rotary", "prompt", "prompt", "shared", "shared"])
    c = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16", "bf16"]), "kv": rng.choice([1, 2, 4, 8]),
         "dim": rng.choice([64, 96, 128, 128, 192, 256])}
    values = c["kv"] * c["dim"]
    if op == "rotary":
        return {**c, "seqs": _spread(rng, 1, 100), "longest": _spread(rng, 1, 600), "held": rng.choice([0, 10, 1000, 100_000]),
                "group": rng.choice([1, 3, 4, 8]), "rotary": rng.choice([c["dim"], c["dim"], c["dim"] // 2]),
                "interleaved": rng.random() < 0.4, "page": rng.choice([16, 32, 64, 128]),
                "theta": rng.choice([10000.0, 500000.0])}
    c["group"] = rng.choice([1, 3, 4, 8, 16])
    if op == "prompt":
        seqs = _spread(rng, 1, 40)
        # the products of all pairs of positions stay below the largest listed case's
        longest = _spread(rng, 8, int(min(8000, (4e11 / (seqs * values * c["group"])) ** 0.5)))
        return {**c, "seqs": seqs, "longest": longest, "window": rng.choice([0, 0, 0, 700])}
    seqs, queries = _spread(rng, 2, 256), rng.choice([1, 1, 1, 2, 4])
    rows = seqs * queries * c["group"] * values
    prefix = _spread(rng, 100, int(max(200, min(64_000, 8e9 / rows))))
    return {**c, "seqs": seqs, "queries": queries, "prefix": prefix, "page": rng.choice([16, 32, 64, 128]),
            "longest": max(queries, _spread(rng, 8, int(max(16, min(4000, 1e8 / (seqs * values))))))}


def _lengths(case, low, high, salt):
    """A length for each sequence, of [low, high] with high among them: by the case alone."""
    rng = random.Random("%d %d %d %d" % (case["seqs"], low, high, salt))
    return [high] + [rng.randint(low, high) for _ in range(case["seqs"] - 1)]


def _plan(case):
    """(tokens held before, tokens added) of each sequence; (own positions held, 0) behind a prefix."""
    if case["op"] == "rotary":
        return _lengths(case, 0, case["held"], 1), _lengths(case, min(1, case["longest"]), case["longest"], 2)
    if case["op"] == "prompt":
        return [0] * case["seqs"], _lengths(case, 0, case["longest"], 2)
    return _lengths(case, min(case["queries"], case["longest"]), case["longest"], 1), [0] * case["seqs"]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    held, added = _plan(case)
    seqs, kv, dim, heads = case["seqs"], case["kv"], case["dim"], case["kv"] * case["group"]
    total = sum(added)
    starts = [sum(added[:i]) for i in range(seqs + 1)]

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    # keys have channels of unlike magnitude, queries the inverse ones: scores of a spread near one
    channel = torch.exp(0.5 * normal(kv, dim))
    inverse = (1 / channel).repeat_interleave(case["group"], 0)
    state = {"case": case}
    if case["op"] != "shared":
        # what one product of q|k|v gives: slices of its rows
        qkv = torch.cat([normal(total, heads, dim) * inverse, normal(total, kv, dim) * channel, normal(total, kv, dim)], 1)
        q, k, v = qkv.to(dtype).split([heads, kv, kv], 1)
        state |= {"q": q, "k": k, "v": v, "starts": _ints(starts), "longest": max(added)}
    if case["op"] == "prompt":
        return state

    # a pool of pages in which the sequences' pages lie in no order, filled over its whole length with what was put there
    page = case["page"]
    shared = -(-case["prefix"] // page) if case["op"] == "shared" else 0
    begins = [h // page if case["op"] == "rotary" else 0 for h in held]  # the first page that is read or written
    ends = [-(-(h + a) // page) for h, a in zip(held, added)]
    width = max(ends) + 1
    need = [e - b for b, e in zip(begins, ends)]
    pages = shared + sum(need) + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    slot = torch.arange(width, device=DEV)
    first = torch.tensor([shared + sum(need[:i]) - begins[i] for i in range(seqs)], device=DEV)
    table = order[(first[:, None] + slot).clamp(min=0, max=pages - 1)]
    k, ks = _page_codes(normal(pages, kv, page, dim) * channel[:, None] * torch.exp(0.3 * normal(pages, 1, 1, 1)))
    v, vs = _page_codes(normal(pages, kv, page, dim) * torch.exp(0.3 * normal(pages, 1, 1, 1)))
    state |= {"k_pages": k, "k_scales": ks, "v_pages": v.transpose(2, 3).contiguous(), "v_scales": vs,
              "table": table.contiguous(), "lens": _ints(held)}
    if case["op"] == "rotary":
        i = torch.arange(case["rotary"] // 2, device=DEV, dtype=torch.float64)
        return {**state, "freqs": (case["theta"] ** (-2 * i / case["rotary"])).float()}
    q = normal(seqs, case["queries"], heads, dim) * inverse
    return {**state, "q": q.to(dtype), "prefix": order[:shared].contiguous(), "prefix_len": _ints([case["prefix"]])}


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "rotary":
        return _rotary(state)
    return {"out": _prompt(state) if case["op"] == "prompt" else _shared(state)}


def _run_own(case, s):
    import quantized_weight_decode_gemv_amd as qwg

    if case["op"] == "prompt":
        return {"out": qwg.prompt_attend(s["q"], s["k"], s["v"], starts=s["starts"], max_len=s["longest"],
                                         window=case["window"])}
    pages = s["k_pages"], s["k_scales"], s["v_pages"], s["v_scales"]
    if case["op"] == "shared":
        return {"out": qwg.kv8_attend_shared(s["q"], *pages, s["prefix"], s["prefix_len"], s["table"], s["lens"])}
    one = s["longest"] == 1
    keys = None if one else torch.empty(s["k"].shape, dtype=s["k"].dtype, device=s["k"].device)
    q = qwg.kv8_append_rotary(s["q"], s["k"], s["v"], s["freqs"], *pages, s["table"], s["lens"],
                              starts=None if one else s["starts"], max_new=s["longest"],
                              interleaved=case["interleaved"], k_out=keys)
    return _values(s, q, keys)


def _values(s, q, keys):
    """Rotated queries and keys, and the pool as the values it holds: fp8 codes, and a power of two for each page and head."""
    found = {"q": q, "k": s["k_pages"].view(torch.float8_e4m3fn), "v": s["v_pages"].view(torch.float8_e4m3fn),
             "k_exponents": s["k_scales"], "v_exponents": s["v_scales"]}
    return found if s["longest"] == 1 else {**found, "keys": keys}


def _power(exponent):
    """2^exponent in 64 bits, made from its bits (exp2 need not be exact, and a tie's rounding shows it)."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _page_exponent(largest):
    """The biased exponent of the smallest power of two that brings `largest` to 448 or less."""
    bits = largest.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=0)


def _page_codes(x):
    """[pages, heads, tokens, channels] values -> e4m3 codes, and an exponent for each page and head."""
    e = _page_exponent(x.abs().amax((-1, -2)))
    return (x.double() * _power(127 - e)[..., None, None]).float().to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.uint8)


def _turn(x, cos, sin, case):
    """[tokens, heads, channels] in 32 bits, the first `rotary` channels rotated in pairs."""
    half = case["rotary"] // 2
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if case["interleaved"] else (turned[..., :half], turned[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1), rest], -1)


def _rotary(s):
    case = s["case"]
    page, seqs = case["page"], case["seqs"]
    begin, held, added = s["starts"][:-1].long(), s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    tokens = torch.arange(s["q"].shape[0], device=held.device)
    of = torch.searchsorted(s["starts"][1:].long(), tokens, right=True)
    angle = (held[of] + tokens - begin[of]).double()[:, None, None] * s["freqs"].double()  # far positions: 64 bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q, k = _turn(s["q"].float(), cos, sin, case), _turn(s["k"].float(), cos, sin, case)
    # every page that any sequence's new tokens reach: [seqs, pages]
    at = (held // page)[:, None] + torch.arange(-(-s["longest"] // page) + 1, device=held.device)
    touched = (at * page < (held + added)[:, None]) & (added > 0)[:, None]
    ids = s["table"].gather(1, at.clamp(max=s["table"].shape[1] - 1)).long()[touched]
    of = torch.arange(seqs, device=held.device)[:, None].expand_as(at)[touched]
    where = at[touched][:, None] * page + torch.arange(page, device=held.device)  # positions of the slots
    old = where < held[of][:, None]
    new = ~old & (where < (held + added)[of][:, None])
    token = (begin[of][:, None] + where - held[of][:, None]).clamp(0, tokens.shape[0] - 1)
    for x, pages, scales, turned in ((k, s["k_pages"], s["k_scales"], False), (s["v"].float(), s["v_pages"], s["v_scales"], True)):
        codes = pages[ids].transpose(2, 3) if turned else pages[ids]  # [touched, heads, slots, channels]
        is_old, is_new = old[:, None, :, None], new[:, None, :, None]
        fresh = torch.where(is_new, x[token].transpose(1, 2), 0.0)
        before = torch.where(old.any(1)[:, None], scales[ids].int(), 0)
        after = torch.maximum(before, _page_exponent(fresh.abs().amax((-1, -2))))
        kept = codes.view(torch.float8_e4m3fn).double() * _power(before - after)[..., None, None]
        put = fresh.double() * _power(127 - after)[..., None, None]
        put = torch.where(is_old, kept, put).float().to(torch.float8_e4m3fn).view(torch.uint8)
        codes = torch.where(is_old | is_new, put, codes)
        pages[ids] = codes.transpose(2, 3) if turned else codes
        scales[ids] = after.to(torch.uint8)
    return _values(s, q.to(s["q"].dtype), k.to(s["k"].dtype))


def _prompt(s):
    case, starts = s["case"], s["starts"].long()
    group, longest = case["group"], s["longest"]
    at = torch.arange(longest, device=starts.device)
    token = (starts[:-1, None] + at).clamp(max=max(0, s["q"].shape[0] - 1))  # [seqs, positions]
    q = s["q"][token].float().unflatten(2, (-1, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    held = at < (starts[1:] - starts[:-1])[:, None]
    k = s["k"][token].float().transpose(1, 2)
    v = torch.where(held[..., None, None], s["v"][token].float(), 0.0).transpose(1, 2)
    hidden = at > at[:, None]
    if case["window"]:
        hidden |= at <= at[:, None] - case["window"]
    score = (q @ k.transpose(2, 3)).unflatten(2, (group, longest))  # [seqs, kv, group, queries, positions]
    p = score.mul_(case["dim"] ** -0.5).masked_fill_(hidden, -torch.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    out = (p.flatten(2, 3) @ v).unflatten(2, (group, longest)) / p.sum(-1, keepdim=True)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [seqs, positions, heads, channels]
    tokens = torch.arange(s["q"].shape[0], device=starts.device)
    of = torch.searchsorted(starts[1:], tokens, right=True)
    return out[of, tokens - starts[of]].to(s["q"].dtype)


def _shared(s):
    case, q = s["case"], s["q"]
    seqs, queries, heads, dim = q.shape
    kv, group = case["kv"], case["group"]

    def values(pages, scales, ids, turned):
        x = pages[ids].view(torch.float8_e4m3fn).float() * _power(scales[ids].int() - 127).float()[..., None, None]
        return (x.transpose(-1, -2) if turned else x).transpose(-3, -4).flatten(-3, -2)  # [.., kv, positions, channels]

    pages = (s["k_pages"], s["k_scales"], False), (s["v_pages"], s["v_scales"], True)
    kp, vp = (values(p, e, s["prefix"].long(), t) for p, e, t in pages)  # [kv, positions, channels]
    ko, vo = (values(p, e, s["table"].long(), t) for p, e, t in pages)  # [seqs, kv, positions, channels]
    x = q.float().unflatten(2, (kv, group)) * dim ** -0.5
    # the last position of the whole that each query sees
    last = s["prefix_len"].long() + s["lens"].long()[:, None] - queries + torch.arange(queries, device=q.device)
    at = torch.arange(kp.shape[1], device=q.device)
    seen_p = (at < s["prefix_len"]) & (at <= last[..., None])  # [seqs, queries, positions]
    at = torch.arange(ko.shape[2], device=q.device)
    seen_o = s["prefix_len"] + at <= last[..., None]
    rows = x.permute(2, 0, 1, 3, 4).flatten(1, 3)  # [kv, rows, channels]
    sp = (rows @ kp.transpose(1, 2)).unflatten(1, (seqs, queries, group))
    sp = sp.masked_fill_(~seen_p[:, :, None], -torch.inf)
    mine = x.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seqs, kv, rows, channels]
    so = (mine @ ko.transpose(2, 3)).unflatten(2, (queries, group))
    so = so.masked_fill_(~seen_o[:, None, :, None], -torch.inf)
    top = torch.maximum(sp.amax(-1), so.amax(-1).transpose(0, 1))  # [kv, seqs, queries, group]
    pp = sp.sub_(top[..., None]).exp_()
    po = so.sub_(top.transpose(0, 1)[..., None]).exp_()
    total = pp.sum(-1) + po.sum(-1).transpose(0, 1)
    vp = torch.where((torch.arange(vp.shape[1], device=q.device) < s["prefix_len"])[:, None], vp, 0.0)
    vo = torch.where((at < s["lens"][:, None])[:, None, :, None], vo, 0.0)
    out = (pp.flatten(1, 3) @ vp).unflatten(1, (seqs, queries, group))
    out = out + (po.flatten(2, 3) @ vo).unflatten(2, (queries, group)).transpose(0, 1)
    out = out / total[..., None]
    return out.permute(1, 2, 0, 3, 4).flatten(2, 3).to(q.dtype)


def work(case):
    held, added = _plan(case)
    size, kv, heads, dim = SIZE[case["dtype"]], case["kv"], case["kv"] * case["group"], case["dim"]
    if case["op"] == "rotary":
        n = sum(added) * dim
        keys = kv if max(added) > 1 else 0
        return {"bytes": n * (size * (2 * heads + 2 * kv + keys) + 2 * kv), "flops": n * (3 * (heads + kv) + 6 * kv)}
    if case["op"] == "prompt":
        w = case["window"] or max(added)
        seen = sum(n * (n + 1) // 2 - max(0, n - w) * (max(0, n - w) + 1) // 2 for n in added)
        return {"bytes": 2 * size * sum(added) * dim * (heads + kv), "flops": 4 * seen * heads * dim}
    positions = case["seqs"] * case["prefix"] + sum(held)
    rows = case["seqs"] * case["queries"] * heads
    return {"bytes": (case["prefix"] + sum(held)) * kv * dim * 2 + 2 * size * rows * dim,
            "flops": 4 * positions * case["queries"] * heads * dim}


def _two_to(e):
    return torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device=e.device)[e.long() + 400]


def _e8m0(scales):
    return _two_to(scales.long() - 127)[..., None, None]


def _exact_e4m3(a):
    _, e = torch.frexp(a)
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return torch.round(a / step) * step


def _exact_turn(x, position, s):
    """A token's heads as complex numbers, multiplied by exp(i angle)."""
    case, x = s["case"], x.double()
    n = case["rotary"]
    angle = position.double()[:, None] * s["freqs"].double()[None]
    pair = x[..., :n].reshape(*x.shape[:-1], n // 2, 2) if case["interleaved"] else x[..., :n].reshape(*x.shape[:-1], 2, n // 2).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    pair = torch.view_as_real(z)
    turned = pair.reshape(*x.shape[:-1], n) if case["interleaved"] else pair.transpose(-1, -2).reshape(*x.shape[:-1], n)
    return torch.cat([turned, x[..., n:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    held, added = _plan(case)
    if case["op"] == "prompt":
        return {"out": _exact_prompt(s, added)}
    if case["op"] == "shared":
        return {"out": _exact_shared(s, held)}
    page, table = case["page"], s["table"].tolist()
    starts = s["starts"].tolist()
    position = torch.cat([torch.arange(h, h + n, device=DEV) for h, n in zip(held, added)])
    found = {"q": _exact_turn(s["q"], position, s), "keys": _exact_turn(s["k"], position, s)}
    for name, values in (("k", found["keys"]), ("v", s["v"].double())):
        codes = s[name + "_pages"].view(torch.float8_e4m3fn).double()
        codes = codes.transpose(2, 3).contiguous() if name == "v" else codes
        exponents = s[name + "_scales"].double() - 127
        for i, (h, n) in enumerate(zip(held, added)):
            x = values[starts[i]:starts[i + 1]].transpose(0, 1)  # [heads, tokens, channels]
            done = 0
            while done < n:
                p, slot = table[i][(h + done) // page], (h + done) % page
                part = x[:, done:done + page - slot]
                m, e = torch.frexp(part.abs().amax((1, 2)))
                want = (e - 9 + (m > 0.875)).double().clamp(min=-127)
                if slot:
                    want = torch.maximum(want, exponents[p])
                    codes[p, :, :slot] = _exact_e4m3(codes[p, :, :slot] * _two_to(exponents[p] - want)[:, None, None])
                exponents[p] = want
                codes[p, :, slot:slot + part.shape[1]] = _exact_e4m3(part * _two_to(-want)[:, None, None])
                done += part.shape[1]
        found[name] = codes.transpose(2, 3).contiguous() if name == "v" else codes
    found |= {"k_exponents": None, "v_exponents": None}
    return {k: v for k, v in found.items() if k != "keys" or s["longest"] > 1}


def _exact_prompt(s, added):
    case = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    begin = 0
    for n in added:
        for head in range(s["q"].shape[1]):
            k, v = (s[name][begin:begin + n, head // case["group"]].double() for name in ("k", "v"))
            for t in range(0, n, 2048):  # queries t .. t + 2047 and the keys that one of them sees
                end = min(n, t + 2048)
                low = max(0, t - case["window"] + 1) if case["window"] else 0
                q = s["q"][begin + t:begin + end, head].double() / case["dim"] ** 0.5
                mine, other = torch.arange(t, end, device=DEV)[:, None], torch.arange(low, end, device=DEV)[None]
                seen = (other <= mine) & (other > mine - case["window"]) if case["window"] else other <= mine
                w = torch.softmax((q @ k[low:end].T).masked_fill(~seen, -torch.inf), -1)
                out[begin + t:begin + end, head] = w @ v[low:end]
        begin += n
    return out


def _exact_shared(s, held):
    case = s["case"]
    kv, page, queries = case["kv"], case["page"], case["queries"]

    def both(ids, count):
        k = s["k_pages"][ids].view(torch.float8_e4m3fn).double() * _e8m0(s["k_scales"][ids])
        v = s["v_pages"][ids].view(torch.float8_e4m3fn).double() * _e8m0(s["v_scales"][ids])
        return (k.permute(1, 0, 2, 3).reshape(kv, -1, case["dim"])[:, :count],
                v.permute(1, 0, 3, 2).reshape(kv, -1, case["dim"])[:, :count])

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    kp, vp = both(s["prefix"].long(), case["prefix"])
    for i, h in enumerate(held):
        ko, vo = both(s["table"][i, :-(-h // page)].long(), h)
        k, v = torch.cat([kp, ko], 1), torch.cat([vp, vo], 1)
        for t in range(queries):
            end = case["prefix"] + h - queries + t + 1
            q = s["q"][i, t].double().reshape(kv, case["group"], -1)
            w = torch.softmax(q @ k[:, :end].transpose(1, 2) / case["dim"] ** 0.5, -1)
            out[i, t] = (w @ v[:, :end]).reshape(-1, case["dim"])
    return out
