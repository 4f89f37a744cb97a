"""Cases of the microscaled (MXFP4) and 8-bit cache operators, and their plain forms.

Each case is one operator at one size: `run` computes it in elementary torch operations, or, with `own` set, through the
package's entry points. `exact` computes it in 64 bits from the definitions.

Sizes are TinyLlama-1.1B's (hidden 2048, feed-forward 5632, 32 query and 4 key/value heads of 64, 32000 words) where a case
is small, and generic ones of larger decoders (hidden 4096, feed-forward 14336, 8 key/value heads of 128) beyond.
"""
import random

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the activations of a few decoding sequences, before a product of two microscaled matrices
        {"name": "encode 5x2048 bf16", "op": "encode", "dtype": "bf16", "rows": 5, "n": 2048},
        # the LM head's weights, encoded when a model is loaded
        {"name": "encode 32000x2048 f32", "op": "encode", "dtype": "f32", "rows": 32000, "n": 2048},
        # one token's query projection
        {"name": "gemm 1x2048x2048 f32", "op": "gemm", "dtype": "f32", "batch": 1, "n_in": 2048, "n_out": 2048},
        # one token's LM head
        {"name": "gemm 1x2048x32000 bf16", "op": "gemm", "dtype": "bf16", "batch": 1, "n_in": 2048, "n_out": 32000},
        # a larger decoder's feed-forward product for eleven sequences
        {"name": "gemm 11x4096x14336 f16", "op": "gemm", "dtype": "f16", "batch": 11, "n_in": 4096, "n_out": 14336},
        # a prompt of 509 tokens through the gate projection
        {"name": "matmul 509x2048x5632 bf16", "op": "matmul", "dtype": "bf16", "rows": 509, "n_in": 2048, "n_out": 5632},
        # a long prompt through a larger decoder's gate and up projections
        {"name": "matmul 8192x4096x28672 bf16", "op": "matmul", "dtype": "bf16", "rows": 8192, "n_in": 4096,
         "n_out": 28672},
        # one decoding step's keys and values of 33 sequences
        {"name": "append 33x1 f32", "op": "append", "dtype": "f32", "seqs": 33, "longest": 1, "held": 700, "kv": 4,
         "dim": 64, "page": 16},
        # the keys and values of prompts of ragged lengths, some of them continued
        {"name": "append 9x2000 bf16", "op": "append", "dtype": "bf16", "seqs": 9, "longest": 2000, "held": 150, "kv": 8,
         "dim": 128, "page": 64},
        # one sequence's attention early in a conversation
        {"name": "attend 1x517 f32", "op": "attend", "dtype": "f32", "seqs": 1, "longest": 517, "queries": 1, "window": 0,
         "kv": 4, "group": 8, "dim": 64, "page": 16},
        # a served batch of ragged lengths
        {"name": "attend 32x8192 bf16", "op": "attend", "dtype": "bf16", "seqs": 32, "longest": 8192, "queries": 1,
         "window": 0, "kv": 8, "group": 4, "dim": 128, "page": 64},
        # one very long context, four tokens checked at once
        {"name": "attend 1x131071x4 f16", "op": "attend", "dtype": "f16", "seqs": 1, "longest": 131071, "queries": 4,
         "window": 0, "kv": 8, "group": 8, "dim": 128, "page": 32},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["encode", "gemm", "gemm", "matmul", "append", "attend", "attend"])
    c = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if op == "encode":
        n = 32 * _spread(rng, 1, 448)
        return {**c, "rows": _spread(rng, 1, min(32000, 50_000_000 // n)), "n": n}
    if op == "gemm":
        return {**c, "batch": _spread(rng, 1, 16), "n_in": 32 * _spread(rng, 2, 448), "n_out": _spread(rng, 16, 32000)}
    if op == "matmul":
        return {**c, "rows": _spread(rng, 1, 6000), "n_in": 32 * _spread(rng, 2, 256), "n_out": _spread(rng, 32, 16000)}
    c |= {"kv": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 96, 128, 192, 256]), "page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        return {**c, "seqs": _spread(rng, 1, 64), "longest": _spread(rng, 1, 600), "held": rng.choice([0, 10, 100, 1000])}
    seqs = _spread(rng, 1, 64)
    longest = _spread(rng, 1, min(100_000, 200_000_000 // (seqs * c["kv"] * c["dim"])))
    return {**c, "seqs": seqs, "longest": longest, "queries": rng.choice([1, 1, 1, 2, 5]),
            "window": rng.choice([0, 0, 0, 1000]), "group": rng.choice([1, 3, 4, 8, 16])}


def _lengths(case, low, high, salt):
    """A length for each sequence, of [low, high] with high among them: by the case alone."""
    rng = random.Random("%d %d %d %d" % (case["seqs"], low, high, salt))
    return [high] + [rng.randint(low, high) for _ in range(case["seqs"] - 1)]


def _plan(case):
    """(tokens held before, tokens added) of each sequence of an append case; (tokens held, 0) of an attend case."""
    if case["op"] == "append":
        return _lengths(case, 0, case["held"], 1), _lengths(case, min(1, case["longest"]), case["longest"], 2)
    return _lengths(case, case["longest"] // 4, case["longest"], 1), [0] * case["seqs"]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if case["op"] == "encode":
        # rows of unlike magnitude, a few large channels: activations and weights of a trained model
        x = normal(case["rows"], case["n"]) * torch.exp(0.5 * normal(case["rows"], 1)) * torch.exp(0.7 * normal(case["n"]))
        return {"case": case, "x": x.to(dtype)}
    if case["op"] in ("gemm", "matmul"):
        codes, scales = _encode(normal(case["n_out"], case["n_in"]) * (0.02 * torch.exp(0.3 * normal(case["n_out"], 1))))
        x = normal(case["batch"] if case["op"] == "gemm" else case["rows"], case["n_in"]) * torch.exp(0.7 * normal(case["n_in"]))
        return {"case": case, "codes": codes, "scales": scales, "x": x.to(dtype)}

    # a pool of pages in which the sequences' pages lie in no order, filled over its whole length with what was put there
    held, added = _plan(case)
    page, kv, dim = case["page"], case["kv"], case["dim"]
    width = max(-(-(h + a) // page) for h, a in zip(held, added)) + 1
    need = [-(-(h + a) // page) for h, a in zip(held, added)]
    pages = sum(need) + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    slot = torch.arange(width, device=DEV)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
    table = order[(first[:, None] + slot).clamp(max=pages - 1)]
    channel = torch.exp(0.5 * normal(kv, 1, dim))
    k, ks = _page_codes(normal(pages, kv, page, dim) * channel * torch.exp(0.3 * normal(pages, 1, 1, 1)))
    v, vs = _page_codes(normal(pages, kv, page, dim) * torch.exp(0.3 * normal(pages, 1, 1, 1)))
    state = {"case": case, "k_pages": k, "k_scales": ks, "v_pages": v.transpose(2, 3).contiguous(), "v_scales": vs,
             "table": table.contiguous(), "lens": torch.tensor(held, dtype=torch.int32, device=DEV)}
    if case["op"] == "append":
        total = sum(added)
        starts = [sum(added[:i]) for i in range(len(added) + 1)]
        return {**state, "k": (normal(total, kv, dim) * channel.transpose(0, 1)).to(dtype), "v": normal(total, kv, dim).to(dtype),
                "starts": torch.tensor(starts, dtype=torch.int32, device=DEV), "longest": max(added)}
    heads = kv * case["group"]
    return {**state, "q": (normal(case["seqs"], case["queries"], heads, dim) / channel.transpose(0, 1).repeat_interleave(case["group"], 1)).to(dtype)}


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "encode":
        return {"values": _decode(*_encode(state["x"]))}
    if case["op"] == "gemm":
        return {"y": (state["x"].float() @ _decode(state["codes"], state["scales"]).T).to(state["x"].dtype)}
    if case["op"] == "matmul":
        x = _decode(*_encode(state["x"]))
        return {"y": (x @ _decode(state["codes"], state["scales"]).T).to(state["x"].dtype)}
    if case["op"] == "append":
        return _append(state)
    return {"out": _attend(state)}


def _run_own(case, s):
    import quantized_weight_decode_gemv_amd as qwg

    if case["op"] == "encode":
        return {"values": qwg.dequant_mxfp4(*qwg.encode_mxfp4(s["x"]))}
    if case["op"] == "gemm":
        return {"y": qwg.gemm_mxfp4(s["codes"], s["scales"], s["x"])}
    if case["op"] == "matmul":
        codes, scales = qwg.encode_mxfp4(s["x"])
        return {"y": qwg.matmul_mxfp4(codes, scales, s["codes"], s["scales"], dtype=s["x"].dtype)}
    pages = s["k_pages"], s["k_scales"], s["v_pages"], s["v_scales"]
    if case["op"] == "append":
        qwg.kv8_append(s["k"], s["v"], *pages, s["table"], s["lens"], starts=s["starts"], max_new=s["longest"])
        return _values(s)
    return {"out": qwg.kv8_attend(s["q"], *pages, s["table"], s["lens"], window=case["window"])}


def _values(s):
    """The pool as the values it holds: fp8 codes, and a power of two for each page and head."""
    return {"k": s["k_pages"].view(torch.float8_e4m3fn), "v": s["v_pages"].view(torch.float8_e4m3fn),
            "k_exponents": s["k_scales"], "v_exponents": s["v_scales"]}


def _encode(x):
    """Rows of values -> (4-bit codes, two to a byte, the first in the low half; a power of two for each 32 values)."""
    b = x.float().unflatten(-1, (-1, 32))
    largest = b.abs().amax(-1)
    exponent = ((largest.view(torch.int32) >> 23) - 2).clamp(min=0)
    a = (b.double() * _power(127 - exponent)[..., None]).float().abs()
    code = (a > 0.25).to(torch.uint8)
    code = code + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), exponent.to(torch.uint8)


def _decode(codes, scales):
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = value[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()].unflatten(-1, (-1, 32))
    return (v * _power(scales.int() - 127).float()[..., None]).flatten(-2)


def _page_exponent(largest):
    """The biased exponent of the smallest power of two that brings `largest` to 448 or less."""
    bits = largest.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=0)


def _power(exponent):
    """2^exponent in 64 bits, made from its bits (exp2 need not be exact, and a tie's rounding shows it)."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _page_codes(x):
    """[pages, heads, tokens, channels] values -> e4m3 codes, and an exponent for each page and head."""
    e = _page_exponent(x.abs().amax((-1, -2)))
    return (x.double() * _power(127 - e)[..., None, None]).float().to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.uint8)


def _append(s):
    case = s["case"]
    page, seqs = case["page"], case["seqs"]
    held, added = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    # every page that any sequence's new tokens may reach: [seqs, pages]
    at = (held // page)[:, None] + torch.arange(-(-s["longest"] // page) + 1, device=held.device)
    touched = (at * page < (held + added)[:, None]) & (added > 0)[:, None]
    ids = s["table"].gather(1, at.clamp(max=s["table"].shape[1] - 1)).long()[touched]
    of = torch.arange(seqs, device=held.device)[:, None].expand_as(at)[touched]
    where = at[touched][:, None] * page + torch.arange(page, device=held.device)  # positions of the slots
    old = where < held[of][:, None]
    new = ~old & (where < (held + added)[of][:, None])
    token = (s["starts"][:-1].long()[of][:, None] + where - held[of][:, None]).clamp(0, s["k"].shape[0] - 1)
    for x, pages, scales, turned in ((s["k"], s["k_pages"], s["k_scales"], False), (s["v"], s["v_pages"], s["v_scales"], True)):
        codes = pages[ids].transpose(2, 3) if turned else pages[ids]  # [touched, heads, slots, channels]
        is_old, is_new = old[:, None, :, None], new[:, None, :, None]
        fresh = torch.where(is_new, x.float()[token].transpose(1, 2), 0.0)
        before = torch.where(old.any(1)[:, None], scales[ids].int(), 0)
        after = torch.maximum(before, _page_exponent(fresh.abs().amax((-1, -2))))
        kept = codes.view(torch.float8_e4m3fn).double() * _power(before - after)[..., None, None]
        put = fresh.double() * _power(127 - after)[..., None, None]
        put = torch.where(is_old, kept, put).float().to(torch.float8_e4m3fn).view(torch.uint8)
        codes = torch.where(is_old | is_new, put, codes)
        pages[ids] = codes.transpose(2, 3) if turned else codes
        scales[ids] = after.to(torch.uint8)
    return _values(s)


def _attend(s):
    case, q = s["case"], s["q"]
    seqs, queries, heads, dim = q.shape
    kv, group = case["kv"], case["group"]
    table = s["table"].long()
    k = s["k_pages"].view(torch.float8_e4m3fn).float() * _power(s["k_scales"].int() - 127).float()[..., None, None]
    v = s["v_pages"].view(torch.float8_e4m3fn).float() * _power(s["v_scales"].int() - 127).float()[..., None, None]
    k = k[table].transpose(1, 2).flatten(2, 3)  # [seqs, kv, positions, dim]
    v = v.transpose(2, 3)[table].transpose(1, 2).flatten(2, 3)
    at = torch.arange(k.shape[2], device=q.device)
    mine = (s["lens"].long()[:, None] - queries + torch.arange(queries, device=q.device))[..., None]
    seen = (at <= mine) & ((at > mine - case["window"]) if case["window"] else True)  # [seqs, queries, positions]
    seen = seen[:, None, :, None, :]
    x = q.float().unflatten(2, (kv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (x @ k.transpose(2, 3)).unflatten(2, (queries, group)) * dim ** -0.5
    score = torch.where(seen, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    held = (at < s["lens"][:, None])[:, None, :, None]
    out = p.flatten(2, 3) @ torch.where(held, v, 0.0)
    out = out.unflatten(2, (queries, group)) / torch.where(total == 0, 1.0, total)
    return out.permute(0, 2, 1, 3, 4).flatten(2, 3).to(q.dtype)


def work(case):
    if case["op"] == "encode":
        n = case["rows"] * case["n"]
        return {"bytes": n * (SIZE[case["dtype"]] + 4), "flops": 3 * n}  # the values in, and those they became
    if case["op"] in ("gemm", "matmul"):
        m = case.get("batch") or case["rows"]
        weights = case["n_in"] * case["n_out"]
        return {"bytes": weights * 17 // 32 + SIZE[case["dtype"]] * m * (case["n_in"] + case["n_out"]), "flops": 2 * m * weights}
    held, added = _plan(case)
    if case["op"] == "append":
        n = sum(added) * case["kv"] * case["dim"] * 2
        return {"bytes": n * (SIZE[case["dtype"]] + 1), "flops": 3 * n}
    rows = case["seqs"] * case["queries"] * case["kv"] * case["group"]
    seen = [min(h, case["window"] + case["queries"] - 1) if case["window"] else h for h in held]
    return {"bytes": sum(seen) * case["kv"] * case["dim"] * 2 + 2 * SIZE[case["dtype"]] * rows * case["dim"],
            "flops": 4 * sum(seen) * case["queries"] * case["kv"] * case["group"] * case["dim"]}


def _two_to(e):
    return torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device=e.device)[e.long() + 400]


def _e8m0(scales):
    return _two_to(scales.long() - 127)


def _exact_mx(x):
    """Each block of 32 values divided by its power of two and brought to the nearest of the fifteen magnitudes."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))  # amax = m 2^e with m in [1/2, 1)
    step = _two_to((e - 3).clamp(min=-127))
    a = b.abs() / step
    low = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))  # the spacing at a; torch.round takes ties to even
    return (torch.sign(b) * (torch.round(a / low) * low).clamp(max=6.0) * step).reshape(x.shape)


def _exact_weights(s):
    codes = torch.stack([s["codes"] % 16, s["codes"] // 16], -1).reshape(s["codes"].shape[0], -1)
    e, m = (codes // 2 % 4).double(), (codes % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * _two_to(e - 1)) * (1 - 2 * (codes // 8).double())
    return v * _e8m0(s["scales"]).repeat_interleave(32, 1)


def _exact_e4m3(a):
    _, e = torch.frexp(a)
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return torch.round(a / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "encode":
        return {"values": _exact_mx(s["x"])}
    if case["op"] in ("gemm", "matmul"):
        x = s["x"].double() if case["op"] == "gemm" else _exact_mx(s["x"])
        return {"y": torch.cat([part @ _exact_weights(s).T for part in x.split(2048)])}
    held, added = _plan(case)
    page = case["page"]
    table = s["table"].tolist()
    if case["op"] == "append":
        found = {}
        for name, turned in (("k", False), ("v", True)):
            codes = s[name + "_pages"].view(torch.float8_e4m3fn).double()
            codes = codes.transpose(2, 3).contiguous() if turned else codes
            exponents = s[name + "_scales"].double() - 127
            start = 0
            for i, (h, n) in enumerate(zip(held, added)):
                x = s[name][start:start + n].double().transpose(0, 1)  # [heads, tokens, channels]
                start += n
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
            found[name] = codes.transpose(2, 3).contiguous() if turned else codes
        return {**found, "k_exponents": None, "v_exponents": None}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    queries, group = case["queries"], case["group"]
    for i, h in enumerate(held):
        ids = torch.tensor(table[i][:-(-h // page)], device=DEV, dtype=torch.long)
        k = s["k_pages"][ids].view(torch.float8_e4m3fn).double() * _e8m0(s["k_scales"][ids])[..., None, None]
        v = s["v_pages"][ids].view(torch.float8_e4m3fn).double() * _e8m0(s["v_scales"][ids])[..., None, None]
        k = k.permute(1, 0, 2, 3).reshape(case["kv"], -1, case["dim"])[:, :h]
        v = v.permute(1, 0, 3, 2).reshape(case["kv"], -1, case["dim"])[:, :h]
        for t in range(queries):
            last = h - queries + t + 1  # the positions below it are seen
            begin = max(0, last - case["window"]) if case["window"] else 0
            if last > begin:
                q = s["q"][i, t].double().reshape(case["kv"], group, -1)
                w = torch.softmax(q @ k[:, begin:last].transpose(1, 2) / case["dim"] ** 0.5, -1)
                out[i, t] = (w @ v[:, begin:last]).reshape(-1, case["dim"])
    return {"out": out}
