"""Rotation on the way into the 8-bit cache, against plain 64-bit implementations.

A rotated value a cos - b sin: sine and cosine are off by 2^-25 (their fp32 rounding, the angle's own error being
below 2^-34 at the positions used here), each product by half an fp32 step of its own, the sum by another:
(|a| + |b|) (2^-25 + 2^-24) + 2^-24 |result| and less, so (|a| + |b|) 2^-22.5 and half a step of the type cover it.
Keys go to their page from 64 bits: a code is that of the exact key, or of a key 2^-33 (|a| + |b|) from it, the error
of its angle; so is the page's exponent."""
import numpy as np
import pytest
import torch

import layer_ref
import mx_ref as ref
import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import TYPES, assert_pages, dev, pages, tables, typed

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def frequencies(rotary, theta=10000.0):
    return (theta ** (-2 * np.arange(rotary // 2) / rotary)).astype(np.float32)


def assert_rotated(got, x, positions, freqs, interleaved, t):
    want, size = layer_ref.rotate(x, positions, freqs, interleaved)
    got = got.cpu().double().numpy().reshape(want.shape)
    tol = size * 2.0 ** -22.5 + torch.finfo(t).eps / 2 * np.abs(want) + (2.0 ** -25 if t is torch.float16 else 0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"
    still = 2 * len(freqs)
    assert np.array_equal(got[..., still:], x[..., still:])
    return want, size


def assert_keys(codes, exponents, c, want, size, table, held, starts):
    """Pages `c` (before the call) with the exact keys put into them, against codes and exponents after it."""
    codes, exponents = codes.cpu().numpy(), exponents.cpu().numpy()
    slack = size * 2.0 ** -33
    touched = np.zeros(codes.shape[:3], bool)
    for s, h in enumerate(held):
        for i in range(starts[s + 1] - starts[s]):
            page, slot = divmod(h + i, codes.shape[2])
            if h < 0 or page >= table.shape[1] or not 0 <= table[s, page] < len(codes):
                continue
            p, n = table[s, page], min(codes.shape[2] - slot, starts[s + 1] - starts[s] - i)
            touched[p, :, slot] = True
            if i == 0 or slot == 0:  # the page's exponent, from all its new keys
                part = slice(starts[s] + i, starts[s] + i + n)
                for head in range(codes.shape[1]):
                    may = [max(ref.page_exponent(np.abs(want[part, head]) + d * slack[part, head]), c.ks[p, head] if slot else 0)
                           for d in (-1, 0, 1)]
                    assert exponents[p, head] in may
                    if slot:  # what was there before has the page's new scale
                        old = ref.encode_e4m3_keeping_nan(c.k[p, head, :slot], int(c.ks[p, head]) - int(exponents[p, head]))
                        got = codes[p, head, :slot]
                        old = c.k[p, head, :slot] if exponents[p, head] == c.ks[p, head] else old
                        assert np.array_equal(np.where(got == 255, 127, got), np.where(old == 255, 127, old))
                        touched[p, head, :slot] = True
            for head in range(codes.shape[1]):
                may = layer_ref.codes_of(want[starts[s] + i, head], slack[starts[s] + i, head], int(exponents[p, head]))
                got = codes[p, head, slot]
                fits = [(got == m) | ((got & 127) + (m & 127) == 0) for m in may]  # (a zero may have either sign)
                assert np.logical_or.reduce(fits).all(), (s, i, head)
    assert np.array_equal(codes[~touched], c.k[~touched])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,rotary,page,kv,group,interleaved", [
    (64, 64, 16, 2, 8, False), (64, 16, 128, 1, 1, True), (96, 96, 32, 1, 3, True), (96, 48, 16, 2, 5, False),
    (128, 128, 64, 2, 4, False), (128, 64, 32, 1, 9, False), (192, 192, 64, 1, 2, False), (256, 256, 16, 2, 1, True),
    (256, 128, 128, 1, 4, False)])
def test_rotary_matches(t, dim, rotary, page, kv, group, interleaved):
    rng = np.random.default_rng(dim + page + rotary)
    held = [0, 1, page - 1, page, 5, 0, 3 * page + 2, 120_001, 40]
    new = [1, 1, 1, 2 * page + 3, 0, page, 1, 21, 70]
    total = [h + n for h, n in zip(held, new)]
    # entries of pages that are neither read nor written are no pages at all
    need = [-(-n // page) - h // page if n > h else 0 for h, n in zip(held, total)]
    table = np.full((len(held), max(total) // page + 2), -7, np.int32)
    order, at = rng.permutation(sum(need) + 2).astype(np.int32), 0
    for s, (h, n) in enumerate(zip(held, need)):
        table[s, h // page:h // page + n] = order[at:at + n]
        at += n
    c = ref.Cache(len(order), kv, dim, page, rng)
    c.ks[...], c.vs[...] = 120, 120  # of what the pages held before
    starts = np.concatenate([[0], np.cumsum(new)])
    tokens = starts[-1] + 2  # two rows more than are used
    spread = np.exp(2 * rng.standard_normal((tokens, 1, 1)))
    (q, qd), (k, kd), (v, vd) = (typed(rng.standard_normal((tokens, n, dim)) * spread, t) for n in (kv * group, kv, kv))
    freqs = frequencies(rotary)
    got = pages(c)
    mark = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    args = dev(table), dev(np.array(held, np.int32))
    first = dev(starts.astype(np.int32))
    out = qwg.kv8_append_rotary(q, k, v, dev(freqs), *got, *args, starts=first, interleaved=interleaved, out=mark[0], k_out=mark[1])
    assert out is mark[0] and (out[-2:] == 7).all() and (mark[1][-2:] == 7).all()
    n = starts[-1]
    positions = np.concatenate([np.arange(h, e) for h, e in zip(held, total)])
    assert_rotated(out[:n], qd[:n], positions, freqs, interleaved, t)
    want, size = assert_rotated(mark[1][:n], kd[:n], positions, freqs, interleaved, t)
    assert_keys(got[0], got[1], c, want, size, table, held, starts)
    k_before, ks_before = c.k.copy(), c.ks.copy()
    c.append(kd, vd, table, held, starts)
    c.k, c.ks = got[0].cpu().numpy(), got[1].cpu().numpy()  # (the keys are checked above)
    assert_pages(got, c)
    # the launch sized for one token, with no keys asked for: the same
    c.k, c.ks = k_before, ks_before
    before = ref.Cache(len(order), kv, dim, page, np.random.default_rng(0))
    before.k[...], before.ks[...], before.vs[...], before.v[...] = k_before, ks_before, 120, 0
    again = pages(before)
    out2 = qwg.kv8_append_rotary(q, k, v, dev(freqs), *again, *args, starts=first, max_new=1, interleaved=interleaved)
    assert torch.equal(out2[:n], out[:n]) and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_in_place_on_a_fused_result(t, interleaved):
    # one token of each sequence, q turned in place, the tokens at an odd distance and any address
    rng = np.random.default_rng(5)
    kv, group, dim, page, seqs = 2, 3, 96, 16, 5
    heads = kv * group
    width = (heads + 2 * kv) * dim
    flat, d = typed(rng.standard_normal(seqs * (width + 3) + 1), t)
    x, xd = flat[1:].view(seqs, width + 3)[:, :width], d[1:].reshape(seqs, width + 3)[:, :width]
    q, k, v = (y.unflatten(1, (-1, dim)) for y in x.split([heads * dim, kv * dim, kv * dim], 1))
    qd, kd = xd[:, :heads * dim].reshape(seqs, heads, dim), xd[:, heads * dim:(heads + kv) * dim].reshape(seqs, kv, dim)
    lens = np.array([0, 9, 15, 16, 31], np.int32)
    table, n_pages = tables(rng, lens + 1, page)
    c = ref.Cache(n_pages, kv, dim, page, rng)
    c.ks[...], c.vs[...] = 118, 118
    got = pages(c)
    freqs = frequencies(96)
    rest = flat.clone()
    out = qwg.kv8_append_rotary(q, k, v, dev(freqs), *got, dev(table), dev(lens), interleaved=interleaved, out=q)
    assert out.data_ptr() == q.data_ptr()
    want, size = layer_ref.rotate(kd, lens, freqs, interleaved)
    assert_rotated(out, qd, lens, freqs, interleaved, t)
    assert_keys(got[0], got[1], c, want, size, table, lens, np.arange(seqs + 1))
    rest[1:].view(seqs, width + 3)[:, :heads * dim] = q.flatten(1)
    assert torch.equal(rest, flat)  # nothing else was written


@pytest.mark.parametrize("t", TYPES)
def test_rotary_behind_a_prefix_and_far_away(t):
    rng = np.random.default_rng(6)
    kv, dim, page = 1, 64, 32
    lens, new = np.array([3, 0], np.int32), 40
    table, n_pages = tables(rng, lens + new, page)
    c = ref.Cache(n_pages, kv, dim, page)
    (q, qd), (k, kd) = (typed(rng.standard_normal((2, new, n, dim)), t) for n in (2, 1))
    freqs = frequencies(64, 500000.0)
    for before in (0, 17, 1_000_003, -5):
        got = pages(c)
        keys = torch.empty_like(k)
        out = qwg.kv8_append_rotary(q, k, k, dev(freqs), *got, dev(table), dev(lens), k_out=keys,
                                    prefix_len=dev(np.array([before], np.int32)))
        positions = np.concatenate([np.arange(h, h + new) + before for h in lens])
        assert_rotated(out, qd.reshape(-1, 2, dim), positions, freqs, False, t)
        assert_rotated(keys, kd.reshape(-1, 1, dim), positions, freqs, False, t)
    plain = pages(c)
    qwg.kv8_append(k, k, *plain, dev(table), dev(lens))
    assert torch.equal(plain[2], got[2]) and torch.equal(plain[3], got[3])  # values do not turn


def test_rotary_without_pages_and_with_values_that_are_none():
    rng = np.random.default_rng(7)
    heads, dim, page = 2, 64, 16
    table = np.array([[3, 99], [-1, 2], [4, 5], [0, 1]], np.int32)
    held, starts = np.array([10, 10, 30, -4], np.int32), np.array([0, 20, 40, 50, 60], np.int32)
    c = ref.Cache(6, heads, dim, page, np.random.default_rng(1))
    c.ks[...], c.vs[...] = 120, 120
    got = pages(c)
    k, kd = typed(rng.standard_normal((60, heads, dim)), torch.float32)
    freqs = frequencies(64)
    keys = torch.empty_like(k)
    out = qwg.kv8_append_rotary(k, k, k, dev(freqs), *got, dev(table), dev(held), starts=dev(starts), k_out=keys)
    positions = np.concatenate([np.arange(h, h + n) for h, n in zip(held, np.diff(starts))])
    # tokens that have no page, or no position, still turn
    want, size = assert_rotated(out, kd, positions, freqs, False, torch.float32)
    assert torch.equal(out, keys)
    assert_keys(got[0], got[1], c, want, size, table, held, starts)
    # a NaN or an infinity reaches its pair alone, and does not count for the page's exponent
    k[3, 0, 5], k[4, 1, 40] = float("nan"), float("inf")
    out = qwg.kv8_append_rotary(k, k, k, dev(freqs), *got, dev(table), dev(held), starts=dev(starts))
    none = ~torch.isfinite(out)
    assert none[3, 0, [5, 37]].all() and none[4, 1, [40, 8]].all() and none.sum() == 4
    assert (got[0][3, 0, 13, [5, 37]] & 127 == 127).all() and (got[0][3, 1, 14, [8, 40]] & 127 == 127).all()
    assert got[1][3, 0] < 140


@pytest.mark.parametrize("t", TYPES)
def test_rotary_captured_and_replayed(t):
    rng = np.random.default_rng(8)
    kv, group, dim, page, seqs = 2, 4, 128, 16, 3
    table, n_pages = tables(rng, [64] * seqs, page)
    freqs = dev(frequencies(128))
    lens = dev(np.array([0, 5, 31], np.int32))
    q, k = (typed(rng.standard_normal((seqs, n, dim)), t)[0] for n in (kv * group, kv))
    cache, plain = (qwg.kv8_pages(n_pages, kv, dim, page, device=DEV) for _ in range(2))
    tab, at = dev(table), lens.clone()
    qwg.kv8_append_rotary(q, k, k, freqs, *plain, tab, lens)
    for x in plain:
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qwg.kv8_append_rotary(q, k, k, freqs, *cache, tab, lens)
        lens += 1
    for step in range(20):
        for x in (q, k):
            x.copy_(typed(rng.standard_normal(x.shape), t)[0])
        graph.replay()
        want = qwg.kv8_append_rotary(q, k, k, freqs, *plain, tab, at)
        at += 1
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(at, lens)
        for a, b in zip(cache, plain):
            assert torch.equal(a, b)


def test_rotary_refusals():
    cache = qwg.kv8_pages(4, 2, 64, 16, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    k, q, f = torch.zeros(2, 2, 64, device=DEV), torch.zeros(2, 4, 64, device=DEV), torch.ones(32, device=DEV)
    qkv = torch.zeros(2, 8, 64, device=DEV)

    def call(q=q, k=k, v=k, f=f, **more):
        return qwg.kv8_append_rotary(q, k, v, f, *cache, table, lens, **more)

    bad = [lambda: call(q.half()), lambda: call(q[:1]), lambda: call(q[:, :3]), lambda: call(q.cpu()), lambda: call(f=f.double()),
           lambda: call(f=f[:12]), lambda: call(f=torch.ones(40, device=DEV)), lambda: call(f=f[:0]), lambda: call(f=f.cpu()),
           lambda: call(out=q[:1]), lambda: call(out=q.half()), lambda: call(k_out=q), lambda: call(k_out=k.half()),
           lambda: call(v=k[:1]), lambda: call(prefix_len=lens), lambda: call(prefix_len=3), lambda: call(q.unflatten(0, (2, 1))),
           lambda: call(q.transpose(1, 2).contiguous().transpose(1, 2))]
    for one in bad:
        with pytest.raises(ValueError):
            one()
    # results over what the call still reads
    for one in (lambda: call(k_out=k), lambda: call(v=qkv[:, 4:6], out=qkv[:, 2:6]), lambda: call(qkv[:, :4], out=qkv[:, 1:5]),
                lambda: call(k=qkv[:, 4:6], k_out=qkv[:, 5:7]), lambda: call(out=qkv[:, :4], k_out=qkv[:, 3:5]),
                lambda: call(qkv[:, :4], out=qkv.view(-1)[:512].view(2, 4, 64))):
        with pytest.raises(qwg.QwgError) as e:
            one()
        assert e.value.status == 11
    call(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], out=qkv[:, :4])  # slices of one result interleave
    torch.cuda.synchronize()
