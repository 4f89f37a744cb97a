"""Attention behind a shared prefix against plain 64-bit implementations, and the calls of a layer in a row.

The bound is that of attention over the cache (test_kv8_gpu), with a probability of the 16-bit types rounded to fp16: 2^-11
of it; and where it is below 2^-14 (times its page's scale, against the largest such product of the row) 2^-25 of that
product, each of at most 448 codes: a page's largest is over 224, so n 2^-24 of the largest |v| covers them. Over many
outputs the two roundings add up as independent errors of at most half a step, evenly spread: a third of their
squares."""
import numpy as np
import pytest
import torch

import layer_ref
import mx_ref as ref
import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import TYPES, assert_attend, dev, pages, typed
from test_prompt_gpu import assert_prompt
from test_rotary_gpu import assert_rotated, frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def assert_shared(out, want, weight, size, v_top, t, n):
    dim = want.shape[-1]
    got = out.cpu().double().numpy().reshape(want.shape)
    p = 0 if t is torch.float32 else 2.0 ** -11
    tol = (4 * (3 * dim / 32 + 36) * 2.0 ** -24 * size + 2.0 ** -17 * (1 + n / 4096) + p) * weight
    tol = tol + torch.finfo(t).eps / 2 * np.abs(want) + (2.0 ** -25 if t is torch.float16 else 0)
    tol = tol + (0 if t is torch.float32 else 2.0 ** -24 * n * v_top)
    bad = ~(np.abs(got - want) <= tol)
    if t is not torch.float32 and want.size > 20000:
        half = torch.finfo(t).eps / 2
        assert np.linalg.norm(got - want) <= ((half ** 2 + 2.0 ** -22) / 3) ** 0.5 * np.linalg.norm(want)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def filled(rng, prefix_len, lens, heads, dim, page, spread=1.0, width=None):
    """A pool with a prefix and each sequence's own positions; stale bytes and tables' spare entries elsewhere."""
    each = [prefix_len] + list(lens)
    need = [-(-n // page) for n in each]
    order, at = rng.permutation(sum(need) + 2).astype(np.int32), 0
    table = np.full((len(each), max(need + [width or 1]) + 1), -7, np.int32)
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    c = ref.Cache(len(order), heads, dim, page, rng)
    starts = np.concatenate([[0], np.cumsum(each)])
    x = [rng.standard_normal((starts[-1], heads, dim)) * np.exp(spread * rng.standard_normal((starts[-1], 1, 1))) for _ in "kv"]
    c.append(x[0], x[1], table, np.zeros(len(each), int), starts)
    own = table[1:, :max(need[1:] + [1]) + 1].copy()
    return c, table[0, :need[0] + 1].copy(), own, np.array(lens, np.int32)


def attend(q, c, prefix, prefix_len, table, lens, **more):
    return qwg.kv8_attend_shared(q, *pages(c), dev(prefix), dev(np.array([prefix_len], np.int32)), dev(table), dev(np.asarray(lens, np.int32)), **more)


def wide(prefix, q, c):
    """The table, with entries that are no pages behind the prefix's, as wide as it takes for many rows to be
    taken on large tiles (15 * 2^20 rows and positions): the launch goes by what a table may hold."""
    rows = q.numel() // q.shape[-1]
    return np.concatenate([prefix, np.full(-(-(15 << 20) // (rows * c.page)), -9, np.int32)])


LENS = [0, 1, 2, 15, 16, 17, 64, 130, 3]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,q_len,prefix", [
    (64, 16, 2, 8, 1, 300), (64, 128, 1, 1, 1, 65), (96, 32, 2, 3, 2, 257), (128, 64, 2, 4, 1, 640), (128, 16, 1, 16, 3, 1),
    (128, 32, 1, 8, 5, 1100), (192, 64, 1, 5, 1, 64), (256, 128, 1, 2, 4, 333), (256, 16, 2, 17, 1, 15), (64, 64, 3, 7, 7, 2000)])
def test_shared_matches(t, dim, page, kv, group, q_len, prefix):
    rng = np.random.default_rng(dim + page + group)
    c, pre, table, lens = filled(rng, prefix, LENS, kv, dim, page)
    q, qd = typed(rng.standard_normal((len(LENS), q_len, kv * group, dim)), t)
    out = attend(q, c, pre, prefix, table, lens)
    assert out.is_contiguous() and out.shape == q.shape
    want = layer_ref.shared(qd, c, pre, prefix, table, lens, dim ** -0.5)
    assert_shared(out, *want, t, prefix + max(LENS))
    assert torch.equal(out, attend(q, c, pre, prefix, table, lens))


# (rows per key/value head fill three quarters and more of tiles of 256, or not)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,seqs,q_len,prefix", [
    (64, 16, 1, 8, 30, 1, 5000), (128, 64, 2, 4, 60, 1, 3000), (128, 128, 1, 1, 250, 1, 1501), (96, 32, 1, 3, 70, 1, 2100),
    (64, 64, 1, 16, 31, 1, 700), (96, 16, 2, 2, 50, 2, 300), (128, 32, 1, 3, 33, 5, 64), (64, 128, 1, 5, 40, 1, 999),
    (192, 16, 1, 16, 20, 1, 900), (256, 64, 2, 2, 65, 1, 1025)])
def test_shared_by_many_sequences(t, dim, page, kv, group, seqs, q_len, prefix):
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 40, seqs)
    lens[seqs // 2] = 700
    c, pre, table, lens = filled(rng, prefix, lens, kv, dim, page, spread=0.3)
    q, qd = typed(rng.standard_normal((seqs, q_len, kv * group, dim)), t)
    want = layer_ref.shared(qd, c, pre, prefix, table, lens, dim ** -0.5)
    for width in (pre, wide(pre, q, c)):
        out = attend(q, c, width, prefix, table, lens)
        assert_shared(out, *want, t, prefix + 700)
        assert torch.equal(out, attend(q, c, width, prefix, table, lens))


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_shared_scales_on_large_tiles(t, scale):
    rng = np.random.default_rng(31)
    c, pre, table, lens = filled(rng, 500, [9] * 30, 1, 64, 16, spread=0.3)
    q, qd = typed(rng.standard_normal((30, 1, 8, 64)), t)
    out = attend(q, c, wide(pre, q, c), 500, table, lens, scale=scale)
    assert_shared(out, *layer_ref.shared(qd, c, pre, 500, table, lens, scale), t, 509)


@pytest.mark.parametrize("t", TYPES)
def test_shared_is_attention_over_the_whole(t):
    # a prefix of whole pages: the same as attention over tables that begin with them
    rng = np.random.default_rng(3)
    c, pre, table, lens = filled(rng, 640, [5, 100, 64, 1], 2, 128, 64)
    q, qd = typed(rng.standard_normal((4, 2, 8, 128)), t)
    out = attend(q, c, pre, 640, table, lens, scale=0.05)
    full = np.concatenate([np.repeat(pre[None, :10], 4, 0), table], 1)
    whole = qwg.kv8_attend(q, *pages(c), dev(full), dev(lens + 640), scale=0.05)
    assert_attend(whole, *ref.attend(qd, c, full, lens + 640, 0.05), t, 128)
    assert_shared(out, *layer_ref.shared(qd, c, pre, 640, table, lens, 0.05), t, 740)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("times", [1, 10])
def test_shared_prefixes_of_no_and_of_bad_length(t, times):
    rng = np.random.default_rng(4)
    c, pre, table, lens = filled(rng, 40, [20, 0, 33, 2] * times, 1, 64, 16)
    q, qd = typed(rng.standard_normal((4 * times, 3, 2, 64)), t)  # (240 rows are taken on a large tile)
    widths = [pre, wide(pre, q, c)]
    for n in (0, 1, 2, 40):
        want = layer_ref.shared(qd, c, pre, n, table, lens, 0.125)
        for width in widths:
            out = attend(q, c, width, n, table, lens)
            assert_shared(out, *want, t, 100)
            if n == 0:
                assert (out[1] == 0).all() and (out[3, 0] == 0).all()  # rows that see nothing
    for width in widths:
        for n in (-1, 16 * len(width) + 1):
            assert torch.isnan(attend(q, c, width, n, table, lens)).all()
        bad = lens.copy()
        bad[1:3] = [-1, 16 * table.shape[1] + 1]
        out = attend(q, c, width, 40, table, bad)
        assert torch.isnan(out[1:3]).all()
        keep = [0] + list(range(3, 4 * times))
        want = layer_ref.shared(qd, c, pre, 40, table, lens, 0.125)
        assert_shared(out[keep], *(w if np.ndim(w) == 0 else w[keep] for w in want), t, 100)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("seqs,tiled", [(3, False), (60, False), (60, True)])
def test_shared_bad_pages_and_nan_reach_the_rows_that_see_them(t, seqs, tiled):
    rng = np.random.default_rng(5)
    c, pre, table, lens = filled(rng, 100, [10] * seqs, 1, 64, 16)
    q, qd = typed(rng.standard_normal((seqs, 2, 2, 64)), t)

    def call(q=q, pre=pre, table=table):
        return attend(q, c, wide(pre, q, c) if tiled else pre, 100, table, lens)

    want = layer_ref.shared(qd, c, pre, 100, table, lens, 0.125)
    bad = table.copy()
    bad[1, 0] = 1 << 20  # one sequence's own page
    out = call(table=bad)
    assert torch.isnan(out[1]).all()
    keep = [s for s in range(seqs) if s != 1]
    assert_shared(out[keep], *(w if np.ndim(w) == 0 else w[keep] for w in want), t, 110)
    broken = pre.copy()
    broken[2] = -1
    assert torch.isnan(call(pre=broken)).all()
    # a NaN in the last position of the prefix: the rows of a sequence whose first query stands before it do not see it
    p, slot = pre[99 // 16], 99 % 16
    c.v[p, 0, 7, slot] = 0x7F
    lens[2] = 0  # two queries, none of them own: the first is at position 98, the second at 99
    nan = torch.isnan(call().cpu())
    assert not nan[2, 0].any() and nan[..., 7].sum() == nan.sum() == 2 * (2 * seqs - 1)
    # NaN codes behind the prefix's end, in the same page, are nobody's
    c.v[p, 0, 7, slot] = 0x30
    c.v[p, 0, :, slot + 1:], c.k[p, 0, slot + 1:] = 0x7F, 0x7F
    assert_shared(call(), *layer_ref.shared(qd, c, pre, 100, table, lens, 0.125), t, 110)
    # a NaN in one query
    q[0, 1, 1, 9] = float("nan")
    out = call().cpu()
    assert torch.isnan(out[0, 1, 1]).all() and torch.isnan(out).sum() == 64
    # scales that are none
    q[0, 1, 1, 9] = 0
    for scales in (c.ks, c.vs):
        kept, scales[pre[1], 0] = scales[pre[1], 0], 255
        assert torch.isnan(call()).all()
        scales[pre[1], 0] = kept
    assert not torch.isnan(call()).any()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("step", [12, 40])
@pytest.mark.parametrize("seqs", [2, 100])
def test_shared_pages_of_unlike_scales(t, step, seqs):
    # pages of V whose scales lie far apart, and a softmax that picks the small ones
    rng = np.random.default_rng(6)
    c, pre, table, lens = filled(rng, 256, [8] * seqs, 1, 64, 16, spread=0)
    c.vs[pre[:16], 0] = 120 + step * (np.arange(16) % 3 - 1)  # 2^-7 times a code, and far below and above
    at = 35  # (its page has the middle scale)
    q, qd = typed(np.repeat(ref.E4M3[c.k[pre[at // 16], 0, at % 16]][None, None] / 8, seqs, 0).repeat(2, 1), t)
    for scale in (0.05, 1.0, 4.0, 16.0):  # sharper and sharper
        want, weight, size, _ = layer_ref.shared(qd[:, None], c, pre, 256, table, lens, scale)
        # the weights' errors, those of fp16's smallest against the largest product of a row, and the type's own
        tol = (np.expm1(4 * 42 * 2.0 ** -24 * size) + 2.0 ** -11 + 2.0 ** -15) * weight + 2.0 ** -24 * 264 * weight.max(-1, keepdims=True)
        tol = tol + torch.finfo(t).eps / 2 * np.abs(want) + (2.0 ** -25 if t is torch.float16 else 0)
        for width in (pre, wide(pre, q, c)):
            got = attend(q, c, width, 256, table, lens, scale=scale).cpu().double().numpy().reshape(want.shape)
            big = np.abs(want) >= torch.finfo(t).max  # (an fp16 result of the largest scale is infinite)
            assert (np.abs(got - want)[~big] <= tol[~big]).all() and np.isinf(got[big]).all()


def test_shared_graphs_and_streams_do_not_share_a_workspace():
    rng = np.random.default_rng(11)
    c, pre, table, lens = filled(rng, 5000, [300, 1200], 2, 64, 16, spread=0.3)
    pre = np.concatenate([pre, np.full(100, -7, np.int32)])
    args = *pages(c), dev(pre), dev(np.array([5000], np.int32)), dev(table), dev(lens)
    qs = [typed(rng.standard_normal((2, 8, 64)), torch.bfloat16)[0] for _ in range(3)]
    want = [qwg.kv8_attend_shared(q, *args).clone() for q in qs]
    graphs, outs = [], []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qwg.kv8_attend_shared(q, *args))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        last = qwg.kv8_attend_shared(qs[2], *args)
        torch.cuda.synchronize()
        for o, w in zip(outs + [last], want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("t", TYPES)
def test_a_prompt_and_answers_to_it(t):
    """A layer's calls: a prompt through rotation and attention, then answers sampled behind it, token by token."""
    rng = np.random.default_rng(12)
    kv, group, dim, page, seqs, n = 2, 4, 64, 16, 3, 75
    heads, width, hidden = kv * group, (kv * group + 2 * kv) * dim, 128
    w, scales = qwg.encode_mxfp4(dev(0.1 * rng.standard_normal((width, hidden)).astype(np.float32)))
    freqs = frequencies(dim)
    cache = qwg.kv8_pages(5 + seqs * 2, kv, dim, page, device=DEV)
    order = rng.permutation(5 + seqs * 2).astype(np.int32)
    prefix, table = order[:5].copy(), order[5:].reshape(seqs, 2).copy()
    x = typed(rng.standard_normal((n, hidden)), t)[0]
    qkv = qwg.matmul_mxfp4(*qwg.encode_mxfp4(x), w, scales, dtype=t)
    q, k, v = (y.unflatten(1, (-1, dim)) for y in qkv.split([heads * dim, kv * dim, kv * dim], 1))
    qd, kd, vd = (y.cpu().double().numpy() for y in (q, k, v))
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    keys = torch.empty_like(k.contiguous())
    turned = qwg.kv8_append_rotary(q, k, v, dev(freqs), *cache, dev(prefix[None]), none, k_out=keys)
    positions = np.arange(n)
    assert_rotated(turned, qd, positions, freqs, False, t)
    assert_rotated(keys, kd, positions, freqs, False, t)
    out = qwg.prompt_attend(turned, keys, v)
    rd, rk = (y.cpu().double().numpy() for y in (turned, keys))
    assert_prompt(out, *layer_ref.prompt(rd, rk, vd, [0, n], dim ** -0.5), t, n, np.abs(vd).max())
    held = dev(np.array([n], np.int32))
    lens = torch.zeros(seqs, dtype=torch.int32, device=DEV)
    plain = ref.Cache(len(order), kv, dim, page)
    for step in range(20):
        qkv = qwg.gemm_mxfp4(w, scales, typed(rng.standard_normal((seqs, hidden)), t)[0])
        q, k, v = (y.unflatten(1, (-1, dim)) for y in qkv.split([heads * dim, kv * dim, kv * dim], 1))
        qd = q.cpu().double().numpy()
        turned = qwg.kv8_append_rotary(q, k, v, dev(freqs), *cache, dev(table), lens, prefix_len=held, out=q)
        assert_rotated(turned, qd, np.full(seqs, n + step), freqs, False, t)
        lens += 1
        out = qwg.kv8_attend_shared(turned, *cache, dev(prefix), held, dev(table), lens)
        plain.k, plain.ks, plain.v, plain.vs = (y.cpu().numpy() for y in cache)
        rd = turned.cpu().double().numpy()[:, None]
        assert_shared(out, *layer_ref.shared(rd, plain, prefix, n, table, [step + 1] * seqs, dim ** -0.5), t, n + step)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("own,tiled", [(30, False), (30, True), (6000, False)])
def test_shared_in_place(t, own, tiled):
    rng = np.random.default_rng(own)
    c, pre, table, lens = filled(rng, 400, [own] * 32, 1, 64, 128)
    q = typed(rng.standard_normal((32, 2, 4, 64)), t)[0]
    pre = wide(pre, q, c) if tiled else pre
    want = attend(q, c, pre, 400, table, lens)
    args = *pages(c), dev(pre), dev(np.array([400], np.int32)), dev(table), dev(lens)
    assert qwg.kv8_attend_shared(q, *args, out=q) is q and torch.equal(q, want)
    rows = torch.zeros(33, 2, 4, 64, dtype=t, device=DEV)
    with pytest.raises(qwg.QwgError):
        qwg.kv8_attend_shared(rows[:32], *args, out=rows[1:])


def test_shared_refusals():
    cache = qwg.kv8_pages(4, 2, 64, 16, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    pre, n, q = table[0].contiguous(), lens[:1], torch.zeros(2, 4, 64, device=DEV)

    def call(q=q, pre=pre, n=n, table=table, lens=lens, **more):
        return qwg.kv8_attend_shared(q, *cache, pre, n, table, lens, **more)

    for one in (lambda: call(q[:1]), lambda: call(q[:, :3]), lambda: call(q.cpu()), lambda: call(pre=pre.long()), lambda: call(pre=table),
                lambda: call(pre=pre[:0]), lambda: call(n=lens), lambda: call(n=5), lambda: call(lens=lens[:1]),
                lambda: call(table=table[0]), lambda: call(out=q[:1]), lambda: call(q.int()), lambda: call(q.transpose(1, 2))):
        with pytest.raises(ValueError):
            one()
    many = torch.zeros(65535, 32, 64, device=DEV, dtype=torch.float16)
    with pytest.raises(qwg.QwgError):  # more rows than a call takes
        call(many, table=torch.zeros(65535, 1, dtype=torch.int32, device=DEV), lens=torch.zeros(65535, dtype=torch.int32, device=DEV))
