"""The 8-bit key/value cache against plain 64-bit implementations.

Append is exact, bytes and exponents. Attention's bound per output: a score s = scale q.k carries
at most (3 D/32 + 36) 2^-24 scale sum |q k| (3 D/32 accumulations of 32 products each), a probability twice
that and some roundings of its own, so an output is off by at most

    (4 (3 D/32 + 36) 2^-24 scale sum |q k| + 2^-17 + (2^-15 for the 16-bit types)) sum p |v|

plus half a step of its type: 2^-17 covers 64 additions' roundings in the sums over positions, exp2 and
the division, 2^-15 the 16 bits of a probability that the 16-bit types keep."""
import numpy as np
import pytest
import torch

import mx_ref as ref
import quantized_weight_decode_gemv_amd as qwg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def typed(a, t):
    x = torch.from_numpy(np.asarray(a, np.float32)).to(t)
    return x.to(DEV), x.double().numpy()


def pages(c):
    return dev(c.k), dev(c.ks), dev(c.v), dev(c.vs)


def assert_pages(got, c, what=""):
    for name, g, w in zip(("k", "k scales", "v", "v scales"), got, (c.k, c.ks, c.v, c.vs)):
        g = g.cpu().numpy()
        if name in "kv":  # a NaN has two codes
            g, w = np.where(g == 255, 127, g), np.where(w == 255, 127, w)
        assert np.array_equal(g, w), f"{what} {name}: {np.argwhere(g != w)[:4].tolist()}"


def tables(rng, lens, page, spare=2, extra=1):
    """A page table whose pages lie in no order, entries past a sequence's own no pages at all."""
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(need) + extra), -7, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def filled(rng, lens, heads, dim, page, spread=1.0):
    """A cache holding lens positions of each sequence, stale bytes everywhere else."""
    table, n = tables(rng, lens, page)
    c = ref.Cache(n, heads, dim, page, rng)
    starts = np.concatenate([[0], np.cumsum(lens)])
    x = [rng.standard_normal((starts[-1], heads, dim)) * np.exp(spread * rng.standard_normal((starts[-1], 1, 1))) for _ in "kv"]
    c.append(x[0], x[1], table, np.zeros(len(lens), int), starts)
    return c, table


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 4), (96, 32, 1), (128, 64, 2), (192, 128, 3), (256, 16, 2)])
def test_append_matches(t, dim, page, heads):
    rng = np.random.default_rng(dim + page)
    held = [0, 1, page - 1, page, 5, 0, 3 * page + 2, 40]
    new = [1, 1, 1, 2 * page + 3, 0, page, 1, 200]
    total = [h + n for h, n in zip(held, new)]
    table, n_pages = tables(rng, total, page)
    c = ref.Cache(n_pages, heads, dim, page, rng)
    first = np.concatenate([[0], np.cumsum(held)])
    old = rng.standard_normal((2, first[-1], heads, dim))
    c.append(old[0], old[1], table, np.zeros(len(held), int), first)
    starts = np.concatenate([[0], np.cumsum(new)])
    # magnitudes up and down, so that some pages' scales rise and others' stay; two rows more than are used
    x = rng.standard_normal((2, starts[-1] + 2, heads, dim)) * np.exp(2 * rng.standard_normal((1, starts[-1] + 2, 1, 1)))
    (k, kd), (v, vd) = typed(x[0], t), typed(x[1], t)
    got = pages(c)
    before = [g.clone() for g in got]
    qwg.kv8_append(k, v, *got, dev(table), dev(np.array(held, np.int32)), starts=dev(starts.astype(np.int32)))
    c.append(kd, vd, table, held, starts)
    assert_pages(got, c)
    # the same with the launch sized for the longest, then for one token
    for most in (max(new), 1):
        again = [b.clone() for b in before]
        qwg.kv8_append(k, v, *again, dev(table), dev(np.array(held, np.int32)), starts=dev(starts.astype(np.int32)), max_new=most)
        for a, b in zip(again, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("t", TYPES)
def test_append_one_token_at_a_time_of_a_fused_result(t):
    rng = np.random.default_rng(3)
    heads, dim, page, seqs = 2, 64, 16, 3
    lens = np.array([0, 5, 14], np.int32)
    table, n_pages = tables(rng, lens + 20, page)
    c = ref.Cache(n_pages, heads, dim, page, rng)
    got = pages(c)
    c.append(np.zeros((19, heads, dim)) + 1, np.zeros((19, heads, dim)) + 1, table, np.zeros(3, int), [0, 0, 5, 19])
    got = pages(c)
    for step in range(20):
        qkv, d = typed(rng.standard_normal((seqs, 8 * dim)) * np.exp(rng.standard_normal()), t)
        q, k, v = qkv.split([4 * dim, heads * dim, heads * dim], dim=1)
        qwg.kv8_append(k.unflatten(1, (heads, dim)), v.unflatten(1, (heads, dim)), *got, dev(table), dev(lens))
        c.append(d[:, 4 * dim:6 * dim].reshape(seqs, heads, dim), d[:, 6 * dim:].reshape(seqs, heads, dim), table, lens, [0, 1, 2, 3])
        lens = lens + 1
    assert_pages(got, c)


def test_append_borders_and_special_values():
    rng = np.random.default_rng(4)
    heads, dim, page = 1, 64, 16
    # page maxima at and next to 1.75 2^e, ties of every size, subnormal and huge magnitudes
    tops = [np.ldexp(m, e) for e in (-149, -140, -127, -119, -118, -8, 0, 100, 127)
            for m in (1.0, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), 1.99) if np.ldexp(m, e) < 3.4e38]
    table = np.arange(len(tops) + 3, dtype=np.int32)[:, None]
    x = np.zeros((len(table), heads, dim))
    for i, top in enumerate(tops):
        step = np.arange(dim) / 128.0
        x[i, 0] = np.float32(top * step) * np.where(np.arange(dim) % 2, 1, -1)
        x[i, 0, 7] = np.float32(top)
    x[-3, 0, :4] = [np.nan, np.inf, -np.inf, 2.0]     # the other values keep their scale
    x[-2, 0, 0] = np.nan                              # all others zero
    c = ref.Cache(len(table), heads, dim, page, rng)
    got = pages(c)
    k, kd = typed(x, torch.float32)
    lens = np.zeros(len(table), np.int32)
    qwg.kv8_append(k, k, *got, dev(table), dev(lens))
    c.append(kd, kd, table, lens, np.arange(len(table) + 1))
    assert_pages(got, c)
    # a larger token later: every kept code is rounded to the page's new scale, subnormals and NaN among them
    y, yd = typed(x * np.array([1.0, 3.0, 300.0, 1e6])[np.arange(len(table)) % 4, None, None], torch.float32)
    qwg.kv8_append(y, y, *got, dev(table), dev(lens + 1))
    c.append(yd, yd, table, lens + 1, np.arange(len(table) + 1))
    assert_pages(got, c)


def test_append_leaves_out_what_has_no_page():
    rng = np.random.default_rng(5)
    heads, dim, page = 2, 64, 16
    table = np.array([[3, 99], [-1, 2], [4, 5], [0, 1]], np.int32)
    held, starts = np.array([10, 10, 30, -4], np.int32), np.array([0, 20, 40, 50, 60], np.int32)
    c = ref.Cache(6, heads, dim, page, np.random.default_rng(1))
    c.ks[...], c.vs[...] = 120, 120
    got = pages(c)
    k, kd = typed(rng.standard_normal((60, heads, dim)), torch.bfloat16)
    qwg.kv8_append(k, k, *got, dev(table), dev(held), starts=dev(starts))
    c.append(kd, kd, table, held, starts)
    assert_pages(got, c)


# ---------------------------------------------------------------- attend

def assert_attend(out, want, weight, size, t, dim):
    got = out.cpu().double().numpy().reshape(want.shape)
    tol = (4 * (3 * dim / 32 + 36) * 2.0 ** -24 * size + 2.0 ** -17 + (0 if t is torch.float32 else 2.0 ** -15)) * weight
    tol = tol + torch.finfo(t).eps / 2 * np.abs(want) + (2.0 ** -25 if t is torch.float16 else 0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 255, 257, 700]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,q_len,window", [
    (64, 16, 2, 8, 1, 0), (64, 128, 1, 1, 1, 0), (96, 32, 2, 3, 2, 0), (128, 64, 2, 4, 1, 0), (128, 16, 1, 16, 3, 0),
    (128, 32, 1, 8, 5, 20), (192, 64, 1, 5, 1, 0), (256, 128, 1, 2, 4, 1), (256, 16, 2, 17, 1, 300), (64, 64, 3, 7, 7, 64)])
def test_attend_matches(t, dim, page, kv, group, q_len, window):
    rng = np.random.default_rng(dim + page + group)
    c, table = filled(rng, LENS, kv, dim, page)
    q, qd = typed(rng.standard_normal((len(LENS), q_len, kv * group, dim)), t)
    lens = np.array(LENS, np.int32)
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens), window=window)
    want = ref.attend(qd, c, table, lens, dim ** -0.5, window)
    assert_attend(out, *want, t, dim)
    # another split of the positions: the same bound
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens), window=window, max_len=1)
    assert_attend(out, *want, t, dim)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,length", [(64, 16, 20011), (128, 64, 33000), (256, 32, 9001)])
def test_attend_long_and_split(t, dim, page, length):
    rng = np.random.default_rng(length)
    lens = [length, 77, length // 3]
    c, table = filled(rng, lens, 1, dim, page, spread=0.3)
    q, qd = typed(2 * rng.standard_normal((3, 2, 4, dim)), t)
    want = ref.attend(qd, c, table, lens, 0.3 * dim ** -0.5, 0)
    n = dev(np.array(lens, np.int32))
    out = qwg.kv8_attend(q, *pages(c), dev(table), n, scale=0.3 * dim ** -0.5)
    # 2^-17 covers 64 additions; a lane here adds at most length / 64 + 16 partial sums, with their errors in both signs
    assert_attend(out, want[0], want[1] * (1 + length / 64 / 64), want[2], t, dim)
    assert torch.equal(out, qwg.kv8_attend(q, *pages(c), dev(table), n, scale=0.3 * dim ** -0.5))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,q_len", [(64, 16, 1, 4, 1), (64, 32, 1, 17, 1), (96, 64, 1, 2, 9), (128, 16, 2, 4, 1),
                                                     (64, 32, 2, 17, 1), (96, 16, 2, 3, 1), (128, 128, 1, 5, 4), (192, 64, 1, 2, 1),
                                                     (192, 32, 1, 1, 17), (256, 16, 1, 3, 1)])
def test_attend_many_short_sequences(t, dim, page, kv, group, q_len):
    rng = np.random.default_rng(dim * group)
    lens = rng.integers(0, 300, 300).astype(np.int32)
    c, table = filled(rng, lens, kv, dim, page)
    q, qd = typed(rng.standard_normal((300, q_len, kv * group, dim)), t)
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens))
    assert_attend(out, *ref.attend(qd, c, table, lens, dim ** -0.5, 0), t, dim)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,window", [(64, 16, 512), (128, 64, 1000), (128, 128, 4097), (256, 32, 961), (96, 16, 2500)])
def test_attend_window_of_a_long_sequence(t, dim, page, window):
    rng = np.random.default_rng(window)
    lens = np.array([9001, 3, window, window + 62, 0, 4 * window - 1], np.int32)
    c, table = filled(rng, lens, 1, dim, page, spread=0.3)
    q, qd = typed(rng.standard_normal((len(lens), 3, 4, dim)), t)
    want = ref.attend(qd, c, table, lens, dim ** -0.5, window)
    for most in (None, 16):
        out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens), window=window, max_len=most)
        assert_attend(out, want[0], want[1] * (1 + window / 64 / 64), want[2], t, dim)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,kv,group,q_len", [(192, 1, 13, 3), (256, 2, 5, 8), (256, 1, 16, 5)])
def test_attend_many_rows_of_wide_heads(t, dim, kv, group, q_len):
    rng = np.random.default_rng(dim + group)
    lens = np.array([2600, 70, 1, 40000 // kv], np.int32)  # enough to take two tiles of rows at once
    c, table = filled(rng, lens, kv, dim, 32, spread=0.3)
    q, qd = typed(rng.standard_normal((len(lens), q_len, kv * group, dim)), t)
    want = ref.attend(qd, c, table, lens, dim ** -0.5, 0)
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens))
    assert_attend(out, want[0], want[1] * (1 + lens.max() / 64 / 64), want[2], t, dim)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [512, 513, 1008, 1024, 1025])
def test_attend_one_sequence_around_the_first_split(dim, length):
    rng = np.random.default_rng(dim + length)
    lens = np.array([length], np.int32)
    c, table = filled(rng, lens, 2, dim, 16)
    table = table[:, :-(-length // 16)]
    q, qd = typed(rng.standard_normal((1, 1, 6, dim)), torch.bfloat16)
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens))
    assert_attend(out, *ref.attend(qd, c, table, lens, dim ** -0.5, 0), torch.bfloat16, dim)


@pytest.mark.parametrize("t", TYPES)
def test_attend_nan_in_a_query_stays_in_its_row(t):
    rng = np.random.default_rng(12)
    lens = np.array([90, 5], np.int32)
    c, table = filled(rng, lens, 2, 64, 16)
    q, qd = typed(rng.standard_normal((2, 3, 8, 64)), t)
    want, weight, size = ref.attend(qd, c, table, lens, 0.125, 0)
    q[0, 1, 2, 7], q[1, 2, 5, 0] = float("nan"), float("inf")
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens))
    for at in ((0, 1, 2), (1, 2, 5)):
        assert torch.isnan(out[at]).all()
        out[at] = torch.from_numpy(want[at]).to(out)  # the others are as they were
    assert_attend(out, want, weight, size, t, 64)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("size", [30.0, 3000.0])
def test_attend_sharp_softmax_and_slices(t, size):
    # scores far apart: one position takes all, and the row maximum changes from block to block
    rng = np.random.default_rng(8)
    lens = np.array([513, 64], np.int32)
    c, table = filled(rng, lens, 2, 128, 64)
    qkv, d = typed(size * rng.standard_normal((2, 12 * 128)), t)
    out = qwg.kv8_attend(qkv[:, :8 * 128].unflatten(1, (8, 128)), *pages(c), dev(table), dev(lens))
    assert out.is_contiguous() and out.shape == (2, 8, 128)
    want, weight, s = ref.attend(d[:, None, :8 * 128].reshape(2, 1, 8, 128), c, table, lens, 128 ** -0.5)
    # where the winner is in doubt the bound is void: keep the outputs for which it says something
    tol = 4 * (3 * 4 + 36) * 2.0 ** -24 * s
    sure = (tol < 0.05)[..., 0]
    got = out.cpu().double().numpy().reshape(want.shape)
    assert sure.any() or size > 100
    full = (2 * np.expm1(tol) + 2.0 ** -14) * weight + torch.finfo(t).eps * np.abs(want)
    assert (np.abs(got - want) <= full)[sure].all() and np.isfinite(got).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("where", ["k", "v"])
def test_attend_nan_reaches_the_rows_that_see_it(t, where):
    rng = np.random.default_rng(9)
    lens = np.array([40, 100, 100], np.int32)
    c, table = filled(rng, lens, 1, 64, 16)
    bad_at = [38, 99, 60]  # seen by some queries, by the last alone, by all (or, in a window, by some)
    for s, pos in enumerate(bad_at):
        p = table[s, pos // 16]
        if where == "k":
            c.k[p, 0, pos % 16, 5] = 0x7F
        else:
            c.v[p, 0, 5, pos % 16] = 0xFF
    q, qd = typed(rng.standard_normal((3, 4, 2, 64)), t)
    for window in (0, 41):
        out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens), window=window).cpu()
        for s, pos in enumerate(bad_at):
            for row in range(4):
                last = lens[s] - 4 + row
                sees = pos <= last and (not window or pos > last - window)
                nan = torch.isnan(out[s, row])
                if where == "k":
                    assert bool(nan.all()) == sees and bool(nan.any()) == sees, (window, s, row)
                else:  # the channel alone
                    assert bool(nan[:, 5].all()) == sees and not nan[:, 6:].any() and not nan[:, :5].any(), (window, s, row)


@pytest.mark.parametrize("t", TYPES)
def test_attend_bad_pages_and_lengths_are_loud(t):
    rng = np.random.default_rng(10)
    lens = np.array([70, 70, 70, 70], np.int32)
    c, table = filled(rng, lens, 1, 64, 16)
    q, qd = typed(rng.standard_normal((4, 2, 2, 64)), t)
    want = ref.attend(qd, c, table, lens, 0.125, 8)
    table = table.copy()
    table[0, 0] = 1 << 20      # outside the window of 8: no row sees it
    table[1, 4] = -1           # positions 64 ..: every row's
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens), window=8)
    assert bool(torch.isnan(out[1]).all())
    keep = [0, 2, 3]
    assert_attend(out[keep], *(w[keep] for w in want), t, 64)
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens))
    assert bool(torch.isnan(out[:2]).all()) and not torch.isnan(out[2:]).any()
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(np.array([-1, 16 * table.shape[1] + 1, 70, 0], np.int32)))
    assert bool(torch.isnan(out[:2]).all()) and not torch.isnan(out[2:]).any() and (out[3] == 0).all()


def test_graphs_and_streams_do_not_share_a_workspace():
    rng = np.random.default_rng(11)
    lens = [9000, 5000]
    c, table = filled(rng, lens, 2, 64, 16, spread=0.3)
    got, tab, n = pages(c), dev(table), dev(np.array(lens, np.int32))
    qs = [typed(rng.standard_normal((2, 8, 64)), torch.bfloat16)[0] for _ in range(3)]
    want = [qwg.kv8_attend(q, *got, tab, n).clone() for q in qs]
    graphs, outs = [], []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qwg.kv8_attend(q, *got, tab, n))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        last = qwg.kv8_attend(qs[2], *got, tab, n)
        torch.cuda.synchronize()
        for o, w in zip(outs + [last], want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("t", TYPES)
def test_decode_steps_with_microscaled_projections(t):
    """q|k|v product, append, attention and o product of a few decoding steps, as a program runs them."""
    rng = np.random.default_rng(12)
    hidden, kv, group, dim, page, seqs = 256, 2, 4, 64, 16, 3
    wide = (kv * group + 2 * kv) * dim
    w_qkv, s_qkv = qwg.encode_mxfp4(dev(0.1 * rng.standard_normal((wide, hidden)).astype(np.float32)))
    w_o, s_o = qwg.encode_mxfp4(dev(0.1 * rng.standard_normal((hidden, kv * group * dim)).astype(np.float32)))
    qkv_w = ref.decode_mxfp4(w_qkv.cpu().numpy(), s_qkv.cpu().numpy())
    o_w = ref.decode_mxfp4(w_o.cpu().numpy(), s_o.cpu().numpy())
    lens = np.zeros(seqs, np.int32)
    table, n_pages = tables(rng, [64] * seqs, page)
    cache = qwg.kv8_pages(n_pages, kv, dim, page, device=DEV)
    plain = ref.Cache(n_pages, kv, dim, page)
    tab = dev(table)
    for new in (21, 1, 1, 1):  # a prompt, then single tokens
        x, xd = typed(rng.standard_normal((seqs * new, hidden)), t)
        if new > 1:
            a, b = qwg.encode_mxfp4(x)
            qkv = qwg.matmul_mxfp4(a, b, w_qkv, s_qkv, dtype=t)
            xd = ref.decode_mxfp4(*ref.encode_mxfp4(xd))
        else:
            qkv = qwg.gemm_mxfp4(w_qkv, s_qkv, x)
        want = xd @ qkv_w.T
        assert (np.abs(qkv.cpu().double().numpy() - want) <= 2e-6 * (np.abs(xd) @ np.abs(qkv_w).T) + torch.finfo(t).eps / 2 * np.abs(want) * 1.01).all()
        q, k, v = qkv.view(seqs, new, -1).split([kv * group * dim, kv * dim, kv * dim], dim=2)
        k, v, q = (y.unflatten(2, (-1, dim)) for y in (k, v, q))
        qwg.kv8_append(k, v, *cache, tab, dev(lens))
        kd, vd, qd = (y.cpu().double().numpy() for y in (k, v, q))
        plain.append(kd.reshape(-1, kv, dim), vd.reshape(-1, kv, dim), table, lens, np.arange(seqs + 1) * new)
        assert_pages(cache, plain)
        lens = lens + new
        out = qwg.kv8_attend(q, *cache, tab, dev(lens))
        assert_attend(out, *ref.attend(qd, plain, table, lens, dim ** -0.5), t, dim)
        if new == 1:
            y = qwg.gemm_mxfp4(w_o, s_o, out.flatten(1))
            od = out.flatten(1).cpu().double().numpy()
            want = od @ o_w.T
            assert (np.abs(y.cpu().double().numpy() - want) <= 2e-6 * (np.abs(od) @ np.abs(o_w).T) + torch.finfo(t).eps / 2 * np.abs(want) * 1.01).all()


def test_refusals():
    cache = qwg.kv8_pages(4, 2, 64, 16, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    k = torch.zeros(2, 2, 64, device=DEV)
    q = torch.zeros(2, 4, 64, device=DEV)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    other = (cache[0], cache[1], cache[2][:, :, :32].contiguous(), cache[3])
    bad = [
        lambda: qwg.kv8_append(k, k.half(), *cache, table, lens), lambda: qwg.kv8_append(k[:1], k, *cache, table, lens),
        lambda: qwg.kv8_append(k[:1], k[:1], *cache, table, lens), lambda: qwg.kv8_append(k[:, :1], k[:, :1], *cache, table, lens),
        lambda: qwg.kv8_append(k, k, *cache, table.long(), lens), lambda: qwg.kv8_append(k, k, *cache, table, lens[:1]),
        lambda: qwg.kv8_append(k, k, *cache, table, lens, starts=starts[:2]), lambda: qwg.kv8_append(k, k, *other, table, lens),
        lambda: qwg.kv8_append(k, k, *cache, table, lens, starts=starts, max_new=0),
        lambda: qwg.kv8_append(k[:1].expand(2, 2, 64), k, *cache, table, lens), lambda: qwg.kv8_append(k.int(), k.int(), *cache, table, lens),
        lambda: qwg.kv8_attend(q[:1], *cache, table, lens), lambda: qwg.kv8_attend(q[:, :3], *cache, table, lens),
        lambda: qwg.kv8_attend(q, *cache, table, lens, window=-1), lambda: qwg.kv8_attend(q, *cache, table, lens, out=q[:1]),
        lambda: qwg.kv8_attend(q.transpose(1, 2), *cache, table, lens), lambda: qwg.kv8_attend(q.cpu(), *cache, table, lens),
        lambda: qwg.kv8_attend(q, *other, table, lens), lambda: qwg.kv8_pages(4, 2, 80, 16), lambda: qwg.kv8_pages(4, 2, 64, 8),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shift,gap", [(1, 0), (0, 3), (8, 8)])
def test_values_at_any_address(t, shift, gap):
    # keys, values and queries that start on their type's alignment alone, tokens at an odd distance
    rng = np.random.default_rng(13)
    heads, dim, page = 2, 96, 32
    lens, new = np.array([3, 40], np.int32), 37
    table, n_pages = tables(rng, lens + new, page)
    c = ref.Cache(n_pages, heads, dim, page, rng)
    c.append(rng.standard_normal((43, heads, dim)), rng.standard_normal((43, heads, dim)), table, np.zeros(2, int), [0, 3, 43])
    got = pages(c)
    width = heads * dim
    flat, d = typed(rng.standard_normal(2 * new * (width + gap) + shift), t)
    x = flat[shift:].view(2 * new, width + gap)[:, :width].unflatten(1, (heads, dim))
    xd = d[shift:].reshape(2 * new, width + gap)[:, :width].reshape(-1, heads, dim)
    qwg.kv8_append(x, x, *got, dev(table), dev(lens))
    c.append(xd, xd, table, lens, [0, new, 2 * new])
    assert_pages(got, c)
    q, qd = x[:4].unflatten(0, (2, 2)), xd[:4].reshape(2, 2, heads, dim)
    assert_attend(qwg.kv8_attend(q, *got, dev(table), dev(lens + new)), *ref.attend(qd, c, table, lens + new, dim ** -0.5), t, dim)
