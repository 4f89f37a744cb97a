"""Attention over prompts against plain 64-bit implementations.

A score is a sum of D products: in fp32 off by at most (D + 4) 2^-24 of scale sum |q k|; a probability by twice that, by
the rounding of its exponent (below 150, so 2^-16.7 of it) and exp2's; the sums over n positions by n 2^-24 each; so an
output by (4 (D + 4) 2^-24 size + 2 n 2^-24 + 2^-15 + P) sum p |v|, P being the rounding of a probability to the type (half
a step: 2^-8, 2^-11, none), and half a step of the type. An fp16 probability below 2^-14 is off by up to 2^-25 of the
largest. Over many outputs the two roundings add up as independent errors of at most half a step, evenly spread:
sqrt(2/3) of half a step in the 2-norm."""
import numpy as np
import pytest
import torch

import layer_ref
import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import TYPES, dev, typed

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def assert_prompt(out, want, weight, size, t, n, v_top):
    dim = want.shape[-1]
    got = out.cpu().double().numpy().reshape(want.shape)
    half = torch.finfo(t).eps / 2
    p = 0 if t is torch.float32 else half
    tol = (4 * (dim + 4) * 2.0 ** -24 * size + 2 * n * 2.0 ** -24 + 2.0 ** -15 + p) * weight + half * np.abs(want)
    if t is torch.float16:
        tol = tol + 2.0 ** -25 * (1 + n * v_top)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"
    if t is not torch.float32 and want.size > 20000:
        assert np.linalg.norm(got - want) <= (2 / 3) ** 0.5 * half * np.linalg.norm(want)


def fused(rng, tokens, heads, kv, dim, t, gap=0, shift=0):
    width = (heads + 2 * kv) * dim
    flat, d = typed(rng.standard_normal(tokens * (width + gap) + shift), t)
    x, xd = flat[shift:].view(tokens, width + gap)[:, :width], d[shift:].reshape(tokens, width + gap)[:, :width]
    cut = [heads * dim, kv * dim, kv * dim]
    return ([y.unflatten(1, (-1, dim)) for y in x.split(cut, 1)],
            [y.reshape(tokens, -1, dim) for y in np.split(xd, np.cumsum(cut)[:-1], 1)])


LENS = [0, 1, 2, 31, 32, 33, 0, 63, 64, 65, 130, 257]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,kv,group,window", [
    (64, 2, 8, 0), (64, 1, 1, 0), (64, 1, 32, 50), (96, 2, 3, 0), (96, 1, 5, 33), (128, 2, 4, 0), (128, 1, 1, 1),
    (128, 1, 16, 64), (192, 1, 5, 0), (192, 2, 1, 100), (256, 2, 2, 0), (256, 1, 7, 20)])
def test_prompt_matches(t, dim, kv, group, window):
    rng = np.random.default_rng(dim + group + window)
    starts = np.concatenate([[0], np.cumsum(LENS)]).astype(np.int32)
    (q, k, v), (qd, kd, vd) = fused(rng, starts[-1] + 3, kv * group, kv, dim, t)  # three rows more than are used
    mark = torch.full(q.shape, 7.0, dtype=t, device=DEV)
    want, weight, size = layer_ref.prompt(qd, kd, vd, starts, dim ** -0.5, window)
    for most in (None, 1, max(LENS)):
        out = qwg.prompt_attend(q, k, v, starts=dev(starts), window=window, out=mark, max_len=most)
        assert out is mark and (out[-3:] == 7).all()
        assert_prompt(out[:-3], want[:-3], weight[:-3], size[:-3], t, max(LENS), np.abs(vd).max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,heads,kv,length,window", [(64, 4, 1, 1301, 0), (128, 2, 1, 1111, 0), (256, 1, 1, 900, 0), (128, 4, 2, 1500, 200),
                                                        (64, 1, 1, 2500, 1000), (96, 3, 3, 700, 0), (192, 2, 2, 700, 128)])
def test_prompt_of_one_long_sequence(t, dim, heads, kv, length, window):
    rng = np.random.default_rng(length)
    (q, k, v), (qd, kd, vd) = fused(rng, length, heads, kv, dim, t)
    out = qwg.prompt_attend(2 * q, k, v, window=window, scale=0.4 * dim ** -0.5)
    assert out.is_contiguous() and out.shape == q.shape
    want = layer_ref.prompt(2 * qd, kd, vd, [0, length], 0.4 * dim ** -0.5, window)
    assert_prompt(out, *want, t, length, np.abs(vd).max())
    assert torch.equal(out, qwg.prompt_attend(2 * q, k, v, window=window, scale=0.4 * dim ** -0.5))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,seqs,length", [(64, 300, 9), (128, 70, 40), (96, 130, 1), (256, 65, 3)])
def test_prompt_of_many_short_sequences(t, dim, seqs, length):
    # as many tokens each: four dimensions, no starts
    rng = np.random.default_rng(seqs)
    (q, k, v), (qd, kd, vd) = fused(rng, seqs * length, 6, 2, dim, t)
    out = qwg.prompt_attend(*(x.unflatten(0, (seqs, length)) for x in (q, k, v)))
    assert out.shape == (seqs, length, 6, dim)
    want = layer_ref.prompt(qd, kd, vd, np.arange(seqs + 1) * length, dim ** -0.5)
    assert_prompt(out, *want, t, length, np.abs(vd).max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shift,gap", [(1, 0), (0, 3), (8, 8)])
def test_prompt_values_at_any_address(t, shift, gap):
    rng = np.random.default_rng(13)
    (q, k, v), (qd, kd, vd) = fused(rng, 150, 4, 2, 96, t, gap, shift)
    starts = np.array([0, 61, 150], np.int32)
    want = layer_ref.prompt(qd, kd, vd, starts, 96 ** -0.5)
    assert_prompt(qwg.prompt_attend(q, k, v, starts=dev(starts)), *want, t, 89, np.abs(vd).max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("size", [30.0, 3000.0])
def test_prompt_sharp_softmax(t, size):
    # scores far apart: one position takes all, and the row maximum changes from block to block
    rng = np.random.default_rng(8)
    (q, k, v), (qd, kd, vd) = fused(rng, 400, 4, 2, 128, t)
    q, qd = typed(size * qd, t)
    out = qwg.prompt_attend(q, k, v)
    want, weight, s = layer_ref.prompt(qd, kd, vd, [0, 400], 128 ** -0.5)
    tol = 4 * 132 * 2.0 ** -24 * s  # where the winner is in doubt the bound is void
    sure = (tol < 0.05)[..., 0]
    got = out.cpu().double().numpy()
    assert sure.any() or size > 100
    full = (2 * np.expm1(tol) + 2.0 ** -13 + torch.finfo(t).eps) * weight + torch.finfo(t).eps * np.abs(want) + 2.0 ** -20
    assert (np.abs(got - want) <= full)[sure].all() and np.isfinite(got).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30])
def test_prompt_scales(t, scale):
    rng = np.random.default_rng(9)
    (q, k, v), (qd, kd, vd) = fused(rng, 200, 4, 2, 64, t)
    for window in (0, 70):
        want = layer_ref.prompt(qd, kd, vd, [0, 200], scale, window)
        assert_prompt(qwg.prompt_attend(q, k, v, scale=scale, window=window), *want, t, 200, np.abs(vd).max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,group,window", [(64, 2, 0), (64, 2, 41), (128, 8, 0), (96, 1, 90), (256, 3, 0)])
def test_prompt_what_is_not_finite_reaches_the_rows_that_see_it(t, dim, group, window):
    rng = np.random.default_rng(dim + window)
    starts = np.array([0, 200, 330], np.int32)
    (q, k, v), (qd, kd, vd) = fused(rng, 330, group, 1, dim, t)
    # in the values of one channel each; the first and last tokens of neighbouring sequences among them
    marks = [(0, 3, "nan"), (77, 5, "inf"), (130, 6, "-inf"), (199, 7, "nan"), (200, 8, "inf"), (329, 9, "-inf"), (140, 6, "inf")]
    for at, c, x in marks:
        v[at, 0, c] = float(x)
    out = qwg.prompt_attend(q, k, v, starts=dev(starts), window=window).cpu().double().numpy()
    clean = vd.copy()
    for at, c, _ in marks:
        clean[at, 0, c] = 0
    want, weight, size = layer_ref.prompt(qd, kd, clean, starts, dim ** -0.5, window)
    for at, c, x in marks:
        b, e = (0, 200) if at < 200 else (200, 330)
        stop = min(e, at + window) if window else e
        want[at:stop, :, c] += float(x)  # infinities of both signs are none
    assert np.array_equal(np.isnan(out), np.isnan(want)) and np.array_equal(np.isinf(out), np.isinf(want))
    assert np.array_equal(out[np.isinf(out)], want[np.isinf(out)])
    fine = np.isfinite(want)
    got = torch.from_numpy(np.where(fine, out, 0))
    assert_prompt(got, np.where(fine, want, 0), weight, size, t, 200, np.abs(clean).max())
    # in a key and in a query: the rows that see it, and the one row
    k[150, 0, 1], q[20, 0, 2] = float("nan"), float("inf")
    v.copy_(torch.from_numpy(clean))
    out = qwg.prompt_attend(q, k, v, starts=dev(starts), window=window).cpu()
    nan = torch.isnan(out).all(-1)
    assert torch.equal(nan, torch.isnan(out).any(-1))
    sees = np.zeros(nan.shape, bool)
    sees[150:min(200, 150 + window) if window else 200] = True
    sees[20, 0] = True
    assert np.array_equal(nan.numpy(), sees)


@pytest.mark.parametrize("t", TYPES)
def test_prompt_on_other_streams_and_in_graphs(t):
    rng = np.random.default_rng(11)
    (q, k, v), _ = fused(rng, 500, 8, 2, 64, t)
    starts = dev(np.array([0, 180, 500], np.int32))
    want = qwg.prompt_attend(q, k, v, starts=starts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qwg.prompt_attend(q, k, v, starts=starts)
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = qwg.prompt_attend(q, k, v, starts=starts)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)


def test_prompt_starts_that_are_none():
    # starts out of order or out of range: no more than the tokens there are is read or written
    rng = np.random.default_rng(12)
    (q, k, v), (qd, kd, vd) = fused(rng, 100, 2, 1, 64, torch.float32)
    out = torch.full(q.shape, 7.0, device=DEV)
    qwg.prompt_attend(q, k, v, starts=dev(np.array([-5, 40, 40, 30, 1000], np.int32)), out=out)
    want = layer_ref.prompt(qd, kd, vd, [0, 40], 0.125)
    assert_prompt(out[:30], *(w[:30] for w in want), torch.float32, 40, np.abs(vd).max())


@pytest.mark.parametrize("long", [0, 7, 8, 511, 512, 1023, 1301])
def test_prompt_among_many_sequences(long):
    # short and empty ones, one of several tiles, the last ones empty
    rng = np.random.default_rng(long)
    lens = rng.integers(0, 3, 1400)
    lens[1310:], lens[long] = 0, 150
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = int(starts[-1])
    (q, k, v), (qd, kd, vd) = fused(rng, n, 2, 1, 64, torch.float16)
    out = qwg.prompt_attend(q, k, v, starts=dev(starts))
    assert_prompt(out, *layer_ref.prompt(qd, kd, vd, starts, 0.125), torch.float16, 150, np.abs(vd).max())


@pytest.mark.parametrize("seqs,each", [(700, 1), (70, 65), (3, 130), (1, 33)])
def test_prompt_of_equal_lengths(seqs, each):
    rng = np.random.default_rng(seqs)
    (q, k, v), (qd, kd, vd) = fused(rng, seqs * each, 6, 2, 64, torch.bfloat16)
    parts = (x.unflatten(0, (seqs, each)) for x in (q, k, v))
    out = qwg.prompt_attend(*parts)
    want = layer_ref.prompt(qd, kd, vd, np.arange(seqs + 1) * each, 0.125)
    assert_prompt(out.flatten(0, 1), *want, torch.bfloat16, each, np.abs(vd).max())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim", [64, 192])
def test_prompt_in_place(t, dim):
    rng = np.random.default_rng(dim)
    q, k, v = (typed(rng.standard_normal((300, heads, dim)), t)[0] for heads in (6, 2, 2))
    want = qwg.prompt_attend(q, k, v, window=100)
    assert qwg.prompt_attend(q, k, v, window=100, out=q) is q and torch.equal(q, want)
    rows = torch.zeros(301, 2, dim, dtype=t, device=DEV)
    for bad in (lambda: qwg.prompt_attend(rows[:300], k, v, out=rows[1:]), lambda: qwg.prompt_attend(k, rows[1:], v, out=rows[:300]),
                lambda: qwg.prompt_attend(k, k, rows[:300], out=rows[:300])):
        with pytest.raises(qwg.QwgError):
            bad()


def test_prompt_refusals():
    q, k = torch.zeros(6, 4, 64, device=DEV), torch.zeros(6, 2, 64, device=DEV)
    starts = torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV)
    bad = [lambda: qwg.prompt_attend(q, k, k.half()), lambda: qwg.prompt_attend(q, k[:5], k[:5]), lambda: qwg.prompt_attend(q[:, :3], k, k),
           lambda: qwg.prompt_attend(q, k, k[:, :1]), lambda: qwg.prompt_attend(q.cpu(), k, k), lambda: qwg.prompt_attend(q, k, k, starts=starts.long()),
           lambda: qwg.prompt_attend(q, k, k, starts=starts[:1]), lambda: qwg.prompt_attend(q, k, k, window=-1),
           lambda: qwg.prompt_attend(q, k, k, max_len=-1), lambda: qwg.prompt_attend(q, k, k, out=q[:3]),
           lambda: qwg.prompt_attend(q.int(), k.int(), k.int()), lambda: qwg.prompt_attend(q[..., :32], k[..., :32], k[..., :32]),
           lambda: qwg.prompt_attend(q[:0], k[:0], k[:0]), lambda: qwg.prompt_attend(q[:1].expand(6, 4, 64), k, k),
           lambda: qwg.prompt_attend(q[0], k[0], k[0]), lambda: qwg.prompt_attend(q[:, :, ::2], k[:, :, ::2], k[:, :, ::2])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
