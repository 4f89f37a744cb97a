"""How exact attention over the 8-bit cache is, on inputs that leave no other error to hide behind.

Keys and values are powers of two or small whole numbers, exact as codes, and scores are exact in fp32
sums, so that each test's tolerance holds the roundings that it names and nothing else."""
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


def cache_of(k, v, page):
    """One sequence's k and v [positions, dim], exact as codes of scale 1, in pages in reversed order."""
    n, dim = k.shape
    need = -(-n // page)
    c = ref.Cache(need, 1, dim, page, np.random.default_rng(n))
    c.ks[...], c.vs[...] = 127, 127
    table = np.arange(need, dtype=np.int32)[::-1][None].copy()
    for pos in range(n):
        c.k[table[0, pos // page], 0, pos % page] = ref.encode_e4m3(k[pos])
        c.v[table[0, pos // page], 0, :, pos % page] = ref.encode_e4m3(v[pos])
    got_k, got_v = c.rows(table, 0, n)
    assert np.array_equal(got_k[0], k) and np.array_equal(got_v[0], v)
    return (dev(c.k), dev(c.ks), dev(c.v), dev(c.vs)), dev(table), dev(np.array([n], np.int32))


def first_against_the_rest(q0, dim, page, n, key, first, rest, scale):
    """out of queries that are q0 in channel 0 over a position of `key` there and n of zero: the first
    has weight 1 and value `first`, the others weight exp(-scale q0 key) and value `rest`."""
    k, v = np.zeros((n + 1, dim)), np.full((n + 1, dim), float(rest))
    k[0, 0], v[0] = key, first
    q = torch.zeros(1, len(q0), dim, dtype=q0.dtype, device=DEV)
    q[0, :, 0] = q0
    pages, table, lens = cache_of(k, v, page)
    out = qwg.kv8_attend(q, *pages, table, lens, scale=scale)
    p = np.exp(-scale * key * q0.cpu().double().numpy())
    return out[0].cpu().double().numpy(), ((first + n * rest * p) / (1 + n * p))[:, None]


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 16), (64, 64, 48), (96, 32, 16), (128, 64, 16), (128, 16, 48), (192, 16, 16),
                                            (256, 128, 16), (256, 32, 40)])
def test_probabilities_of_the_16_bit_types_are_rounded_to_nearest(t, dim, page, heads):
    # 64 positions of weight p a little below 1 against one of weight 1 and the opposite value: the
    # output, 64 (p - 1) / (1 + 64 p), shows p's own error. p lies in [1/2, 1), where two roundings to 8 bits
    # leave 2^-18; exp2 leaves 2^-24, and 16 additions of up to 64 in fp32, over 65, 2^-20.
    # (Cut off to 16 bits p is off by up to 2^-16, by 2^-17 on average.)
    q0 = (1 + 3 * torch.rand(heads, generator=torch.Generator().manual_seed(dim + heads))).to(t).to(DEV)
    got, want = first_against_the_rest(q0, dim, page, 64, 64.0, -64.0, 1.0, 2.0 ** -18)
    tol = 2.0 ** -18 + 2.0 ** -24 + 2.0 ** -20 + torch.finfo(t).eps / 2 * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,heads,n,window,bad", [
    (64, 16, 2, 70, 8, [0, 1, 2]),       # before the window, in the block where it begins
    (128, 32, 20, 60, 3, [0]),
    (256, 16, 3, 70, 8, [1]),
    (64, 16, 2, 65, 0, [4]),             # a last page that the newest query alone sees
    (128, 64, 40, 129, 0, [2]),
    (96, 128, 1, 129, 100, [1]),
    (192, 16, 17, 33, 0, [2]),
    (64, 16, 4, 33, 16, [0, 2]),         # both
    (64, 16, 4, 32, 16, [0]),            # a page whose last position the older query alone sees
])
def test_a_nan_scale_reaches_the_rows_that_see_its_page(t, dim, page, heads, n, window, bad):
    rng = np.random.default_rng(n + dim)
    k, v = rng.integers(-4, 5, (2, n, dim)).astype(np.float64)
    pages, table, lens = cache_of(k, v, page)
    q = torch.from_numpy(rng.standard_normal((1, 2, heads, dim))).to(t).to(DEV)
    want = qwg.kv8_attend(q, *pages, table, lens, window=window)
    sees = []
    for r in range(2):
        last = n - 2 + r
        first = max(0, last - window + 1) if window else 0
        sees.append(any(p * page <= last and first < (p + 1) * page for p in bad))
    assert not all(sees)
    ids = table[0, torch.tensor(bad, device=DEV)].long()
    for which in (1, 3):  # K's scale, then V's
        spoiled = list(pages)
        spoiled[which] = pages[which].clone()
        spoiled[which][ids] = 255
        got = qwg.kv8_attend(q, *spoiled, table, lens, window=window)
        for r in range(2):
            assert bool(torch.isnan(got[0, r]).all()) if sees[r] else torch.equal(got[0, r], want[0, r]), (which, r)


def fp32_queries(low, high, heads, seed):
    """Queries whose significand ends in eight ones, spread over [low, high] when multiplied by 64 * 2^-6."""
    x = torch.linspace(low, high, heads, dtype=torch.float32) * (1 + 0.01 * torch.rand(heads, generator=torch.Generator().manual_seed(seed)))
    return (x.view(torch.int32) | 0xFF).view(torch.float32)


def fp32_tolerance(x):
    """Relative, of the output n p / (1 + n p) with p = exp(-x), in fp32: the score is exact, its product with
    the scale and log2 e is off by 1.5 u x (u = 2^-24), exp2 by 2 u, so numerator and denominator by
    3 u x + 4 u together; at most 12 u in the numerator's sums (6 instructions and the join), 8 u in the
    denominator's and 4 u in the division. In all (3 x + 28) u."""
    return (3 * x + 32) * 2.0 ** -24


@pytest.mark.parametrize("dim,page,heads", [(64, 16, 16), (64, 64, 48), (96, 32, 16), (96, 16, 40), (128, 64, 16), (128, 16, 48),
                                            (192, 16, 16), (192, 64, 48), (256, 128, 16), (256, 32, 40)])
@pytest.mark.parametrize("low,high", [(0.02, 1.0), (4.0, 9.0)])
def test_fp32_queries_and_probabilities_keep_all_their_bits(dim, page, heads, low, high):
    # near scores show a probability's own error, far ones (where n p is 1 or less) a query's: sixteen bits
    # of a probability are up to 2^-16 of it too small, sixteen of these queries 255 2^-24, x times that in p
    q0 = fp32_queries(low, high, heads, dim + heads)
    got, want = first_against_the_rest(q0.to(DEV), dim, page, 64, 64.0, 0.0, 1.0, 2.0 ** -6)
    tol = fp32_tolerance(q0.double().numpy())[:, None] * want
    assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()


@pytest.mark.parametrize("dim,page,heads", [(64, 16, 16), (128, 64, 48), (256, 32, 40)])
def test_fp16_queries_keep_all_their_bits(dim, page, heads):
    # eleven bits, the last three of them ones: eight would be 7 2^-10 off, x times that in p. The tolerance of
    # fp32, 2^-17 for a probability's own rounding (p may lie anywhere) and half a step of the output
    q0 = (torch.linspace(4.0, 9.0, heads).half().view(torch.int16) | 7).view(torch.float16)
    got, want = first_against_the_rest(q0.to(DEV), dim, page, 64, 64.0, 0.0, 1.0, 2.0 ** -6)
    tol = (fp32_tolerance(q0.double().numpy())[:, None] + 2.0 ** -17 + 2.0 ** -11) * want
    assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / tol).max()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,n", [(64, 16, 700), (96, 32, 3000), (128, 64, 3000), (192, 16, 1100), (256, 128, 3000)])
@pytest.mark.parametrize("steep", [7, 15])
def test_one_position_takes_all(t, dim, page, n, steep):
    # scores are whole multiples of 2^(steep - 3), the largest at least seven of them above every other: e^-112 and
    # less is 0 in fp32, so a row is the value of its position, exactly; of two with one score, their mean
    rng = np.random.default_rng(n + dim)
    k = rng.integers(-8, 9, (n, dim)).astype(np.float64)
    v = ref.E4M3[rng.integers(0, 127, (n, dim)) + 128 * rng.integers(0, 2, (n, dim))]
    # in the first and last positions of blocks of 64 and of splits; the last two heads have two winners
    at = [[0], [63], [64], [255], [256], [n // 2], [n - 1], [1, n - 2], [200, n // 2 + 1]]
    q = torch.zeros(1, len(at), dim, dtype=t, device=DEV)
    for h, where in enumerate(at):
        q[0, h, 7 * h] = 2.0 ** steep if h % 2 else -2.0 ** steep
        k[where, 7 * h] = 15 if h % 2 else -15
    pages, table, lens = cache_of(k, v, page)
    want = torch.from_numpy(np.stack([v[where].sum(0) / len(where) for where in at])).to(t)
    for most in (None, n):  # splits by the table and by the length
        got = qwg.kv8_attend(q, *pages, table, lens, scale=0.125, max_len=most)
        assert torch.equal(got[0].cpu(), want)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("scale", [0, 5, 12, 20])
def test_the_smallest_values(t, dim, page, scale):
    # a probability times its page's V scale loses what lies below 2^-133, in each of n positions: 2^-133 times
    # the sum of the codes' values at most, the largest probability being 1 before the division
    rng = np.random.default_rng(scale + dim)
    n = 3 * page + 5
    k, v = rng.integers(-4, 5, (n, dim)).astype(np.float64), rng.integers(1, 9, (n, dim)).astype(np.float64)
    pages, table, lens = cache_of(k, v, page)
    pages[3].fill_(scale)
    q = torch.from_numpy(rng.standard_normal((1, 8, dim))).to(t).to(DEV)
    got = qwg.kv8_attend(q, *pages, table, lens)[0].cpu().double().numpy()
    x = q[0].cpu().double().numpy() @ k.T * dim ** -0.5
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    small = 2.0 ** (scale - 127)
    want = p @ (v * small)
    # a score: 3 D/32 + 36 roundings of sum |q k|; a probability twice that, as does their sum; 2^-17 for a
    # probability's own rounding in the 16-bit types and 2^-17 for the sums, exp2 and the division
    size = (np.abs(q[0].cpu().double().numpy()) @ np.abs(k.T)).max(1, keepdims=True) * dim ** -0.5
    tol = (4 * (3 * dim / 32 + 36) * 2.0 ** -24 * size + 2.0 ** -16 + torch.finfo(t).eps / 2) * want + 2.0 ** -133 * v.sum(0) + 2.0 ** -133
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
