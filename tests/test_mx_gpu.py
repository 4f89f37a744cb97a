"""MXFP4 encoder, decoder and products against plain 64-bit implementations.

The encoder and the decoder are exact. A product's bound per output is 2e-6 sum |w x| (the library's
bound for a product in fp32 sums) plus half a step of the output type."""
import numpy as np
import pytest
import torch

import mx_ref as ref
import quantized_weight_decode_gemv_amd as qwg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def gen(seed):
    return np.random.default_rng(seed)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def typed(a, t):
    """(tensor of type t, its values in float64)"""
    x = torch.from_numpy(np.asarray(a, np.float32)).to(t)
    return x.to(DEV), x.double().numpy()


def weights(rng, n_out, n_in):
    codes = rng.integers(0, 256, (n_out, n_in // 2), dtype=np.uint8)
    scales = rng.integers(118, 130, (n_out, n_in // 32), dtype=np.uint8)
    return codes, scales, ref.decode_mxfp4(codes, scales)


def half_step(t):
    return 0.0 if t is torch.float64 else torch.finfo(t).eps / 2


def assert_product(y, w, x, t, what=""):
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    got = y.cpu().double().numpy()
    # the smallest step of the type too: fp16 results below 2^-14 are spaced 2^-24
    tol = 2e-6 * size * (1 + half_step(t)) + half_step(t) * np.abs(want) + float(torch.finfo(t).smallest_normal) * torch.finfo(t).eps / 2
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


# ---------------------------------------------------------------- encoder and decoder

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 32), (3, 96), (7, 2048), (65, 5632), (129, 65536)])
def test_encode_matches(t, rows, n):
    rng = gen(rows + n)
    x, v = typed(rng.standard_normal((rows, n)) * np.exp(rng.standard_normal((rows, 1))), t)
    codes, scales = qwg.encode_mxfp4(x)
    wc, ws = ref.encode_mxfp4(v)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(codes.cpu().numpy(), wc)
    back = qwg.dequant_mxfp4(codes, scales)
    assert np.array_equal(back.cpu().double().numpy(), ref.decode_mxfp4(wc, ws))


def test_encode_borders():
    # every tie and its neighbours, at scales from the smallest to the largest
    steps = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99])
    v = np.concatenate([steps, np.nextafter(np.float32(steps), np.float32(0)), np.nextafter(np.float32(steps), np.float32(9)), [0.0, 4.0]])
    assert v.size == 32
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -60, 0, 1, 60, 120, 124):
        rows.append(np.float32(np.ldexp(v, e)) * np.where(np.arange(32) % 3, 1, -1))
        rows.append(np.where(np.arange(32) == 5, np.float32(np.ldexp(1.0, e)), 0))
    rows.append(np.zeros(32))
    rows.append(-np.zeros(32))
    x, d = typed(np.stack(rows), torch.float32)
    codes, scales = qwg.encode_mxfp4(x)
    wc, ws = ref.encode_mxfp4(d)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(codes.cpu().numpy(), wc)
    back = qwg.dequant_mxfp4(codes, scales).cpu().double().numpy()
    assert np.array_equal(back, np.float32(ref.decode_mxfp4(wc, ws)).astype(np.float64))


@pytest.mark.parametrize("t", TYPES)
def test_encode_nan_and_infinity_spoil_their_block_alone(t):
    rng = gen(5)
    v = rng.standard_normal((4, 128))
    v[0, 40], v[1, 0], v[2, 127] = np.nan, np.inf, -np.inf
    x, d = typed(v, t)
    codes, scales = qwg.encode_mxfp4(x)
    wc, ws = ref.encode_mxfp4(d)
    assert np.array_equal(scales.cpu().numpy(), ws) and (ws == 255).sum() == 3
    assert np.array_equal(codes.cpu().numpy(), wc)
    back = qwg.dequant_mxfp4(codes, scales, dtype=t).cpu()
    assert int(torch.isnan(back).sum()) == 3 * 32


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("offset,gap", [(0, 64), (1, 0), (3, 5), (8, 8)])
def test_encode_rows_that_lie_apart(t, offset, gap):
    rng = gen(9)
    x, v = typed(rng.standard_normal((6, offset + 96 + gap)), t)
    codes, scales = qwg.encode_mxfp4(x[:, offset:offset + 96])
    wc, ws = ref.encode_mxfp4(v[:, offset:offset + 96])
    assert np.array_equal(codes.cpu().numpy(), wc) and np.array_equal(scales.cpu().numpy(), ws)


@pytest.mark.parametrize("t", TYPES)
def test_dequant_every_code_at_every_scale(t):
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1)).reshape(256, 256)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    got = qwg.dequant_mxfp4(dev(codes), dev(scales), dtype=t).cpu()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(np.float32(ref.decode_mxfp4(codes, scales))).to(t)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


def test_encode_more_blocks_than_one_grid():
    # 65,536 columns: 8192 lanes a row; 33,000 rows are more than one pass of the grid
    x = torch.randn(33000, 64, device=DEV).repeat(1, 1024)
    codes, scales = qwg.encode_mxfp4(x)
    small_c, small_s = qwg.encode_mxfp4(x[:, :64])
    assert torch.equal(codes.view(33000, 1024, 32), small_c[:, None].expand(-1, 1024, -1))
    assert torch.equal(scales.view(33000, 1024, 2), small_s[:, None].expand(-1, 1024, -1))


# ---------------------------------------------------------------- few rows

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("batch", [1, 2, 5, 6, 8, 11, 16])
@pytest.mark.parametrize("n_out,n_in", [(1, 32), (17, 96), (64, 512), (300, 544), (33, 2080)])
def test_gemm_matches(t, batch, n_out, n_in):
    rng = gen(1000 * batch + n_out)
    c, s, w = weights(rng, n_out, n_in)
    x, v = typed(rng.standard_normal((batch, n_in)), t)
    assert_product(qwg.gemm_mxfp4(dev(c), dev(s), x), w, v, t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("batch,n_out,n_in", [(1, 2048, 2048), (1, 32000, 2048), (3, 2048, 5632), (16, 5000, 8192),
                                              (1, 16, 65536), (16, 40, 65504), (1, 70000, 64)])
def test_gemm_larger(t, batch, n_out, n_in):
    rng = gen(n_out + n_in)
    c, s, w = weights(rng, n_out, n_in)
    x, v = typed(rng.standard_normal((batch, n_in)), t)
    assert_product(qwg.gemm_mxfp4(dev(c), dev(s), x), w, v, t)


def test_gemv_is_the_first_row_and_repeats():
    rng = gen(3)
    c, s, w = weights(rng, 777, 1056)
    x, v = typed(rng.standard_normal(1056), torch.float32)
    y = qwg.gemv_mxfp4(dev(c), dev(s), x)
    assert_product(y[None], w, v[None], torch.float32)
    assert torch.equal(y, qwg.gemv_mxfp4(dev(c), dev(s), x))
    assert torch.equal(y, qwg.gemm_mxfp4(dev(c), dev(s), x[None])[0])


@pytest.mark.parametrize("t", TYPES)
def test_gemm_scales_at_any_address_and_one_hot(t):
    rng = gen(4)
    c, s, w = weights(rng, 50, 256)
    flat = torch.zeros(s.size + 3, dtype=torch.uint8, device=DEV)
    odd = flat[3:].view(50, 8)
    odd.copy_(dev(s))
    assert odd.data_ptr() % 4
    for k in (0, 31, 32, 100, 255):
        x = torch.zeros(2, 256, dtype=t, device=DEV)
        x[1, k] = 1
        y = qwg.gemm_mxfp4(dev(c), odd, x).cpu().double().numpy()
        assert (y[0] == 0).all()
        assert np.array_equal(y[1], w[:, k])  # a weight is exact in every type here


def test_gemm_special_values():
    rng = gen(6)
    c, s, w = weights(rng, 40, 128)
    s[7, 2] = 255                      # a NaN block: its row alone
    c[9] = 0x22                        # a row of ones
    s[9] = 127
    x = rng.standard_normal((3, 128)).astype(np.float32)
    x[1, 5] = np.inf                   # an infinity stays one: its parts are (inf, 0, 0)
    x[2, 6] = np.nan
    y = qwg.gemm_mxfp4(dev(c), dev(s), dev(x)).cpu().numpy()
    assert np.isnan(y[:, 7]).all() and np.isfinite(np.delete(y[0], 7)).all()
    assert y[1, 9] == np.inf and np.isnan(y[2]).all()
    assert np.isfinite(y[0, 9])


def test_gemm_extreme_magnitudes():
    # weights from 2^-128 to 2^126, activations that bring the products back to 1: exact
    c = np.full((254, 16), 0x11, np.uint8)          # 1/2
    s = np.arange(254, dtype=np.uint8)[:, None]
    for e in (0, 1, 2, 20, 127, 200, 252):
        x = np.zeros((1, 32), np.float32)
        x[0, 3] = np.ldexp(1.0, min(127 - e + 1, 127))
        y = qwg.gemm_mxfp4(dev(c), dev(s), dev(x)).cpu().double().numpy()[0]
        assert y[e] == np.ldexp(0.5, e - 127) * float(x[0, 3])


# ---------------------------------------------------------------- many rows

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n_out,n_in", [(1, 1, 32), (1, 300, 96), (2, 17, 2048), (37, 129, 544), (128, 128, 512),
                                             (129, 257, 1056), (200, 64, 4096), (300, 520, 288)])
def test_matmul_matches(t, rows, n_out, n_in):
    rng = gen(rows * 7 + n_in)
    c, s, w = weights(rng, n_out, n_in)
    ac, asc, a = weights(rng, rows, n_in)
    y = qwg.matmul_mxfp4(dev(ac), dev(asc), dev(c), dev(s), dtype=t)
    assert y.shape == (rows, n_out) and y.dtype == t
    assert_product(y, w, a, t)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,n_out,n_in", [(509, 2048, 5632), (1025, 1030, 1024), (2048, 3000, 256), (16, 20000, 320), (3600, 3170, 96),
                                             (3, 64, 65536)])
def test_matmul_larger(t, rows, n_out, n_in):
    rng = gen(rows + n_out)
    c, s, w = weights(rng, n_out, n_in)
    ac, asc, a = weights(rng, rows, n_in)
    assert_product(qwg.matmul_mxfp4(dev(ac), dev(asc), dev(c), dev(s), dtype=t), w, a, t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,n_out,n_in", [(1, 5, 2080), (33, 31, 2304), (32, 256, 2048), (250, 1000, 2176), (257, 1000, 2176),
                                             (70, 90, 16416)])
def test_matmul_of_few_tiles_and_long_rows(t, rows, n_out, n_in):
    rng = gen(rows + n_in)
    c, s, w = weights(rng, n_out, n_in)
    ac, asc, a = weights(rng, rows, n_in)
    assert_product(qwg.matmul_mxfp4(dev(ac), dev(asc), dev(c), dev(s), dtype=t), w, a, t)
    # scales at an odd address, and a NaN block of each: its row and its column alone
    s[0, 63], asc[0, 1] = 255, 255
    odd = torch.zeros(s.size + 1, dtype=torch.uint8, device=DEV)[1:].view(s.shape)
    odd.copy_(dev(s))
    y = qwg.matmul_mxfp4(dev(ac), dev(asc), dev(c), odd, dtype=t)
    assert torch.isnan(y[0]).all() and torch.isnan(y[:, 0]).all()
    if rows > 1:
        assert_product(y[1:, 1:], w[1:], a[1:], t)


def test_matmul_nan_blocks_and_odd_scales():
    rng = gen(8)
    c, s, w = weights(rng, 70, 256)
    ac, asc, a = weights(rng, 40, 256)
    s[3, 1], asc[5, 7] = 255, 255
    odd = torch.zeros(s.size + 1, dtype=torch.uint8, device=DEV)[1:].view(s.shape)
    odd.copy_(dev(s))
    y = qwg.matmul_mxfp4(dev(ac), dev(asc), dev(c), odd, dtype=torch.float32).cpu().numpy()
    nan = np.zeros((40, 70), bool)
    nan[5], nan[:, 3] = True, True
    assert np.array_equal(np.isnan(y), nan)
    w[3], a[5] = 0, 0
    want, size = a @ w.T, np.abs(a) @ np.abs(w).T
    assert (np.abs(np.where(nan, 0, y) - want) <= 2e-6 * size).all()


# ---------------------------------------------------------------- together

def test_streams_graphs_and_a_step_together():
    """Encode, both products and their replays from two graphs on two streams, beside eager work."""
    rng = gen(10)
    c, s, w = weights(rng, 640, 512)
    wc, ws = dev(c), dev(s)
    xs = [torch.randn(33, 512, device=DEV, dtype=torch.bfloat16) for _ in range(2)]

    def step(x):
        a, b = qwg.encode_mxfp4(x)
        return qwg.matmul_mxfp4(a, b, wc, ws), qwg.gemm_mxfp4(wc, ws, x[:7])

    want = [[y.clone() for y in step(x)] for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            for y in o:
                y.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = step(xs[0])
        torch.cuda.synchronize()
        for o, e in zip(outs + [eager], want + [want[0]]):
            for y, z in zip(o, e):
                assert torch.equal(y, z)


def test_refusals():
    x = torch.zeros(2, 64, device=DEV)
    c, s = qwg.encode_mxfp4(x)
    bad = [
        lambda: qwg.encode_mxfp4(x[:, :48]), lambda: qwg.encode_mxfp4(x.double()), lambda: qwg.encode_mxfp4(x.t()),
        lambda: qwg.encode_mxfp4(x[:0]), lambda: qwg.encode_mxfp4(x[0]), lambda: qwg.encode_mxfp4(x[:1].expand(2, 64)),
        lambda: qwg.encode_mxfp4(x, codes=c[:1]), lambda: qwg.dequant_mxfp4(c, s[:, :1]),
        lambda: qwg.dequant_mxfp4(c, s, dtype=torch.float64), lambda: qwg.dequant_mxfp4(c.int(), s),
        lambda: qwg.gemm_mxfp4(c, s, torch.zeros(17, 64, device=DEV)), lambda: qwg.gemm_mxfp4(c, s, x[:, :32]),
        lambda: qwg.gemm_mxfp4(c, s, x.int()), lambda: qwg.gemm_mxfp4(c, s, x, out=x), lambda: qwg.gemm_mxfp4(c, s, x.cpu()),
        lambda: qwg.gemv_mxfp4(c, s, x), lambda: qwg.matmul_mxfp4(c, s, c[:, :16].contiguous(), s[:, :1].contiguous()),
        lambda: qwg.matmul_mxfp4(c, s, c, s, dtype=torch.int8), lambda: qwg.matmul_mxfp4(c, s, c, s.cpu()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
