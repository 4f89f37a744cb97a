"""Rounding errors of the MXFP4 products where they add up most: long rows of terms of one sign that
repeat, so that every addition to a growing fp32 sum is rounded the same way.

With u = 2^-24 and n additions to one sum the error is at most n u sum |w x|. A wavefront of the product of few
rows adds at most 64 results of its matrix instructions to one sum, and 32 such sums, before up to 16
wavefronts' sums meet: 112 u (2e-6 for one row on such inputs, as documented). Several column tiles on
one row tile (more than 5 rows of fp32 or 8 of fp16, n_out of 4096 at most) keep one sum, as does the product
of two MXFP4 matrices, whose instructions take 128 terms each, so (16 + n_in/32) u and (16 + n_in/64) u, 16 for
what is rounded within an instruction and where sums meet."""
import pytest
import torch

import quantized_weight_decode_gemv_amd as qwg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
ROWS = 64  # distinct ones
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def repeated(g, n_in, spread, period):
    """[ROWS, n_in] positive weights that repeat after `period`, block scales over 2^spread, and their values."""
    c = (torch.randint(0, 256, (ROWS, period // 2), device=DEV, generator=g, dtype=torch.uint8) & 0x77) | 0x11
    s = (127 - torch.randint(0, spread + 1, (ROWS, period // 32), device=DEV, generator=g)).to(torch.uint8)
    codes, scales = c.repeat(1, n_in // period), s.repeat(1, n_in // period)
    v = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[torch.stack([codes & 7, codes >> 4], -1).flatten(1).long()]
    return codes, scales, v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


@pytest.mark.parametrize("n_in,n_out,batch,bound", [
    (14336, 32000, 1, 2e-6), (65536, 4096, 1, 2e-6), (65536, 32000, 1, 2e-6), (14336, 70016, 1, 2e-6),
    (14336, 70016, 5, 112 * U), (14336, 70016, 16, 112 * U), (65536, 8192, 16, 112 * U), (512, 4096, 16, 32 * U), (14336, 4096, 16, (16 + 14336 / 32) * U),
    (65536, 640, 11, (16 + 65536 / 32) * U)])
def test_gemm_terms_of_one_sign(n_in, n_out, batch, bound):
    g = torch.Generator(device=DEV).manual_seed(n_in + n_out + batch)
    for spread, period in ((0, 32), (3, 512), (12, 128)):
        c, s, w = repeated(g, n_in, spread, period)
        x = (torch.rand(batch, period, device=DEV, generator=g) + 0.5).repeat(1, n_in // period)
        y = qwg.gemm_mxfp4(c.repeat(n_out // ROWS, 1), s.repeat(n_out // ROWS, 1), x)
        want = x.double() @ w.T  # = sum |w x|
        for at in (0, n_out - ROWS):
            off = ((y[:, at:at + ROWS].double() - want).abs() / want).max()
            assert float(off) <= bound * (1 + U) + U, (spread, period, at, float(off))


@pytest.mark.parametrize("rows,n_out,n_in", [(64, 64, 65536), (192, 1024, 14336), (1024, 1024, 14336), (4096, 4096, 14336),
                                             (1024, 1024, 65536), (1024, 1024, 512), (640, 2048, 2048)])
def test_matmul_terms_of_one_sign(rows, n_out, n_in):
    g = torch.Generator(device=DEV).manual_seed(rows + n_in)
    for spread, period in ((8, 256), (14, 512), (20, 128)):
        c, s, w = repeated(g, n_in, spread, period)
        a, b, x = repeated(g, n_in, spread, period)
        y = qwg.matmul_mxfp4(a.repeat(rows // ROWS, 1), b.repeat(rows // ROWS, 1), c.repeat(n_out // ROWS, 1),
                             s.repeat(n_out // ROWS, 1), dtype=torch.float32)
        want = x @ w.T
        for i, j in ((0, 0), (rows - ROWS, n_out - ROWS)):
            off = ((y[i:i + ROWS, j:j + ROWS].double() - want).abs() / want).max()
            assert float(off) <= (16 + n_in / 64) * U + U, (spread, period, float(off))


@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
def test_views_that_start_between_16_bytes_are_refused(t):
    c, s = qwg.encode_mxfp4(torch.randn(4, 64, device=DEV))
    x = torch.zeros(72, device=DEV, dtype=t)
    odd = torch.zeros(4 * 32 + 1, device=DEV, dtype=torch.uint8)[1:].view(4, 32)
    cache = qwg.kv8_pages(2, 1, 64, 16, device=DEV)
    pages = torch.zeros(2 * 16 * 64 + 1, device=DEV, dtype=torch.uint8)[1:].view(2, 1, 16, 64)
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    k = torch.zeros(1, 1, 64, device=DEV, dtype=t)
    for call in (lambda: qwg.gemm_mxfp4(c, s, x[1:65].view(1, 64)), lambda: qwg.gemv_mxfp4(c, s, x[1:65]),
                 lambda: qwg.gemm_mxfp4(odd, s, x[:64].view(1, 64)), lambda: qwg.matmul_mxfp4(odd, s, c, s, dtype=t),
                 lambda: qwg.matmul_mxfp4(c, s, odd, s, dtype=t), lambda: qwg.dequant_mxfp4(odd, s, dtype=t),
                 lambda: qwg.dequant_mxfp4(c[:1], s[:1], dtype=t, out=x[1:65].view(1, 64)),
                 lambda: qwg.kv8_append(k, k, pages, *cache[1:], table, lens),
                 lambda: qwg.kv8_attend(k, pages, *cache[1:], table, lens)):
        with pytest.raises(qwg.QwgError):
            call()


@pytest.mark.parametrize("batch,n_out", [(1, 640), (7, 640), (16, 8192)])
@pytest.mark.parametrize("e", [-104, -110, -116, -122, -126, -131])
def test_gemm_smallest_fp32_activations(batch, n_out, e):
    # an activation's bits below 2^-133, the last of its three parts' smallest, are left out; the output's
    # own step, 2^-149, is finer than that of any term
    g = torch.Generator(device=DEV).manual_seed(batch - e)
    c, s, w = repeated(g, 1024, 3, 512)
    x = (1 + torch.rand(batch, 1024, device=DEV, generator=g)) * 2.0 ** e
    y = qwg.gemm_mxfp4(c.repeat(n_out // ROWS, 1), s.repeat(n_out // ROWS, 1), x)[:, :ROWS].double()
    want = x.double() @ w.T
    assert bool(((y - want).abs() <= (16 + 1024 / 32) * U * want + 2.0 ** -133 * w.sum(1) + 2.0 ** -149 * 32).all())
