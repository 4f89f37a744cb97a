"""The MXFP4 encoder and decoder where a launch's workgroups take more than one turn: 2^20 of them hold
2^30 units of 16 bytes of values (the runs), 65,535 rows of them (rows that lie apart)."""
import pytest
import torch

import quantized_weight_decode_gemv_amd as qwg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("t,rows", [(torch.bfloat16, 131072), (torch.float32, 65536)])
def test_more_units_than_one_turn_of_the_grid(t, rows):
    # rows x 65536 values are 2^30 units; sixteen rows more take the second turn
    g = torch.Generator(device=DEV).manual_seed(rows)
    few = (torch.randn(16, 65536, device=DEV, generator=g) * torch.exp(torch.randn(16, 2048, device=DEV, generator=g)).repeat_interleave(32, 1)).to(t)
    want_codes, want_scales = qwg.encode_mxfp4(few)
    times = rows // 16 + 1
    x = few.repeat(times, 1)
    assert x.numel() * x.element_size() > 16 << 30
    codes, scales = qwg.encode_mxfp4(x)
    assert bool((codes.view(times, 16, -1) == want_codes).all()) and bool((scales.view(times, 16, -1) == want_scales).all())
    want = qwg.dequant_mxfp4(want_codes, want_scales, dtype=t)
    x.zero_()
    qwg.dequant_mxfp4(codes, scales, dtype=t, out=x)
    assert bool((x.view(times, 16, -1) == want).all())


@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("offset,gap", [(0, 64), (1, 7)])
def test_more_rows_that_lie_apart_than_one_turn_of_the_grid(t, offset, gap):
    rows, n = 65600, 64
    g = torch.Generator(device=DEV).manual_seed(gap)
    x = torch.randn(rows, offset + n + gap, device=DEV, generator=g).to(t)
    codes, scales = qwg.encode_mxfp4(x[:, offset:offset + n])
    want_codes, want_scales = qwg.encode_mxfp4(x[:, offset:offset + n].contiguous())
    assert torch.equal(codes, want_codes) and torch.equal(scales, want_scales)
