"""Prompt attention under scales of zero and below the normal fp32 numbers, where the products of queries and keys are large.

The bound is test_prompt_gpu's: the scale is held to 2^-149 where it is that small, which moves scores of 2^123 and less, as
here, by 2^-26."""
import numpy as np
import pytest
import torch

import layer_ref
import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import typed
from test_prompt_gpu import assert_prompt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -123, 2.0 ** -128, -2.0 ** -130, 2.0 ** -149])
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 60)])
def test_prompt_of_large_products_under_small_scales(t, scale, dim, window):
    rng = np.random.default_rng(dim)
    (q, qd), (k, kd) = (typed(2.0 ** 59 * np.clip(rng.standard_normal((150, n, dim)), -3, 3), t) for n in (4, 2))
    v, vd = typed(rng.standard_normal((150, 2, dim)), t)
    want = layer_ref.prompt(qd, kd, vd, [0, 150], scale, window)
    assert_prompt(qwg.prompt_attend(q, k, v, scale=scale, window=window), *want, t, 150, np.abs(vd).max())
