"""A scale that is NaN makes every row that sees a position NaN, in all attention calls."""
import numpy as np
import pytest
import torch

import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import TYPES, dev, filled as filled_alone, pages, typed
from test_prompt_gpu import fused
from test_shared_gpu import attend, filled, wide

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 40), (256, 0)])
def test_prompt_under_a_scale_that_is_nan(t, dim, window):
    rng = np.random.default_rng(dim)
    (q, k, v), _ = fused(rng, 203, 4, 2, dim, t)
    out = torch.full(q.shape, 7.0, dtype=t, device=q.device)
    qwg.prompt_attend(q, k, v, starts=dev(np.array([0, 1, 1, 200], np.int32)), scale=NAN, window=window, out=out)
    assert torch.isnan(out[:200]).all() and (out[200:] == 7).all()


@pytest.mark.parametrize("t", TYPES)
def test_cache_attention_under_a_scale_that_is_nan(t):
    rng = np.random.default_rng(3)
    c, table = filled_alone(rng, [5, 0, 100], 1, 64, 16)
    q = typed(rng.standard_normal((3, 2, 64)), t)[0]
    out = qwg.kv8_attend(q, *pages(c), dev(table), dev(np.array([5, 0, 100], np.int32)), scale=NAN)
    assert torch.isnan(out[[0, 2]]).all() and (out[1] == 0).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("tiled", [False, True])
def test_shared_under_a_scale_that_is_nan(t, tiled):
    rng = np.random.default_rng(4)
    c, pre, table, lens = filled(rng, 100, [9, 0, 30, 1] * 15, 1, 64, 16)
    q = typed(rng.standard_normal((60, 1, 4, 64)), t)[0]
    pre = wide(pre, q, c) if tiled else pre
    assert torch.isnan(attend(q, c, pre, 100, table, lens, scale=NAN)).all()
