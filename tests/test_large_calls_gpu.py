"""Rotation, prompts and shared prefixes at sizes whose offsets pass 32 bits, and at the largest number of rows."""
import numpy as np
import pytest
import torch

import layer_ref
import mx_ref as ref
import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import dev, typed
from test_prompt_gpu import assert_prompt
from test_rotary_gpu import assert_keys, assert_rotated, frequencies
from test_shared_gpu import assert_shared, attend, filled, wide

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def doubles(x):
    return x.cpu().double().numpy()


def test_two_to_the_thirty_second_query_values():
    # 16,384 sequences of 128 and 129 tokens: rotated in place, appended, attended over
    seqs, heads, dim, page, t = 1 << 14, 32, 64, 128, torch.float16
    each = np.full(seqs, 128, np.int32)
    each[1::2] = 129
    starts = np.concatenate([[0], np.cumsum(each)]).astype(np.int32)
    n = int(starts[-1])
    assert n * heads * dim > 1 << 32
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    q, k, v = (torch.randn(n, h, dim, dtype=t, device=DEV, generator=g) for h in (heads, 1, 1))
    cache = qwg.kv8_pages(2 * seqs, 1, dim, page, device=DEV)
    table = torch.arange(2 * seqs, dtype=torch.int32, device=DEV).flip(0).view(seqs, 2).contiguous()
    lens = torch.full((seqs,), 5, dtype=torch.int32, device=DEV)
    cache[1].fill_(100), cache[3].fill_(100)
    keys, freqs = torch.empty_like(k), frequencies(dim)
    looked_at = [0, 1, seqs // 2 + 1, seqs - 2, seqs - 1]
    before = {s: doubles(q[starts[s]:starts[s + 1]]) for s in looked_at}
    out = qwg.kv8_append_rotary(q, k, v, dev(freqs), *cache, table, lens, starts=dev(starts), max_new=129, out=q, k_out=keys)
    assert out.data_ptr() == q.data_ptr()
    attended = qwg.prompt_attend(q, keys, v, starts=dev(starts))
    for s in looked_at:
        at, m = slice(starts[s], starts[s + 1]), int(each[s])
        positions = np.arange(5, 5 + m)
        assert_rotated(q[at], before[s], positions, freqs, False, t)
        want, size = assert_rotated(keys[at], doubles(k[at]), positions, freqs, False, t)
        c = ref.Cache(2, 1, dim, page)
        c.ks[...] = 100
        two = table[s].long()
        assert_keys(cache[0][two], cache[1][two], c, want, size, np.array([[0, 1]]), [5], [0, m])
        want, weight, size = layer_ref.prompt(doubles(q[at]), doubles(keys[at]), doubles(v[at]), [0, m], dim ** -0.5)
        assert_prompt(attended[at], want, weight, size, t, m, np.abs(doubles(v[at])).max())


@pytest.mark.parametrize("t", [torch.float32, torch.float16])
@pytest.mark.parametrize("dim,tiled", [(64, False), (64, True), (256, False)])
def test_shared_by_as_many_rows_as_a_call_takes(t, dim, tiled):
    # sequences may share their own pages too, where nothing is appended: eight kinds of them
    rng = np.random.default_rng(dim)
    c, pre, table, lens = filled(rng, 100, [1, 2, 15, 16, 0, 3, 9, 16], 4, dim, 16, spread=0.3)
    times = 4096
    table, lens = np.tile(table, (times, 1)), np.tile(lens, times)
    seqs = len(lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    q = torch.randn(seqs, 32, dim, dtype=t, device=DEV, generator=g)
    assert seqs * 32 == 1 << 20
    out = attend(q, c, wide(pre, q, c) if tiled else pre, 100, table, lens)
    for s in (0, seqs // 2 - 8, seqs - 8):
        at = slice(s, s + 8)
        want = layer_ref.shared(doubles(q[at])[:, None], c, pre, 100, table[at], lens[at], dim ** -0.5)
        assert_shared(out[at], *want, t, 116)
