"""Attention over the 8-bit cache by a prompt's tokens, and with tables far wider than what the sequences
hold, as a program has that keeps one table, or one captured graph, while they grow."""
import numpy as np
import pytest
import torch

import mx_ref as ref
import quantized_weight_decode_gemv_amd as qwg
from test_kv8_gpu import TYPES, assert_attend, dev, filled, pages, typed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,q_len,window", [(64, 16, 1, 4, 300, 0), (64, 64, 2, 1, 300, 100), (96, 32, 1, 3, 130, 0),
                                                            (128, 64, 1, 4, 257, 64), (128, 128, 1, 2, 300, 0), (192, 16, 1, 2, 200, 33),
                                                            (256, 32, 1, 3, 150, 0), (256, 64, 2, 1, 300, 1)])
def test_attend_by_a_prompt(t, dim, page, kv, group, q_len, window):
    # a prompt alone, one after others' tokens, shorter ones (whose first rows see nothing), none
    rng = np.random.default_rng(dim + q_len)
    lens = np.array([q_len, q_len + 211, q_len - 100, 1, 0], np.int32)
    c, table = filled(rng, lens, kv, dim, page)
    q, qd = typed(rng.standard_normal((len(lens), q_len, kv * group, dim)), t)
    want, weight, size = ref.attend(qd, c, table, lens, dim ** -0.5, window)
    for most in (None, int(lens.max())):
        out = qwg.kv8_attend(q, *pages(c), dev(table), dev(lens), window=window, max_len=most)
        assert_attend(out, want, weight, size, t, dim)
        assert bool((out[2, :100] == 0).all()) and bool((out[3, :-1] == 0).all()) and bool((out[4] == 0).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,q_len,window", [(64, 16, 2, 8, 1, 0), (128, 64, 2, 4, 3, 0), (128, 128, 1, 8, 5, 900),
                                                            (256, 32, 1, 4, 1, 0), (64, 16, 1, 1, 40, 0)])
def test_attend_with_a_table_wider_than_the_lengths(t, dim, page, kv, group, q_len, window):
    rng = np.random.default_rng(page + q_len)
    lens = np.array([1300, 0, 65, q_len, 517], np.int32)
    c, table = filled(rng, lens, kv, dim, page)
    wide = np.full((len(lens), 131072 // page), -7, np.int32)
    wide[:, :table.shape[1]] = table
    q, qd = typed(rng.standard_normal((len(lens), q_len, kv * group, dim)), t)
    want = ref.attend(qd, c, table, lens, dim ** -0.5, window)
    for most in (None, 1300):
        out = qwg.kv8_attend(q, *pages(c), dev(wide), dev(lens), window=window, max_len=most)
        assert_attend(out, *want, t, dim)


def test_a_captured_step_follows_lengths_that_grow():
    """Append and attention captured once, for a wide table, and replayed while the sequences grow past
    one split: every replay against eager calls on a copy of the cache."""
    rng = np.random.default_rng(5)
    kv, group, dim, page, seqs, t = 2, 4, 128, 64, 3, torch.bfloat16
    lens = np.array([0, 900, 4000], np.int32)
    c, narrow = filled(rng, lens + 64, kv, dim, page, spread=0.3)
    table = np.full((seqs, 1024), -1, np.int32)
    table[:, :narrow.shape[1]] = narrow
    cache, table, n = pages(c), dev(table), dev(lens)
    k, v = (torch.empty(seqs, kv, dim, dtype=t, device=n.device) for _ in "kv")
    q = torch.empty(seqs, kv * group, dim, dtype=t, device=n.device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qwg.kv8_append(k, v, *cache, table, n)
        n.add_(1)
        out = qwg.kv8_attend(q, *cache, table, n)
    n.copy_(dev(lens))
    plain = [x.clone() for x in cache]
    for step in range(6):
        for x in (k, v, q):
            x.copy_(typed(rng.standard_normal(x.shape), t)[0])
        before = n.clone()
        graph.replay()
        qwg.kv8_append(k, v, *plain, table, before)
        want = qwg.kv8_attend(q, *plain, table, before + 1)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(n, before + 1)
        for x, y in zip(cache, plain):
            assert torch.equal(x, y)
        if step == 2:  # on by more than a page
            n.add_(40)
