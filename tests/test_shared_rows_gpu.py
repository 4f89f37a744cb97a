"""Attention behind a shared prefix where each sequence's own positions are one part: their launch joins the prefix's parts
too, with two to eight wavefronts and one or two tiles of rows to a workgroup by the heads' width, the rows and the sequences.

The bounds are test_shared_gpu's."""
import ctypes

import numpy as np
import pytest
import torch

import layer_ref
import quantized_weight_decode_gemv_amd as qwg
from quantized_weight_decode_gemv_amd._mx import Kv8Desc
from test_kv8_gpu import TYPES, typed
from test_shared_gpu import assert_shared, attend, filled

pytestmark = pytest.mark.gpu


def shared(q, c, prefix, prefix_len, table, lens, scale):
    """layer_ref.shared, the rows of a sequence and key/value head together."""
    seqs, q_len, heads, dim = q.shape
    out, weight, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3] + (1,))
    kp, vp = c.rows(prefix[None], 0, prefix_len)
    kv, group = kp.shape[0], heads // kp.shape[0]
    v_top = np.abs(vp).max(initial=0)
    for s in range(seqs):
        ko, vo = c.rows(table, s, lens[s])
        v_top = max(v_top, np.abs(vo).max(initial=0))
        n = prefix_len + lens[s]
        seen = np.repeat(np.arange(n) <= (n - q_len + np.arange(q_len))[:, None], group, 0)
        for g in range(kv):
            at = slice(g * group, (g + 1) * group)
            found = layer_ref.softmax_rows(q[s, :, at].reshape(-1, dim), np.concatenate([kp[g], ko[g]]), np.concatenate([vp[g], vo[g]]), seen, scale)
            out[s, :, at], weight[s, :, at] = (x.reshape(q_len, group, dim) for x in found[:2])
            size[s, :, at, 0] = found[2].reshape(q_len, group)
    return out, weight, size, v_top


def one_part(q, c, prefix, table):
    """Whether the own positions are one part: then no room is needed for what their parts sum."""
    seqs, q_len, heads, dim = q.shape
    desc = Kv8Desc(1 << 12, 1 << 12, 1 << 12, 1 << 12, len(c.k), c.k.shape[1], dim, c.page)
    kind = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[q.dtype]

    def room(width):
        return qwg.lib().qwg_kv8_attend_shared_workspace(ctypes.byref(desc), kind, len(prefix), width, seqs, q_len, heads)

    return room(table.shape[1]) == room(1)


# sequences that hold up to what their table of `width` pages takes
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim,page,kv,group,q_len,seqs,width,prefix", [
    (256, 64, 2, 16, 4, 32, 16, 1500), (256, 64, 1, 48, 1, 128, 16, 1300), (256, 128, 1, 40, 1, 160, 24, 300), (256, 32, 1, 40, 1, 300, 16, 200),
    (256, 64, 2, 4, 1, 30, 6, 1100), (256, 16, 1, 2, 1, 300, 6, 1100), (192, 64, 2, 20, 2, 48, 16, 1100), (192, 16, 1, 33, 1, 300, 32, 200),
    (192, 32, 1, 3, 3, 20, 7, 1300), (128, 64, 2, 4, 5, 10, 8, 1500), (128, 32, 2, 20, 1, 150, 8, 300), (128, 64, 4, 4, 1, 90, 12, 1200),
    (96, 16, 2, 17, 1, 260, 4, 300), (96, 32, 1, 17, 2, 9, 10, 2000), (64, 64, 2, 18, 1, 140, 12, 400), (64, 16, 1, 17, 2, 9, 20, 2000),
    (64, 16, 2, 4, 1, 300, 6, 700)])
def test_shared_joined_by_the_own_positions_launch(t, dim, page, kv, group, q_len, seqs, width, prefix):
    rng = np.random.default_rng(dim + page + group)
    lens = rng.integers(0, 3 * page, seqs)
    lens[:4] = 0, width * page, 1, width * page - 1
    lens = np.minimum(lens, width * page)
    c, pre, table, lens = filled(rng, prefix, lens, kv, dim, page, spread=0.3)
    table = table[:, :width].copy()
    q, qd = typed(rng.standard_normal((seqs, q_len, kv * group, dim)), t)
    assert one_part(q, c, pre, table)
    want = shared(qd, c, pre, prefix, table, lens, dim ** -0.5)
    out = attend(q, c, pre, prefix, table, lens)
    assert_shared(out, *want, t, prefix + width * page)
    assert torch.equal(out, attend(q, c, pre, prefix, table, lens))
