"""What the rotary append, prompt attention and attention behind a shared prefix refuse, on the host alone."""
import ctypes

import pytest
import torch

import quantized_weight_decode_gemv_amd as qwg
from quantized_weight_decode_gemv_amd._mx import Kv8Desc

P, NULL, SHAPE, ALIGN, TYPE, OVERLAP = 1 << 20, 1, 2, 3, 10, 11
CACHE = dict(k_pages=P, v_pages=P, k_scales=P, v_scales=P, n_pages=8, n_kv_heads=2, head_dim=64, page_tokens=16)
ROTARY = dict(q_out=16 * P, q_out_stride=512, k_out=None, k_out_stride=0, q=2 * P, q_stride=512, k=3 * P, k_stride=128,
              v=4 * P, v_stride=128, type=0, n_heads=8, freqs=P, rotary=64, interleaved=0, prefix_len=None, n_tokens=4,
              starts=None, table=P, width=3, lens=P, n_seqs=2, max_new=2, stream=None)
PROMPT = dict(out=16 * P, q=2 * P, q_stride=512, k=3 * P, k_stride=128, v=4 * P, v_stride=128, type=0, n_tokens=4, starts=None,
              n_seqs=2, max_len=0, n_heads=8, n_kv=2, dim=64, scale=0.1, window=0, stream=None)
SHARED = dict(out=16 * P, q=2 * P, type=0, q_stride=512, prefix=P, prefix_width=3, prefix_len=P, table=P, width=2, lens=P, n_seqs=2,
              q_len=1, n_heads=8, scale=0.1, workspace=P, bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    *[({x: None}, NULL) for x in ("q_out", "q", "k", "v", "freqs", "table", "lens")],
    ({"type": 3}, TYPE), ({"n_heads": 3}, SHAPE), ({"n_heads": 0}, SHAPE), ({"n_heads": 1 << 17}, SHAPE), ({"rotary": 0}, SHAPE),
    ({"rotary": 24}, SHAPE), ({"rotary": 80}, SHAPE), ({"q_stride": 511}, SHAPE), ({"q_out_stride": 511}, SHAPE), ({"k_stride": 127}, SHAPE),
    ({"v_stride": 0}, SHAPE), ({"k_out": 32 * P, "k_out_stride": 127}, SHAPE), ({"n_tokens": 0}, SHAPE), ({"n_tokens": 3}, SHAPE),
    ({"n_tokens": 1 << 31}, SHAPE), ({"max_new": 0}, SHAPE), ({"width": 0}, SHAPE), ({"width": 1 << 27}, SHAPE), ({"n_seqs": 65536}, SHAPE),
    ({"q": 2 * P + 2}, ALIGN), ({"q_out": 16 * P + 1}, ALIGN), ({"freqs": P + 2}, ALIGN), ({"prefix_len": P + 2}, ALIGN), ({"k_out": 32 * P + 2, "k_out_stride": 128}, ALIGN),
    ({"q_out": 3 * P}, OVERLAP), ({"q_out": 4 * P}, OVERLAP), ({"q_out": 2 * P + 64}, OVERLAP), ({"q_out": 2 * P, "q_out_stride": 600}, OVERLAP),
    ({"k_out": 3 * P, "k_out_stride": 128}, OVERLAP), ({"k_out": 2 * P + 2048, "k_out_stride": 512}, OVERLAP),
    ({"k_out": 16 * P + 4096, "k_out_stride": 128}, OVERLAP), ({"k_out": 3 * P - 256, "k_out_stride": 128}, OVERLAP),
    # slices of one fused result of 768 values, the last overlapping the queries by one value
    ({"q_stride": 768, "k_stride": 768, "v_stride": 768, "k": 2 * P + 2048, "v": 2 * P + 2560, "q_out": 2 * P + 4, "q_out_stride": 768}, OVERLAP)])
def test_rotary_refuses(change, status):
    L = qwg.lib()
    assert L.qwg_kv8_append_rotary(ctypes.byref(Kv8Desc(**CACHE)), *{**ROTARY, **change}.values()) == status
    assert L.qwg_kv8_append_rotary(None, *ROTARY.values()) == NULL
    assert L.qwg_kv8_append_rotary(ctypes.byref(Kv8Desc(**{**CACHE, "head_dim": 80})), *ROTARY.values()) == SHAPE


@pytest.mark.parametrize("change,status", [
    *[({x: None}, NULL) for x in ("out", "q", "k", "v")], ({"type": -1}, TYPE), ({"dim": 80}, SHAPE), ({"n_kv": 0}, SHAPE), ({"n_kv": 3}, SHAPE),
    ({"n_kv": 2048, "n_heads": 2048}, SHAPE), ({"n_heads": 0}, SHAPE), ({"n_seqs": 0}, SHAPE), ({"n_seqs": 3}, SHAPE), ({"n_tokens": 0}, SHAPE),
    ({"n_tokens": 1 << 28, "starts": P}, SHAPE), ({"n_seqs": 1 << 22, "starts": P}, SHAPE), ({"n_tokens": 1 << 62, "starts": P}, SHAPE),
    ({"n_seqs": 1 << 62, "starts": P}, SHAPE), ({"max_len": -1}, SHAPE), ({"window": -1}, SHAPE), ({"q_stride": 511}, SHAPE), ({"k_stride": 127}, SHAPE),
    ({"v_stride": -128}, SHAPE), ({"q": 2 * P + 2}, ALIGN), ({"out": 16 * P + 2}, ALIGN), ({"starts": P + 2}, ALIGN), ({"v": 4 * P + 1, "type": 2}, ALIGN),
    ({"out": 3 * P}, OVERLAP), ({"out": 4 * P}, OVERLAP), ({"out": 3 * P - 4096}, OVERLAP), ({"out": 2 * P + 4}, OVERLAP),
    ({"out": 2 * P, "q_stride": 768}, OVERLAP), ({"out": 4 * P + 1024}, OVERLAP)])
def test_prompt_refuses(change, status):
    assert qwg.lib().qwg_prompt_attend(*{**PROMPT, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    *[({x: None}, NULL) for x in ("out", "q", "prefix", "prefix_len", "table", "lens", "workspace")], ({"type": 7}, TYPE),
    ({"q_stride": 511}, SHAPE), ({"prefix_width": 0}, SHAPE), ({"prefix_width": 1 << 27}, SHAPE), ({"width": 0}, SHAPE), ({"n_seqs": 0}, SHAPE),
    ({"n_seqs": 65536}, SHAPE), ({"n_seqs": 65535, "n_heads": 18}, SHAPE), ({"q_len": 0}, SHAPE), ({"n_heads": 7}, SHAPE), ({"bytes": 15}, SHAPE),
    ({"workspace": P + 8}, ALIGN), ({"prefix_len": P + 2}, ALIGN), ({"prefix": P + 1}, ALIGN), ({"out": P + 2}, ALIGN),
    ({"out": 2 * P + 4}, OVERLAP), ({"out": 2 * P + 4092}, OVERLAP), ({"out": 2 * P, "q_stride": 600}, OVERLAP)])
def test_shared_refuses(change, status):
    L, desc = qwg.lib(), Kv8Desc(**CACHE)
    args = {**SHARED, **change}
    assert L.qwg_kv8_attend_shared(ctypes.byref(desc), *args.values()) == status
    size = L.qwg_kv8_attend_shared_workspace(ctypes.byref(desc), *(args[x] for x in ("type", "prefix_width", "width", "n_seqs", "q_len", "n_heads")))
    shape = set(change) & {"type", "prefix_width", "width", "n_seqs", "q_len", "n_heads"}
    assert size == -status if shape else size > 0 and size % 16 == 0


def test_binding_refuses_what_is_not_on_a_device():
    x, u, i = torch.zeros(2, 2, 64), torch.zeros(1, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: qwg.kv8_append_rotary(x, x, x, x, u, u, u, u, i, i), lambda: qwg.prompt_attend(x, x, x),
                 lambda: qwg.kv8_attend_shared(x, u, u, u, u, i, i, i, i), lambda: qwg.prompt_attend(None, x, x)):
        with pytest.raises(ValueError):
            call()


def test_statuses_have_words():
    text = {qwg.lib().qwg_strerror(s) for s in range(12)}
    assert len(text) == 12 and qwg.lib().qwg_strerror(12) not in text
