"""CPU tier of the MXFP4 and 8-bit cache calls: host-side refusals (no HIP call is reached), and the
tests' plain implementations against hand-worked values."""
import ctypes

import numpy as np
import pytest

import mx_ref as ref
from quantized_weight_decode_gemv_amd import _mx
from test_abi_cpu import FAKE, L, declared_symbols  # noqa: F401


def desc(**kw):
    d = dict(k_pages=FAKE, v_pages=FAKE, k_scales=FAKE, v_scales=FAKE, n_pages=4, n_kv_heads=2, head_dim=64, page_tokens=16)
    return ctypes.byref(_mx.Kv8Desc(*{**d, **kw}.values()))


def test_the_calls_are_declared():
    names = declared_symbols()
    for want in ("qwg_encode_mxfp4", "qwg_dequant_mxfp4", "qwg_gemv_mxfp4", "qwg_gemm_mxfp4", "qwg_matmul_mxfp4",
                 "qwg_kv8_append", "qwg_kv8_attend", "qwg_kv8_attend_workspace"):
        assert want in names


@pytest.mark.parametrize("change,status", [
    ({"codes": None}, 1), ({"scales": None}, 1), ({"x": None}, 1), ({"type": 3}, 10), ({"type": -1}, 10),
    ({"n_rows": 0}, 2), ({"n_rows": (1 << 24) + 1}, 2), ({"n_in": 48}, 2), ({"n_in": 0}, 2), ({"n_in": 65536 + 32}, 2),
    ({"stride": 32}, 2), ({"codes": FAKE + 8}, 3), ({"x": FAKE + 2}, 3)])
def test_encode_refusals(L, change, status):  # noqa: F811
    a = {**dict(codes=FAKE, scales=FAKE + 1, x=FAKE + 4, type=0, n_rows=1, n_in=64, stride=64, stream=None), **change}
    assert L.qwg_encode_mxfp4(*a.values()) == status


@pytest.mark.parametrize("change,status", [
    ({"codes": None}, 1), ({"dst": None}, 1), ({"type": 9}, 10), ({"n": 0}, 2), ({"n": 33}, 2), ({"dst": FAKE + 4}, 3), ({"codes": FAKE + 4}, 3)])
def test_dequant_refusals(L, change, status):  # noqa: F811
    a = {**dict(codes=FAKE, scales=FAKE, dst=FAKE, type=1, n=64, stream=None), **change}
    assert L.qwg_dequant_mxfp4(*a.values()) == status


@pytest.mark.parametrize("change,status", [
    ({"y": None}, 1), ({"x": None}, 1), ({"w": None}, 1), ({"s": None}, 1), ({"type": 3}, 10), ({"n_in": 40}, 2),
    ({"n_out": 0}, 2), ({"n_out": (1 << 24) + 1}, 2), ({"batch": 0}, 4), ({"batch": 17}, 4), ({"x": FAKE + 8}, 3),
    ({"w": FAKE + 8}, 3), ({"y": FAKE + 1}, 3)])
def test_gemm_refusals(L, change, status):  # noqa: F811
    a = {**dict(y=FAKE, x=FAKE, type=1, w=FAKE, s=FAKE, n_in=64, n_out=4, batch=2, stream=None), **change}
    assert L.qwg_gemm_mxfp4(*a.values()) == status
    if status != 4:
        del a["batch"]
        assert L.qwg_gemv_mxfp4(*a.values()) == status


@pytest.mark.parametrize("change,status", [
    ({"c": None}, 1), ({"a": None}, 1), ({"ws": None}, 1), ({"type": 3}, 10), ({"n_in": 40}, 2), ({"n_rows": 0}, 2),
    ({"n_out": 0}, 2), ({"a": FAKE + 4}, 3), ({"w": FAKE + 4}, 3), ({"c": FAKE + 1}, 3)])
def test_matmul_refusals(L, change, status):  # noqa: F811
    a = {**dict(c=FAKE, type=2, a=FAKE, as_=FAKE, w=FAKE, ws=FAKE, n_rows=3, n_in=64, n_out=4, stream=None), **change}
    assert L.qwg_matmul_mxfp4(*a.values()) == status


CACHES = [({"k_pages": None}, 1), ({"v_scales": None}, 1), ({"n_pages": 0}, 2), ({"n_kv_heads": 0}, 2), ({"head_dim": 80}, 2),
          ({"page_tokens": 8}, 2), ({"page_tokens": 48}, 2), ({"k_pages": FAKE + 8}, 3), ({"v_pages": FAKE + 8}, 3)]


@pytest.mark.parametrize("cache,change,status", [(c, {}, s) for c, s in CACHES] + [({}, c, s) for c, s in [
    ({"k": None}, 1), ({"v": None}, 1), ({"table": None}, 1), ({"lens": None}, 1), ({"type": 3}, 10), ({"n_tokens": 0}, 2),
    ({"n_tokens": 5, "starts": None}, 2), ({"width": 0}, 2), ({"n_seqs": 0}, 2), ({"n_seqs": 65536, "n_tokens": 65536}, 2),
    ({"k_stride": 127}, 2), ({"v_stride": 127}, 2), ({"max_new": 0}, 2), ({"k": FAKE + 1}, 3), ({"lens": FAKE + 2}, 3)]])
def test_append_refusals(L, cache, change, status):  # noqa: F811
    a = {**dict(k=FAKE, v=FAKE, type=1, k_stride=128, v_stride=128, n_tokens=4, starts=FAKE, table=FAKE, width=2, lens=FAKE, n_seqs=2,
                max_new=4, stream=None), **change}
    assert L.qwg_kv8_append(desc(**cache), *a.values()) == status
    assert L.qwg_kv8_append(None, *a.values()) == 1


@pytest.mark.parametrize("cache,change,status", [(c, {}, s) for c, s in CACHES] + [({}, c, s) for c, s in [
    ({"out": None}, 1), ({"q": None}, 1), ({"table": None}, 1), ({"lens": None}, 1), ({"type": 5}, 10), ({"q_stride": 200}, 2),
    ({"width": 0}, 2), ({"n_seqs": 0}, 2), ({"q_len": 0}, 2), ({"n_heads": 3}, 2), ({"n_heads": 0}, 2), ({"q_len": 20000}, 2),
    ({"window": -1}, 2), ({"max_len": -1}, 2), ({"q": FAKE + 1}, 3), ({"ws": FAKE + 8}, 3),
    ({"width": 4096, "ws": None}, 1), ({"width": 4096, "bytes": 16}, 2)]])
def test_attend_refusals(L, cache, change, status):  # noqa: F811
    a = {**dict(out=FAKE, q=FAKE, type=1, q_stride=256, table=FAKE, width=2, lens=FAKE, n_seqs=2, q_len=1, n_heads=4, scale=1.0,
                window=0, max_len=0, ws=FAKE, bytes=0, stream=None), **change}
    assert L.qwg_kv8_attend(desc(**cache), *a.values()) == status


def test_attend_workspace(L):  # noqa: F811
    size = L.qwg_kv8_attend_workspace
    assert size(desc(), 2, 2, 1, 4, 0, 0) == 0              # 32 positions: one workgroup a head
    assert size(desc(), 65536, 1, 1, 8, 0, 0) > 0
    assert size(desc(), 65536, 1, 1, 8, 512, 0) == 0        # a window of 512: the same
    for dim, width in ((64, 64), (128, 64), (192, 32), (256, 32)):  # 1024 and 512 positions on pages of 16
        for seqs, most in ((1, 0), (1, 1), (300, 0)):
            assert size(desc(head_dim=dim), width, seqs, 4, 32, 0, most) == 0
    assert 0 < size(desc(), 65536, 1, 1, 8, 8192, 0) < size(desc(), 65536, 1, 1, 8, 0, 0)
    assert size(desc(head_dim=80), 2, 2, 1, 4, 0, 0) == -2 and size(None, 2, 2, 1, 4, 0, 0) == -1
    assert size(desc(), 2, 2, 1, 3, 0, 0) == -2 and size(desc(), 2, 2, 1, 4, -1, 0) == -2


def test_binding_refuses_cpu_tensors():
    import torch
    import quantized_weight_decode_gemv_amd as qwg
    x, u = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8)
    for call in (lambda: qwg.encode_mxfp4(x), lambda: qwg.dequant_mxfp4(u, u), lambda: qwg.gemm_mxfp4(u, u, x),
                 lambda: qwg.gemv_mxfp4(u, u, x[0]), lambda: qwg.matmul_mxfp4(u, u, u, u),
                 lambda: qwg.kv8_append(x, x, u, u, u, u, u, u), lambda: qwg.kv8_attend(x, u, u, u, u, u, u)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- the plain implementations

def test_mxfp4_by_hand():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, -5.0, 3.5, 2.5, 0.25, 0.75, -1.25, 7.9]   # ties to even; 7.9 saturates
    c, s = ref.encode_mxfp4(x)
    assert s[0, 0] == 127
    codes = np.stack([c & 15, c >> 4], -1).reshape(-1)[:8]
    assert codes.tolist() == [7, 8 + 6, 6, 4, 0, 2, 8 + 2, 7]
    assert ref.decode_mxfp4(c, s)[0, :8].tolist() == [6, -4, 4, 2, 0, 1, -1, 6]
    x[0, 8] = 8.0                                              # doubles the scale
    assert ref.encode_mxfp4(x)[1][0, 0] == 128
    x[0, 9] = np.inf
    assert ref.encode_mxfp4(x)[1][0, 0] == 255


def test_e4m3_by_hand():
    assert ref.E4M3[0x7E] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[0x38] == 1 and np.isnan(ref.E4M3[0x7F])
    assert np.array_equal(ref.encode_e4m3(ref.E4M3[:127]), np.arange(127))
    assert ref.encode_e4m3(np.array([1.0625, 1.1875, 2.0 ** -10, 1.5 * 2.0 ** -9, np.inf])).tolist() == [0x38, 0x3A, 0, 2, 127]
    assert [ref.page_exponent(np.array([v])) for v in (448.0, 449.0, 0.0, 1.75, 1.0)] == [127, 128, 0, 119, 119]


@pytest.mark.parametrize("n_rows,n_out", [(1 << 24, 1 << 24), (1 << 24, (1 << 14) + 1), ((1 << 19) + 1, 1 << 19)])
def test_matmul_refuses_more_outputs_than_a_launch_takes(L, n_rows, n_out):  # noqa: F811
    # the size is refused as such, before any HIP call
    assert L.qwg_matmul_mxfp4(FAKE, 2, FAKE, FAKE, FAKE, FAKE, n_rows, 64, n_out, None) == 2


def test_the_binding_asks_for_a_workspace_wherever_one_is_needed(L):  # noqa: F811
    """Up to the positions that the binding takes for short, and the header names, the workspace is 0
    whatever the sequences, heads, query tokens, window and known length are."""
    assert tuple(_mx._ALONE) == _mx.KV8_HEAD_DIMS
    for dim, most in _mx._ALONE.items():
        assert most == (1024 if dim <= 128 else 512)
        for page in _mx.KV8_PAGE_TOKENS:
            for kv, group, q_len in ((1, 1, 1), (1, 16, 1), (8, 4, 1), (2, 17, 3), (8, 1, 128), (1024, 1, 1)):
                c = desc(head_dim=dim, page_tokens=page, n_kv_heads=kv)
                for seqs in (1, 2, 9, 33, 64, 300, 65535):
                    for window in (0, 1, 100, most, 1 << 40):
                        for known in (0, 1, most // 2, most, 1 << 40):
                            for width in (1, most // page):
                                assert L.qwg_kv8_attend_workspace(c, width, seqs, q_len, kv * group, window, known) == 0
        # and one twice as long needs one, for one sequence at least
        c = desc(head_dim=dim, page_tokens=128, n_kv_heads=1)
        assert L.qwg_kv8_attend_workspace(c, 2 * most // 128, 1, 1, 1, 0, 0) > 0


def test_a_known_length_of_one_split_costs_no_workspace(L):  # noqa: F811
    """max_len shapes the split: where it makes every sequence one split, the workspace that the table's
    width still asks for is no larger than without it."""
    size = L.qwg_kv8_attend_workspace
    for dim in _mx.KV8_HEAD_DIMS:
        for page in (16, 128):
            c = desc(head_dim=dim, page_tokens=page, n_kv_heads=8)
            for seqs in (1, 8, 32, 200):
                for q_len in (1, 5, 1024):
                    for positions in (1024, 2048, 5120, 131072):
                        for known in (1, 100, 512):
                            for window in (0, 3000):
                                a = (positions // page, seqs, q_len, 32, window)
                                assert 0 <= size(c, *a, known) <= size(c, *a, 0), (dim, page, seqs, q_len, positions, known, window)
