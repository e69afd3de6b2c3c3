"""Calls of the 8-bit cache's operators that a machine without a GPU can decide:
those without rows, through the C ABI and through the binding.  As in
test_binding_host.py host tensors stand in for device tensors."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

import lossless_ultra_long_b200 as L
from test_binding_host import on_dev, workspace, zeros

STREAM = types.SimpleNamespace(cuda_stream=0)
D, HKV, HQ = 64, 2, 8
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host-memory stand-ins are for machines without a GPU")


@pytest.fixture(autouse=True)
def _current_device_zero(monkeypatch):
    from lossless_ultra_long_b200 import build
    build.build()
    if not torch.cuda.is_available():
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(L, "_raw_stream", lambda index: 0)


def bf16(*shape):
    return zeros(shape, torch.bfloat16)


def cache(n_q8=64, n_tail=5, cap=128, tail=100):
    k8, v8 = (on_dev(torch.zeros(HKV, cap, D, dtype=torch.uint8).view(torch.float8_e4m3fn)) for _ in "kv")
    scales = (zeros((HKV, cap // 64), torch.uint8) for _ in "kv")
    return L.KvCacheQ8(k8, v8, *scales, bf16(HKV, tail, D), bf16(HKV, tail, D), n_q8=n_q8, n_tail=n_tail)


# ------------------------------------------------------------------ without rows
def test_empty_calls_need_no_addresses():
    lib = L.library()
    assert lib.ts_kv_quantize_q8(None, None, 0, 2, 64, 0, 0, None, None, None, None, 0, 0, None) == 0
    st = L._Q8Cache(0, 0, 0, 0, 0, 0, 0, 0, 0, 2, 64, 0, 0)
    assert lib.ts_kv_gather_q8(ctypes.byref(st), None, 0, None, None, 0, 1 << 20, 256, None) == 0
    for parent in (None, 1 << 20):
        assert lib.ts_rope_append(None, 512, None, 128, None, 128, 8, 2, 64, 0, parent, 0, None, 0, 0, 1.0,
                                  None, None, None, 0, 0, None) == 0
    # what an empty call says is still checked
    assert lib.ts_kv_quantize_q8(None, None, 0, 2, 64, 1, 0, None, None, None, None, 0, 0, None) == 1
    assert lib.ts_kv_quantize_q8(None, None, 0, 2, 96, 0, 0, None, None, None, None, 0, 0, None) == 2
    assert lib.ts_rope_append(None, 512, None, 128, None, 128, 8, 2, 64, 0, None, 0, None, 0, 0, 1.0,
                              None, None, None, 10, 11, None) == 1
    assert lib.ts_kv_gather_q8(ctypes.byref(st), None, 0, None, None, 0, None, 256, None) == 3
    # and one row needs them
    assert lib.ts_rope_append(None, 512, None, 128, None, 128, 8, 2, 64, 1, None, 0, None, 0, 0, 1.0,
                              None, None, None, 10, 0, None) == 1
    assert lib.ts_kv_gather_q8(ctypes.byref(st), None, 1, None, None, 1, 1 << 20, 256, None) == 1


@no_gpu
def test_empty_calls_of_the_binding():
    kc, vc = bf16(HKV, 9, D), bf16(HKV, 9, D)
    q, k, v = bf16(0, HQ, D), bf16(0, HKV, D), bf16(0, HKV, D)
    ws = dict(q_out=bf16(0, HQ, D), stream=STREAM)
    for parent in (None, []):
        assert L.rope_append(q, k, v, kc, vc, 9, 3, zeros(D // 2), parent=parent, **ws).shape == (0, HQ, D)
    c = cache()
    assert c.append(q, k, v, zeros(D // 2), **ws).shape == (0, HQ, D) and c.n_tail == 5
    kp, vp = L.kv_gather_q8(c, zeros((HKV, 0), torch.int32), k_partial=bf16(HKV, 0, D),
                            v_partial=bf16(HKV, 0, D), workspace=workspace(256), stream=STREAM)
    assert kp.shape == vp.shape == (HKV, 0, D)
    none = cache(n_q8=0, n_tail=0, cap=0, tail=0)
    L.kv_quantize_q8(none.k_tail, none.v_tail, 0, 0, none.k8, none.v8, none.k_scale, none.v_scale, 0, stream=STREAM)
    assert none.fold(stream=STREAM) == 0


# ------------------------------------------------------------- what a call would misread
@no_gpu
def test_a_short_acceptance_result_is_refused():
    """The kernel reads up to 2 + n_tree entries."""
    c = cache(n_tail=5, tail=100)
    for n in (0, 2, 14):
        with pytest.raises(ValueError, match="entries"):
            c.commit(zeros(n, torch.int32), 13, 0, workspace=workspace(256), stream=STREAM)
    with pytest.raises(L.TsError) as e:          # enough of them: accepted, there is no device
        c.commit(zeros(15, torch.int32), 13, 0, workspace=workspace(256), stream=STREAM)
    assert e.value.status == 4


@pytest.mark.parametrize("parent", [
    np.array([-1, 0, 2 ** 32]), np.array([-1, 2 ** 32 - 1, 0]), [-1, 0, 0.5], np.array([-1.0, 0.0, 1.5]),
    (-1, 0, math.nan), torch.tensor([-1, 0, 2 ** 33 + 1]), np.array([2 ** 32 - 1, 0, 0], dtype=np.uint32),
    [-1, 0, 1 << 70], [-1, None, 0], "abc", np.array([[-1, 0, 0]]), [-1, [0], 0],
], ids=str)
def test_a_tree_that_is_not_32_bit_integers_is_refused(parent):
    """(2^32 would be node 0 in 32 bits, 1.5 node 1)"""
    with pytest.raises((ValueError, TypeError, OverflowError)):
        L._parent_arg(parent, 3)


def test_a_tree_in_other_types_and_strides():
    wide = np.array([[-1, 7], [0, 7], [1, 7]])
    for parent in (wide[:, 0], wide.astype(np.int32)[:, 0], np.array([-1.0, 0.0, 1.0]), torch.tensor([-1, 0, 1]).to(
            torch.int16), np.array([-1, 0, 1], dtype=">i4"), [np.int64(-1), 0, True]):
        keep, address = L._parent_arg(parent, 3)
        assert list((ctypes.c_int32 * 3).from_address(address)) == [-1, 0, 1]
        del keep


@no_gpu
@pytest.mark.parametrize("name,at", [("pos0", 2 ** 64 + 5), ("row0", 2 ** 64), ("n_rows", 2 ** 32 + 64),
                                     ("from", 2 ** 64), ("dst", 2 ** 64), ("n_sink", 2 ** 32 + 4),
                                     ("budget", 2 ** 32 + 60), ("budget", 2 ** 63)])
def test_integers_past_the_c_types_are_refused(name, at):
    """(cut to their low bits these would be valid calls)"""
    c, f = cache(n_q8=64, n_tail=5), {"pos0": 5, "row0": 0, "n_rows": 64, "from": 0, "dst": 0, "n_sink": 4, "budget": 60}

    def rope():
        L.rope_append(bf16(4, HQ, D), bf16(4, HKV, D), bf16(4, HKV, D), c.k_tail, c.v_tail, f["row0"], f["pos0"],
                      zeros(D // 2), q_out=bf16(4, HQ, D), stream=STREAM)

    def quantize():
        L.kv_quantize_q8(c.k_tail, c.v_tail, f["from"], f["n_rows"], c.k8, c.v8, c.k_scale, c.v_scale, f["dst"],
                         stream=STREAM)

    def select():
        L.kv_select_from_scores_q8(zeros((HQ, 69)), c, f["n_sink"], f["budget"], k_partial=bf16(HKV, 69, D),
                                   v_partial=bf16(HKV, 69, D), idx_out=zeros((HKV, f["keep"]), torch.int32),
                                   workspace=workspace(), stream=STREAM)

    call = {"pos0": rope, "row0": rope, "n_sink": select, "budget": select}.get(name, quantize)
    f["keep"] = 64
    with pytest.raises(L.TsError) as e:          # accepted as it is, there is no device
        call()
    assert e.value.status == 4
    f[name], f["keep"] = at, 69
    with pytest.raises(ValueError, match="bit integer"):
        call()


def test_positions_past_64_bits_are_refused():
    lib, A = L.library(), 1 << 20
    for n_tok, pos0 in ((1, 2 ** 63 - 1), (4, 2 ** 63 - 4)):
        assert lib.ts_rope_append(A, 512, A, 128, A, 128, 8, 2, 64, n_tok, None, pos0, A, 64, 0, 1.0, 2 * A, A, A,
                                  10, 0, None) == 1
