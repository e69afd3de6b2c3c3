"""On which stream a call makes the buffers that it is not given: the one that it
runs on.  As in test_binding_host.py host tensors stand in for device tensors, and
each call ends at its first CUDA runtime call."""
import contextlib
import types

import pytest
import torch

import lossless_ultra_long_b200 as L
from lossless_ultra_long_b200 import inputs as I
from test_binding_host import D, HKV, HQ, N_CTX, T, VOCAB, _attn_inputs, on_dev, workspace, zeros

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-memory stand-ins are for machines without a GPU")

STREAM = types.SimpleNamespace(cuda_stream=0)
Q8 = dict(n_q8=1984, n_tail=64)


def cache():
    k8, v8 = (on_dev(torch.zeros(HKV, 1984, D, dtype=torch.uint8).view(torch.float8_e4m3fn)) for _ in "kv")
    scales = (zeros((HKV, 31), torch.uint8) for _ in "kv")
    return L.KvCacheQ8(k8, v8, *scales, *(zeros((HKV, 128, D), torch.bfloat16) for _ in "kv"), **Q8)


def rows(heads):
    return zeros((T, heads, D), torch.bfloat16)


CALLS = {
    "tree_verify_attn": lambda s: L.tree_verify_attn(*_attn_inputs(), N_CTX, I.bfs_tree(T), stream=s),
    "kv_importance_select": lambda s: L.kv_importance_select(
        zeros((HQ, D), torch.bfloat16), *_attn_inputs()[1:], N_CTX, 16, 240, want_scores=True, stream=s),
    "kv_select_from_scores": lambda s: L.kv_select_from_scores(
        zeros((HQ, N_CTX)), *_attn_inputs()[1:], N_CTX, 16, 240, want_scores=True, stream=s),
    "penalize_accept": lambda s: L.penalize_accept(
        zeros((T, VOCAB)), zeros(16, torch.int32), 1.2, I.bfs_tree(T), zeros(T, torch.int32), stream=s),
    "penalize_sample_accept": lambda s: L.penalize_sample_accept(
        zeros((T, VOCAB)), zeros((T, VOCAB)), 0.7, None, 1.2, I.bfs_tree(T), zeros(T, torch.int32), stream=s),
    "kv_commit_path": lambda s: L.kv_commit_path(*_attn_inputs()[1:], N_CTX, T, zeros(2 + T, torch.int32), stream=s),
    "selftest_bounded_wait": lambda s: L.selftest_bounded_wait(stream=s),
    "rope_append": lambda s: L.rope_append(rows(HQ), rows(HKV), rows(HKV), *_attn_inputs()[1:], 5, 7,
                                           zeros(D // 2), stream=s),
    "tree_verify_attn_q8": lambda s: L.tree_verify_attn_q8(rows(HQ), cache(), I.bfs_tree(T), stream=s),
    "kv_gather_q8": lambda s: L.kv_gather_q8(cache(), zeros((HKV, 9), torch.int32), stream=s),
    "kv_select_from_scores_q8": lambda s: L.kv_select_from_scores_q8(
        zeros((HQ, N_CTX)), cache(), 16, 240, want_scores=True, stream=s),
    "KvCacheQ8.append": lambda s: cache().append(rows(HQ), rows(HKV), rows(HKV), zeros(D // 2),
                                                 parent=I.bfs_tree(T).tolist(), stream=s),
    "KvCacheQ8.commit": lambda s: cache().commit(zeros(2 + T, torch.int32), T, 3, stream=s),
}
MADE = {"tree_verify_attn": 2, "kv_importance_select": 5, "kv_select_from_scores": 5, "penalize_accept": 3,
        "penalize_sample_accept": 3, "kv_commit_path": 1, "selftest_bounded_wait": 1, "rope_append": 1,
        "tree_verify_attn_q8": 2, "kv_gather_q8": 3, "kv_select_from_scores_q8": 5, "KvCacheQ8.append": 1,
        "KvCacheQ8.commit": 1}


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_makes_its_buffers_on_its_stream(monkeypatch, name, given):
    on, made = [], []
    L.library()
    real_zeros, real_empty, real_like = torch.zeros, torch.empty, torch.empty_like

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    def device_buffer(*size, dtype=None, device=None):
        if device is None:
            return real_zeros(*size, dtype=dtype)
        size = size[0] if len(size) == 1 else size
        made.append(on[-1] if on else None)
        n = real_empty(size, dtype=dtype, device="meta").nbytes
        # on the library's borders, as device memory is
        return on_dev(workspace(max(n, 256))[:n].as_subclass(torch.Tensor).view(dtype).reshape(size))

    def like(x):
        return device_buffer(x.shape, dtype=x.dtype, device="cuda:0")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: STREAM)
    monkeypatch.setattr(L, "_raw_stream", lambda index: 0)
    call = CALLS[name]
    for n, f in (("zeros", device_buffer), ("empty", device_buffer), ("empty_like", like)):
        monkeypatch.setattr(torch, n, f)
    with pytest.raises(L.TsError) as e:
        call(STREAM if given else None)
    assert e.value.status == 4, name          # it was accepted, there is no device
    assert len(made) == MADE[name], made
    assert all(s is (STREAM if given else None) for s in made), made
