"""The 8-bit cache over many chunks of a prompt, and its tail's bookkeeping."""
import numpy as np
import pytest
import torch

import lossless_ultra_long_b200 as L
import q8_plain as P8

pytestmark = pytest.mark.gpu


def folded(rows):
    """bf16 rows [H, n, D] as they come out of the cache: full blocks through 8 bits."""
    n = rows.shape[1] // 64 * 64
    codes, byte = P8.quantize(rows[:, :n])
    return torch.cat([codes * P8.factors(byte).repeat_interleave(64, 1)[..., None], rows[:, n:].double()], 1)


@pytest.mark.parametrize("tail_rows,chunks", [
    (1024, [1000, 984, 961, 23, 1000]),   # behind 40, 0, 1 and 24 rows up to the tail's end
    (1024, [625, 800, 70, 900]), (512, [449] * 5), (128, [65, 65, 1, 65, 64, 65]), (256, [193, 250, 193, 193]),
    (64, [40, 24, 64, 1, 63, 1]),
])
@pytest.mark.parametrize("stream", [False, True])
def test_chunks_of_a_prompt(tail_rows, chunks, stream):
    hkv, d = 2, 64
    rng = np.random.default_rng(tail_rows)
    total = sum(chunks)
    cache = L.KvCacheQ8.empty(hkv, d, total, tail_rows=tail_rows)
    k, v = (P8.bf16(rng, hkv, total, d) for _ in "kv")
    dk, dv = (x.transpose(0, 1).contiguous().cuda() for x in (k, v))
    s = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    at = 0
    for n in chunks:
        cache.append(None, dk[at:at + n], dv[at:at + n], None, stream=s)
        at += n
        before = cache.n_tail
        assert cache.fold(stream=s) == before // 64 * 64
        assert cache.n_ctx == at and cache.n_tail == at % 64 and cache.tail_row0 == 0
    torch.cuda.synchronize()
    idx = torch.arange(total, dtype=torch.int32, device="cuda").expand(hkv, -1).contiguous()
    kp, vp = L.kv_gather_q8(cache, idx)
    assert torch.equal(kp.cpu().double(), folded(k)) and torch.equal(vp.cpu().double(), folded(v))


@pytest.mark.parametrize("row0,n_tail", [(10, 50), (50, 10), (1, 63), (30, 64), (5, 200)])
def test_fold_moves_what_is_left_to_the_start(row0, n_tail):
    """Also where the rows' old and new places overlap."""
    hkv, d, cap = 3, 128, 300
    rng = np.random.default_rng(row0)
    k, v = (P8.bf16(rng, hkv, cap, d) for _ in "kv")
    k8, v8 = (torch.zeros(hkv, 256, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.zeros(hkv, 4, dtype=torch.uint8, device="cuda") for _ in "kv")
    cache = L.KvCacheQ8(k8, v8, ks, vs, k.cuda(), v.cuda(), n_tail=n_tail, tail_row0=row0)
    rows = cache.fold()
    assert rows == n_tail // 64 * 64 and (cache.n_q8, cache.n_tail, cache.tail_row0) == (rows, n_tail - rows, 0)
    idx = torch.arange(n_tail, dtype=torch.int32, device="cuda").expand(hkv, -1).contiguous()
    kp, vp = L.kv_gather_q8(cache, idx)
    assert torch.equal(kp.cpu().double(), folded(k[:, row0:row0 + n_tail]))
    assert torch.equal(vp.cpu().double(), folded(v[:, row0:row0 + n_tail]))
