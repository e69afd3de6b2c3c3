"""The 8-bit cache's attention on the GPU, beyond the plain forms' sizes: the same
call twice, long tails with keys that are no numbers."""
import math

import numpy as np
import pytest
import torch

import lossless_ultra_long_b200 as L
import q8_plain as P8

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ the same call twice
def random_call(seed, hq, hkv, d, n_q8, n_tail, t):
    """A call on a cache made on the device: (queries, cache, tree)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes():
        x = torch.randint(0, 256, (hkv, n_q8, d), generator=g, device="cuda", dtype=torch.uint8)
        return (x & 0xBF).view(torch.float8_e4m3fn)      # magnitudes of at most 1.875

    def scales():
        return torch.randint(124, 129, (hkv, n_q8 // 64), generator=g, device="cuda",
                             dtype=torch.uint8)

    def tail():
        return torch.randn(hkv, n_tail + t, d, generator=g, device="cuda").to(torch.bfloat16)

    cache = L.KvCacheQ8(codes(), codes(), scales(), scales(), tail(), tail(), n_q8=n_q8, n_tail=n_tail)
    q = torch.randn(t, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    return q, cache, P8.parents("bfs", t)


@pytest.mark.parametrize("hq,hkv,d,n_q8,n_tail,t", [
    (8, 2, 64, 192, 20, 1), (8, 2, 64, 1984, 64, 13), (8, 2, 64, 20480, 64, 40),
    (32, 8, 128, 1984, 63, 40), (32, 8, 128, 32704, 63, 1), (32, 8, 128, 102336, 37, 1),
    (32, 8, 128, 102336, 51, 13), (32, 8, 128, 32704, 63, 32), (32, 8, 128, 102336, 51, 40),
    (40, 8, 128, 32704, 63, 40), (32, 32, 128, 32768, 0, 4), (8, 1, 128, 16384, 300, 64),
    (74, 74, 128, 448, 700, 3),
], ids=lambda x: str(x))
@pytest.mark.parametrize("root", [False, True])
def test_the_same_call_gives_the_same_bits(hq, hkv, d, n_q8, n_tail, t, root):
    """Whichever split is faster, and whatever runs beside the call."""
    q, cache, parent = random_call(n_q8 + t, hq, hkv, d, n_q8, n_tail, t)
    ws = L.new_workspace(L.tree_verify_attn_q8_workspace_size(hq, hkv, d, n_q8, n_tail, t))
    first = None
    noise, side = torch.zeros(1 << 24, device="cuda"), torch.cuda.Stream()
    for rep in range(24):
        rs = torch.empty(hq, n_q8 + n_tail, device="cuda") if root else None
        if rep >= 12:                     # something else on the memory system
            with torch.cuda.stream(side):
                noise.add_(1.0)
        out = L.tree_verify_attn_q8(q, cache, parent, workspace=ws, root_scores_out=rs)
        if first is None:
            first = out, rs
        assert torch.equal(out, first[0]), rep
        assert not root or torch.equal(rs, first[1]), rep
    assert L.workspace_status(ws) == 0
    torch.cuda.synchronize()


# --------------------------------------------------- values that are no numbers
@pytest.mark.parametrize("hq,hkv,n_tail,t", [(74, 74, 2500, 3), (592, 74, 2000, 12), (592, 74, 1900, 16),
                                             (296, 74, 1500, 40)])
def test_many_tail_tiles_with_keys_that_are_no_numbers(hq, hkv, n_tail, t):
    """Each CTA takes more tail tiles than it has places for their notes."""
    d = 128
    c = P8.cache_inputs(96, hkv, d, 0, n_tail, t)
    rng = np.random.default_rng(97)
    bad = torch.from_numpy(rng.random((hkv, n_tail)) < 0.02)
    c["k_tail"][:, :n_tail][bad] = math.nan
    q, parent = P8.bf16(rng, t, hq * d).reshape(t, hq, d), P8.parents("random", t, 2)
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=0, n_tail=n_tail)
    g = hq // hkv
    k = torch.where(bad[..., None], 0.0, c["k_tail"][:, :n_tail].double())
    mask = bad.repeat_interleave(g, 0)
    want = torch.einsum("hgd,hnd->hgn", q[0].double().reshape(hkv, g, d), k).reshape(hq, -1) * d ** -0.5 / math.log(2)
    mag = torch.einsum("hgd,hnd->hgn", q[0].double().abs().reshape(hkv, g, d), k.abs()).reshape(hq, -1)
    bound = mag * d ** -0.5 / math.log(2) * ((d + 8) * 2.0 ** -23 + 2.0 ** -20) + 1e-30
    for _ in range(8):
        rs = torch.zeros(hq, n_tail, device="cuda")
        out = L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs)
        got = rs.double().cpu()
        assert torch.equal(torch.isnan(got), mask)
        assert bool(((got - want).abs() <= bound)[~mask].all())
        assert bool(torch.isnan(out).all())
