"""The 8-bit cache's attention on the GPU: the same call twice, tail rows of very
different sizes, rows that hold no numbers, blocks of zeros; the rotation of long
prompts."""
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


# ------------------------------------------------- tail rows far apart in size
def near(q, k, v, n_ctx, parent, scale):
    """(out, bound) as P8.attention, with every score's error taken at its own
    position: eta_j = (sum of its magnitudes) * per + 2^-18, so that a position
    without weight does not widen the bound.  Weights w_j e^(+-eta_j) move the
    result by at most sum w_j (e^eta_j - e^-eta_j) |v_j - out| / sum w_j e^-eta_j."""
    t, hq, d = q.shape
    g = hq // k.shape[0]
    per = (d + 8) * 2.0 ** -23 + 2.0 ** -20
    vis = P8.sees(parent)
    out = torch.empty(t, hq, d, dtype=torch.float64)
    bound = torch.empty_like(out)
    for h in range(hq):
        kh, vh, qd = k[h // g], v[h // g], q[:, h].cpu().double()
        for i in range(t):
            at = torch.cat([torch.arange(n_ctx), n_ctx + vis[i].nonzero()[:, 0]])
            x = kh[at] @ qd[i] * scale
            eta = kh[at].abs() @ qd[i].abs() * abs(scale) * per + 2.0 ** -18
            x = x - torch.logsumexp(x, 0)
            w, more, less = x.exp(), (x + eta).exp(), (x - eta).exp()
            o = w @ vh[at]
            off = (vh[at] - o).abs()
            move = torch.maximum(w @ vh[at].abs(), w @ off)
            out[i, h] = o
            bound[i, h] = (2.0 ** -8 * (move + o.abs()) * (1 + 2.0 ** -7) +
                           (more - less) @ off / less.sum() + 1e-30)
    return out, bound


KERNELS = [(8, 2, 64, 128), (16, 4, 128, 2176), (148, 74, 128, 640)]   # general, general, tcgen05


@pytest.mark.parametrize("hq,hkv,d,n_q8", KERNELS)
@pytest.mark.parametrize("size", [1e5, 1e30])
def test_a_large_unseen_key_changes_nothing(hq, hkv, d, n_q8, size):
    """Finite keys and values of a branch that a node does not see."""
    t, n_tail = 13, 30
    c = P8.cache_inputs(90, hkv, d, n_q8, n_tail, t)
    q, parent, scale = P8.bf16(np.random.default_rng(91), t, hq * d).reshape(t, hq, d), P8.parents("bfs", t), d ** -0.5
    c["k_tail"][:, n_tail + 2] *= size
    c["k_tail"][:, n_tail + 12, 5] = -size
    c["v_tail"][:, n_tail + 12] *= size
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=n_tail)
    rs = torch.empty(hq, n_q8 + n_tail, device="cuda")
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs).double().cpu()
    k, v = (P8.cache_rows(c, n, n_q8, 0, n_tail + t) for n in "kv")
    vis = P8.sees(parent)
    free = ~(vis[:, 2] | vis[:, 12])
    assert bool(free.any()) and not bool(free.all())
    want, bound = near(q, k, v, n_q8 + n_tail, parent, scale)
    assert bool(((out - want).abs() <= bound)[free].all()), float(((out - want).abs() / bound)[free].max())
    _, _, wr, br = P8.attention(q[:1], k[:, :n_q8 + n_tail + 1], v[:, :n_q8 + n_tail + 1], n_q8 + n_tail, [-1], scale)
    assert bool(((rs.double().cpu() - wr).abs() <= br).all())


@pytest.mark.parametrize("hq,hkv,d,n_q8", KERNELS + [(74, 74, 128, 0)])
@pytest.mark.parametrize("power", [20, 60])
def test_tail_keys_of_very_different_sizes(hq, hkv, d, n_q8, power):
    """Context rows in the tail from 2^-power to 2^power; the large ones point
    away from every query, the root's scores are right at each."""
    t, n_tail = 4, 330
    c = P8.cache_inputs(92, hkv, d, n_q8, n_tail, t)
    rng = np.random.default_rng(93)
    q = P8.bf16(rng, t, hq * d).reshape(t, hq, d)
    q[:] = q[:1, :1]
    away = -(q[0, 0].double() / q[0, 0].double().norm())
    size = torch.from_numpy(rng.integers(-power, power + 1, (hkv, n_tail, 1)).astype(np.float64))
    rows = c["k_tail"][:, :n_tail].double()
    rows = torch.where(size > 0, rows.norm(dim=-1, keepdim=True) * away, rows) * 2.0 ** size
    c["k_tail"][:, :n_tail] = rows.to(torch.bfloat16)
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=n_tail)
    rs = torch.empty(hq, n_q8 + n_tail, device="cuda")
    parent = P8.parents("chain", t)
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs).double().cpu()
    k, v = (P8.cache_rows(c, n, n_q8, 0, n_tail + t) for n in "kv")
    want, bound = near(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
    assert bool(((out - want).abs() <= bound).all()), float(((out - want).abs() / bound).max())
    _, _, wr, br = P8.attention(q[:1], k[:, :n_q8 + n_tail + 1], v[:, :n_q8 + n_tail + 1],
                                n_q8 + n_tail, [-1], d ** -0.5)
    err = (rs.double().cpu() - wr).abs()
    assert bool((err <= br).all()), float((err / br).max())


# --------------------------------------------------- values that are no numbers
@pytest.mark.parametrize("hq,hkv,d,n_q8", KERNELS + [(74, 74, 128, 0)])
@pytest.mark.parametrize("what", [math.inf, math.nan])
def test_root_scores_do_not_depend_on_values(hq, hkv, d, n_q8, what):
    """A row of V that is no number makes the outputs NaN, not a score; a row
    of K its own score."""
    t, n_tail = 5, 150
    c = P8.cache_inputs(94, hkv, d, n_q8, n_tail, t)
    q, parent = P8.bf16(np.random.default_rng(95), t, hq * d).reshape(t, hq, d), P8.parents("bfs", t)
    c["v_tail"][:, 7, 3] = what
    c["v_tail"][:, 140, d - 1] = -what
    c["v_tail"][0, n_tail + 3, 0] = what
    c["k_tail"][hkv - 1, 99, 1] = what
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=n_tail)
    rs = torch.zeros(hq, n_q8 + n_tail, device="cuda")
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs)
    assert bool(torch.isnan(out).all())
    k = P8.cache_rows(c, "k", n_q8, 0, n_tail + t)
    bad = n_q8 + 99
    k[hkv - 1, bad] = 0.0
    _, _, wr, br = P8.attention(q[:1], k[:, :n_q8 + n_tail + 1], torch.zeros_like(k[:, :n_q8 + n_tail + 1]),
                                n_q8 + n_tail, [-1], d ** -0.5)
    got = rs.double().cpu()
    last = slice(hq - hq // hkv, hq)
    assert bool(torch.isnan(got[last, bad]).all())
    got[last, bad] = 0.0
    assert bool(((got - wr).abs() <= br).all()), float(((got - wr).abs() / br).max())


@pytest.mark.parametrize("hq,hkv,d,n_q8,n_tail", [(8, 2, 64, 2048, 9), (74, 74, 128, 4096, 9), (740, 37, 128, 2048, 9),
                                                  (600, 20, 128, 6144, 9)])
@pytest.mark.parametrize("what", [-math.inf, math.nan])
def test_a_row_that_sees_no_number_is_nan_where_scores_rise(hq, hkv, d, n_q8, n_tail, what):
    """Scores that outgrow a split's reference (its rows are computed again) beside
    one element of a branch's value, or key, that is no number."""
    t, rise = 5, 200.0
    q = P8.bf16(np.random.default_rng(85), t, hq * d).reshape(t, hq, d)
    q[:] = q[:1, :1]
    dirn = q[0, 0].double() / q[0, 0].double().norm()
    ramp = torch.linspace(0, 1, n_q8, dtype=torch.float64) * rise * math.sqrt(d) / float(q[0, 0].double().norm())
    parent = [-1, 0, 0, 1, 2]
    vis = P8.sees(parent)
    for flip in (False, True):
        c = P8.cache_inputs(86, hkv, d, n_q8, n_tail, t)
        rows = (ramp.flip(0) if flip else ramp)[None, :, None] * dirn
        codes, byte = P8.quantize(rows.expand(hkv, n_q8, d).to(torch.bfloat16))
        c["k8"], c["k_scale"] = codes.float().to(torch.float8_e4m3fn), byte
        k, v = (P8.cache_rows(c, x, n_q8, 0, n_tail + t) for x in "kv")
        want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
        c["v_tail"][:, n_tail + 2, 7] = what
        c["k_tail"][:, n_tail + 3, d - 2] = what
        cache = L.KvCacheQ8(**{x: y.cuda() for x, y in c.items()}, n_q8=n_q8, n_tail=n_tail)
        out = L.tree_verify_attn_q8(q.cuda(), cache, parent).double().cpu()
        hit = vis[:, 2] | vis[:, 3]
        assert bool(torch.isnan(out[hit]).all()), flip
        assert bool(((out - want).abs() <= bound)[~hit].all()), flip


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


@pytest.mark.parametrize("hq,hkv,d,n_q8", KERNELS)
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_root_scores_of_a_block_that_is_no_number(hq, hkv, d, n_q8, which):
    """A block of K has NaN for its scores, a block of V its keys' own."""
    n_tail, t = 9, 4
    c = P8.cache_inputs(87, hkv, d, n_q8, n_tail, t)
    q = P8.bf16(np.random.default_rng(88), t, hq * d).reshape(t, hq, d)
    k = P8.cache_rows(c, "k", n_q8, 0, n_tail)
    c[which][1, 1] = 255
    cache = L.KvCacheQ8(**{x: y.cuda() for x, y in c.items()}, n_q8=n_q8, n_tail=n_tail)
    rs = torch.zeros(hq, n_q8 + n_tail, device="cuda")
    L.tree_verify_attn_q8(q.cuda(), cache, P8.parents("chain", t), root_scores_out=rs)
    got = rs.double().cpu().reshape(hkv, hq // hkv, -1)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[1, :, 64:128] = which == "k_scale"
    assert torch.equal(torch.isnan(got), nan)
    kk = torch.cat([k, torch.zeros(hkv, 1, d, dtype=torch.float64)], 1)
    _, _, wr, br = P8.attention(q[:1], kk, torch.zeros_like(kk), n_q8 + n_tail, [-1], d ** -0.5)
    err = (got - wr.reshape(got.shape)).abs()
    assert bool((err <= br.reshape(got.shape))[~nan].all())


@pytest.mark.parametrize("hq,hkv,d,n_q8", KERNELS)
@pytest.mark.parametrize("what", [math.inf, math.nan])
def test_a_query_that_is_no_number_reaches_its_own_row(hq, hkv, d, n_q8, what):
    n_tail, t = 9, 5
    c = P8.cache_inputs(89, hkv, d, n_q8, n_tail, t)
    q = P8.bf16(np.random.default_rng(84), t, hq * d).reshape(t, hq, d)
    k, v = (P8.cache_rows(c, x, n_q8, 0, n_tail + t) for x in "kv")
    parent = P8.parents("bfs", t)
    want, bound, wr, br = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
    q[0, 1, 5], q[3, hq - 1, d - 1] = what, what
    cache = L.KvCacheQ8(**{x: y.cuda() for x, y in c.items()}, n_q8=n_q8, n_tail=n_tail)
    rs = torch.zeros(hq, n_q8 + n_tail, device="cuda")
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs).double().cpu()
    hit = torch.zeros(t, hq, dtype=torch.bool)
    hit[0, 1] = hit[3, hq - 1] = True
    assert bool(torch.isnan(out[hit]).all())
    assert bool(((out - want).abs() <= bound)[~hit].all())
    rest = [h for h in range(hq) if h != 1]
    assert bool(((rs.double().cpu() - wr).abs() <= br)[rest].all())


# ------------------------------------------------------- one large element in a row
@pytest.mark.parametrize("hq,hkv,d,n_q8", KERNELS)
@pytest.mark.parametrize("power", [6, 12, 20])
def test_small_elements_beside_a_large_one(hq, hkv, d, n_q8, power):
    """Queries with one element 2^power times the others, where every key has a zero,
    and tail keys with another where every query has one.  Down to 2^-14 of the
    largest the others count in full, a smaller one may be off by 2^-21 of it."""
    t, n_tail = 5, 70
    c = P8.cache_inputs(98, hkv, d, n_q8, n_tail, t)
    rng = np.random.default_rng(99)
    q = P8.bf16(rng, t, hq * d).reshape(t, hq, d)
    x = c["k8"].view(torch.uint8)
    x[:, :, 3] = 0
    x[:, :, 9] = 0
    c["k_tail"][:, :, 3] = 0.0
    c["k_tail"][:, :, 9] = 2.0 ** power
    q[..., 3] = 2.0 ** power
    q[..., 9] = 0.0
    cache = L.KvCacheQ8(**{k: y.cuda() for k, y in c.items()}, n_q8=n_q8, n_tail=n_tail)
    n, parent, scale = n_q8 + n_tail, P8.parents("chain", t), d ** -0.5
    rs = torch.empty(hq, n, device="cuda")
    L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs)
    k = P8.cache_rows(c, "k", n_q8, 0, n_tail)
    g = hq // hkv
    q0 = q[0].double().reshape(hkv, g, d)
    want = torch.einsum("hgd,hnd->hgn", q0, k).reshape(hq, n) * scale / math.log(2)
    mag = torch.einsum("hgd,hnd->hgn", q0.abs(), k.abs()).reshape(hq, n)
    # (an element is split without loss from 2^-6 of the scaled row on, whose largest is
    # at most 448 and lies above 224: at least 2^-14 of it)
    far = 2.0 ** -21 * (q0.abs().amax(-1)[..., None] * k.abs().sum(-1)[:, None] +
                        q0.abs().sum(-1)[..., None] * k.abs().amax(-1)[:, None]).reshape(hq, n)
    bound = (mag * ((d + 8) * 2.0 ** -23 + 2.0 ** -20) + (far if power > 6 else 0.0)) * scale / math.log(2) + 1e-30
    err = (rs.double().cpu() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


# ----------------------------------------------------------- values near nothing
def test_weights_over_blocks_of_zeros_count():
    """2^20 positions whose values are zeros (the least scale), each with a
    weight 2^-26.1 of the one position that has a value: together 1.4 % of the sum."""
    d, n = 128, 1 << 20
    zeros = torch.zeros(1, n, d, dtype=torch.uint8).view(torch.float8_e4m3fn)
    byte = torch.full((1, n // 64), 27, dtype=torch.uint8)
    k_tail, v_tail = torch.zeros(1, 1, d), torch.ones(1, 1, d)
    q = torch.zeros(1, 1, d)
    q[..., 0] = 1.0
    k_tail[..., 0] = 26.125
    c = dict(k8=zeros, v8=zeros.clone(), k_scale=byte, v_scale=byte.clone(),
             k_tail=k_tail.to(torch.bfloat16), v_tail=v_tail.to(torch.bfloat16))
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n, n_tail=0)
    out = L.tree_verify_attn_q8(q.to(torch.bfloat16).cuda(), cache, [-1], softmax_scale=math.log(2))
    want = 1.0 / (1.0 + n * 2.0 ** -26.125)
    # its one rounding, the weights' (each way) and the sum of 2^20 terms in 32 bits
    assert float((out.double().cpu() - want).abs().max()) <= (2.0 ** -8 + 2.0 ** -8 * (1 - want)) * want + 2.0 ** -12


# ------------------------------------------------------------ rotation of long prompts
@pytest.mark.parametrize("hq,hkv,d,rot,inter,n", [
    (8, 2, 128, 128, False, 2303), (8, 2, 128, 128, True, 8190), (4, 2, 64, 64, False, 8190),
    (4, 2, 64, 32, True, 2303), (5, 1, 128, 64, False, 4801), (3, 3, 64, 20, False, 2303),
    (0, 2, 128, 96, True, 8190),
])
def test_rope_append_of_long_prompts(hq, hkv, d, rot, inter, n):
    """Runs of several tokens per CTA, the last one short."""
    rng = np.random.default_rng(n + rot)
    fused = P8.bf16(rng, n, (hq + 2 * hkv) * d).reshape(n, hq + 2 * hkv, d)
    q, k, v = fused.cuda().split([hq, hkv, hkv], 1)
    freq, m = L.rope_inv_freq(rot, 500000.0, "wavelength", 8.0, 1.0, 4.0, 8192.0)
    cap, row0, pos0 = n + 5, 2, 24571
    kc, vc = (torch.full((hkv, cap, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = L.rope_append(q if hq else None, k, v, kc, vc, row0, pos0, freq.cuda(), interleaved=inter, mscale=m)
    cq, ck, cv = fused.split([hq, hkv, hkv], 1)
    for x, y in ((cq, got), (ck, kc[:, row0:row0 + n].transpose(0, 1))):
        if x.shape[1] == 0:
            continue
        want = P8.rotate(x, range(pos0, pos0 + n), freq, inter, m)
        bound = 2.0 ** -8 * want.abs() + P8.rotate_bound(x, freq, inter, m)
        assert bool(((y.cpu().double() - want).abs() <= bound).all())
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
    assert torch.equal(vc[:, row0:row0 + n].cpu(), cv.transpose(0, 1))
    for x in (kc, vc):
        assert bool((x[:, :row0] == 3.0).all()) and bool((x[:, row0 + n:] == 3.0).all())


# ------------------------------------------------------------ captured calls
def test_graphs_that_share_a_workspace_and_one_that_makes_its_own():
    """Two captured calls of different shapes on one workspace, replayed in turn, and
    one whose workspace and output were made while it was captured."""
    shapes = [(16, 4, 128, 8128, 40, 13), (8, 2, 64, 192, 20, 1), (160, 40, 128, 1024, 20, 40)]
    ws = L.new_workspace(max(L.tree_verify_attn_q8_workspace_size(*s) for s in shapes))
    jobs = []
    for i, shape in enumerate(shapes):
        q, cache, parent = random_call(7 + i, *shape)
        eager = L.tree_verify_attn_q8(q, cache, parent)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = L.tree_verify_attn_q8(q, cache, parent, workspace=ws if i < 2 else None)
        jobs.append((graph, out, eager, cache, q))
    for _ in range(5):
        for graph, out, _, _, _ in jobs:
            out.zero_()
            graph.replay()
        for _, out, eager, _, _ in jobs:
            assert torch.equal(out, eager)
    assert L.workspace_status(ws) == 0
