"""The 8-bit cache's operators on the GPU against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import lossless_ultra_long_b200 as L
import q8_plain as P8

pytestmark = pytest.mark.gpu


def make(seed, hkv, d, n_q8, n_tail, t, **kw):
    c = P8.cache_inputs(seed, hkv, d, n_q8, n_tail, t, **kw)
    row0 = kw.get("tail_row0", 0)
    dev = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=n_tail,
                      tail_row0=row0)
    return c, dev


def queries(seed, t, hq, d):
    return P8.bf16(np.random.default_rng(1000 + seed), t, hq * d).reshape(t, hq, d)


def check_attention(seed, hq, hkv, d, n_q8, n_tail, t, tree, root=True, scale=None, **kw):
    row0 = kw.get("tail_row0", 0)
    c, cache = make(seed, hkv, d, n_q8, n_tail, t, **kw)
    q = queries(seed, t, hq, d)
    parent = P8.parents(tree, t, seed)
    n = n_q8 + n_tail
    rs = torch.full((hq, n), math.nan, device="cuda") if root else None
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent, root_scores_out=rs, softmax_scale=scale)
    k = P8.cache_rows(c, "k", n_q8, row0, n_tail + t)
    v = P8.cache_rows(c, "v", n_q8, row0, n_tail + t)
    want, bound, wr, br = P8.attention(q, k, v, n, parent, d ** -0.5 if scale is None else scale)
    err = (out.double().cpu() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    if root:
        err = (rs.double().cpu() - wr).abs()
        assert bool((err <= br).all()), float((err / br).max())


# (hq, hkv, d, n_q8, n_tail, t, tree)
SHAPES = [
    (1, 1, 64, 0, 0, 1, "chain"),        # a token that sees only itself
    (8, 2, 64, 0, 5, 1, "chain"),        # all of the context in the tail
    (8, 2, 64, 64, 0, 4, "chain"),       # no context in the tail
    (8, 2, 64, 192, 20, 1, "chain"),
    (8, 2, 64, 1984, 64, 13, "bfs"),
    (8, 1, 64, 640, 63, 64, "random"),
    (3, 3, 64, 448, 1, 7, "star"),
    (36, 4, 64, 128, 130, 33, "random"),
    (2, 1, 128, 0, 0, 64, "random"),
    (4, 4, 128, 64, 127, 2, "chain"),
    (32, 8, 128, 1024, 37, 1, "chain"),
    (32, 8, 128, 1984, 63, 40, "bfs"),
    (40, 8, 128, 2112, 29, 40, "bfs"),   # 200 query rows per KV head
    (8, 1, 128, 4096, 300, 64, "random"),   # 512 rows, a tail of several tiles
    (5, 1, 128, 2048, 0, 13, "bfs"),
    (64, 64, 128, 2176, 3, 4, "chain"),
    (12, 1, 128, 3200, 64, 11, "random"),
    (32, 8, 128, 8128, 51, 40, "bfs"),
    (32, 8, 128, 8192, 0, 4, "chain"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_attention(shape):
    check_attention(sum(map(len, map(str, shape))), *shape)


def test_attention_rows_outside_the_cache_are_not_read():
    check_attention(3, 8, 2, 64, 320, 17, 9, "random", cap=512, tail_cap=200, tail_row0=70)
    check_attention(4, 16, 4, 128, 2240, 17, 9, "random", cap=2560, tail_cap=200, tail_row0=70)
    check_attention(4, 148, 74, 128, 704, 17, 9, "random", cap=768, tail_cap=200, tail_row0=70)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_attention_scales(scale):
    check_attention(5, 8, 2, 64, 128, 9, 5, "bfs", scale=scale)
    check_attention(6, 8, 2, 128, 2176, 9, 5, "bfs", scale=scale)
    check_attention(6, 74, 74, 128, 640, 9, 5, "bfs", scale=scale)


@pytest.mark.parametrize("hq,hkv,d,n_q8", [(8, 2, 64, 128), (16, 4, 128, 2176), (148, 74, 128, 640)])
def test_unseen_rows_may_hold_anything(hq, hkv, d, n_q8):
    """NaN and infinities in a branch reach its own nodes alone."""
    t, n_tail = 13, 30
    c, _ = make(7, hkv, d, n_q8, n_tail, t)
    parent = P8.parents("bfs", t)
    q = queries(7, t, hq, d)
    clean = L.tree_verify_attn_q8(q.cuda(), make(7, hkv, d, n_q8, n_tail, t)[1], parent)
    c["k_tail"][:, n_tail + 2, 3] = math.nan
    c["v_tail"][:, n_tail + 3, 5] = math.inf
    c["v_tail"][:, n_tail + 12, :] = -math.inf
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=n_tail)
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent).float().cpu()
    vis = P8.sees(parent)
    hit = vis[:, 2] | vis[:, 3] | vis[:, 12]
    assert bool(hit.any()) and not bool(hit.all())
    assert bool(torch.isnan(out[hit]).all())
    k, v = (P8.cache_rows(P8.cache_inputs(7, hkv, d, n_q8, n_tail, t), n, n_q8, 0, n_tail + t)
            for n in "kv")
    want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
    assert bool(((out.double() - want).abs() <= bound)[~hit].all())
    assert bool(torch.isfinite(clean).all())


@pytest.mark.parametrize("hq,hkv,d,n_q8", [(8, 2, 64, 128), (16, 4, 128, 2176), (148, 74, 128, 640)])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_a_block_that_is_not_a_number_reaches_its_head(hq, hkv, d, n_q8, which):
    c, _ = make(8, hkv, d, n_q8, 9, 4)
    c[which][1, 1] = 255
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=9)
    out = L.tree_verify_attn_q8(queries(8, 4, hq, d).cuda(), cache, P8.parents("chain", 4))
    nan = torch.isnan(out).reshape(4, hkv, -1)
    assert bool(nan[:, 1].all()) and not bool(nan[:, [0] + list(range(2, hkv))].any())


@pytest.mark.parametrize("hq,hkv,d,n_q8", [(8, 2, 64, 192), (16, 4, 128, 2176), (148, 74, 128, 640)])
def test_extreme_scales(hq, hkv, d, n_q8):
    """Values far apart: tiny values of V in one block, large ones in another; small keys."""
    c, _ = make(9, hkv, d, n_q8, 9, 4)
    c["v_scale"][:, 0] = 127 - 100
    c["v_scale"][:, 1] = 127 + 60
    c["k_scale"][:, 2] = 127 - 100
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=9)
    q, parent = queries(9, 4, hq, d), P8.parents("chain", 4)
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent)
    k, v = (P8.cache_rows(c, n, n_q8, 0, 13) for n in "kv")
    want, bound, _, _ = P8.attention(q, k, v, n_q8 + 9, parent, d ** -0.5)
    assert bool(((out.double().cpu() - want).abs() <= bound).all())


@pytest.mark.parametrize("hq,hkv,d,n_q8,n_tail", [(8, 2, 64, 2048, 9), (16, 4, 128, 4096, 9),
                                                  (32, 8, 128, 2176, 150), (74, 74, 128, 1024, 9),
                                                  (37, 37, 128, 2048, 150)])
@pytest.mark.parametrize("rise", [30.0, 200.0])
def test_scores_that_rise_along_the_context(hq, hkv, d, n_q8, n_tail, rise):
    """Keys whose score grows by `rise` nats towards either end: the first
    tile a kernel meets says nothing about the largest score."""
    t = 5
    q = queries(10, t, hq, d)
    q[:] = q[:1, :1]
    dirn = q[0, 0].double() / q[0, 0].double().norm()
    for flip in (False, True):
        c, _ = make(10, hkv, d, n_q8, n_tail, t)
        ramp = torch.linspace(0, 1, n_q8, dtype=torch.float64)
        ramp = ramp.flip(0) if flip else ramp
        size = rise * math.sqrt(d) / float(q[0, 0].double().norm())
        rows = (ramp[None, :, None] * size * dirn).expand(hkv, n_q8, d).to(torch.bfloat16)
        codes, byte = P8.quantize(rows)
        c["k8"] = codes.float().to(torch.float8_e4m3fn)
        c["k_scale"] = byte
        cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=n_q8, n_tail=n_tail)
        parent = P8.parents("random", t, 1)
        out = L.tree_verify_attn_q8(q.cuda(), cache, parent)
        k, v = (P8.cache_rows(c, n, n_q8, 0, n_tail + t) for n in "kv")
        want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
        err = (out.double().cpu() - want).abs()
        assert bool((err <= bound).all()), (flip, float((err / bound).max()))


@pytest.mark.parametrize("shapes", [
    [(16, 4, 128, 2176, 9, 13), (8, 2, 64, 320, 20, 5), (16, 4, 128, 4096, 63, 40)],
    [(74, 74, 128, 640, 9, 13), (8, 2, 64, 320, 20, 5), (120, 40, 128, 1024, 63, 60)],
], ids=["short", "long"])
def test_attention_reuses_a_workspace_and_a_graph(shapes):
    """One workspace over calls of other shapes; a captured call replayed with
    new contents of the same buffers, while a second graph has its own."""
    ws = L.new_workspace(max(L.tree_verify_attn_q8_workspace_size(*s) for s in shapes))
    for i, (hq, hkv, d, n_q8, n_tail, t) in enumerate(shapes + shapes):
        c, cache = make(20 + i, hkv, d, n_q8, n_tail, t)
        q, parent = queries(20 + i, t, hq, d), P8.parents("bfs", t)
        out = L.tree_verify_attn_q8(q.cuda(), cache, parent, workspace=ws)
        k, v = (P8.cache_rows(c, n, n_q8, 0, n_tail + t) for n in "kv")
        want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
        assert bool(((out.double().cpu() - want).abs() <= bound).all()), i
        assert L.workspace_status(ws) == 0

    graphs = []
    for seed, (hq, hkv, d, n_q8, n_tail, t) in ((30, shapes[0]), (31, shapes[2])):
        _, cache = make(seed, hkv, d, n_q8, n_tail, t)
        q = queries(seed, t, hq, d).cuda()
        out = torch.empty_like(q)
        own = L.new_workspace(L.tree_verify_attn_q8_workspace_size(hq, hkv, d, n_q8, n_tail, t))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.tree_verify_attn_q8(q, cache, P8.parents("bfs", t), out=out, workspace=own)
        # (the graph's replays use the workspace, too: it must live as long)
        graphs.append((g, q, cache, out, own, t))
    for rep in range(3):
        for j, (g, q, cache, out, own, t) in enumerate(graphs):
            q.copy_(queries(40 + rep, t, q.shape[1], q.shape[2]))
            g.replay()
        torch.cuda.synchronize()
        for j, (g, q, cache, out, own, t) in enumerate(graphs):
            eager = L.tree_verify_attn_q8(q, cache, P8.parents("bfs", t))
            # both within one bound of the truth; they differ by summation order
            assert float((out.float() - eager.float()).abs().max()) <= 2.0 ** -6 * float(
                eager.float().abs().max()), (rep, j)


def test_attention_on_another_stream():
    hq, hkv, d, n_q8, n_tail, t = 16, 4, 128, 2176, 9, 13
    c, cache = make(50, hkv, d, n_q8, n_tail, t)
    q, parent = queries(50, t, hq, d), P8.parents("bfs", t)
    s = torch.cuda.Stream()
    dq = q.cuda()
    ws = L.new_workspace(L.tree_verify_attn_q8_workspace_size(hq, hkv, d, n_q8, n_tail, t))
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(dq)
    L.tree_verify_attn_q8(dq, cache, parent, out=out, workspace=ws, stream=s)
    s.synchronize()
    k, v = (P8.cache_rows(c, n, n_q8, 0, n_tail + t) for n in "kv")
    want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
    assert bool(((out.double().cpu() - want).abs() <= bound).all())


# ----------------------------------------------------------------- quantisation
@pytest.mark.parametrize("hkv,d,rows,row0,dst,cap,src_cap", [
    (1, 64, 64, 0, 0, 64, 64), (8, 128, 64, 13, 128, 256, 100), (2, 64, 640, 3, 64, 768, 650),
    (3, 128, 192, 0, 0, 192, 192),
])
def test_quantize(hkv, d, rows, row0, dst, cap, src_cap):
    rng = np.random.default_rng(rows + d)
    k, v = (P8.bf16(rng, hkv, src_cap, d, spread=1.5) for _ in range(2))
    if rows >= 192:
        k[0, row0 + 5, 7] = math.inf                       # block 0: not a number
        v[hkv - 1, row0 + 64, 0] = math.nan
        k[0, row0 + 64:row0 + 128] = 0                     # an empty block
        v[0, row0 + 128:row0 + 192] *= 2.0 ** -112         # below the least scale
        k[hkv - 1, row0 + 128:row0 + 192] = 3.3e38         # the largest scale
        k[hkv - 1, row0, :] = 2.0 ** -133                  # subnormal
    k8, v8 = (torch.full((hkv, cap, d), 0x55, dtype=torch.uint8, device="cuda").view(
        torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((hkv, cap // 64), 7, dtype=torch.uint8, device="cuda") for _ in range(2))
    L.kv_quantize_q8(k.cuda(), v.cuda(), row0, rows, k8, v8, ks, vs, dst)
    for x, codes, sc in ((k, k8, ks), (v, v8, vs)):
        want, byte = P8.quantize(x[:, row0:row0 + rows])
        got = codes.float().cpu().double()
        assert torch.equal(got[:, dst:dst + rows], want)
        assert torch.equal(sc[:, dst // 64:(dst + rows) // 64].cpu(), byte)
        rest = codes.view(torch.uint8).cpu()
        assert bool((rest[:, :dst] == 0x55).all()) and bool((rest[:, dst + rows:] == 0x55).all())
        assert bool((sc[:, :dst // 64] == 7).all()) and bool((sc[:, (dst + rows) // 64:] == 7).all())


# ----------------------------------------------------------------------- gather
@pytest.mark.parametrize("hkv,d,n_q8,n_tail,keep,cap", [
    (1, 64, 0, 5, 5, 5), (2, 64, 1984, 64, 256, 300), (8, 128, 1024, 0, 1, 1),
    (3, 128, 640, 100, 700, 741),
])
def test_gather(hkv, d, n_q8, n_tail, keep, cap):
    c, cache = make(60, hkv, d, n_q8, n_tail, 0, cap=n_q8 + 64, tail_cap=n_tail + 9, tail_row0=4)
    rng = np.random.default_rng(keep)
    idx = torch.from_numpy(np.stack([np.sort(rng.permutation(n_q8 + n_tail)[:keep])
                                     for _ in range(hkv)]).astype(np.int32))
    kp, vp = (torch.full((hkv, cap, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = L.new_workspace(256)
    L.kv_gather_q8(cache, idx.cuda(), k_partial=kp, v_partial=vp, workspace=ws)
    assert L.workspace_status(ws) == 0
    for got, name in ((kp, "k"), (vp, "v")):
        every = P8.cache_rows(c, name, n_q8, 4, n_tail)
        want = torch.gather(every, 1, idx.long()[..., None].expand(-1, -1, d))
        assert torch.equal(got[:, :keep].cpu().double(), want)     # exact: 4 bits and a power of two
        assert bool((got[:, keep:] == 3.0).all())


def test_gather_flags_bad_positions():
    c, cache = make(61, 2, 64, 128, 10, 0)
    idx = torch.tensor([[0, 137, 138], [-1, 5, 2 ** 31 - 1]], dtype=torch.int32)
    ws = L.new_workspace(256)
    kp, vp = L.kv_gather_q8(cache, idx.cuda(), workspace=ws)
    assert L.workspace_status(ws) == 6
    want = P8.cache_rows(c, "k", 128, 0, 10)
    assert torch.equal(kp[0, :2].cpu().double(), want[0, [0, 137]])
    assert torch.equal(kp[1, 1].cpu().double(), want[1, 5])
    for x in (kp, vp):
        assert bool((x[0, 2] == 0).all()) and bool((x[1, [0, 2]] == 0).all())


def test_gather_keeps_a_bad_block_bad():
    c, _ = make(62, 2, 64, 128, 0, 0)
    c["v_scale"][1, 1] = 255
    cache = L.KvCacheQ8(**{k: x.cuda() for k, x in c.items()}, n_q8=128, n_tail=0)
    idx = torch.tensor([[3, 100], [63, 64]], dtype=torch.int32).cuda()
    kp, vp = L.kv_gather_q8(cache, idx)
    assert bool(torch.isfinite(kp).all()) and bool(torch.isfinite(vp[0]).all())
    assert bool(torch.isfinite(vp[1, 0]).all()) and bool(torch.isnan(vp[1, 1]).all())


# ----------------------------------------------------------------------- rotation
@pytest.mark.parametrize("hq,hkv,d,rot,inter,n,tree,pos0", [
    (8, 2, 64, 64, False, 1, "chain", 0), (8, 2, 64, 64, True, 13, "bfs", 2048),
    (32, 8, 128, 128, False, 40, "bfs", 102387), (32, 8, 128, 64, False, 64, "random", 131071),
    (5, 1, 128, 128, True, 7, "random", 99999), (3, 3, 64, 20, False, 9, None, 77),
    (3, 3, 64, 22, True, 9, None, 77), (2, 1, 128, 2, False, 3, None, 1 << 20),
    (2, 1, 128, 0, False, 3, None, 5), (4, 2, 128, 126, False, 300, None, 50000),
    (0, 2, 128, 128, False, 5, "chain", 9), (16, 8, 128, 128, False, 1000, None, 0),
])
def test_rope_append(hq, hkv, d, rot, inter, n, tree, pos0):
    rng = np.random.default_rng(n)
    fused = P8.bf16(rng, n, (hq + 2 * hkv) * d).reshape(n, hq + 2 * hkv, d)
    dev = fused.cuda()
    q, k, v = dev.split([hq, hkv, hkv], 1)
    freq, m = L.rope_inv_freq(rot, 10000.0, "yarn", 8.0, 4096.0, 32.0, 1.0)
    cap, row0 = n + 11, 6
    kc, vc = (torch.full((hkv, cap, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    parent = P8.parents(tree, n, 3) if tree else None
    got = L.rope_append(q if hq else None, k, v, kc, vc, row0, pos0, freq.cuda(), parent=parent,
                        interleaved=inter, mscale=m)
    pos = [pos0 + x for x in (P8.depths(parent) if tree else range(n))]
    cq, ck, cv = fused.split([hq, hkv, hkv], 1)
    for x, y in ((cq, got), (ck, kc[:, row0:row0 + n].transpose(0, 1))):
        if x.shape[1] == 0:
            assert y is None
            continue
        want = P8.rotate(x, pos, freq, inter, m)
        bound = 2.0 ** -8 * want.abs() + P8.rotate_bound(x, freq, inter, m)
        err = (y.cpu().double() - want).abs()
        assert bool((err <= bound).all()), float((err - bound).max())
        if rot < d:
            assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
    assert torch.equal(vc[:, row0:row0 + n].cpu(), cv.transpose(0, 1))
    for x in (kc, vc):
        assert bool((x[:, :row0] == 3.0).all()) and bool((x[:, row0 + n:] == 3.0).all())


def test_rope_in_place():
    rng = np.random.default_rng(5)
    q, k, v = (P8.bf16(rng, 6, h * 64).reshape(6, h, 64) for h in (8, 2, 2))
    freq = L.rope_inv_freq(64, 10000.0)[0].cuda()
    kc, vc = (torch.zeros(2, 6, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dq = q.cuda()
    want = L.rope_append(dq, k.cuda(), v.cuda(), kc, vc, 0, 100, freq)
    got = L.rope_append(dq, k.cuda(), v.cuda(), kc, vc, 0, 100, freq, q_out=dq)
    assert got.data_ptr() == dq.data_ptr() and torch.equal(got, want)


def test_rope_far_positions_past_32_bits_of_elements():
    """Rows far down a long cache: offsets past 2^31 elements."""
    hkv, d, n = 2, 128, 4
    cap = (1 << 24) + 100     # 2 heads x 16.8M rows x 128: 8.6 GB
    kc = torch.empty((hkv, cap, d), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(6)
    k, v = (P8.bf16(rng, n, hkv * d).reshape(n, hkv, d) for _ in range(2))
    freq = L.rope_inv_freq(d, 10000.0)[0]
    vc = torch.empty_like(kc)
    L.rope_append(None, k.cuda(), v.cuda(), kc, vc, cap - n, (1 << 33) + 7, freq.cuda())
    want = P8.rotate(k, [(1 << 33) + 7 + i for i in range(n)], freq, False, 1.0)
    bound = 2.0 ** -8 * want.abs() + P8.rotate_bound(k, freq, False, 1.0)
    got = kc[:, cap - n:].transpose(0, 1).cpu().double()
    # the angle itself: 2^33 turns lose 2^-20 of 64 bits' 2^-53, still far below 2^-21
    assert bool(((got - want).abs() <= bound).all())
    assert torch.equal(vc[:, cap - n:].transpose(0, 1).cpu(), v)


# ------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("hq,hkv,d,prompt", [(8, 2, 64, 500), (16, 4, 128, 2300), (80, 40, 128, 900)])
def test_steps(hq, hkv, d, prompt):
    """A prompt, then steps of a drafted tree: append, verify, select, gather,
    accept, commit, fold; every step's attention against the cache that the
    plain forms keep, and the draft cache against the same positions."""
    rng = np.random.default_rng(9)
    t, vocab, n_sink, budget = 13, 512, 4, 60
    parent = P8.parents("bfs", t)
    freq, m = L.rope_inv_freq(d, 500000.0, "wavelength", 8.0, 1.0, 4.0, 8192.0)
    dfreq = freq.cuda()
    cache = L.KvCacheQ8.empty(hkv, d, prompt + 512, tail_rows=prompt + 64)
    ctx = {"k": torch.zeros(hkv, 0, d, dtype=torch.float64),
           "v": torch.zeros(hkv, 0, d, dtype=torch.float64)}
    fused = P8.bf16(rng, prompt, (hq + 2 * hkv) * d).reshape(prompt, -1, d)
    q, k, v = fused.cuda().split([hq, hkv, hkv], 1)
    cache.append(q, k, v, dfreq, mscale=m)
    tail = {n: getattr(cache, n + "_tail")[:, :prompt].cpu() for n in "kv"}
    assert torch.equal(tail["v"], fused[:, hq + hkv:].transpose(0, 1))
    folded = 0

    def fold():
        nonlocal folded
        n = cache.fold()
        for name in "kv":
            if n:
                codes, byte = P8.quantize(tail[name][:, :n])
                ctx[name] = torch.cat([ctx[name], codes * P8.factors(byte).repeat_interleave(64, 1)[..., None]], 1)
                tail[name] = tail[name][:, n:]
        folded += n

    fold()
    for step in range(9):
        fused = P8.bf16(rng, t, (hq + 2 * hkv) * d).reshape(t, -1, d)
        q, k, v = fused.cuda().split([hq, hkv, hkv], 1)
        n = cache.n_ctx
        assert n == ctx["k"].shape[1] + tail["k"].shape[1]
        tq = cache.append(q, k, v, dfreq, parent=parent, mscale=m)
        rs = torch.empty((hq, n), device="cuda")
        out = L.tree_verify_attn_q8(tq, cache, parent, root_scores_out=rs)
        at = cache.tail_row0 + cache.n_tail
        tree = {x: getattr(cache, x + "_tail")[:, at:at + t].cpu() for x in "kv"}
        kk, vv = (torch.cat([ctx[x], tail[x].double(), tree[x].double()], 1) for x in "kv")
        want, bound, wr, br = P8.attention(tq.cpu(), kk, vv, n, parent, d ** -0.5)
        assert bool(((out.double().cpu() - want).abs() <= bound).all()), step
        assert bool(((rs.double().cpu() - wr).abs() <= br).all()), step
        idx, kp, vp, _ = L.kv_select_from_scores_q8(rs, cache, n_sink, budget)
        ii = idx.cpu().long()
        assert bool((ii[:, 1:] > ii[:, :-1]).all()) and torch.equal(ii[0, :n_sink], torch.arange(n_sink))
        assert torch.equal(kp.cpu().double(), torch.gather(kk, 1, ii[..., None].expand(-1, -1, d)))
        assert torch.equal(vp.cpu().double(), torch.gather(vv, 1, ii[..., None].expand(-1, -1, d)))
        logits = torch.from_numpy(rng.standard_normal((t, vocab)).astype(np.float32)).cuda()
        top = logits.argmax(-1).cpu().tolist()
        tokens = [0] + [top[parent[i]] if (i % 3) == step % 3 else vocab + i for i in range(1, t)]
        acc, _ = L.penalize_accept(logits, None, 1.0, parent,
                                   torch.tensor(tokens, dtype=torch.int32, device="cuda"))
        a = acc.cpu().tolist()
        cache.commit(acc, t, a[0])
        path = a[2:3 + a[0]]
        for x in "kv":
            tail[x] = torch.cat([tail[x], tree[x][:, path]], 1)
        for _ in range(3):    # plain decoding in between: more rows
            one = P8.bf16(rng, 5, (hq + 2 * hkv) * d).reshape(5, -1, d)
            q, k, v = one.cuda().split([hq, hkv, hkv], 1)
            before = cache.tail_row0 + cache.n_tail
            cache.append(q, k, v, dfreq, mscale=m)
            for x in "kv":
                tail[x] = torch.cat([tail[x], getattr(cache, x + "_tail")[:, before:before + 5].cpu()], 1)
        fold()
    assert folded > prompt // 64 * 64


def test_select_is_the_bf16_caches_select():
    """The same scores select the same positions as on a bf16 cache."""
    hq, hkv, d, n_q8, n_tail = 16, 4, 128, 2176, 24
    c, cache = make(70, hkv, d, n_q8, n_tail, 0)
    n = n_q8 + n_tail
    rs = torch.from_numpy(np.random.default_rng(70).standard_normal((hq, n)).astype(np.float32)).cuda()
    k, v = (P8.cache_rows(c, x, n_q8, 0, n_tail).to(torch.bfloat16).cuda() for x in "kv")
    for call in (lambda: L.kv_select_from_scores_q8(rs, cache, 0, 0),
                 lambda: L.kv_select_from_scores(rs, k, v, n, 0, 0)):
        with pytest.raises(L.TsError):     # nothing to keep: neither takes the empty result
            call()
    for sink, budget in ((16, 240), (0, 1), (5, 0), (64, n)):
        idx, kp, vp, sc = L.kv_select_from_scores_q8(rs, cache, sink, budget, want_scores=True)
        wi, wk, wv, ws = L.kv_select_from_scores(rs, k, v, n, sink, budget, want_scores=True)
        assert torch.equal(idx, wi) and torch.equal(kp, wk) and torch.equal(vp, wv)
        assert torch.equal(sc, ws)


def test_a_cache_on_another_device_is_refused():
    _, cache = make(71, 2, 64, 64, 3, 4)
    with pytest.raises(ValueError):
        L.tree_verify_attn_q8(torch.zeros(4, 8, 64, dtype=torch.bfloat16), cache, [-1, 0, 1, 2])
    with pytest.raises(ValueError):
        L.tree_verify_attn_q8(torch.zeros(4, 8, 64, device="cuda"), cache, [-1, 0, 1, 2])
    with pytest.raises(ValueError):
        L.tree_verify_attn_q8(torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda"), cache,
                              [-1, 0, 1, 2])


# ------------------------------------------- both attention kernels' borders
BORDERS = [
    (16, 4, 128, 704, 60, 3, "bfs"),      # 767 positions: the last of the short kernel's
    (16, 4, 128, 704, 60, 4, "bfs"),      # 768
    (32, 8, 128, 768, 0, 1, "chain"),
    (4, 4, 128, 0, 900, 5, "random"),     # bf16 rows alone: up to 64 query rows a head,
    (24, 8, 128, 0, 777, 40, "random"),   # up to 128,
    (32, 8, 128, 0, 1500, 40, "bfs"),     # up to 192
    (24, 8, 128, 832, 130, 40, "random"),
    (16, 1, 128, 1024, 63, 4, "star"),    # 64 rows a head
    (13, 1, 128, 1024, 63, 5, "star"),    # 65
    (32, 1, 128, 1024, 63, 6, "random"),  # 192
    (50, 1, 128, 1024, 10, 5, "bfs"),     # whole nodes of 50 rows: groups of 2, 2 and 1
    (130, 1, 128, 1024, 10, 2, "bfs"),    # a node's rows fit no block
    (10, 1, 128, 1024, 10, 13, "random"),   # root scores of more than 8 heads
    (160, 160, 128, 832, 10, 3, "bfs"),   # more KV heads than SMs
    (74, 74, 128, 832, 10, 3, "bfs"),
]


# the tcgen05 kernel: more than two tiles of 64 positions in turn per split,
# which many KV heads make of a short context
BORDERS += [
    (74, 74, 128, 192, 60, 4, "bfs"),       # 256 positions are four tiles of 64, two in turn:
    (74, 74, 128, 192, 61, 4, "bfs"),       # the general kernel's; one more
    (74, 74, 128, 320, 0, 1, "chain"),
    (148, 148, 128, 192, 0, 1, "chain"),    # a head is one CTA's
    (74, 74, 128, 0, 400, 5, "random"),     # bf16 rows alone: up to 64 query rows a head,
    (111, 37, 128, 0, 600, 40, "random"),   # up to 128,
    (148, 37, 128, 0, 800, 40, "bfs"),      # up to 192
    (111, 37, 128, 576, 130, 40, "random"),
    (592, 37, 128, 640, 63, 4, "star"),     # 64 rows a head
    (481, 37, 128, 640, 63, 5, "star"),     # 65
    (74, 37, 128, 640, 63, 64, "random"),   # 128
    (222, 74, 128, 448, 63, 43, "random"),  # 129: too few for a second block with the root's
    (259, 37, 128, 640, 63, 19, "random"),  # 133, the same
    (370, 74, 128, 448, 63, 27, "random"),  # 135: enough
    (185, 37, 128, 640, 63, 40, "random"),  # 200: two groups of nodes
    (1000, 20, 128, 640, 10, 5, "bfs"),     # whole nodes of 50 rows: groups of 2, 2 and 1
    (74, 74, 128, 704, 300, 64, "chain"),   # a tail of several tiles
]


@pytest.mark.parametrize("root", [False, True])
@pytest.mark.parametrize("shape", BORDERS, ids=lambda s: "-".join(map(str, s)))
def test_attention_borders(shape, root):
    check_attention(sum(map(len, map(str, shape))), *shape, root=root)


def test_attention_of_a_million_positions():
    """A head's scale bytes in shared memory (2 x 16 KB), 8-bit tiles numbered
    past 2^13; the plain form takes one head."""
    check_attention(80, 1, 1, 128, 1 << 20, 5, 2, "chain")


@pytest.mark.parametrize("n_q8", [128, 1024])
def test_attention_past_32_bits_of_elements(n_q8):
    """A head's rows start past element 2^31 of the codes and of the tail."""
    hkv, d, cap, n_tail, t = 18, 128, 1 << 20, 9, 4
    c = P8.cache_inputs(81, hkv, d, n_q8, n_tail, t)
    k8, v8 = (torch.zeros(hkv, cap, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = [torch.zeros(hkv, cap // 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k_tail, v_tail = (torch.zeros(hkv, cap, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for dst, name in ((k8, "k8"), (v8, "v8")):
        dst[:, :n_q8] = c[name].view(torch.uint8).cuda()[:, :n_q8]
    for dst, name in zip(scales, ("k_scale", "v_scale")):
        dst[:, :n_q8 // 64] = c[name].cuda()[:, :n_q8 // 64]
    row0 = cap - n_tail - t
    for dst, name in ((k_tail, "k_tail"), (v_tail, "v_tail")):
        dst[:, row0:] = c[name].cuda()
    cache = L.KvCacheQ8(k8.view(torch.float8_e4m3fn), v8.view(torch.float8_e4m3fn), *scales, k_tail,
                        v_tail, n_q8=n_q8, n_tail=n_tail, tail_row0=row0)
    q, parent = queries(81, t, 2 * hkv, d), P8.parents("bfs", t)
    out = L.tree_verify_attn_q8(q.cuda(), cache, parent)
    k, v = (P8.cache_rows(c, x, n_q8, 0, n_tail + t) for x in "kv")
    want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
    assert bool(((out.double().cpu() - want).abs() <= bound).all())

    # the same rows gathered, and the tail's last 64 quantised behind the codes
    idx = torch.arange(n_q8 + n_tail, dtype=torch.int32, device="cuda").expand(hkv, -1).contiguous()
    kp, vp = L.kv_gather_q8(cache, idx)
    assert torch.equal(kp.double().cpu(), k[:, :n_q8 + n_tail])
    assert torch.equal(vp.double().cpu(), v[:, :n_q8 + n_tail])
    L.kv_quantize_q8(k_tail, v_tail, cap - 64, 64, cache.k8, cache.v8, *scales, cap - 64)
    for rows, codes, byte in ((k_tail, cache.k8, scales[0]), (v_tail, cache.v8, scales[1])):
        wc, wb = P8.quantize(rows[:, cap - 64:].cpu())
        assert torch.equal(codes[:, cap - 64:].float().double().cpu(), wc)
        assert torch.equal(byte[:, -1:].cpu(), wb)


def test_attention_on_two_streams_at_once():
    """Calls on two streams, each with its workspace, in no order between them."""
    jobs = []
    for seed, (hq, hkv, d, n_q8, n_tail, t) in ((82, (16, 4, 128, 8192, 9, 13)),
                                               (83, (16, 4, 128, 4096, 63, 40)),
                                               (84, (8, 2, 64, 2048, 9, 5)),
                                               (85, (74, 74, 128, 640, 9, 13)),
                                               (86, (80, 40, 128, 1024, 9, 40))):
        c, cache = make(seed, hkv, d, n_q8, n_tail, t)
        q, parent = queries(seed, t, hq, d), P8.parents("bfs", t)
        k, v = (P8.cache_rows(c, n, n_q8, 0, n_tail + t) for n in "kv")
        want, bound, _, _ = P8.attention(q, k, v, n_q8 + n_tail, parent, d ** -0.5)
        ws = L.new_workspace(L.tree_verify_attn_q8_workspace_size(hq, hkv, d, n_q8, n_tail, t))
        jobs.append((torch.cuda.Stream(), q.cuda(), cache, parent, ws, want, bound))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, q, cache, parent, ws, _, _ in jobs:
            out = torch.empty_like(q)
            L.tree_verify_attn_q8(q, cache, parent, out=out, workspace=ws, stream=s)
            outs.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        _, _, _, _, ws, want, bound = jobs[i % len(jobs)]
        assert L.workspace_status(ws) == 0
        assert bool(((out.double().cpu() - want).abs() <= bound).all()), i


def test_a_cache_keeps_its_rows_in_bounds():
    cache = L.KvCacheQ8.empty(2, 64, 64, tail_rows=140)
    assert cache.n_ctx == 0 and cache.fold() == 0
    fused = torch.zeros(140, 6, 64, dtype=torch.bfloat16, device="cuda")
    q, k, v = fused.split([2, 2, 2], 1)
    freq = L.rope_inv_freq(64, 1e4)[0].cuda()
    with pytest.raises(L.TsError):           # one row more than the tail has
        cache.append(torch.cat([q, q[:1]]), torch.cat([k, k[:1]]), torch.cat([v, v[:1]]), freq)
    cache.append(q, k, v, freq)
    assert (cache.n_q8, cache.n_tail) == (0, 140)
    with pytest.raises(L.TsError):           # two blocks, room for one
        cache.fold()
    assert (cache.n_q8, cache.n_tail, cache.tail_row0) == (0, 140, 0)
    accept = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):          # a tree behind the tail's end
        cache.commit(accept, 1, 0)
    cache = L.KvCacheQ8.empty(2, 64, 64, tail_rows=140)
    for n_tree, n_accepted in ((4, 4), (4, -1), (0, 0)):
        with pytest.raises(ValueError):
            cache.commit(accept, n_tree, n_accepted)
    for kw in ({"n_q8": 63}, {"n_q8": 128}, {"n_q8": -64}, {"n_tail": 141}, {"n_tail": -1},
               {"tail_row0": -1}, {"n_tail": 100, "tail_row0": 41}):
        with pytest.raises(ValueError):
            L.KvCacheQ8(cache.k8, cache.v8, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail,
                        **kw)
