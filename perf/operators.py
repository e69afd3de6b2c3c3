"""The 8-bit KV cache's operators, with their plain forms.

One verification step over a cache held in 8 bits goes through four
operators: the rotation of the step's queries and keys with the append of its
K/V rows, the tree attention over the 8-bit blocks and the bf16 tail, the
gather of selected rows into the bf16 draft cache, and the quantisation of
the blocks that filled up.  ``own`` false computes each from elementary torch
operations; ``own`` true makes the framework's calls.

Cache format: rows in blocks of 64; a block of one KV head holds e4m3 codes
and one power-of-two scale, stored as its biased exponent (byte b is
2^(b - 127), 255 marks a block with a non-finite value).  The newest context
rows and the draft tree's rows are bf16, in a tail.
"""
import math

import torch

own = False

BLOCK = 64
LOG2E = 1.4426950408889634
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token over a short context: latency alone
        dict(name="attn_d64_n212_t1", op="attn", hq=8, hkv=2, d=64, n_q8=192, n_tail=20, t=1,
             tree="chain", root=False),
        # the small workload: a 13-node tree over 2048 positions, head_dim 64
        dict(name="attn_d64_n2048_t13", op="attn", hq=8, hkv=2, d=64, n_q8=1984, n_tail=64, t=13,
             tree="bfs", root=True),
        # plain decoding (a tree of one node) at 100K positions
        dict(name="attn_gqa_n102400_t1", op="attn", hq=32, hkv=8, d=128, n_q8=102336, n_tail=37,
             t=1, tree="chain", root=False),
        # the 40-node verification step at 32K, as the context is built up
        dict(name="attn_gqa_n32768_t40", op="attn", hq=32, hkv=8, d=128, n_q8=32704, n_tail=63,
             t=40, tree="bfs", root=True),
        # the headline step: 40 nodes over 100K positions, with the root scores
        dict(name="attn_gqa_n102400_t40", op="attn", hq=32, hkv=8, d=128, n_q8=102336, n_tail=51,
             t=40, tree="bfs", root=True),
        # a chain of 4 with a head per query head (no sharing) at 100K positions
        dict(name="attn_mha_n102400_t4", op="attn", hq=32, hkv=32, d=128, n_q8=102400, n_tail=0,
             t=4, tree="chain", root=False),
        # a step's rows: 40 nodes at their depths, behind a 100K context, frequencies stretched
        dict(name="rope_gqa_t40", op="rope", hq=32, hkv=8, d=128, rot=128, inter=False, t=40,
             tree="bfs", pos0=102387, row0=51, cap=256, scaled="wavelength"),
        # a prompt's chunk, interleaved pairs, half of each head rotated
        dict(name="rope_prompt_8190", op="rope", hq=40, hkv=8, d=128, rot=64, inter=True, t=8190,
             tree="prompt", pos0=24576, row0=2, cap=8192, scaled="yarn"),
        # the one block that a step fills
        dict(name="quant_one_block", op="quant", hkv=8, d=128, rows=64, row0=13, src_cap=256,
             n_q8=102336, cap=102464),
        # a 32K prompt's cache turned to 8 bits
        dict(name="quant_n32768", op="quant", hkv=8, d=128, rows=32768, row0=0, src_cap=32800,
             n_q8=0, cap=32768),
        # the small workload's draft cache
        dict(name="gather_d64_keep256", op="gather", hkv=2, d=64, n_q8=1984, n_tail=64, keep=256),
        # sinks and the best of 100K positions for the draft pass
        dict(name="gather_n102400_keep4096", op="gather", hkv=8, d=128, n_q8=102336, n_tail=51,
             keep=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rope", "quant", "gather"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 16, 32])
    g = rng.choice([1, 2, 4, 5, 8])
    if op == "attn":
        t = rng.choice([1, 2, 4, 13, 40, rng.randint(1, 64)])
        # no more bytes and no more products than the largest listed case
        n = _log(rng, 1, min(8 * 102400 // max(8, hkv), 32 * 40 * 102400 // (hkv * g * t)))
        n_tail = min(n, rng.choice([0, rng.randint(0, 63), rng.randint(0, 63),
                                    rng.randint(64, 300)]))
        n_q8 = (n - n_tail) // BLOCK * BLOCK
        return dict(op=op, hq=hkv * g, hkv=hkv, d=d, n_q8=n_q8, n_tail=n_tail, t=t,
                    tree=rng.choice(["bfs", "chain", "random"]), root=rng.random() < 0.5)
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(0, d // 2)])
        t = _log(rng, 1, 8192)
        tree = "prompt" if t > 64 or rng.random() < 0.3 else rng.choice(["bfs", "chain", "random"])
        row0 = rng.randint(0, 200)
        return dict(op=op, hq=min(hkv * g, 40), hkv=min(hkv, 8), d=d, rot=rot,
                    inter=rng.random() < 0.5, t=t, tree=tree, pos0=rng.randint(0, 131072),
                    row0=row0, cap=row0 + t + rng.randint(0, 60),
                    scaled=rng.choice(["plain", "linear", "wavelength", "yarn"]))
    if op == "quant":
        rows = BLOCK * _log(rng, 1, 512 * 8 // max(8, hkv))
        row0, n_q8 = rng.randint(0, 100), BLOCK * rng.randint(0, 40)
        return dict(op=op, hkv=hkv, d=d, rows=rows, row0=row0, src_cap=row0 + rows + rng.randint(0, 9),
                    n_q8=n_q8, cap=n_q8 + rows + BLOCK * rng.randint(0, 3))
    n = _log(rng, 64, 8 * 131072 // max(8, hkv))
    n_tail = min(n, rng.randint(0, 150))
    n_q8 = (n - n_tail) // BLOCK * BLOCK
    return dict(op=op, hkv=hkv, d=d, n_q8=n_q8, n_tail=n_tail,
                keep=min(n_q8 + n_tail, _log(rng, 1, 4096)))


def work(case):
    c = case
    if c["op"] == "attn":
        n = c["n_q8"] + c["n_tail"]
        cache = 2 * c["hkv"] * (c["n_q8"] * c["d"] + c["n_q8"] // BLOCK)
        tail = 4 * c["hkv"] * c["d"] * (c["n_tail"] + c["t"])
        rows = 4 * c["t"] * c["hq"] * c["d"]
        root = 4 * c["hq"] * n if c["root"] else 0
        return {"bytes": cache + tail + rows + root,
                "flops": 4 * c["hq"] * c["t"] * c["d"] * (n + c["t"])}
    if c["op"] == "rope":
        heads = c["hq"] + 2 * c["hkv"]
        return {"bytes": 4 * c["t"] * heads * c["d"] + 2 * c["rot"],
                "flops": 3 * c["t"] * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "quant":
        n = c["hkv"] * c["rows"] * c["d"]
        return {"bytes": 2 * (3 * n + c["hkv"] * c["rows"] // BLOCK), "flops": 4 * n}
    # a kept row is read at one or two bytes a value and written at two; int32 positions
    n, total = c["hkv"] * c["keep"] * c["d"], c["n_q8"] + c["n_tail"]
    read = (c["n_q8"] + 2 * c["n_tail"]) / total
    return {"bytes": int(2 * n * (2 + read)) + 4 * c["hkv"] * c["keep"], "flops": 2 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(0x8B17 + seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _parents(case, seed):
    """Parent of each tree node; a prompt has none."""
    t = case["t"]
    if case["tree"] == "prompt":
        return None
    if case["tree"] == "chain":
        return [i - 1 for i in range(t)]
    if case["tree"] == "bfs":
        return [(i - 1) // 3 for i in range(t)]
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(t, generator=g).tolist()
    return [-1] + [int(u[i] * i) for i in range(1, t)]


def _rows(g, hkv, n, d, spread):
    """bf16 rows whose size differs from block to block and from channel to channel."""
    x = _randn(g, hkv, n, d)
    x *= torch.exp(spread * _randn(g, hkv, (n + BLOCK - 1) // BLOCK, 1)) \
        .repeat_interleave(BLOCK, 1)[:, :n]
    x *= torch.exp(spread * _randn(g, 1, 1, d))
    return x.to(torch.bfloat16)


def _two_to(e):
    """2^e in 32 bits, exactly (e from -126 to 127)"""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x):
    """(codes, scale bytes) of bf16 rows [H, 64 m, D]: per block of 64 rows the
    least power of two that brings the largest magnitude to 448 or below."""
    h, n, d = x.shape
    b = x.float().reshape(h, n // BLOCK, BLOCK * d)
    top = b.abs().amax(-1)
    fine = torch.isfinite(top)
    m, e = torch.frexp(torch.where(fine, top, torch.ones_like(top)))
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp_min(-100)
    e = torch.where(top == 0, torch.full_like(e, -100), e)
    y = torch.where(fine[..., None], b * _two_to(-e)[..., None], torch.zeros_like(b))
    byte = torch.where(fine, e + 127, torch.full_like(e, 255))
    return y.to(torch.float8_e4m3fn).reshape(h, n, d), byte.to(torch.uint8)


def _factors(byte):
    f = _two_to(byte.to(torch.int32).clamp(1, 254) - 127)
    return torch.where(byte == 255, torch.full_like(f, float("nan")), f)


def _frequencies(case):
    """The table of a rotary embedding's frequencies, stretched for long contexts or not."""
    rot = case["rot"]
    f = torch.tensor([500000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    m = 1.0
    if case["scaled"] == "linear":
        f = f / 4
    elif case["scaled"] == "wavelength" and rot:
        s = ((8192 * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        f = f * (s + (1 - s) / 8)
    elif case["scaled"] == "yarn" and rot:
        at = [rot * math.log(8192 / (2 * math.pi * r)) / (2 * math.log(500000.0)) for r in (32, 1)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        s = 1 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (s + (1 - s) / 16)
        m = 0.1 * math.log(16) + 1
    return f.float().to(DEV), m


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if own:
        import lossless_ultra_long_b200 as L
    if c["op"] in ("attn", "gather"):
        tail = c["n_tail"] + c.get("t", 0)
        k8, ks = _encode(_rows(g, c["hkv"], c["n_q8"], c["d"], 0.25))
        v8, vs = _encode(_rows(g, c["hkv"], c["n_q8"], c["d"], 0.5))
        kt, vt = _rows(g, c["hkv"], tail, c["d"], 0.25), _rows(g, c["hkv"], tail, c["d"], 0.5)
        s.update(k8=k8, v8=v8, k_scale=ks, v_scale=vs, k_tail=kt, v_tail=vt)
        if own:
            s["cache"] = L.KvCacheQ8(k8, v8, ks, vs, kt, vt, n_q8=c["n_q8"], n_tail=c["n_tail"])
    if c["op"] == "attn":
        s["q"] = _randn(g, c["t"], c["hq"], c["d"]).to(torch.bfloat16)
        s["parent"] = _parents(c, seed)
        sees = torch.zeros(c["t"], c["t"], dtype=torch.bool)
        for i, p in enumerate(s["parent"]):
            sees[i] = sees[p] if i else False
            sees[i, i] = True
        s["sees"] = sees.to(DEV)
        if own:
            s["out"] = torch.empty_like(s["q"])
            s["ws"] = L.new_workspace(L.tree_verify_attn_q8_workspace_size(
                c["hq"], c["hkv"], c["d"], c["n_q8"], c["n_tail"], c["t"]))
            s["scores"] = torch.empty((c["hq"], c["n_q8"] + c["n_tail"]), dtype=torch.float32,
                                      device=DEV) if c["root"] else None
    elif c["op"] == "rope":
        # one projection's output: queries, keys and values of a token side by side
        heads = c["hq"] + 2 * c["hkv"]
        x = _randn(g, c["t"], heads, c["d"]).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        s["k_cache"], s["v_cache"] = (_randn(g, c["hkv"], c["cap"], c["d"]).to(torch.bfloat16)
                                      for _ in range(2))
        s["freq"], s["m"] = _frequencies(c)
        s["parent"] = _parents(c, seed)
        depth = list(range(c["t"])) if s["parent"] is None else [0] * c["t"]
        if s["parent"] is not None:
            for i in range(1, c["t"]):
                depth[i] = depth[s["parent"][i]] + 1
        s["pos"] = c["pos0"] + torch.tensor(depth, device=DEV)
        if own:
            s["q_out"] = torch.empty((c["t"], c["hq"], c["d"]), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "quant":
        s["k"], s["v"] = (_rows(g, c["hkv"], c["src_cap"], c["d"], 0.5) for _ in range(2))
        shape = (c["hkv"], c["cap"], c["d"])
        s["k8"], s["v8"] = (torch.zeros(shape, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
        s["k_scale"], s["v_scale"] = (torch.zeros(shape[0], shape[1] // BLOCK, dtype=torch.uint8,
                                                  device=DEV) for _ in range(2))
    else:
        n = c["n_q8"] + c["n_tail"]
        pick = torch.rand(c["hkv"], n, generator=g, device=DEV).argsort(-1)[:, :c["keep"]]
        s["idx"] = pick.sort(-1).values.to(torch.int32)
        if own:
            shape = (c["hkv"], c["keep"], c["d"])
            s["kp"], s["vp"] = (torch.empty(shape, dtype=torch.bfloat16, device=DEV)
                                for _ in range(2))
            s["ws"] = L.new_workspace(256)
    return s


# --------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"attn": _attn, "rope": _rope, "quant": _quant, "gather": _gather}[c["op"]](s, c)


def _run_own(s, c):
    import lossless_ultra_long_b200 as L
    if c["op"] == "attn":
        out = L.tree_verify_attn_q8(s["q"], s["cache"], s["parent"], out=s["out"],
                                    workspace=s["ws"], root_scores_out=s["scores"])
        return (out, s["scores"]) if c["root"] else (out,)
    if c["op"] == "rope":
        q = L.rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], c["row0"], c["pos0"],
                          s["freq"], parent=s["parent"], interleaved=c["inter"], mscale=s["m"],
                          q_out=s["q_out"])
        return q, s["k_cache"], s["v_cache"]
    if c["op"] == "quant":
        L.kv_quantize_q8(s["k"], s["v"], c["row0"], c["rows"], s["k8"], s["v8"], s["k_scale"],
                         s["v_scale"], c["n_q8"])
        return s["k8"], s["v8"], s["k_scale"], s["v_scale"]
    return L.kv_gather_q8(s["cache"], s["idx"], k_partial=s["kp"], v_partial=s["vp"],
                          workspace=s["ws"])


def _plain(codes, byte):
    """8-bit rows [H, n, D] in 32 bits."""
    return codes.float() * _factors(byte).repeat_interleave(BLOCK, 1)[..., None]


def _attn(s, c):
    t, hq, d, hkv = c["t"], c["hq"], c["d"], c["hkv"]
    n = c["n_q8"] + c["n_tail"]
    k = torch.cat([_plain(s["k8"], s["k_scale"]), s["k_tail"].float()], 1)
    v = torch.cat([_plain(s["v8"], s["v_scale"]), s["v_tail"].float()], 1)
    q = s["q"].float().reshape(t, hkv, hq // hkv, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
    x = torch.matmul(q, k.transpose(1, 2)) * (d ** -0.5)           # [Hkv, T G, n + T]
    root = (x[:, :hq // hkv, :n] * LOG2E).reshape(hq, n) if c["root"] else None
    x = x.reshape(hkv, t, hq // hkv, n + t)
    x[..., n:] = x[..., n:].masked_fill(~s["sees"][None, :, None, :], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(hkv, -1, n + t)
    o = torch.matmul(p, v).reshape(hkv, t, hq // hkv, d).permute(1, 0, 2, 3).reshape(t, hq, d)
    out = o.to(torch.bfloat16)
    return (out, root) if c["root"] else (out,)


def _turn(x, cos, sin, rot, inter):
    a = x.float()
    r, rest = a[..., :rot], a[..., rot:]
    if inter:
        u, w = r[..., 0::2], r[..., 1::2]
        y = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([y, rest], -1).to(torch.bfloat16)


def _rope(s, c):
    angle = s["pos"].double()[:, None, None] * s["freq"].double()    # far positions: 64 bits
    cos, sin = (torch.cos(angle) * s["m"]).float(), (torch.sin(angle) * s["m"]).float()
    q = _turn(s["q"], cos, sin, c["rot"], c["inter"])
    k = _turn(s["k"], cos, sin, c["rot"], c["inter"])
    s["k_cache"][:, c["row0"]:c["row0"] + c["t"]] = k.transpose(0, 1)
    s["v_cache"][:, c["row0"]:c["row0"] + c["t"]] = s["v"].transpose(0, 1)
    return q, s["k_cache"], s["v_cache"]


def _quant(s, c):
    rows, blocks = slice(c["row0"], c["row0"] + c["rows"]), c["rows"] // BLOCK
    at, to = slice(c["n_q8"], c["n_q8"] + c["rows"]), c["n_q8"] // BLOCK
    k8, ks = _encode(s["k"][:, rows])
    v8, vs = _encode(s["v"][:, rows])
    s["k8"][:, at], s["k_scale"][:, to:to + blocks] = k8, ks
    s["v8"][:, at], s["v_scale"][:, to:to + blocks] = v8, vs
    return s["k8"], s["v8"], s["k_scale"], s["v_scale"]


def _gather(s, c):
    n8, at = c["n_q8"], s["idx"].long()
    head = torch.arange(c["hkv"], device=DEV)[:, None]
    old = (at < n8)[..., None]
    tail = (at - n8).clamp_min(0)

    def rows(codes, byte, new):
        if n8 == 0:
            return new[head, tail]
        i = at.clamp_max(n8 - 1)
        x = (codes[head, i].float() * _factors(byte)[head, i // BLOCK][..., None]).to(torch.bfloat16)
        return torch.where(old, x, new[head, tail]) if c["n_tail"] else x

    return rows(s["k8"], s["k_scale"], s["k_tail"]), rows(s["v8"], s["v_scale"], s["v_tail"])


# ------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)

    def power(e):
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)

    if c["op"] == "attn":
        d, g, n = c["d"], c["hq"] // c["hkv"], c["n_q8"] + c["n_tail"]
        out = torch.empty(c["t"], c["hq"], d, dtype=torch.float64, device=DEV)
        root = torch.empty(c["hq"], n, dtype=torch.float64, device=DEV) if c["root"] else None
        for j in range(c["hkv"]):
            k, v = (torch.cat([
                codes[j].double() * power(byte[j].long() - 127).repeat_interleave(BLOCK)[:, None],
                tail[j].double()]) for codes, byte, tail in
                ((s["k8"], s["k_scale"], s["k_tail"]), (s["v8"], s["v_scale"], s["v_tail"])))
            for h in range(j * g, (j + 1) * g):
                x = s["q"][:, h].double() @ k.T / math.sqrt(d)
                if root is not None:
                    root[h] = x[0, :n] / math.log(2.0)
                for i in range(c["t"]):
                    path, a = [], i
                    while a >= 0:
                        path.append(n + a)
                        a = s["parent"][a]
                    at = torch.cat([torch.arange(n, device=DEV), torch.tensor(path, device=DEV)])
                    w = torch.softmax(x[i, at], 0)
                    out[i, h] = w[:n] @ v[:n] + w[n:] @ v[at[n:]]
        return (out, root) if c["root"] else (out,)
    if c["op"] == "rope":
        f = s["freq"].double()
        z = torch.polar(torch.full_like(s["pos"][:, None].double() * f, s["m"]),
                        s["pos"][:, None].double() * f)[:, None]

        def turned(x):
            y, r = x.double().clone(), c["rot"]
            if r:
                a, b = (y[..., 0:r:2], y[..., 1:r:2]) if c["inter"] else (y[..., :r // 2], y[..., r // 2:r])
                w = torch.complex(a.contiguous(), b.contiguous()) * z
                if c["inter"]:
                    y[..., 0:r:2], y[..., 1:r:2] = w.real, w.imag
                else:
                    y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
            return y

        k, v = s["k_cache"].double(), s["v_cache"].double()
        k[:, c["row0"]:c["row0"] + c["t"]] = turned(s["k"]).transpose(0, 1)
        v[:, c["row0"]:c["row0"] + c["t"]] = s["v"].double().transpose(0, 1)
        return turned(s["q"]), k, v
    if c["op"] == "quant":
        def codes(x, old):
            # nearest multiple of e4m3's spacing at that size, ties to even, block by block
            y = old.double().clone()
            for b in range(c["rows"] // BLOCK):
                z = x[:, c["row0"] + b * BLOCK:c["row0"] + (b + 1) * BLOCK].double()
                top = z.abs().amax((1, 2), keepdim=True)
                m, e = torch.frexp(top / 448)
                per = power(e - (m == 0.5).to(e.dtype))
                size = torch.frexp((z / per).abs().clamp_min(2.0 ** -6))[1] - 1
                step = power(size - 3)
                y[:, c["n_q8"] + b * BLOCK:c["n_q8"] + (b + 1) * BLOCK] = torch.round(z / per / step) * step
            return y
        return codes(s["k"], s["k8"]), codes(s["v"], s["v8"]), None, None
    rows = []
    for codes, byte, tail in ((s["k8"], s["k_scale"], s["k_tail"]), (s["v8"], s["v_scale"], s["v_tail"])):
        per = power(byte.long() - 127).repeat_interleave(BLOCK, 1)[..., None]
        every = torch.cat([codes.double() * per, tail.double()], 1)
        rows.append(torch.gather(every, 1, s["idx"].long()[..., None].expand(-1, -1, c["d"])))
    return tuple(rows)
