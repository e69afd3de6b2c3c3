"""The 8-bit cache's operators on a machine without a GPU: refusals of the
C ABI and of the binding, the frequency tables, and the plain forms' own
checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import lossless_ultra_long_b200 as L
import q8_plain as P8

P = ctypes.c_void_p
A = 1 << 20   # an aligned address that nothing reads: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    from lossless_ultra_long_b200 import build
    build.build()
    return L.library()


def _cache(**over):
    f = dict(k8=A, v8=A, k_scale=A, v_scale=A, q8_cap=256, k_tail=A, v_tail=A, tail_cap=128,
             tail_row0=0, n_heads_kv=2, head_dim=64, n_q8=192, n_tail=20)
    f.update(over)
    return L._Q8Cache(*[f[n] for n, _ in L._Q8Cache._fields_])


def _attn(lib, cache, q=A, hq=8, t=4, parent=(-1, 0, 0, 1), scale=0.125, out=A, root=None, ws=A,
          ws_bytes=1 << 30):
    par = np.array(parent, np.int32) if parent is not None else None
    return lib.ts_tree_verify_attn_q8(
        ctypes.byref(cache) if cache is not None else None, q, hq, t,
        par.ctypes.data_as(P) if par is not None else None, scale, out, root, ws, ws_bytes, None)


@pytest.mark.parametrize("over,code", [
    (dict(k8=0), 1), (dict(v_scale=0), 1), (dict(q8_cap=128), 1), (dict(q8_cap=250), 1),
    (dict(n_q8=100), 1), (dict(n_q8=-64), 1), (dict(n_tail=-1), 1), (dict(tail_cap=23), 1),
    (dict(tail_row0=105), 1), (dict(tail_row0=-1), 1), (dict(k_tail=0), 1), (dict(k8=A + 8), 1),
    (dict(v_tail=A + 2), 1), (dict(n_heads_kv=3), 1), (dict(n_heads_kv=0), 1),
    (dict(head_dim=96), 2), (dict(n_q8=2 ** 31 - 64, q8_cap=2 ** 31), 1),
])
def test_attention_refuses_bad_caches(lib, over, code):
    assert _attn(lib, _cache(**over)) == code


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=A + 8), 1), (dict(out=A + 2), 1),
    (dict(hq=7), 1), (dict(parent=None), 1), (dict(parent=(-1, 0, 2, 1)), 1),
    (dict(parent=(0, 0, 0, 1)), 1), (dict(t=0), 1),
    (dict(t=65, parent=[-1] + list(range(64))), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(root=A + 2), 1), (dict(ws=None), 3), (dict(ws=A + 128), 3),
    (dict(ws_bytes=64), 3),
])
def test_attention_refuses_bad_arguments(lib, over, code):
    assert _attn(lib, _cache(), **over) == code


def test_attention_refuses_no_cache(lib):
    assert _attn(lib, None) == 1


def test_workspace_size(lib):
    f = L.tree_verify_attn_q8_workspace_size
    assert f(32, 8, 128, 102336, 51, 40) > 256
    assert f(8, 2, 64, 0, 0, 1) >= 256
    for bad in ((7, 2, 64, 64, 0, 1), (8, 2, 96, 64, 0, 1), (8, 2, 64, 65, 0, 1),
                (8, 2, 64, 64, -1, 1), (8, 2, 64, 64, 0, 65), (8, 2, 64, -64, 0, 1)):
        assert f(*bad) == 0


@pytest.mark.parametrize("over", [
    dict(k=None), dict(v8=None), dict(k_scale=None), dict(n_rows=100), dict(dst=100),
    dict(cap=100), dict(n_rows=-64), dict(dst=192), dict(row0=5), dict(row0=-1), dict(k=A + 8),
    dict(v8=A + 4), dict(hkv=0), dict(n_rows=128, src_cap=100),
])
def test_quantize_refusals(lib, over):
    f = dict(k=A, v=A, src_cap=128, hkv=2, d=64, row0=0, n_rows=128, k8=A, v8=A, k_scale=A,
             v_scale=A, cap=256, dst=64)
    f.update(over)
    assert lib.ts_kv_quantize_q8(f["k"], f["v"], f["src_cap"], f["hkv"], f["d"], f["row0"],
                                 f["n_rows"], f["k8"], f["v8"], f["k_scale"], f["v_scale"],
                                 f["cap"], f["dst"], None) == 1


def test_empty_calls_do_nothing(lib):
    assert lib.ts_kv_quantize_q8(A, A, 128, 2, 64, 0, 0, A, A, A, A, 256, 0, None) == 0
    c = _cache()
    assert lib.ts_kv_gather_q8(ctypes.byref(c), A, 0, A, A, 0, A, 256, None) == 0
    assert lib.ts_rope_append(A, 512, A, 128, A, 128, 8, 2, 64, 0, None, 0, A, 64, 0, 1.0, A, A, A,
                              10, 10, None) == 0


@pytest.mark.parametrize("over,code", [
    (dict(idx=None), 1), (dict(n=5, cap=4), 1), (dict(n=-1), 1), (dict(kp=A + 8), 1),
    (dict(ws=None), 3), (dict(ws_bytes=128), 3),
])
def test_gather_refusals(lib, over, code):
    f = dict(idx=A, n=4, kp=A, vp=A, cap=4, ws=A, ws_bytes=256)
    f.update(over)
    c = _cache()
    assert lib.ts_kv_gather_q8(ctypes.byref(c), f["idx"], f["n"], f["kp"], f["vp"], f["cap"],
                               f["ws"], f["ws_bytes"], None) == code


@pytest.mark.parametrize("over,code", [
    (dict(rs=None), 1), (dict(hq=7), 1), (dict(sink=-1), 1), (dict(budget=-1), 1),
    (dict(cap=10), 1), (dict(rs=A + 4), 1), (dict(hq=32), 2), (dict(ws_bytes=256), 3),
    (dict(cache=dict(n_q8=0, n_tail=0)), 1),
])
def test_select_refusals(lib, over, code):
    f = dict(rs=A, hq=8, sink=4, budget=60, idx=A, kp=A, vp=A, cap=64, ws=A, ws_bytes=1 << 30)
    f.update(over)
    c = _cache(**f.get("cache", {}))
    assert lib.ts_kv_select_from_scores_q8(
        f["rs"], ctypes.byref(c), f["hq"], f["sink"], f["budget"], None, f["idx"], f["kp"],
        f["vp"], f["cap"], f["ws"], f["ws_bytes"], None) == code


@pytest.mark.parametrize("over,code", [
    (dict(k=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(hkv=0), 1),
    (dict(pos0=-1), 1), (dict(row0=-1), 1), (dict(row0=7), 1), (dict(cap=3), 1), (dict(rot=66), 1),
    (dict(rot=31), 1), (dict(rot=-2), 1), (dict(freq=None), 1), (dict(m=math.nan), 1),
    (dict(qs=508), 1), (dict(ks=120), 1), (dict(vs=132), 1), (dict(q=A + 8), 1),
    (dict(parent=(-1, 0, 0, 3)), 1), (dict(d=80), 2), (dict(q_out=A, qs=1024), 1),
    (dict(n=65, cap=100, parent=[-1] + [0] * 64), 1),
])
def test_rope_refusals(lib, over, code):
    f = dict(q=A, qs=512, k=A, ks=128, v=A, vs=128, hq=8, hkv=2, d=64, n=4, parent=(-1, 0, 0, 1),
             pos0=5, freq=A, rot=64, inter=0, m=1.0, q_out=2 * A, kc=A, vc=A, cap=10, row0=2)
    f.update(over)
    par = np.array(f["parent"], np.int32)
    assert lib.ts_rope_append(f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["hq"], f["hkv"],
                              f["d"], f["n"], par.ctypes.data_as(P), f["pos0"], f["freq"],
                              f["rot"], f["inter"], f["m"], f["q_out"], f["kc"], f["vc"],
                              f["cap"], f["row0"], None) == code


# ------------------------------------------------------------ frequency tables
def _table(rot, base, kind, *p):
    f = [base ** (-2 * j / rot) for j in range(rot // 2)]
    if kind == "linear":
        return [x / p[0] for x in f], 1.0
    if kind == "wavelength":
        factor, low, high, ctx = p
        out = []
        for x in f:
            t = ctx * x / (2 * math.pi)
            s = min(max((t - low) / (high - low), 0.0), 1.0)
            out.append(x * s + x / factor * (1 - s))
        return out, 1.0
    if kind == "yarn":
        factor, ctx, fast, slow = p

        def at(turns):
            return rot * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        out = []
        for j, x in enumerate(f):
            r = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            out.append(x / factor * r + x * (1 - r))
        return out, 0.1 * math.log(factor) + 1
    return f, 1.0


@pytest.mark.parametrize("rot,base,kind,params", [
    (128, 10000.0, "plain", ()), (64, 500000.0, "linear", (4.0,)),
    (128, 500000.0, "wavelength", (8.0, 1.0, 4.0, 8192.0)),
    (128, 10000.0, "yarn", (16.0, 4096.0, 32.0, 1.0)), (20, 10000.0, "yarn", (4.0, 32768.0, 32.0, 1.0)),
    (2, 10000.0, "plain", ()), (0, 10000.0, "plain", ()),
])
def test_inv_freq(rot, base, kind, params):
    got, m = L.rope_inv_freq(rot, base, kind, *params)
    want, wm = _table(rot, base, kind, *params) if rot else ([], 1.0)
    assert got.dtype == torch.float32 and got.numel() == rot // 2
    # one rounding to binary32 of a 64-bit value
    np.testing.assert_allclose(got.numpy().astype(np.float64), np.array(want), rtol=2.0 ** -24 * 1.001)
    assert abs(m - wm) <= 2.0 ** -23


@pytest.mark.parametrize("args", [
    (3, 1e4, "plain"), (-2, 1e4, "plain"), (64, 1.0, "plain"), (64, math.inf, "plain"),
    (64, 1e4, "linear", 0.0), (64, 1e4, "wavelength", 8.0, 4.0, 4.0, 8192.0),
    (64, 1e4, "yarn", 4.0, math.nan, 32.0, 1.0),
])
def test_inv_freq_refusals(args):
    with pytest.raises(L.TsError):
        L.rope_inv_freq(*args)


def test_inv_freq_wants_its_parameters():
    with pytest.raises(ValueError):
        L.rope_inv_freq(64, 1e4, "linear")
    with pytest.raises(ValueError):
        L.rope_inv_freq(64, 1e4, "other")


# ------------------------------------------------------- the plain forms themselves
def test_plain_e4m3_is_the_type():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[torch.isfinite(every)]
    assert torch.equal(P8.e4m3(every.double()), every.double())
    x = torch.from_numpy(np.random.default_rng(0).standard_normal(20000) * 40).double().clamp(-448, 448)
    near = every.double()[(x[:, None] - every.double()[None]).abs().argmin(1)]
    assert float((P8.e4m3(x) - x).abs().max()) <= float((near - x).abs().max())
    assert torch.equal(P8.e4m3(x), x.float().to(torch.float8_e4m3fn).double())


def test_plain_scale_is_the_least():
    x = P8.bf16(np.random.default_rng(1), 2, 128, 64)
    codes, byte = P8.quantize(x)
    top = codes.reshape(2, 2, -1).abs().amax(-1)
    assert bool((top <= 448).all()) and bool((top > 200).all())


# ------------------------------------------------------------- the cache's own checks
def test_cache_refuses_host_tensors():
    c = P8.cache_inputs(0, 2, 64, 64, 3, 4)
    with pytest.raises(ValueError):
        L.KvCacheQ8(**c, n_q8=64, n_tail=3)
    with pytest.raises(ValueError):
        L.tree_verify_attn_q8(torch.zeros(4, 8, 64, dtype=torch.bfloat16), None, [-1, 0, 1, 2])


@pytest.mark.parametrize("form", [list, tuple, lambda p: np.array(p, dtype=np.int32),
                                  lambda p: np.array(p, dtype=np.int64), torch.tensor])
def test_a_tree_in_any_form_is_the_same_tree(form):
    parent = [-1, 0, 0, 1, 1]
    keep, address = L._parent_arg(form(parent), 5)
    assert list((ctypes.c_int32 * 5).from_address(address)) == parent
    del keep
    for n in (4, 6):
        with pytest.raises(ValueError):
            L._parent_arg(form(parent), n)
    with pytest.raises((OverflowError, ValueError)):
        L._parent_arg([-1, 1 << 40], 2)
