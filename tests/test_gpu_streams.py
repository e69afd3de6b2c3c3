"""Calls on a stream of their own, with nothing but their inputs given, while the
current stream is busy: their outputs and workspaces are not that stream's."""
import types

import pytest
import torch

import lossless_ultra_long_b200 as L
import q8_plain as P8

pytestmark = pytest.mark.gpu

HQ, HKV, D, N8, TAIL, T, VOCAB = 16, 4, 128, 8192, 40, 13, 4096
N = N8 + TAIL


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device="cuda").manual_seed(5)

    def codes():
        return (torch.randint(0, 256, (HKV, N8, D), generator=g, device="cuda", dtype=torch.uint8) & 0xBF).view(
            torch.float8_e4m3fn)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    s = torch.full((HKV, N8 // 64), 126, dtype=torch.uint8, device="cuda")
    return dict(cache=L.KvCacheQ8(codes(), codes(), s, s.clone(), bf(HKV, TAIL + T, D), bf(HKV, TAIL + T, D),
                                  n_q8=N8, n_tail=TAIL),
                q=bf(T, HQ, D), k=bf(HKV, N + T, D), v=bf(HKV, N + T, D), rows=bf(T, HQ + 2 * HKV, D),
                scores=torch.randn(HQ, N, generator=g, device="cuda"),
                logits=torch.randn(T, VOCAB, generator=g, device="cuda"),
                tokens=torch.arange(T, dtype=torch.int32, device="cuda"),
                window=torch.arange(9, dtype=torch.int32, device="cuda"),
                idx=torch.arange(HKV * 300, dtype=torch.int32, device="cuda").reshape(HKV, 300) * 6,
                freq=L.rope_inv_freq(D, 1e4)[0].cuda())


def _rope(d, stream):
    kc, vc = d["kc"], d["vc"]
    q, k, v = d["rows"].split([HQ, HKV, HKV], 1)
    return L.rope_append(q, k, v, kc, vc, 3, 5, d["freq"], stream=stream), kc, vc


CALLS = {
    "tree_verify_attn": lambda d, s: L.tree_verify_attn(d["q"], d["k"], d["v"], N, d["tree"], stream=s),
    "tree_verify_attn_q8": lambda d, s: L.tree_verify_attn_q8(d["q"], d["cache"], d["tree"], stream=s),
    "kv_select_from_scores": lambda d, s: L.kv_select_from_scores(d["scores"], d["k"], d["v"], N, 16, 600,
                                                                  want_scores=True, stream=s),
    "kv_select_from_scores_q8": lambda d, s: L.kv_select_from_scores_q8(d["scores"], d["cache"], 16, 600,
                                                                        want_scores=True, stream=s),
    "kv_importance_select": lambda d, s: L.kv_importance_select(d["q"][0], d["k"], d["v"], N, 16, 600, stream=s)[:3],
    "kv_gather_q8": lambda d, s: L.kv_gather_q8(d["cache"], d["idx"], stream=s),
    "penalize_accept": lambda d, s: L.penalize_accept(d["logits"], d["window"], 1.2, d["tree"], d["tokens"], stream=s),
    "rope_append": _rope,
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_on_its_own_stream(data, name):
    data["tree"] = P8.parents("bfs", T)
    data["kc"], data["vc"] = (torch.zeros(HKV, 40, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    call, s = CALLS[name], torch.cuda.Stream()
    want = call(data, None)
    want = [x.clone() for x in (want if isinstance(want, tuple) else (want,))]
    torch.cuda.synchronize()
    for where in (torch.cuda.current_stream(), s):     # free memory that is not zero, for each
        with torch.cuda.stream(where):
            junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (256, 1 << 14, 1 << 20, 1 << 23)]
            del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)                      # some 0.2 s of the current stream
    got = call(data, s)
    s.synchronize()     # (a cooperative launch may have waited for the sleep's end)
    got = got if isinstance(got, tuple) else (got,)
    with torch.cuda.stream(s):
        got = [x.clone().cpu() for x in got]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        if name == "tree_verify_attn":   # its tiles are handed out at run time: 1e-4 from call to call
            assert float((x - y.cpu()).abs().max()) <= 2e-4
        else:
            assert torch.equal(x, y.cpu())


def test_a_stream_that_is_only_a_handle(data):
    """Any object with a stream's handle serves, the default stream's 0 among them."""
    data["tree"] = P8.parents("bfs", T)
    s = torch.cuda.Stream()
    want = L.tree_verify_attn_q8(data["q"], data["cache"], data["tree"])
    torch.cuda.synchronize()
    for handle in (s.cuda_stream, 0):
        out = L.tree_verify_attn_q8(data["q"], data["cache"], data["tree"],
                                    stream=types.SimpleNamespace(cuda_stream=handle))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
