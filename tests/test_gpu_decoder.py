"""The decoder's step on the GPU vs the fp64 oracle: embedding sum, attention blocks over a paged cache, dense and MoE
layers, heads, adjusted logits, with the operators called one after another as DecodeStack calls them.

The stack runs free beside the oracle; its layers are dense (one expert), so no route can flip.  Held to the bf16 bar
(max |err| <= 2e-2 x RMS): the layer inputs, the cached keys and values, the queries and the hidden rows are rounded
to bf16, 2^-8 each at most, about ten roundings of independent sign along the way.
"""
import numpy as np
import pytest
import torch

import oracle
from sparse_moe_decoder_b200 import (AttentionWeights, DecodeStack, LogitRules, MoEWeights, PagedCache,
                                     zmoe_get_device_errors)
from tests.gpu_util import assert_close, host, require_gpu

pytestmark = pytest.mark.gpu

T, D_MODEL, F, HQ, HKV, D, N, V = 3, 256, 512, 8, 2, 64, 2, 70
STEPS = 40            # more than two pages, more than the rules' window
WINDOW = 25


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    zmoe_get_device_errors()


def bf(a):
    """bf16-exact float64 values."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).double().numpy()


def params(seed, n_layers=3):
    r = np.random.default_rng(seed)
    n = lambda *s, scale: bf(r.standard_normal(s) * scale)  # noqa: E731
    g = lambda d: (1 + 0.2 * r.standard_normal(d)).astype(np.float32)  # noqa: E731
    layers = [dict(gate=n(1, F, D_MODEL, scale=D_MODEL ** -0.5), up=n(1, F, D_MODEL, scale=D_MODEL ** -0.5),
                   down=n(1, D_MODEL, F, scale=F ** -0.5), gamma=g(D_MODEL)) for _ in range(n_layers)]
    att = [dict(qkv=n((HQ + 2 * HKV) * D, D_MODEL, scale=2 * D_MODEL ** -0.5), o=n(D_MODEL, HQ * D, scale=(HQ * D) ** -0.5),
                gate=n(HQ, D_MODEL, scale=D_MODEL ** -0.5), gamma=g(D_MODEL), qg=g(D), kg=g(D))
           for _ in range(n_layers)]
    att[1] = None     # a layer without attention among them
    return dict(tables=n(N, V, D_MODEL, scale=1.0), gamma0=g(D_MODEL), layers=layers, att=att,
                heads=n(N, V, D_MODEL, scale=3 * D_MODEL ** -0.5), gamma_out=g(D_MODEL),
                inv=10000.0 ** (-np.arange(0, D, 2) / D), codes=r.integers(0, V, (STEPS, T, N)),
                rep=r.uniform(1.0, 1.6, T).astype(np.float32), pre=r.uniform(0, 0.5, T).astype(np.float32),
                bias=r.standard_normal((N, V)).astype(np.float32), ok=r.random((T, N, V)) < 0.7)


def build(p, page=16, n_pages=None, kv=torch.bfloat16):
    dev = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    w = lambda a: torch.from_numpy(a).to("cuda", torch.bfloat16)  # noqa: E731
    layers = [MoEWeights(None, w(L["gate"]), w(L["up"]), w(L["down"]), gamma=dev(L["gamma"])) for L in p["layers"]]
    att = [None if A is None else AttentionWeights(w(A["qkv"]), w(A["o"]), dev(A["gamma"]), HQ, HKV, w(A["gate"]),
                                                   dev(A["qg"]), dev(A["kg"])) for A in p["att"]]
    scale = torch.full((len(layers), HKV), 0.02, device="cuda") if kv == torch.uint8 else None
    cache = PagedCache(len(layers), T, 64, HKV, D, page, n_pages, kv, scale, scale)
    rules = LogitRules(T, N, WINDOW, dev(p["rep"]), dev(p["pre"]), None, dev(p["bias"]), dev(oracle.mask_bits(p["ok"])))
    return DecodeStack(w(p["tables"]), dev(p["gamma0"]), layers, T=T, w_heads=w(p["heads"]),
                       gamma_out=dev(p["gamma_out"]), attention=att, cache=cache, inv_freq=dev(p["inv"]), rules=rules)


class Reference:
    """The same decoder in float64; keys and values are kept as lists of rows."""

    def __init__(self, p):
        self.p = p
        self.kv = [[([], []) for _ in range(T)] for _ in p["layers"]]
        self.frames = []

    def step(self, ids):
        p = self.p
        h = oracle.embed_sum_rmsnorm(ids, p["tables"], p["gamma0"], 1e-6)
        pos = len(self.kv[0][0][0])
        for l, (L, A) in enumerate(zip(p["layers"], p["att"])):
            if A is not None:
                x = oracle.rmsnorm(h, A["gamma"], 1e-6)
                qkv = x @ A["qkv"].T
                q, k, v = (qkv[:, a * D:b * D].reshape(T, b - a, D) for a, b in
                           ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
                q, k, v = oracle.append_rows(q, k, v, [pos] * T, p["inv"], False, A["qg"], A["kg"])
                gate = x @ A["gate"].T
                o = np.zeros((T, HQ, D))
                for t in range(T):
                    keys, values = self.kv[l][t]
                    keys.append(k[t])
                    values.append(v[t])
                    o[t] = oracle.attend(q[t], np.stack(keys), np.stack(values), D ** -0.5, gate[t])[0]
                h = h + o.reshape(T, -1) @ A["o"].T
            x = oracle.rmsnorm(h, L["gamma"], 1e-6)
            h = h + oracle.swiglu_ffn(x, L["gate"][0], L["up"][0], L["down"][0])
        logits = oracle.head_logits(oracle.rmsnorm(h, p["gamma_out"], 1e-6), p["heads"])
        seen = np.stack(self.frames[-WINDOW:], 1) if self.frames else np.zeros((T, 0, N), np.int64)
        return h, oracle.adjust_logits(logits, seen, None, p["rep"], p["pre"], None, p["bias"], p["ok"])


def test_decoder_steps_match_the_oracle():
    p = params(1)
    st, ref = build(p), Reference(p)
    st.cache.reserve(STEPS)
    for i in range(STEPS):
        h = st.step(torch.from_numpy(p["codes"][i].astype(np.int32)).cuda())
        want_h, want_z = ref.step(p["codes"][i])
        assert_close(host(h), want_h, "bf16", f"h of step {i}")
        got = host(st.logits).astype(np.float64)
        assert np.array_equal(np.isneginf(got), ~p["ok"])
        assert_close(np.where(p["ok"], got, 0), np.where(p["ok"], want_z, 0), "bf16", f"logits of step {i}")
        ids = host(st.next_ids)
        assert np.array_equal(ids, oracle.allowed_greedy(got, p["ok"]))
        ref.frames.append(ids)      # the rules remember what was chosen
    assert host(st.cache.lens).tolist() == [STEPS] * T
    hist = host(st.rules.history)
    for t in range(T):
        want = sorted(map(tuple, np.stack(ref.frames[-WINDOW:], 1)[t].tolist()))
        assert sorted(map(tuple, hist[t].tolist())) == want
    assert zmoe_get_device_errors() == 0


def test_decoder_step_captured_and_replayed():
    """The chosen frame feeds the next step without the host: eager steps and replays of one graph agree bit by bit."""
    p = params(2)
    first = torch.from_numpy(p["codes"][0].astype(np.int32)).cuda()

    def run(st, step):
        out = []
        for _ in range(20):
            step()
            out.append((st.h.clone(), st.logits.clone(), st.next_ids.clone()))
        return out

    a, b = build(p), build(p)
    for st in (a, b):
        st.cache.reserve(21)
        st.step(first)              # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(b.next_ids)
    want, got = run(a, lambda: a.step(a.next_ids)), run(b, graph.replay)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))
    assert host(b.cache.lens).tolist() == [21] * T
    assert zmoe_get_device_errors() == 0


def test_decoder_on_another_stream():
    p = params(3)
    a, b = build(p), build(p)
    side = torch.cuda.Stream()
    for st in (a, b):
        st.cache.reserve(6)
    torch.cuda.synchronize()
    for i in range(6):
        codes = torch.from_numpy(p["codes"][i].astype(np.int32)).cuda()
        a.step(codes)
        b.ids.copy_(codes)
        torch.cuda.synchronize()
        b.step(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a.h, b.h) and torch.equal(a.next_ids, b.next_ids)


def test_decoder_with_an_8bit_cache_and_reused_pages():
    """8-bit keys and values: every row is off by at most half a step, so the output differs but little (2^-4 of a
    value, averaged over 64 columns and the tokens); a released sequence starts again as a new one."""
    p = params(4)
    a, b = build(p), build(p, kv=torch.uint8, n_pages=T * 3)
    for st in (a, b):
        st.cache.reserve(40)
    codes = [torch.from_numpy(c.astype(np.int32)).cuda() for c in p["codes"]]
    start = None
    for i in range(40):
        x, y = host(a.step(codes[i])).astype(np.float64), host(b.step(codes[i])).astype(np.float64)
        start = y if i == 0 else start
        assert np.abs(x - y).max() <= 2.0 ** -2 * np.sqrt((x * x).mean())
    with pytest.raises(RuntimeError, match="out of pages"):
        b.cache.reserve(64)
    for s in range(T):
        b.cache.release(s)
    b.cache.reserve(1)
    assert np.array_equal(host(b.step(codes[0])), start.astype(np.float32))
    assert zmoe_get_device_errors() == 0


def test_decoder_without_a_page_counts_an_error():
    p = params(5)
    st = build(p)
    st.step(torch.from_numpy(p["codes"][0].astype(np.int32)).cuda())
    assert zmoe_get_device_errors() > 0
    assert torch.isfinite(st.h).all()


def test_decoder_refusals():
    p = params(6)
    st = build(p)
    args = (st.tables, st.gamma0, st.layers)
    for kw, what in ((dict(attention=st.attention), "cache"), (dict(attention=st.attention[:2], cache=st.cache), "entry"),
                     (dict(attention=st.attention, cache=st.cache, persistent=True), "no attention"),
                     (dict(rules=st.rules), "heads")):
        with pytest.raises(ValueError, match=what):
            DecodeStack(*args, T=T, **kw)
    with pytest.raises(ValueError):
        st.cache.reserve(65)
    with pytest.raises(ValueError):
        PagedCache(1, 1, 16, 1, 64, 24)
    with pytest.raises(ValueError):
        PagedCache(1, 1, 16, 1, 64, 16, dtype=torch.uint8)


def test_decoder_reuses_a_place_while_others_go_on():
    """A sequence that is released while the others go on, and given pages again later, attends to its own tokens alone:
    its rows are a fresh stack's."""
    p = params(7)
    a, b = build(p, n_pages=T + 1), build(p)
    codes = [torch.from_numpy(c.astype(np.int32)).cuda() for c in p["codes"]]
    a.cache.reserve(16)
    b.cache.reserve(16)
    for i in range(5):
        a.step(codes[i])
    a.cache.release(0)
    a.cache.reserve(17, 1)              # sequence 1 goes on in the page that sequence 0 had
    for i in range(5, 11):
        a.step(codes[i])
    assert host(a.cache.lens).tolist() == [0, 11, 11]
    zmoe_get_device_errors()
    a.cache.release(1)
    a.cache.reserve(16, 0)              # and gives it back, with its rows
    for i in range(4):
        x, y = a.step(codes[20 + i]), b.step(codes[20 + i])
        assert_close(host(x)[:1], host(y)[:1].astype(np.float64), "bf16", f"h of the new sequence's step {i}")
        assert host(a.cache.lens)[0] == i + 1


def test_decoder_with_idle_places():
    """Released sequences are padding: they count no errors, the attention leaves their rows, and the others' rows are
    what they are without them."""
    p = params(8)
    a, b = build(p), build(p)
    codes = [torch.from_numpy(c.astype(np.int32)).cuda() for c in p["codes"]]
    for st in (a, b):
        st.cache.reserve(24)
        st.step(codes[0])
    b.cache.release(0)
    b.cache.release(2)
    pages = b.cache.k.clone(), b.cache.v.clone()
    for i in range(1, 20):
        x, y = a.step(codes[i]), b.step(codes[i])
        assert_close(host(y)[1:2], host(x)[1:2].astype(np.float64), "bf16", f"h of step {i}")
    assert zmoe_get_device_errors() == 0
    assert host(b.cache.lens).tolist() == [0, 20, 0]
    mine = b.cache.pages[1]
    others = [i for i in range(b.cache.n_pages) if i not in mine]
    assert torch.equal(b.cache.k[:, others], pages[0][:, others]) and torch.equal(b.cache.v[:, others], pages[1][:, others])
    A, run = b.attention[0], b.att_runners[HQ, HKV, D]
    h = torch.randn((T, D_MODEL), device="cuda")
    got = run.run(h.clone(), A, b.cache, 0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], h[0]) and torch.equal(got[2], h[2]) and not torch.equal(got[1], h[1])


def test_decoder_forgets_the_frames_of_a_released_sequence():
    """Logits and ids of a place that is used again are a fresh stack's, though the other sequences go on and idle
    steps lie between."""
    p = params(9)
    p["rep"][:] = 4.0                   # a penalty that shows
    a, b = build(p), build(p)
    codes = [torch.from_numpy(c.astype(np.int32)).cuda() for c in p["codes"]]
    a.cache.reserve(40)
    b.cache.reserve(40)
    for i in range(7):
        a.step(codes[i])
    a.release(0)
    for i in range(7, 10):
        a.step(codes[i])
    a.cache.reserve(40, 0)
    for i in range(12):
        a.step(codes[20 + i])
        b.step(codes[20 + i])
        ok = p["ok"][:1]
        x, y = host(a.logits)[:1].astype(np.float64), host(b.logits)[:1].astype(np.float64)
        assert_close(np.where(ok, x, 0), np.where(ok, y, 0), "bf16", f"logits of the new sequence's step {i}")
        assert np.array_equal(host(a.next_ids)[0], oracle.allowed_greedy(host(a.logits)[:1], ok)[0])
        # the two may choose otherwise only between logits that are as near as the bar
        if not np.array_equal(host(a.next_ids)[0], host(b.next_ids)[0]):
            break
    assert i >= 5
    assert zmoe_get_device_errors() == 0


def test_rules_of_another_count_are_refused():
    p = params(6)
    st = build(p)
    with pytest.raises(ValueError, match="streams"):
        DecodeStack(st.tables, st.gamma0, st.layers, T=T, w_heads=st.w_heads, gamma_out=st.gamma_out,
                    rules=LogitRules(T + 1, N, WINDOW))


def test_release_without_a_cache():
    p = params(6)
    st = build(p)
    st = DecodeStack(st.tables, st.gamma0, st.layers, T=T, w_heads=st.w_heads, gamma_out=st.gamma_out,
                     rules=LogitRules(T, N, WINDOW, torch.full((T,), 2.0, device="cuda")))
    for i in range(3):
        st.step(torch.from_numpy(p["codes"][i].astype(np.int32)).cuda())
    st.release(1)
    assert host((st.rules.history >= 0).sum((1, 2))).tolist() == [3 * N, 0, 3 * N]


def test_decoder_releases_between_steps_of_another_stream():
    """Steps, releases and pages on a side stream that lags behind the host, with no wait between them."""
    p = params(10)
    codes = [torch.from_numpy(c.astype(np.int32)).cuda() for c in p["codes"]]
    side = torch.cuda.Stream()

    def run(stream, lag):
        st, out = build(p, n_pages=T + 1), []
        st.cache.reserve(16)
        torch.cuda.synchronize()
        for i in range(12):
            if lag:
                with torch.cuda.stream(stream):
                    torch.cuda._sleep(20_000_000)
            if i in (4, 8):
                st.release(i % 3, stream=stream)
                st.cache.reserve(16, i % 3, stream=stream)
            with torch.cuda.stream(stream):
                st.ids.copy_(codes[i])
            st.step(stream=stream)
            with torch.cuda.stream(stream):
                out += [st.h.clone(), st.logits.clone(), st.next_ids.clone(), st.cache.lens.clone()]
        torch.cuda.synchronize()
        return out

    want, got = run(None, False), run(side, True)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert host(got[-1]).tolist() == [12, 8, 4] and zmoe_get_device_errors() == 0


def test_decoder_takes_its_ids_on_the_stream_of_the_step():
    """A step's ids are copied behind the steps before it, also where these lag behind the host."""
    p = params(11)
    codes = [torch.from_numpy(c.astype(np.int32)).cuda() for c in p["codes"]]
    side = torch.cuda.Stream()

    def run(stream, lag):
        st, out = build(p), []
        st.cache.reserve(16)
        st.record_inputs = True
        torch.cuda.synchronize()
        if lag:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(200_000_000)
        for i in range(6):
            st.step(codes[i], stream=stream)
            with torch.cuda.stream(stream):
                out += [st.h.clone(), st.next_ids.clone()] + st.layer_inputs + st.layer_h + st.layer_idx
        torch.cuda.synchronize()
        return out

    want, got = run(None, False), run(side, True)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
