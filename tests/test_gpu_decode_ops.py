"""The decode-step operators on the GPU vs the fp64 oracle: the residual norm with 8-bit output, the append to a
paged cache, the attention over it, the adjusted logits.

Tolerances count roundings: half a step of the output's type relative to the value (HALF), and for what fp32
arithmetic adds before it:
  norm     a sum of d squares in fp32, at most 16 terms in a row and 12 levels, a root and three products, each
           within 2^-23: below 2^-18 relative
  append   sine and cosine within 2^-22 absolute, two products and a sum: 2^-20 of the pair's length; the norm's
           2^-18 where there is one
  scores   a product of D terms in fp32: D 2^-23 of scale * sum |q k|, which is the relative error of exp(score);
           P is carried in two 16-bit terms, 2^-16; the sum over tokens adds 2^-16 more
"""
import numpy as np
import pytest
import torch

import oracle
from sparse_moe_decoder_b200 import (zmoe_add_rmsnorm, zmoe_adjust_logits, zmoe_get_device_errors, zmoe_kv_append,
                                     zmoe_paged_attention, zmoe_paged_attention_workspace_size, zmoe_rmsnorm)
from tests.gpu_util import host, require_gpu

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16
NAN_CODE = 0x7F


@pytest.fixture(autouse=True)
def _no_errors_left():
    require_gpu()
    zmoe_get_device_errors()
    yield


def rnd(seed):
    return np.random.default_rng(seed)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype != torch.float64 else t.cpu().numpy()


# ------------------------------------------------------------------------------------- residual norm

def check_norm(o, h, delta, gamma, eps, x_dtype, group):
    hp = f64(h) + (0 if delta is None else f64(delta))
    if o["h"] is not None:
        got = f64(o["h"])
        assert np.all(np.abs(got - hp) <= HALF[h.dtype] * np.abs(hp) + 2.0 ** -24 * np.abs(hp) + 1e-45)
        hp = got
    else:
        hp = f64(torch.from_numpy(hp.astype(np.float32)).to(h.dtype))
    x = oracle.rmsnorm(hp, f64(gamma), eps)
    if o["x"] is not None:
        assert o["x"].dtype == x_dtype
        assert np.all(np.abs(f64(o["x"]) - x) <= np.abs(x) * (HALF[x_dtype] + 2.0 ** -18) + 1e-38)
    if o["codes"] is not None:
        T, d = x.shape
        parts = np.abs(x).reshape(T, -1, group or d)
        top = parts.max(2)
        s = f64(o["scales"])
        assert s.shape == top.shape
        assert np.all(np.abs(s - np.where(top > 0, top / 448, 1)) <= s * 2.0 ** -17)
        val = oracle.e4m3_decode(o["codes"].cpu().numpy()).reshape(parts.shape) * s[..., None]
        # half a step of E4M3: 2^-4 of the value, 2^-10 scales below the smallest normal number
        tol = (2.0 ** -4 + 2.0 ** -16) * parts + 2.0 ** -10 * s[..., None] * (1 + 2.0 ** -16)
        assert np.all(np.abs(val - x.reshape(parts.shape)) <= tol)
        # the largest magnitude is at the end of the range
        codes = o["codes"].cpu().numpy() & 0x7F
        assert np.all((codes.reshape(parts.shape).max(2) == 0x7E) | (top == 0))


@pytest.mark.parametrize("T,d", [(1, 8), (3, 128), (1, 2048), (77, 2048), (5, 1032), (2, 4096), (9, 5504), (2, 16384),
                                 (1, 32768), (300, 256), (1025, 640)])
@pytest.mark.parametrize("types", ["f32 f32 bf16", "bf16 bf16 bf16", "bf16 f32 f32", "f32 bf16 f32"])
def test_norm_matches_the_formula(T, d, types):
    ht, dt, xt = (F32 if n == "f32" else BF16 for n in types.split())
    r = rnd(T * 31 + d)
    h = dev(r.standard_normal((T, d)) * r.uniform(0.01, 20, (T, 1)), ht)
    delta, gamma = dev(r.standard_normal((T, d)), dt), dev(1 + 0.2 * r.standard_normal(d), F32)
    for group in (0, 128) if d % 128 == 0 else (0,):
        o = zmoe_add_rmsnorm(h, gamma, delta, 1e-6, out_dtype=xt, want_codes=True, group=group)
        check_norm(o, h, delta, gamma, 1e-6, xt, group)
    assert zmoe_get_device_errors() == 0


def test_norm_several_rows_a_block():
    """More 16-bit rows than blocks run at once: a block takes several, the last ones fewer."""
    for T, d, group in ((3001, 2048, 128), (2999, 4096, 0), (5000, 264, 0)):
        r = rnd(T)
        h, delta = (dev(r.standard_normal((T, d)) * s, BF16) for s in (3, 1))
        gamma = dev(1 + 0.2 * r.standard_normal(d), F32)
        check_norm(zmoe_add_rmsnorm(h, gamma, delta, want_codes=True, group=group), h, delta, gamma, 1e-6, BF16, group)


def test_norm_single_outputs_and_no_delta():
    r = rnd(5)
    h, gamma = dev(r.standard_normal((7, 384)), F32), dev(r.standard_normal(384), F32)
    delta = dev(r.standard_normal((7, 384)), F32)
    full = zmoe_add_rmsnorm(h, gamma, delta, want_codes=True)
    for keys in (("h",), ("x",), ("codes", "scales"), ("h", "codes", "scales")):
        outs = {k: torch.zeros_like(full[k]) for k in keys}
        o = zmoe_add_rmsnorm(h, gamma, delta, outs=outs)
        for k in keys:
            assert torch.equal(o[k], full[k])
    o = zmoe_add_rmsnorm(h, gamma, want_codes=True, out_dtype=F32)
    assert o["h"] is None
    check_norm(o, h, None, gamma, 1e-6, F32, 0)
    # without a delta x is zmoe_rmsnorm's row up to the order of its fp32 sums
    w = zmoe_rmsnorm(h, gamma)
    assert np.allclose(f64(o["x"]), f64(w), rtol=2.0 ** -18, atol=0)


def test_norm_in_place():
    r = rnd(6)
    for dt in (F32, BF16):
        h, delta = dev(r.standard_normal((33, 2048)), dt), dev(r.standard_normal((33, 2048)), dt)
        gamma = dev(r.standard_normal(2048), F32)
        want = zmoe_add_rmsnorm(h, gamma, delta)
        a, b = h.clone(), delta.clone()
        x = zmoe_add_rmsnorm(a, gamma, b, outs=dict(h=a, x=torch.empty_like(want["x"])))["x"]
        assert torch.equal(a, want["h"]) and torch.equal(x, want["x"]) and torch.equal(b, delta)
        a = h.clone()
        zmoe_add_rmsnorm(a, gamma, b, outs=dict(h=b))
        assert torch.equal(b, want["h"]) and torch.equal(a, h)


def test_norm_rows_of_zeros_tiny_infinite_and_nan():
    d = 256
    h = np.zeros((6, d), np.float32)
    h[1] = 1e-42                     # below the normal numbers; eps 0 scales it up to one
    h[2, 3], h[2, 5] = np.inf, 2.0
    h[3, 7] = np.nan
    h[4] = 1e-3 * np.arange(d)
    gamma = np.ones(d, np.float32)
    o = zmoe_add_rmsnorm(dev(h), dev(gamma), eps=1e-6, want_codes=True, out_dtype=F32)
    x, codes, s = f64(o["x"]), o["codes"].cpu().numpy(), f64(o["scales"])[:, 0]
    assert not x[0].any() and not codes[0].any() and s[0] == 1
    assert np.isfinite(x[1]).all() and not (codes[1] & 0x7F == NAN_CODE).any() and s[1] > 0
    assert np.isnan(x[2, 3]) and x[2, 5] == 0 and codes[2, 3] & 0x7F == NAN_CODE and codes[2, 5] == 0 and s[2] == 1
    assert np.isnan(x[3]).all() and (codes[3] & 0x7F == NAN_CODE).all() and s[3] == 1
    check_norm({k: v[4:5] if v is not None else None for k, v in o.items()}, dev(h[4:5]), None, dev(gamma), 1e-6, F32, 0)
    # gains so small that max|x| / 448 has no finite reciprocal: the scale stops at 2^-126
    o = zmoe_add_rmsnorm(dev(np.ones((1, d), np.float32)), dev(np.full(d, 1e-40, np.float32)), want_codes=True)
    assert f64(o["scales"])[0, 0] == 2.0 ** -126 and not (o["codes"].cpu().numpy() & 0x7F == NAN_CODE).any()


# ------------------------------------------------------------------------------------- append

def make_cache(r, n_pages, Hkv, page, D, kv):
    if kv == "e4m3":
        k, v = (dev(r.integers(0, 0x7F, (n_pages, Hkv, page, D)).astype(np.uint8)) for _ in range(2))
        return k, v, dev(r.uniform(0.005, 0.02, Hkv), F32), dev(r.uniform(0.005, 0.02, Hkv), F32)
    k, v = (dev(r.standard_normal((n_pages, Hkv, page, D)), BF16) for _ in range(2))
    return k, v, None, None


def decode(cache, scale):
    """The cache's values, [n_pages, Hkv, page, D] float64."""
    if scale is None:
        return f64(cache)
    return oracle.e4m3_decode(cache.cpu().numpy()) * f64(scale)[:, None, None]


def close_rows(got, want, pair, kv, scale, normed):
    """got vs want [..., D], `pair`: the length of each value's pair (its magnitude where nothing turns)."""
    slack = (2.0 ** -20 + (2.0 ** -18 if normed else 0)) * pair
    if kv == "e4m3":
        lim = 448 * scale
        tol = (2.0 ** -4 + 2.0 ** -16) * np.abs(want) + 2.0 ** -10 * scale * (1 + 2.0 ** -16) + slack
        assert np.all(np.abs(got - np.clip(want, -lim, lim)) <= tol)
    else:
        assert np.all(np.abs(got - want) <= HALF[BF16] * np.abs(want) + 1.01 * slack)


def pair_len(y, rot, pairs):
    """The length of the pair that each column belongs to; turning keeps it."""
    n = np.abs(y).copy()
    h = rot // 2
    a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if pairs else (np.arange(h), np.arange(h, rot))
    ln = np.hypot(y[..., a], y[..., b])
    n[..., a], n[..., b] = ln, ln
    return n


def append_case(seed, seqs, pos, Hq, Hkv, D, rot, pairs, norm, src, kv, page, max_pages, packed=True, n_seqs=None):
    r = rnd(seed)
    T = len(pos)
    n_seqs = n_seqs or max(max(seqs) + 1, 1)
    n_pages = n_seqs * max_pages + 1
    kc, vc, ks, vs = make_cache(r, n_pages, Hkv, page, D, kv)
    table = dev(r.permutation(n_pages)[:n_seqs * max_pages].reshape(n_seqs, max_pages).astype(np.int32))
    x = r.standard_normal((T, (Hq + 2 * Hkv) * D)) * 2
    qkv = dev(x, F32 if src == "f32" else BF16)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else None
    k, v = (qkv[:, (Hq + i * Hkv) * D:(Hq + (i + 1) * Hkv) * D].unflatten(1, (Hkv, D)) for i in range(2))
    if not packed:
        q, k, v = (None if t is None else t.contiguous() for t in (q, k, v))
    inv = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1)) if rot else None
    qg = r.uniform(0.5, 1.5, D).astype(np.float32) if norm else None
    kg = r.uniform(0.5, 1.5, D).astype(np.float32) if norm else None
    before = kc.clone(), vc.clone()
    out = zmoe_kv_append(k, v, dev(np.asarray(pos, np.int32)), kc, vc, table, q=q, seq=dev(np.asarray(seqs, np.int32)),
                         inv_freq=None if inv is None else dev(inv), interleaved=pairs,
                         q_gamma=None if qg is None else dev(qg), k_gamma=None if kg is None else dev(kg),
                         k_scale=ks, v_scale=vs,
                         q_out=torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda") if Hq else None)
    qr, kr, vr = oracle.append_rows(None if q is None else f64(q), f64(k), f64(v), pos, inv, pairs, qg, kg)
    flat = oracle.append_rows(None if q is None else f64(q), f64(k), f64(v), [0] * T, inv, pairs, qg, kg)
    tb = table.cpu().numpy()
    stored = np.zeros((n_pages, page), bool)
    K, V = decode(kc, ks), decode(vc, vs)
    for t in range(T):
        if seqs[t] < 0:
            if Hq:
                assert np.all(f64(out[t]) == 7.0)
            continue
        pid, row = tb[seqs[t], pos[t] // page], pos[t] % page
        stored[pid, row] = True
        sk = f64(ks)[:, None] if ks is not None else None
        sv = f64(vs)[:, None] if vs is not None else None
        close_rows(K[pid, :, row], kr[t], pair_len(flat[1][t], rot, pairs), kv, sk, norm)
        close_rows(V[pid, :, row], vr[t], 0 * vr[t], kv, sv, False)
        if Hq:
            close_rows(f64(out[t]), qr[t], pair_len(flat[0][t], rot, pairs), "bf16", None, norm)
    # every other row is as it was
    for new, old in ((kc, before[0]), (vc, before[1])):
        keep = torch.from_numpy(~stored).cuda()
        assert torch.equal(new.transpose(1, 2)[keep], old.transpose(1, 2)[keep])
    assert zmoe_get_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,rot,pairs,norm", [
    (16, 4, 128, 128, False, True), (4, 4, 64, 64, True, False), (6, 2, 64, 32, False, True), (3, 1, 128, 64, True, True),
    (0, 2, 128, 128, False, False), (5, 5, 64, 0, False, False), (1, 1, 64, 16, True, True)])
def test_append_matches_the_formula(Hq, Hkv, D, rot, pairs, norm, src, kv):
    # sequences of several tokens, of one, a padding token between them, the first and last rows of pages
    append_case(Hq + D + rot, [0, 0, 0, 2, -1, 1, 1], [15, 16, 17, 0, 3, 31, 47], Hq, Hkv, D, rot, pairs, norm, src, kv,
                16, 3)


def test_append_many_tokens_and_an_odd_page():
    n = 701   # more than four tokens an SM: blocks of several tokens, the last one short
    append_case(3, [i % 3 for i in range(n)], [5 + i // 3 for i in range(n)], 8, 2, 64, 64, False, True, "bf16", "bf16",
                48, 6)


def test_append_blocks_of_eight_tokens():
    n = 2501
    append_case(13, [i % 5 for i in range(n)], [i // 5 for i in range(n)], 3, 1, 64, 32, True, True, "f32", "e4m3", 32, 16)


def test_append_far_positions():
    append_case(4, [0, 1, 2], [1000003, 524288, 2 ** 21 - 1], 2, 1, 128, 128, True, False, "f32", "bf16", 16384, 128)


def test_append_without_seq_and_unpacked():
    append_case(8, [0, 1, 2], [4, 19, 40], 2, 2, 64, 64, False, False, "bf16", "bf16", 16, 3, packed=False)
    r = rnd(1)
    kc, vc, _, _ = make_cache(r, 6, 2, 16, 64, "bf16")
    kc2, vc2 = kc.clone(), vc.clone()
    table, pos = dev(np.arange(6, dtype=np.int32).reshape(3, 2)), dev(np.array([3, 17, 31], np.int32))
    k, v = dev(r.standard_normal((3, 2, 64)), F32), dev(r.standard_normal((3, 2, 64)), F32)
    zmoe_kv_append(k, v, pos, kc, vc, table)
    zmoe_kv_append(k, v, pos, kc2, vc2, table, seq=dev(np.arange(3, dtype=np.int32)))
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_append_out_of_range_is_counted_and_stores_nothing():
    r = rnd(2)
    kc, vc, _, _ = make_cache(r, 4, 1, 16, 64, "bf16")
    old = kc.clone(), vc.clone()
    table = dev(np.array([[0, 1], [4, -1]], np.int32))                  # sequence 1 has bad pages
    seq = dev(np.array([0, 0, 2, 1, 1, -3], np.int32))
    pos = dev(np.array([-1, 32, 0, 0, 16, 5], np.int32))
    q = dev(r.standard_normal((6, 1, 64)), BF16)
    q_out = torch.full((6, 1, 64), 7.0, dtype=BF16, device="cuda")
    zmoe_kv_append(q, q, pos, kc, vc, table, q=q, seq=seq, q_out=q_out)
    assert zmoe_get_device_errors() == 5
    assert torch.equal(kc, old[0]) and torch.equal(vc, old[1]) and bool((q_out == 7).all())


def test_append_8bit_saturates_and_keeps_nan():
    kc = torch.zeros((1, 1, 16, 64), dtype=torch.uint8, device="cuda")
    vc, one = torch.zeros_like(kc), torch.ones(1, device="cuda")
    k = torch.zeros((1, 1, 64), device="cuda")
    k[0, 0, :4] = torch.tensor([1e6, -1e6, float("nan"), float("inf")])
    zmoe_kv_append(k, k, dev(np.zeros(1, np.int32)), kc, vc, dev(np.zeros((1, 1), np.int32)), k_scale=one, v_scale=one)
    assert kc[0, 0, 0, :4].tolist()[:2] == [0x7E, 0xFE] and kc[0, 0, 0, 2] & 0x7F == NAN_CODE and kc[0, 0, 0, 3] == 0x7E


# ------------------------------------------------------------------------------------- attention

def attn_case(seed, lens, Hq, Hkv, D, kv, page, out_dtype, gate=False, max_pages=None, spread=1.5, poison=True):
    r = rnd(seed)
    B = len(lens)
    cols = max_pages or max(1, -(-max(list(lens) + [1]) // page))
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + 2
    kc, vc, ks, vs = make_cache(r, n_pages, Hkv, page, D, kv)
    if kv == "e4m3":
        kc = torch.where(dev(r.random(kc.shape) < 0.5), kc, kc | 0x80)
        vc = torch.where(dev(r.random(vc.shape) < 0.5), vc, vc | 0x80)
        kc = torch.where((kc & 0x7F) > 0x60, kc & 0x9F, kc)              # values of a few units
        ks = ks * 0.5
    ids = r.permutation(n_pages)
    table = np.full((B, cols), -5, np.int32)                            # what no length reaches is never looked at
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    if poison:   # rows behind each sequence's end, and pages of nobody, hold NaN
        bad = NAN_CODE if kv == "e4m3" else float("nan")
        for b in range(B):
            if need[b] and lens[b] % page:
                kc[table[b, need[b] - 1], :, lens[b] % page:] = bad
                vc[table[b, need[b] - 1], :, lens[b] % page:] = bad
        for p in ids[at:]:
            kc[p], vc[p] = bad, bad
    q = dev(r.standard_normal((B, Hq, D)) * spread, BF16)
    g = dev(r.standard_normal((B, Hq)) * 2, F32) if gate else None
    lse = torch.full((B, Hq), 5.0, device="cuda")
    scale = D ** -0.5
    out = zmoe_paged_attention(q, kc, vc, dev(table), dev(np.asarray(lens, np.int32)), k_scale=ks, v_scale=vs, gate=g,
                               out_dtype=out_dtype, lse=lse)
    K, V = decode(kc, ks), decode(vc, vs)
    got, gl = f64(out), f64(lse)
    for b, n in enumerate(lens):
        n = max(n, 0)
        k = oracle.paged_rows(K, table[b], n) if n else np.zeros((0, Hkv, D))
        v = oracle.paged_rows(V, table[b], n) if n else np.zeros((0, Hkv, D))
        qb = f64(q[b])
        want, wl = oracle.attend(qb, k, v, scale, None if g is None else f64(g[b]))
        if n == 0:
            assert not got[b].any() and np.isneginf(gl[b]).all()
            continue
        kk, vv = np.repeat(k, Hq // Hkv, 1), np.repeat(v, Hq // Hkv, 1)  # [n, Hq, D]
        reach = scale * np.einsum("hd,nhd->nh", np.abs(qb), np.abs(kk)).max(0)          # scale sum |q k|
        score = scale * np.einsum("hd,nhd->nh", qb, kk)
        p = np.exp(score - score.max(0))
        p = p / p.sum(0)
        size = np.einsum("nh,nhd->hd", p, np.abs(vv))                     # sum p |v|
        rel = 2 * D * 2.0 ** -23 * reach + 2.0 ** -15
        assert np.all(np.abs(got[b] - want) <= HALF[out_dtype] * np.abs(want) + rel[:, None] * size)
        assert np.all(np.abs(gl[b] - wl) <= D * 2.0 ** -23 * reach + 2.0 ** -15 + 2.0 ** -22 * np.abs(wl))
    assert zmoe_get_device_errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [0, 33, 0, 1, 700, 0], [2049], [5] * 40])
def test_attention_lengths(lens, D, kv):
    attn_case(len(lens) + D, lens, 8, 2, D, kv, 16, F32)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 4), (7, 7), (15, 3), (9, 1), (16, 1), (17, 1), (24, 2), (40, 1), (64, 4)])
def test_attention_head_layouts(Hq, Hkv, kv):
    attn_case(Hq * 3 + Hkv, [37, 160, 1], Hq, Hkv, 64 if Hq % 2 else 128, kv, 32, BF16 if Hkv == 1 else F32, gate=Hq > 8)


@pytest.mark.parametrize("page", [16, 48, 64, 80, 256])
def test_attention_pages_and_tables(page):
    attn_case(page, [3 * page - 1, page, page + 1, 2 * page], 4, 2, 64, "bf16", page, BF16, gate=True, max_pages=7)


def test_attention_long_and_ragged():
    attn_case(1, [20011, 3, 0, 777, 16], 4, 1, 128, "bf16", 64, F32)
    attn_case(2, [30000, 1], 2, 1, 64, "e4m3", 32, F32, gate=True)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,D", [(12, 64), (16, 128)])
def test_attention_wide_groups_over_long_caches(Hq, D, kv):
    """16 heads at a time, more than one window of pages a piece, a group that ends inside a step."""
    attn_case(Hq, [6007, 2, 1500], Hq, 1, D, kv, 48, F32, gate=True)
    attn_case(Hq + 1, [70001], Hq, 1, D, kv, 16, BF16)


def test_attention_sequences_that_share_pages():
    r = rnd(15)
    kc, vc, _, _ = make_cache(r, 9, 2, 16, 128, "bf16")
    table = np.array([[3, 1, 4, 0], [3, 1, 5, 0], [3, 3, 3, 3]], np.int32)
    lens = [60, 41, 64]
    q = dev(r.standard_normal((3, 4, 128)), BF16)
    out = f64(zmoe_paged_attention(q, kc, vc, dev(table), dev(np.array(lens, np.int32))))
    for b, n in enumerate(lens):
        want, _ = oracle.attend(f64(q[b]), oracle.paged_rows(f64(kc), table[b], n), oracle.paged_rows(f64(vc), table[b], n),
                                128 ** -0.5)
        assert np.allclose(out[b], want, rtol=0, atol=2.0 ** -14)


def test_attention_many_sequences():
    r = rnd(9)
    attn_case(3, r.integers(0, 60, 300).tolist(), 2, 2, 64, "bf16", 16, F32)


def test_attention_peaked_scores():
    """Scores some tens apart: late tokens raise the running maximum by far."""
    attn_case(4, [900, 130], 4, 2, 128, "bf16", 16, F32, spread=12.0)
    attn_case(5, [900, 130], 4, 2, 64, "e4m3", 16, F32, spread=300.0)


def test_attention_long_tail_of_small_weights():
    """One token far above 60000 equal ones, whose weights together still count: 2^-17 each, half a unit."""
    n, D = 60000, 64
    for kv in ("bf16", "e4m3"):
        page = 64
        n_pages = -(-n // page)
        k = np.zeros((n_pages, 1, page, D), np.float32)
        v = np.ones((n_pages, 1, page, D), np.float32)
        k[0, 0, 0, 0] = 17 * np.log(2.0)
        v[0, 0, 0] = -1
        kq = dev(k, BF16) if kv == "bf16" else dev(oracle.e4m3_encode(k))
        vq = dev(v, BF16) if kv == "bf16" else dev(oracle.e4m3_encode(v))
        one = torch.ones(1, device="cuda") if kv == "e4m3" else None
        q = torch.zeros((1, 1, D), dtype=BF16, device="cuda")
        q[0, 0, 0] = 1
        got = f64(zmoe_paged_attention(q, kq, vq, dev(np.arange(n_pages, dtype=np.int32)[None]),
                                       dev(np.array([n], np.int32)), scale=1.0, k_scale=one, v_scale=one))
        top = np.exp(decode(kq, one)[0, 0, 0, 0])
        want = (n - 1 - top) / (n - 1 + top)
        assert np.all(np.abs(got - want) <= 2.0 ** -13)


def test_attention_bad_pages_and_lengths_are_counted():
    r = rnd(11)
    kc, vc, _, _ = make_cache(r, 5, 1, 16, 64, "bf16")
    q = dev(r.standard_normal((3, 2, 64)), BF16)
    table = dev(np.array([[0, 99, 1], [-1, -1, 2], [3, 4, 2]], np.int32))
    lse = torch.zeros((3, 2), device="cuda")
    out = f64(zmoe_paged_attention(q, kc, vc, table, dev(np.array([40, 20, 60], np.int32)), lse=lse))
    assert zmoe_get_device_errors() >= 3
    K, V = f64(kc), f64(vc)
    rows = lambda C, ids, n: np.concatenate([C[p].transpose(1, 0, 2) for p in ids])[:n]  # noqa: E731
    # sequence 0 loses its middle page, 1 has nothing left, 2's length is cut to its three pages
    for b, ids, n in ((0, (0, 1), 24), (2, (3, 4, 2), 48)):
        want, wl = oracle.attend(f64(q[b]), rows(K, ids, n), rows(V, ids, n), 64 ** -0.5)
        assert np.allclose(out[b], want, rtol=0, atol=1e-3) and np.allclose(f64(lse[b]), wl, rtol=0, atol=1e-3)
    assert not out[1].any() and np.isneginf(f64(lse[1])).all()


def test_attention_nan_and_infinite_data_reach_their_rows_only():
    r = rnd(12)
    kc, vc, _, _ = make_cache(r, 3, 1, 16, 64, "bf16")
    kc[0, 0, 2, 5] = float("nan")
    vc[1, 0, 3, 7] = float("inf")
    q = dev(r.standard_normal((3, 2, 64)), BF16)
    out = f64(zmoe_paged_attention(q, kc, vc, dev(np.array([[0], [1], [2]], np.int32)), dev(np.full(3, 16, np.int32))))
    assert np.isnan(out[0]).all()
    assert np.isposinf(out[1, :, 7]).all() and np.isfinite(np.delete(out[1], 7, 1)).all() and np.isfinite(out[2]).all()


@pytest.mark.parametrize("lens", [[20000], [300, 20000, 0, 5000]])
def test_attention_infinite_values_in_a_long_cache(lens):
    """Groups cut into many parts: an infinity stays in its column, a NaN key in its sequence."""
    r = rnd(19)
    n = sum(-(-x // 64) for x in lens)
    kc, vc, _, _ = make_cache(r, n, 1, 64, 128, "bf16")
    need = [-(-x // 64) for x in lens]
    table = np.zeros((len(lens), max(need)), np.int32)
    ids, at = r.permutation(n), 0
    for b, x in enumerate(need):
        table[b, :x] = ids[at:at + x]
        at += x
    long = lens.index(20000)
    vc[table[long, 200], 0, 13, 77] = float("-inf")
    q = dev(r.standard_normal((len(lens), 6, 128)), BF16)
    out = f64(zmoe_paged_attention(q, kc, vc, dev(table), dev(np.array(lens, np.int32))))
    assert np.isneginf(out[long, :, 77]).all() and np.isfinite(np.delete(out[long], 77, 1)).all()
    assert np.isfinite(np.delete(out, long, 0)).all()
    kc[table[long, 3], 0, 5, 0] = float("nan")
    out = f64(zmoe_paged_attention(q, kc, vc, dev(table), dev(np.array(lens, np.int32))))
    assert np.isnan(out[long]).all() and np.isfinite(np.delete(out, long, 0)).all()


def test_attention_is_repeatable_and_its_workspace_needs_no_clearing():
    r = rnd(13)
    lens = np.array([900, 77, 4000, 1], np.int32)
    kc, vc, _, _ = make_cache(r, 320, 2, 16, 128, "bf16")
    table = dev(r.permutation(320)[:4 * 80].reshape(4, 80).astype(np.int32).repeat(4, 1)[:, :250])
    q = dev(r.standard_normal((4, 8, 128)), BF16)
    ws = torch.full((zmoe_paged_attention_workspace_size(4, 8, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    a = zmoe_paged_attention(q, kc, vc, table, dev(lens), workspace=ws).clone()
    for fill in (0, 127, 255):
        ws.fill_(fill)
        assert torch.equal(a, zmoe_paged_attention(q, kc, vc, table, dev(lens), workspace=ws))
        zmoe_paged_attention(q[:1], kc, vc, table[:1], dev(lens[:1]), workspace=ws)


# ------------------------------------------------------------------------------------- logits

def logits_case(seed, T, N, V, L, dtype, rep=True, pre=True, frq=True, bias=True, mask=True, lens=True, inplace=False,
                quantum=None):
    r = rnd(seed)
    z = r.standard_normal((T, N, V)) * 3
    if quantum:
        z = np.round(z / quantum) * quantum                              # many exact ties
    z = dev(z, dtype)
    hist = (r.random((T, L, N)) ** 3 * min(V, 40)).astype(np.int32)
    hist[r.random(hist.shape) < 0.1] = -1
    hl = r.integers(-1, L + 3, T).astype(np.int32) if lens else None
    pen = [r.uniform(a, b, T).astype(np.float32) if on else None
           for on, a, b in ((rep, 0.8, 2), (pre, -0.5, 1), (frq, -0.1, 0.5))]
    bs = r.standard_normal((N, V)).astype(np.float32) if bias else None
    ok = r.random((T, N, V)) < 0.5 if mask else None
    if mask:
        ok[-1, -1] = False                                               # a row whose mask leaves nothing
    src = f64(z)
    d = lambda a: None if a is None else dev(a)  # noqa: E731
    out, ids = zmoe_adjust_logits(z, dev(hist), d(hl), *(d(p) for p in pen), bias=d(bs),
                                  mask=None if ok is None else dev(oracle.mask_bits(ok)), out=z if inplace else None)
    want = oracle.adjust_logits(src, hist, hl, *pen, bias=bs, allowed=ok)
    got = f64(out)
    gone = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), gone)
    # five fp32 roundings of values no larger than `big`, then the type's own
    big = np.abs(src) * 2 + np.abs(np.where(gone, 0, want)) + (L * 0.5 + 1) + (0 if bs is None else np.abs(bs))
    tol = np.where(gone, 0, 5 * 2.0 ** -24 * big + HALF[dtype] * np.abs(np.where(gone, 0, want)) * 1.01)
    assert np.all(np.abs(np.where(gone, 0, got) - np.where(gone, 0, want)) <= tol)
    assert np.array_equal(ids.cpu().numpy(), oracle.allowed_greedy(got, ok))
    assert zmoe_get_device_errors() == 0
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N,V,L", [(1, 9, 1025, 40), (3, 2, 31, 7), (1, 1, 1, 3), (2, 1, 32, 1), (5, 3, 4097, 65),
                                     (1, 1, 40000, 100), (2, 1, 8192, 600)])
def test_logits_match_the_formula(T, N, V, L, dtype):
    logits_case(T + V, T, N, V, L, dtype)


@pytest.mark.parametrize("off", ["rep", "pre", "frq", "bias", "mask", "lens"])
def test_logits_each_step_may_be_left_out(off):
    logits_case(7, 2, 3, 500, 30, F32, **{off: False})


def test_logits_many_middling_rows():
    """More rows than run at once, of a length that goes either way: the same as a few of them alone."""
    r = rnd(23)
    z = dev(r.standard_normal((100, 5, 3001)) * 3, F32)
    hist = dev(r.integers(0, 3001, (100, 70, 5)).astype(np.int32))
    rep, bias = dev(r.uniform(1, 2, 100), F32), dev(r.standard_normal((5, 3001)), F32)
    ok = dev(oracle.mask_bits(r.random((100, 5, 3001)) < 0.7))
    out, ids = zmoe_adjust_logits(z, hist, repetition=rep, bias=bias, mask=ok)
    for i in (0, 57, 99):
        o, j = zmoe_adjust_logits(z[i:i + 1], hist[i:i + 1], repetition=rep[i:i + 1], bias=bias, mask=ok[i:i + 1])
        assert torch.equal(o[0], out[i]) and torch.equal(j[0], ids[i])
    logits_case(24, 100, 5, 3001, 40, F32)


def test_logits_penalties_alone_and_none():
    logits_case(8, 2, 2, 300, 9, BF16, rep=False, frq=False, bias=False, mask=False, lens=False)
    z = dev(rnd(3).standard_normal((2, 2, 77)), F32)
    out, ids = zmoe_adjust_logits(z)
    assert torch.equal(out, z) and torch.equal(ids.long(), z.argmax(2))


def test_logits_in_place_and_ties():
    logits_case(9, 4, 9, 1025, 50, F32, inplace=True, quantum=2.0)
    logits_case(10, 2, 1, 30000, 50, BF16, inplace=True, quantum=4.0, rep=False, pre=False, frq=False, bias=False)


def test_logits_counts_of_a_long_history():
    """More occurrences than a byte holds, of neighbouring ids, and the longest history."""
    L = 65535
    hist = np.zeros((1, L, 1), np.int32)
    hist[0, ::3] = 5
    hist[0, 1::3] = 4
    z = torch.zeros((1, 1, 64), device="cuda")
    out, ids = zmoe_adjust_logits(z, dev(hist), frequency=torch.ones(1, device="cuda"))
    got = f64(out)[0, 0]
    assert got[5] == -21845 and got[4] == -21845 and got[0] == -21845 and not got[6:].any() and ids.item() == 1
    hist[:] = 3
    assert f64(zmoe_adjust_logits(z, dev(hist), frequency=torch.ones(1, device="cuda"))[0])[0, 0, 2:5].tolist() == [0, -65535, 0]


def test_logits_large_vocabulary_crosses_the_counted_chunks():
    V = 8 * 40000 + 7                                                    # each CTA of a cluster counts twice
    z = torch.zeros((1, 1, V), device="cuda")
    at = [0, 32767, 32768, 40000, 40031, 160000, V - 1]
    hist = dev(np.array(at + at[:3], np.int32)[None, :, None])
    z[0, 0, at] = 4.0
    z[0, 0, V - 2] = 3.5
    out, ids = zmoe_adjust_logits(z, hist, frequency=torch.ones(1, device="cuda"))
    assert out[0, 0, at].tolist() == [2, 2, 2, 3, 3, 3, 3] and ids.item() == V - 2
    assert int((out != 0).sum()) == len(at) + 1


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_lie_anywhere(dtype):
    """Logits, biases and outputs that begin at any element, alike and unlike within 16 bytes."""
    r = rnd(17)
    T, N, V = 2, 3, 131
    hist = dev(r.integers(0, V, (T, 20, N)).astype(np.int32))
    rep = torch.full((T,), 1.5, device="cuda")
    z0, b0 = dev(r.standard_normal((T, N, V)), dtype), dev(r.standard_normal((N, V)), F32)
    want, want_ids = zmoe_adjust_logits(z0, hist, repetition=rep, bias=b0)
    for zo in range(0, 9):
        for oo in (zo, 3):
            z, out = (torch.full((T * N * V + 16,), 7.0, dtype=dtype, device="cuda") for _ in range(2))
            b = torch.zeros(N * V + 16, device="cuda")
            zv, ov, bv = z[zo:zo + T * N * V].view(T, N, V), out[oo:oo + T * N * V].view(T, N, V), b[zo % 5:zo % 5 + N * V].view(N, V)
            zv.copy_(z0)
            bv.copy_(b0)
            got, ids = zmoe_adjust_logits(zv, hist, repetition=rep, bias=bv, out=ov)
            assert torch.equal(got, want) and torch.equal(ids, want_ids)
            assert bool((out[:oo] == 7).all()) and bool((out[oo + T * N * V:] == 7).all())


def test_logits_more_counted_ids_than_threads():
    """Rows in place, counted in several chunks, with far more distinct ids in the history than a CTA has threads."""
    r = rnd(18)
    V, L = 60001, 3000
    for dtype in (F32, BF16):
        z = dev(r.standard_normal((2, 1, V)) * 3, dtype)
        src = f64(z)
        hist = r.integers(0, V, (2, L, 1)).astype(np.int32)
        hist[:, :40] = np.arange(V - 40, V)[None, :, None]
        hist[:, 40:80] = np.arange(40)[None, :, None]
        rep, frq = np.full(2, 1.25, np.float32), np.full(2, 0.5, np.float32)
        ok = r.random((2, 1, V)) < 0.6
        out, ids = zmoe_adjust_logits(z, dev(hist), None, dev(rep), None, dev(frq), mask=dev(oracle.mask_bits(ok)), out=z)
        want = oracle.adjust_logits(src, hist, None, rep, None, frq, allowed=ok)
        got = f64(out)
        assert np.array_equal(np.isneginf(got), ~ok)
        w, g = np.where(ok, want, 0), np.where(ok, got, 0)
        assert np.all(np.abs(g - w) <= 4 * 2.0 ** -24 * (2 * np.abs(src) + np.abs(w) + 2) + HALF[dtype] * 1.01 * np.abs(w))
        assert np.array_equal(ids.cpu().numpy(), oracle.allowed_greedy(got, ok))


def test_logits_that_are_all_lowest():
    """Everything that is allowed is -inf or NaN: the lowest allowed -inf, listed or not, in any part of the row."""
    inf = float("inf")
    for V in (5, 300, 1025, 40001):
        z = torch.full((2, 1, V), -inf, device="cuda")
        z[0, 0, :3] = float("nan")
        hist = dev(np.array([[[4]], [[1]]], np.int32))
        ok = np.ones((2, 1, V), bool)
        ok[1, 0, 0] = False
        _, ids = zmoe_adjust_logits(z, hist, presence=torch.ones(2, device="cuda"), mask=dev(oracle.mask_bits(ok)))
        assert ids.flatten().tolist() == [3, 1]
        z[1] = float("nan")
        assert zmoe_adjust_logits(z)[1].flatten().tolist() == [3, -1]


def test_logits_bad_ids_are_counted():
    z = torch.zeros((2, 1, 10), device="cuda")
    hist = dev(np.array([[[3], [10], [-1]], [[99], [4], [3]]], np.int32))
    out, _ = zmoe_adjust_logits(z, hist, presence=torch.ones(2, device="cuda"))
    assert zmoe_get_device_errors() == 2
    assert torch.nonzero(out).tolist() == [[0, 0, 3], [1, 0, 3], [1, 0, 4]]


def test_logits_nan_infinite_and_lowest_values():
    inf, low = float("inf"), torch.finfo(F32).min
    z = torch.tensor([[[float("nan"), 1.0, inf, -inf]], [[-inf, -inf, float("nan"), -inf]], [[low, low, 0.0, low]]],
                     device="cuda")
    mask = dev(np.array([[[0b0011]], [[0b1110]], [[0b1011]]], np.int32))
    out, ids = zmoe_adjust_logits(z, mask=mask)
    assert ids.flatten().tolist() == [1, 1, 0]
    assert out[0, 0, 2] == -inf and bool(torch.isnan(out[0, 0, 0])) and out[2, 0, 2] == -inf
    bias = torch.full((1, 4), low, device="cuda")
    bias[0, 1] = 0
    assert zmoe_adjust_logits(torch.zeros((1, 1, 4), device="cuda"), bias=bias)[1].item() == 1


# ------------------------------------------------------------------------------------- how they are called

def test_no_tokens():
    o = zmoe_add_rmsnorm(torch.zeros((0, 64), device="cuda"), torch.ones(64, device="cuda"), want_codes=True)
    assert o["x"].shape == (0, 64)
    kc, vc, _, _ = make_cache(rnd(0), 2, 1, 16, 64, "bf16")
    e = torch.zeros((0, 1, 64), dtype=BF16, device="cuda")
    i0 = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    assert zmoe_kv_append(e, e, i0, kc, vc, table, q=e).shape == (0, 1, 64)
    assert zmoe_paged_attention(e, kc, vc, table, i0).shape == (0, 1, 64)
    assert zmoe_adjust_logits(torch.zeros((0, 2, 8), device="cuda"))[1].shape == (0, 2)


def test_binding_refusals():
    kc, vc, _, _ = make_cache(rnd(0), 4, 2, 16, 64, "bf16")
    q = torch.zeros((2, 4, 64), dtype=BF16, device="cuda")
    table, lens = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    kv = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    z = torch.zeros((2, 1, 40), device="cuda")
    for call, what in (
        (lambda: zmoe_paged_attention(q, kc, vc, table[:1], lens), ValueError),
        (lambda: zmoe_paged_attention(q, kc, vc[:3], table, lens), ValueError),
        (lambda: zmoe_paged_attention(q, kc, vc, table, lens.long()), TypeError),
        (lambda: zmoe_paged_attention(q.float(), kc, vc, table, lens), TypeError),
        (lambda: zmoe_paged_attention(q[..., :32].contiguous(), kc, vc, table, lens), ValueError),
        (lambda: zmoe_paged_attention(q, kc, vc, table, lens, gate=torch.zeros((2, 3), device="cuda")), ValueError),
        (lambda: zmoe_paged_attention(q, kc, vc, table, lens, out=torch.zeros((2, 4, 32), device="cuda")), ValueError),
        (lambda: zmoe_kv_append(kv, kv, lens, kc, vc, table, seq=lens[:1]), ValueError),
        (lambda: zmoe_kv_append(kv, kv.float(), lens, kc, vc, table), TypeError),
        (lambda: zmoe_kv_append(kv.transpose(1, 2), kv, lens, kc, vc, table), ValueError),
        (lambda: zmoe_kv_append(kv, kv, lens, kc, vc, table, inv_freq=torch.ones(32, device="cuda")), TypeError),
        (lambda: zmoe_kv_append(kv, kv, lens, kc, vc, table, q_out=q), ValueError),
        (lambda: zmoe_add_rmsnorm(q.flatten(1), torch.ones(255, device="cuda")), ValueError),
        (lambda: zmoe_add_rmsnorm(q.flatten(1), torch.ones(256, device="cuda"), kv.flatten(1)), ValueError),
        (lambda: zmoe_adjust_logits(z, torch.zeros((2, 3, 2), dtype=torch.int32, device="cuda")), ValueError),
        (lambda: zmoe_adjust_logits(z, mask=torch.zeros((2, 1, 1), dtype=torch.int32, device="cuda")), ValueError),
        (lambda: zmoe_adjust_logits(z, bias=torch.zeros((2, 40), device="cuda")), ValueError),
    ):
        with pytest.raises(what):
            call()


def step_inputs(seed):
    r = rnd(seed)
    B, Hq, Hkv, D, page = 3, 8, 2, 64, 16
    kc, vc, _, _ = make_cache(r, 60, Hkv, page, D, "bf16")
    table = dev(r.permutation(60).reshape(3, 20).astype(np.int32))
    pos = dev(np.array([40, 0, 310], np.int32))
    h, delta = dev(r.standard_normal((B, 256)), F32), dev(r.standard_normal((B, 256)), F32)
    return dict(kc=kc, vc=vc, table=table, pos=pos, lens=pos + 1, h=h, delta=delta, gamma=torch.ones(256, device="cuda"),
                qkv=dev(r.standard_normal((B, (Hq + 2 * Hkv) * D)), F32),
                inv=dev(10000.0 ** (-np.arange(0, D, 2) / D)), z=dev(r.standard_normal((B, 2, 1025)), F32),
                hist=dev(r.integers(0, 1025, (B, 30, 2)).astype(np.int32)), rep=torch.full((B,), 1.3, device="cuda"),
                ws=torch.empty(zmoe_paged_attention_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda"),
                q=torch.empty((B, Hq, D), dtype=BF16, device="cuda"), o=torch.empty((B, Hq, D), device="cuda"),
                n=dict(h=torch.empty((B, 256), device="cuda"), x=torch.empty((B, 256), dtype=BF16, device="cuda"),
                       codes=torch.empty((B, 256), dtype=torch.uint8, device="cuda"),
                       scales=torch.empty((B, 1), device="cuda")),
                out=torch.empty((B, 2, 1025), device="cuda"), ids=torch.empty((B, 2), dtype=torch.int32, device="cuda"))


def one_step(s, stream=None):
    Hq, Hkv, D = 8, 2, 64
    u = lambda a, b: s["qkv"][:, a * D:b * D].unflatten(1, (b - a, D))  # noqa: E731
    zmoe_add_rmsnorm(s["h"], s["gamma"], s["delta"], outs=s["n"], stream=stream)
    zmoe_kv_append(u(Hq, Hq + Hkv), u(Hq + Hkv, Hq + 2 * Hkv), s["pos"], s["kc"], s["vc"], s["table"], q=u(0, Hq),
                   inv_freq=s["inv"], q_out=s["q"], stream=stream)
    zmoe_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], out=s["o"], workspace=s["ws"], stream=stream)
    zmoe_adjust_logits(s["z"], s["hist"], repetition=s["rep"], out=s["out"], ids=s["ids"], stream=stream)
    return [s["n"]["h"], s["n"]["x"], s["n"]["codes"], s["n"]["scales"], s["q"], s["kc"], s["vc"], s["o"], s["out"], s["ids"]]


def test_other_streams_and_two_at_once():
    want = [[t.clone() for t in one_step(step_inputs(i))] for i in range(2)]
    ins = [step_inputs(i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(ins, streams):
            one_step(s, stream=st)
    torch.cuda.synchronize()
    for s, st, w in zip(ins, streams, want):
        with torch.cuda.stream(st):
            got = one_step(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_captured_and_replayed_with_new_inputs():
    a, b = step_inputs(21), step_inputs(22)
    want_a, want_b = ([t.clone() for t in one_step(step_inputs(i))] for i in (21, 22))
    one_step(step_inputs(23))                                            # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one_step(a)
    for want, src in ((want_a, None), (want_b, b)):
        if src is not None:
            for key, t in a.items():
                if key not in ("n", "ws"):
                    t.copy_(src[key])
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    # positions and lengths are read on the device: a replay after the sequences grew sees them
    b["kc"].copy_(a["kc"])
    b["vc"].copy_(a["vc"])
    for s in (a, b):
        s["pos"].add_(1)
        s["lens"].add_(1)
    graph.replay()
    want = one_step(b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "another stream", "two streams", "host copy", "event"])
def test_captured_behind_anything(before):
    """Each operator as the first call behind a copy, a memset, a fork, a join of two streams: captured, replayed with
    other inputs, and right."""
    def head(s, side, fresh):
        if before == "copy":
            s["h"].copy_(fresh["h"]); s["qkv"].copy_(fresh["qkv"]); s["z"].copy_(fresh["z"])
        elif before == "fill":
            for k in ("h", "qkv", "z"):
                s[k].zero_()
        elif before in ("another stream", "two streams"):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                for k in ("h", "qkv", "z"):
                    s[k].add_(1.0)
            if before == "two streams":
                s["delta"].mul_(1.0)
            main.wait_stream(side)
        elif before == "host copy":
            s["h"].copy_(fresh["pinned"], non_blocking=True)
        elif before == "event":
            torch.cuda.Event().record()

    def calls(s):
        u = lambda a, b: s["qkv"][:, a * 64:b * 64].unflatten(1, (b - a, 64))  # noqa: E731
        return dict(
            norm=lambda: zmoe_add_rmsnorm(s["h"], s["gamma"], s["delta"], outs=s["n"]),
            append=lambda: zmoe_kv_append(u(8, 10), u(10, 12), s["pos"], s["kc"], s["vc"], s["table"], q=u(0, 8),
                                          inv_freq=s["inv"], q_out=s["q"]),
            attn=lambda: zmoe_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], out=s["o"],
                                              workspace=s["ws"]),
            logits=lambda: zmoe_adjust_logits(s["z"], s["hist"], repetition=s["rep"], out=s["out"], ids=s["ids"]))

    side = torch.cuda.Stream()
    for op in ("norm", "append", "attn", "logits"):
        a, b, fresh = step_inputs(31), step_inputs(31), step_inputs(32)
        fresh["pinned"] = fresh["h"].cpu().pin_memory()
        for s in (a, b):
            s["q"].copy_(dev(rnd(3).standard_normal(s["q"].shape), BF16))
        one_step(step_inputs(33))                                        # first use outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            head(b, side, fresh)
            calls(b)[op]()
        for _ in range(3):
            graph.replay()
            head(a, side, fresh)
            torch.cuda.synchronize()
            calls(a)[op]()
            torch.cuda.synchronize()
        if op == "norm":
            assert all(torch.equal(a["n"][k], b["n"][k]) for k in a["n"])
        elif op == "append":
            assert all(torch.equal(a[k], b[k]) for k in ("kc", "vc", "q"))
        elif op == "attn":
            assert torch.equal(a["o"], b["o"])
        else:
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["ids"], b["ids"])
        del graph


def test_chains_without_waiting():
    """Many dependent steps in a row, each kernel launched beside the one before it: as with a wait between all calls."""
    def run(wait):
        s = step_inputs(41)
        s["lens"].copy_(s["pos"] + 1)
        for i in range(60):
            u = lambda a, b: s["qkv"][:, a * 64:b * 64].unflatten(1, (b - a, 64))  # noqa: E731
            steps = [
                lambda: zmoe_add_rmsnorm(s["h"], s["gamma"], s["delta"], outs=dict(h=s["h"], x=s["n"]["x"])),
                lambda: zmoe_kv_append(u(8, 10), u(10, 12), s["pos"], s["kc"], s["vc"], s["table"], q=u(0, 8),
                                       inv_freq=s["inv"], q_out=s["q"]),
                lambda: zmoe_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], out=s["o"], workspace=s["ws"]),
                # the next step's keys come from this step's output, its residual from the logits
                lambda: zmoe_add_rmsnorm(s["o"].view(3, 512), s["ones"], outs=dict(x=s["qkv"][:, :512].contiguous())),
                lambda: s["qkv"][:, :512].copy_(s["o"].view(3, 512)),
                lambda: zmoe_adjust_logits(s["z"], s["hist"], repetition=s["rep"], out=s["z"], ids=s["ids"]),
                lambda: s["pos"].sub_(1).clamp_(min=0),
            ]
            s.setdefault("ones", torch.ones(512, device="cuda"))
            for f in steps:
                f()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [s[k] for k in ("h", "kc", "vc", "o", "z", "ids", "q")]

    a, b = run(True), run(False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_back_to_back_in_place():
    """The same operator on its own output many times over, with nothing in between: what the kernel before wrote is what
    is read, also where rows of different blocks share cache lines."""
    r = rnd(51)
    h0, gamma = dev(r.standard_normal((6000, 24)), F32), torch.ones(24, device="cuda")
    delta = dev(r.standard_normal((6000, 24)), F32)
    z0 = dev(r.standard_normal((301, 3, 1027)), F32)
    bias = dev(r.standard_normal((3, 1027)), F32)
    kc0, vc0, _, _ = make_cache(r, 40, 2, 16, 64, "bf16")
    table, pos = dev(r.permutation(40).reshape(8, 5).astype(np.int32)), dev(np.array([70, 3, 66, 50, 0, 79, 31, 16], np.int32))
    kv = dev(r.standard_normal((8, 2, 64)), BF16)
    ws = torch.empty(zmoe_paged_attention_workspace_size(8, 2, 2, 64), dtype=torch.uint8, device="cuda")

    def run(wait):
        h, z, kc, vc, x, y = h0.clone(), z0.clone(), kc0.clone(), vc0.clone(), kv.clone(), torch.empty_like(kv)
        lens = pos + 1
        torch.cuda.synchronize()
        for i in range(200):
            zmoe_add_rmsnorm(h, gamma, delta, outs=dict(h=h))
            if wait:
                torch.cuda.synchronize()
        for i in range(200):
            zmoe_adjust_logits(z, bias=bias, out=z)
            if wait:
                torch.cuda.synchronize()
        for i in range(200):   # the output of one step is the next one's query, key and value
            zmoe_kv_append(x, x, pos, kc, vc, table, q=x, q_out=y)
            if wait:
                torch.cuda.synchronize()
            zmoe_paged_attention(y, kc, vc, table, lens, out=x, workspace=ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return h, z, kc, vc, x

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, run(False)))


# 65536 ids is what 16 bits number: rows just below and above that many a CTA, in clusters of 1, 2 and 8 CTAs
LONG_ROWS = [(230, 65472, BF16), (230, 65530, BF16), (230, 65536, BF16), (230, 65543, BF16), (256, 128256, BF16),
             (112, 151936, BF16), (288, 65539, F32), (288, 70000, F32), (223, 100003, F32), (1, 524289, F32),
             (1, 600000, F32), (2, 600011, BF16)]


@pytest.mark.parametrize("rows,V,dtype", LONG_ROWS)
@pytest.mark.parametrize("how", ["out", "in place", "history only"])
def test_logits_of_long_rows_without_penalties(rows, V, dtype, how):
    """Every id is written, those at a row's end too, and the greedy id is found among them."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((rows, 1, V), generator=g, device="cuda").to(dtype)
    bias = torch.randn((1, V), generator=g, device="cuda")
    at = V - 1 - torch.arange(rows, device="cuda") % 12                  # the largest logit: one of the last ids
    z[torch.arange(rows, device="cuda"), 0, at] = 64.0
    want = (z.float() + bias).to(dtype)                                  # one fp32 sum, one rounding
    best = want.float().amax(2, keepdim=True)
    want_ids = torch.where(want == best, torch.arange(V, device="cuda"), V).amin(2).int()
    out = z if how == "in place" else torch.full_like(z, 1000.0)
    hist = torch.zeros((rows, 3, 1), dtype=torch.int32, device="cuda") if how == "history only" else None
    got, ids = zmoe_adjust_logits(z, hist, bias=bias, out=out)
    assert torch.equal(got, want) and torch.equal(ids, want_ids) and torch.equal(ids[:, 0], at.int())


def test_logits_of_long_rows_with_masks_and_no_bias():
    """The same with a mask that leaves only ids at the ends, and with one that leaves none."""
    rows, V = 300, 131075
    z = torch.randn((rows, 1, V), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)
    words = torch.zeros((rows, 1, (V + 31) // 32), dtype=torch.int32, device="cuda")
    words[:100, 0, -1] = 0b100                                           # id V - 1 alone
    words[100:200, 0, 0] = 0b10                                          # id 1 alone
    out, ids = zmoe_adjust_logits(z, mask=words, out=torch.full_like(z, 1000.0))
    assert ids.flatten().tolist() == [V - 1] * 100 + [1] * 100 + [-1] * 100
    ok = torch.zeros((rows, 1, V), dtype=torch.bool, device="cuda")
    ok[:100, 0, V - 1] = True
    ok[100:200, 0, 1] = True
    assert torch.equal(out, torch.where(ok, z, float("-inf")))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,top", [(1, 33, 32), (1, 600, 599), (1, 600, 100), (1, 20000, 100), (1, 20000, 19999), (40, 1000, 100)])
@pytest.mark.parametrize("Hq", [8, 16])
def test_attention_nan_far_below_the_largest_score(B, n, top, Hq, kv):
    """exp(score) underflows to 0 where the value is NaN, and 0 x NaN is NaN: in its column of its sequence's heads, however
    the cache is cut (600 tokens: parts that the second kernel joins; 20000: a CTA joins those of its 192 tokens first)."""
    D, page = 64, 16
    cols = -(-n // page)
    r = rnd(n)
    table = r.permutation(B * cols).reshape(B, cols).astype(np.int32)
    k = np.zeros((B * cols, 1, page, D), np.float32)
    v = r.integers(-8, 9, (B * cols, 1, page, D)).astype(np.float32)
    best = table[:, top // page], 0, top % page
    k[best + (0,)] = 16.0                                                # a score of 256, and of 0 elsewhere
    v[table[:, 0], 0, 5, 3] = np.nan
    if kv == "e4m3":
        kc, vc = (torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).cuda() for x in (k, v))
        sc = torch.ones(1, device="cuda")
    else:
        kc, vc, sc = dev(k, BF16), dev(v, BF16), None
    q = torch.zeros((B, Hq, D), dtype=BF16, device="cuda")
    q[:, :, 0] = 16.0
    out = zmoe_paged_attention(q, kc, vc, dev(table), torch.full((B,), n, dtype=torch.int32, device="cuda"), scale=1.0,
                               k_scale=sc, v_scale=sc)
    want = np.repeat(v[best][:, None], Hq, 1)                            # all the weight lies on that token
    want[:, :, 3] = np.nan
    assert np.array_equal(f64(out), want, equal_nan=True)


@pytest.mark.parametrize("types", ["f32 f32 bf16", "bf16 bf16 f32", "f32 bf16 f32", "bf16 f32 bf16"])
@pytest.mark.parametrize("T,d", [(40, 24), (9, 256), (5, 2048), (4, 8192), (4, 32768), (2500, 384)])
def test_norm_rows_at_the_ends_of_the_range(T, d, types):
    """eps 0 scales a row to one, from a largest magnitude of 2^-56 to a sum of squares of 2^127: the squares below 2^-149
    that fp32 loses are d 2^-150 together, 2^-23 of the largest one's 2^-112."""
    ht, dt, xt = (F32 if n == "f32" else BF16 for n in types.split())
    r = rnd(d)
    h = r.uniform(-1, 1, (T, d))
    h[:, 5] = 1.0
    size = np.array([2.0 ** -56, 1e-12, 1.0, 2.0 ** 63 / np.sqrt(d)])[np.arange(T) % 4]
    h, gamma = dev(h * size[:, None], ht), dev(1 + 0.2 * r.standard_normal(d), F32)
    delta = dev(r.uniform(0, 0.01, (T, d)) * size[:, None], dt)
    for group in (0, 128) if d % 128 == 0 else (0,):
        o = zmoe_add_rmsnorm(h, gamma, delta, 0.0, out_dtype=xt, want_codes=True, group=group)
        check_norm(o, h, delta, gamma, 0.0, xt, group)
    # an eps of 2^-126 or more leaves no lower end: rows of subnormal numbers go to 0 as the formula has them
    eps = 2.0 ** -126
    tiny = dev(r.standard_normal((T, d)) * 1e-39, F32)
    check_norm(zmoe_add_rmsnorm(tiny, gamma, None, eps, out_dtype=xt), tiny, None, gamma, eps, xt, 0)


def test_norm_beyond_the_range():
    """Documented: a finite row whose sum of squares passes fp32's range gives 0, codes of 0 and scale 1; without eps a row
    of zeros gives NaN."""
    h = torch.full((2, 256), 1e30, device="cuda")
    h[1] = 0
    o = zmoe_add_rmsnorm(h, torch.ones(256, device="cuda"), eps=0.0, out_dtype=F32, want_codes=True)
    assert not o["x"][0].any() and not o["codes"][0].any() and o["scales"][0].item() == 1
    assert bool(torch.isnan(o["x"][1]).all()) and bool((o["codes"][1] & 0x7F == NAN_CODE).all())


def chained_state():
    r = rnd(61)
    kc, vc, _, _ = make_cache(r, 60, 2, 16, 64, "bf16")
    f = lambda *s: dev(r.standard_normal(s), F32)  # noqa: E731
    pos = dev(np.array([40, 0, 310], np.int32))
    return dict(kc=kc, vc=vc, table=dev(r.permutation(60).reshape(3, 20).astype(np.int32)), pos=pos, lens=pos + 1, h=f(3, 512),
                delta=f(3, 512), gamma=1 + 0.1 * f(512), ones=torch.ones(512, device="cuda"), xkv=f(3, 512), xq=f(3, 512),
                q=torch.empty((3, 8, 64), dtype=BF16, device="cuda"), o=torch.empty((3, 8, 64), device="cuda"),
                bias=f(1, 512), rep=torch.full((3,), 1.3, device="cuda"), frq=torch.full((3,), 0.2, device="cuda"),
                ids=[torch.zeros((3, 1), dtype=torch.int32, device="cuda") for _ in range(2)],
                inv=dev(10000.0 ** (-np.arange(0, 64, 2) / 64)),
                ws=torch.empty(zmoe_paged_attention_workspace_size(3, 8, 2, 64), dtype=torch.uint8, device="cuda"))


def chained_step(s, i, after=lambda: None):
    """Every input that changes is the output of the operator before it or of the step before: the keys and values are the
    norm's, the queries the norm of the attention's output, the residual that output's adjusted values, the history the
    ids of the step before."""
    kv = s["xkv"].view(3, 8, 64)
    zmoe_add_rmsnorm(s["h"], s["gamma"], s["delta"], outs=dict(h=s["h"], x=s["xkv"]))
    after()
    zmoe_kv_append(kv[:, :2], kv[:, 2:4], s["pos"], s["kc"], s["vc"], s["table"], q=s["xq"].view(3, 8, 64), inv_freq=s["inv"],
                   q_out=s["q"])
    after()
    zmoe_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], out=s["o"], workspace=s["ws"])
    after()
    zmoe_add_rmsnorm(s["o"].view(3, 512), s["ones"], outs=dict(x=s["xq"]))
    after()
    zmoe_adjust_logits(s["o"].view(3, 1, 512), s["ids"][i % 2].view(3, 1, 1), repetition=s["rep"], frequency=s["frq"],
                       bias=s["bias"], out=s["delta"].view(3, 1, 512), ids=s["ids"][1 - i % 2])
    after()


def test_chains_through_every_operator():
    """Sixty dependent steps, each kernel launched beside the one whose output it reads: as with a wait between all calls,
    and as two steps captured and replayed."""
    names = ("h", "delta", "xkv", "xq", "q", "o", "kc", "vc")

    def run(after):
        s = chained_state()
        torch.cuda.synchronize()
        for i in range(60):
            chained_step(s, i, after)
        torch.cuda.synchronize()
        return [s[k] for k in names] + s["ids"]

    want = run(torch.cuda.synchronize)
    assert all(bool(torch.isfinite(t.float()).all()) for t in want)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(want, run(lambda: None)))
    s = chained_state()
    chained_step(chained_state(), 0)                                     # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chained_step(s, 0)
        chained_step(s, 1)
    for _ in range(30):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, [s[k] for k in names] + s["ids"]))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_with_a_history_of_no_frames(dtype):
    """The first step of a stream: nothing is penalised yet."""
    z = dev(rnd(71).standard_normal((2, 3, 77)), dtype)
    one = torch.ones(2, device="cuda")
    hist, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 0, 3), (2,)))
    for kw in (dict(repetition=2 * one), dict(presence=one, frequency=one), dict(hist_lens=lens, repetition=2 * one)):
        out, ids = zmoe_adjust_logits(z, hist, **kw)
        assert torch.equal(out, z) and torch.equal(ids.long(), z.float().argmax(2))
    with pytest.raises(Exception, match="penalties need a history"):
        zmoe_adjust_logits(z, repetition=one)


def test_append_refuses_what_is_neither_true_nor_false():
    kc, vc, _, _ = make_cache(rnd(0), 4, 2, 16, 64, "bf16")
    before = kc.clone(), vc.clone()
    kv = torch.ones((2, 2, 64), dtype=BF16, device="cuda")
    pos, table = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="interleaved must be true or false"):
        zmoe_kv_append(kv, kv, pos, kc, vc, table, interleaved=torch.ones(2))
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
