"""The decode-step operators on the CPU: the oracle's pins (closed forms, hand-worked examples, torch's own
functions) and the refusals of the C entry points and of the binding.  Nothing here needs a GPU."""
import math

import numpy as np
import pytest
import torch

import oracle
from sparse_moe_decoder_b200 import build as B
from sparse_moe_decoder_b200 import zmoe as Z

NULL = None
A, A2, A3 = 0x10000, 0x20000, 0x30000   # aligned placeholders, never dereferenced
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    B.build()
    return Z.lib()


# ------------------------------------------------------------------------------------- oracle pins

def test_rotation_by_hand():
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]])
    quarter = np.array([math.pi / 2, math.pi])     # at position 1: a quarter turn, half a turn
    assert np.allclose(oracle.rotate(x, 1, quarter, False), [[-3, -2, 1, -4, 5, 6]])     # pairs (0, 2), (1, 3)
    assert np.allclose(oracle.rotate(x, 1, quarter, True), [[-2, 1, -3, -4, 5, 6]])      # pairs (0, 1), (2, 3)
    assert np.array_equal(oracle.rotate(x, 0, quarter, True), x)


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 32))
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    for pairs in (False, True):
        a = oracle.rotate(q, 107, f, pairs) @ oracle.rotate(k, 100, f, pairs).T
        b = oracle.rotate(q, 7, f, pairs) @ oracle.rotate(k, 0, f, pairs).T
        assert np.allclose(a, b)


def test_attention_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((6, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    out, lse = oracle.attend(q, k, v, 0.3)
    kt, vt = (torch.from_numpy(x).permute(1, 0, 2).repeat_interleave(3, 0) for x in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q)[:, None], kt, vt, scale=0.3)[:, 0]
    assert np.allclose(out, want.numpy())
    assert np.allclose(lse, torch.logsumexp(0.3 * (torch.from_numpy(q)[:, None] @ kt.transpose(1, 2))[:, 0], 1))
    gate = rng.standard_normal(6)
    assert np.allclose(oracle.attend(q, k, v, 0.3, gate)[0], out * torch.sigmoid(torch.from_numpy(gate)).numpy()[:, None])


def test_attention_of_nothing_and_of_one():
    q, v = np.ones((2, 4)), np.arange(8.0).reshape(1, 2, 4)
    out, lse = oracle.attend(q, np.zeros((0, 2, 4)), np.zeros((0, 2, 4)), 1.0)
    assert not out.any() and np.isneginf(lse).all()
    out, lse = oracle.attend(q, np.ones((1, 2, 4)), v, 0.5)
    assert np.array_equal(out, v[0]) and np.allclose(lse, 2.0)


def test_paged_rows_by_hand():
    cache = np.arange(3 * 1 * 2 * 1).reshape(3, 1, 2, 1)      # pages hold (0, 1), (2, 3), (4, 5)
    assert oracle.paged_rows(cache, np.array([2, 0]), 3).ravel().tolist() == [4, 5, 0]


def test_adjusted_logits_by_hand():
    z = np.array([[[2.0, -2.0, 1.0, 0.5]]])
    hist = np.array([[[0], [1], [0], [-1], [3]]])
    got = oracle.adjust_logits(z, hist, [4], [2.0], [0.25], [0.1], np.array([[0, 0, 1.0, 0]]),
                               np.array([[[True, True, True, False]]]))
    assert np.allclose(got[0, 0, :3], [1 - 0.2 - 0.25, -4 - 0.1 - 0.25, 2.0]) and np.isneginf(got[0, 0, 3])
    assert oracle.allowed_greedy(got).tolist() == [[2]]


def test_greedy_ids_ties_nan_and_nothing_allowed():
    z = np.array([[[1.0, 3.0, 3.0], [np.nan, -np.inf, np.nan], [5.0, 1.0, 2.0]]])
    ok = np.array([[[True, True, True], [True, True, True], [False, False, False]]])
    assert oracle.allowed_greedy(z, ok).tolist() == [[1, 1, -1]]
    assert oracle.mask_bits(np.ones((1, 1, 33), bool)).tolist() == [[[-1, 1]]]


# ------------------------------------------------------------------------------------- C entry points

def _norm(L, h=A, ht=F32, delta=A2, dt=F32, gamma=A3, eps=1e-6, T=4, d=256, ho=A, x=A2, xt=BF16, codes=A, scales=A,
          group=0):
    return L.zmoe_add_rmsnorm(h, ht, delta, dt, gamma, eps, T, d, ho, x, xt, codes, scales, group, NULL)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=12), dict(d=0), dict(d=-8), dict(ht=2), dict(dt=7), dict(xt=2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(h=NULL), dict(gamma=NULL), dict(group=64), dict(group=128, d=264), dict(h=A + 4),
    dict(delta=A + 8), dict(codes=A + 8), dict(scales=A + 2), dict(codes=NULL), dict(scales=NULL),
    dict(ho=NULL, x=NULL, codes=NULL, scales=NULL), dict(ho=A2, dt=BF16), dict(ho=A2, ht=BF16),
])
def test_add_rmsnorm_refusals(L, kw):
    assert _norm(L, **kw) == 1
    assert L.zmoe_last_error()


def test_add_rmsnorm_limits(L):
    assert _norm(L, d=32776) == 2
    assert _norm(L, T=0) == 0
    assert _norm(L, T=0, h=NULL, gamma=NULL) == 0


def _append(L, q=A, k=A, v=A, it=BF16, qs=2048, ks=512, vs=512, seq=A, pos=A, freq=A, rot=64, T=4, Hq=16, Hkv=4, D=128,
            q_out=A, kc=A, vc=A, kv=BF16, ksc=NULL, vsc=NULL, table=A, n_seqs=8, max_pages=4, n_pages=32, page=16,
            eps=1e-6, qg=NULL):
    return L.zmoe_kv_append(q, k, v, it, qs, ks, vs, seq, pos, freq, rot, 0, qg, NULL, eps, T, Hq, Hkv, D, q_out, kc, vc,
                            kv, ksc, vsc, table, n_seqs, max_pages, n_pages, page, NULL)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(Hkv=0), dict(Hq=-1), dict(it=2), dict(kv=0), dict(kv=E4M3), dict(kv=E4M3, ksc=A), dict(rot=8),
    dict(rot=144), dict(rot=-16), dict(freq=NULL), dict(page=8), dict(page=24), dict(page=0), dict(max_pages=-1),
    dict(n_pages=-1), dict(eps=-1.0), dict(seq=NULL, n_seqs=3), dict(k=NULL), dict(v=NULL), dict(pos=NULL),
    dict(kc=NULL), dict(vc=NULL), dict(table=NULL), dict(q_out=NULL), dict(q=NULL), dict(qs=1024), dict(ks=516),
    dict(vs=-512), dict(k=A + 8), dict(kc=A + 8), dict(q_out=A + 2), dict(qg=A + 4), dict(pos=A + 2), dict(freq=A + 4),
    dict(max_pages=1 << 28, page=16), dict(Hq=70000, qs=70000 * 128),
])
def test_kv_append_refusals(L, kw):
    assert _append(L, **kw) == 1
    assert L.zmoe_last_error()


def test_kv_append_limits(L):
    for D in (32, 96, 256):
        assert _append(L, D=D, rot=16, qs=16 * D, ks=4 * D, vs=4 * D) == 2
    assert _append(L, T=0) == 0


def _attn(L, q=A, kc=A, vc=A, kv=BF16, ksc=NULL, vsc=NULL, table=A, lens=A, gate=NULL, scale=0.1, B=2, Hq=16, Hkv=4,
          D=128, max_pages=4, n_pages=32, page=16, out=A, ot=F32, lse=NULL, ws=A, nb=1 << 30):
    return L.zmoe_paged_attention(q, kc, vc, kv, ksc, vsc, table, lens, gate, scale, B, Hq, Hkv, D, max_pages, n_pages, page,
                                  out, ot, lse, ws, nb, NULL)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(Hq=15), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(kv=F32), dict(kv=E4M3), dict(ot=2), dict(page=8),
    dict(page=20), dict(max_pages=-1), dict(n_pages=0), dict(scale=float("nan")), dict(q=NULL), dict(kc=NULL),
    dict(vc=NULL), dict(lens=NULL), dict(out=NULL), dict(table=NULL), dict(q=A + 8), dict(kc=A + 8), dict(out=A + 4),
    dict(lens=A + 1), dict(ws=A + 8), dict(max_pages=1 << 28), dict(n_pages=1 << 28, Hkv=4),
])
def test_paged_attention_refusals(L, kw):
    assert _attn(L, **kw) == 1
    assert L.zmoe_last_error()


def test_paged_attention_limits(L):
    assert _attn(L, D=96) == 2
    assert _attn(L, ws=NULL) == 4
    n = L.zmoe_paged_attention_workspace_size(2, 16, 4, 128)
    assert n > 0 and _attn(L, nb=n - 1) == 4
    assert _attn(L, B=0) == 0
    for bad in ((0, 16, 4, 128), (2, 15, 4, 128), (2, 16, 0, 128), (2, 16, 4, 96)):
        assert L.zmoe_paged_attention_workspace_size(*bad) == 0


def _adjust(L, lg=A, dt=F32, hist=A, lens=A, rep=A, pre=A, frq=A, bias=A, mask=A, T=2, N=9, V=1025, hl=16, out=A, ids=A):
    return L.zmoe_adjust_logits(lg, dt, hist, lens, rep, pre, frq, bias, mask, T, N, V, hl, out, ids, NULL)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(N=0), dict(V=0), dict(hl=-1), dict(hl=65536), dict(dt=2), dict(lg=NULL), dict(out=NULL),
    dict(hist=NULL), dict(lg=A + 2), dict(out=A + 1, dt=BF16), dict(bias=A + 2), dict(ids=A + 2), dict(V=0x7fffffff),
    dict(T=1 << 28, N=9),
])
def test_adjust_logits_refusals(L, kw):
    assert _adjust(L, **kw) == 1
    assert L.zmoe_last_error()


def test_adjust_logits_of_no_stream(L):
    assert _adjust(L, T=0) == 0


# ------------------------------------------------------------------------------------- the binding

def _cpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: Z.zmoe_add_rmsnorm(_cpu(2, 16), _cpu(16)),
    lambda: Z.zmoe_kv_append(_cpu(2, 1, 64), _cpu(2, 1, 64), _cpu(2, dtype=torch.int32),
                             _cpu(4, 1, 16, 64, dtype=torch.bfloat16), _cpu(4, 1, 16, 64, dtype=torch.bfloat16),
                             _cpu(2, 2, dtype=torch.int32)),
    lambda: Z.zmoe_paged_attention(_cpu(2, 4, 64, dtype=torch.bfloat16), _cpu(4, 1, 16, 64, dtype=torch.bfloat16),
                                   _cpu(4, 1, 16, 64, dtype=torch.bfloat16), _cpu(2, 2, dtype=torch.int32),
                                   _cpu(2, dtype=torch.int32)),
    lambda: Z.zmoe_adjust_logits(_cpu(1, 9, 1025)),
])
def test_host_tensors_are_rejected(call):
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        call()


def test_compiled_calls_refuse_what_is_no_tensor_and_wrong_counts():
    b, t = Z._calls(), _cpu(2, 4)
    for call, n in ((b.add_rmsnorm, 11), (b.kv_append, 17), (b.paged_attention, 13), (b.adjust_logits, 11)):
        for args in ((t,) * n, (None,) * n, (1,) * n, ("x",) * n):
            with pytest.raises(TypeError, match="must be a CUDA tensor"):
                call(*args)
        for args in ((), (t,) * (n - 1), (t,) * (n + 1)):
            with pytest.raises(TypeError, match=f"{n} arguments wanted, got {len(args)}"):
                call(*args)


def test_missing_compiled_calls_fail_loudly(monkeypatch):
    import sys
    monkeypatch.setattr(Z, "_binding", None)
    monkeypatch.setitem(sys.modules, "sparse_moe_decoder_b200._binding", None)
    monkeypatch.delattr(sys.modules["sparse_moe_decoder_b200"], "_binding", raising=False)
    with pytest.raises(ImportError, match="build it with"):
        Z._calls()
