"""The operators around the MoE path of a decode step, as they are measured.

Four operators of the served decoder: the residual addition with RMSNorm and 8-bit output, the append of
rotated keys and values to a paged cache, the attention of one new token over that cache, and the adjustment
of the codebook logits before the next frame is chosen.  ``run`` makes one pass in plain torch operations
(``own`` false) or through libzmoe's calls (``own`` true); ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TWO_PI = 2.0 * math.pi
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _norm(T, d, h, delta, x, group, name=None):
    """h, delta, x: types; x "none": only the codes are wanted; group: columns that share a scale, 0 a row."""
    c = dict(op="norm", T=T, d=d, h=h, delta=delta, x=x, group=group)
    return dict(name=name, **c) if name else c


def _append(seqs, each, pad, Hq, Hkv, D, rot, pairs, qknorm, src, kv, page, first, name=None):
    """seqs sequences get `each` new tokens at positions from `first` on (each sequence a little further);
    `pad` padding tokens follow; rot: rotated columns; pairs: neighbouring columns make a pair."""
    c = dict(op="append", seqs=seqs, each=each, pad=pad, Hq=Hq, Hkv=Hkv, D=D, rot=rot, pairs=pairs, qknorm=qknorm,
             src=src, kv=kv, page=page, first=first)
    return dict(name=name, **c) if name else c


def _attn(B, longest, ragged, Hq, Hkv, D, kv, page, gate, out, name=None):
    """B sequences of up to `longest` cached tokens (ragged: spread from 1 to that)."""
    c = dict(op="attn", B=B, longest=longest, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, kv=kv, page=page, gate=gate, out=out)
    return dict(name=name, **c) if name else c


def _logits(T, N, V, L, src, bias, mask, name=None):
    """T streams, N codebooks of V ids, L frames of history."""
    c = dict(op="logits", T=T, N=N, V=V, L=L, src=src, bias=bias, mask=mask)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # the pre-norm of one stream's decode step: one row, where latency is all there is
        _norm(1, 2048, "f32", "f32", "bf16", 0, "norm_one_row"),
        # the prefill layer's 16384 tokens: the fp32 residual stream in, the router's bf16 row and the W8A8
        # experts' codes with one scale a token out
        _norm(16384, 2048, "f32", "f32", "bf16", 0, "norm_prefill_rowscale"),
        # a 16-bit residual stream feeding a projection that takes codes in blocks of 128, an odd token count
        _norm(5003, 4096, "bf16", "bf16", "none", 128, "norm_16bit_blocks"),
        # 64 streams, one new token each: the decode step's append with query and key norms
        _append(64, 1, 0, 16, 4, 128, 128, False, True, "bf16", "bf16", 16, 700, "append_decode"),
        # 8 prompts of 2048 tokens, the projection's fp32 output, into a bf16 cache
        _append(8, 2048, 0, 16, 4, 128, 128, False, True, "f32", "bf16", 64, 0, "append_prompts"),
        # continued prompts of odd length far into their sequences, padded batch, 8-bit cache, half of each
        # head rotated, neighbouring pairs
        _append(3, 999, 27, 12, 2, 64, 32, True, False, "bf16", "e4m3", 32, 40000, "append_far_8bit"),
        # one stream a few seconds into its speech: the smallest attention call
        _attn(1, 431, False, 16, 4, 128, "bf16", 16, False, "bf16", "attn_one_stream"),
        # 64 streams of 1 to 4096 frames with the heads' gates: the ordinary decode step
        _attn(64, 4096, True, 16, 4, 128, "bf16", 16, True, "f32", "attn_streams"),
        # a few very long sequences in an 8-bit cache
        _attn(4, 131072, True, 32, 4, 128, "e4m3", 64, False, "bf16", "attn_long_8bit"),
        # the next frame of one stream: 9 codebooks of 1025 ids, repetition over the last 128 frames
        _logits(1, 9, 1025, 128, "f32", True, False, "logits_one_frame"),
        # the same for 64 streams, with a mask of allowed ids for each
        _logits(64, 9, 1025, 512, "f32", True, True, "logits_frames"),
        # a text-sized vocabulary of odd size, 16-bit logits, long history
        _logits(192, 1, 100003, 2048, "bf16", True, True, "logits_vocabulary"),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "logits"])
    if op == "norm":
        group = rng.choice([0, 128])
        d = 128 * _between(rng, 2, 64) if group else 8 * _between(rng, 16, 1024)
        T = _between(rng, 1, max(1, min(16384, 16384 * 2048 // d)))
        h = rng.choice(["f32", "bf16"])
        return _norm(T, d, h, rng.choice(["f32", h]), rng.choice(["bf16", "f32", "none"]), group)
    if op == "append":
        Hkv, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        most = max(1, 16384 * 16 * 128 // (Hq * D))
        seqs = _between(rng, 1, 64)
        each = _between(rng, 1, max(1, min(4096, 16384 // seqs, most // seqs)))
        return _append(seqs, each, rng.choice([0, 5, 27]), Hq, Hkv, D, rng.choice([D, D // 2]),
                       rng.random() < 0.5, rng.random() < 0.5, rng.choice(["f32", "bf16"]),
                       rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 128]), rng.choice([0, 17, 5000, 100000]))
    if op == "attn":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        B = _between(rng, 1, 128)
        longest = _between(rng, 1, max(1, min(131072, 4 * 131072 * 4 * 128 // (B * Hkv * D) // 2)))
        return _attn(B, longest, rng.random() < 0.7, Hkv * rng.choice([1, 3, 4, 8, 16]), Hkv, D,
                     rng.choice(["bf16", "e4m3"]), rng.choice([16, 32, 64, 128]), rng.random() < 0.5,
                     rng.choice(["bf16", "f32"]))
    N = rng.choice([1, 2, 9])
    V = _between(rng, 257, 131072)
    T = _between(rng, 1, max(1, min(256, 192 * 100003 // (N * V))))
    return _logits(T, N, V, _between(rng, 1, 2048), rng.choice(["f32", "bf16"]), rng.random() < 0.5,
                   rng.random() < 0.5)


def _lens(c):
    """The cached tokens of each sequence, spread by the golden ratio."""
    if not c["ragged"]:
        return [c["longest"]] * c["B"]
    return [1 + int((c["longest"] - 1) * math.modf((b + 1) * 0.6180339887498949)[0]) for b in range(c["B"])]


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "e4m3": 1, "none": 0}
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        scales = c["T"] * (c["d"] // c["group"] if c["group"] else 1)
        return dict(bytes=n * (2 * size[c["h"]] + size[c["delta"]] + size[c["x"]] + 1) + 4 * c["d"] + 4 * scales,
                    flops=8 * n)
    if c["op"] == "append":
        T = c["seqs"] * c["each"]
        row = c["Hq"] + 2 * c["Hkv"]
        return dict(bytes=T * c["D"] * (row * size[c["src"]] + 2 * c["Hq"] + 2 * c["Hkv"] * size[c["kv"]]) + 8 * T,
                    flops=8 * T * row * c["D"])
    if c["op"] == "attn":
        n = sum(_lens(c))
        return dict(bytes=2 * n * c["Hkv"] * c["D"] * size[c["kv"]] + 4 * n // c["page"]
                    + c["B"] * c["Hq"] * (c["D"] * (2 + size[c["out"]]) + 4), flops=4 * n * c["Hq"] * c["D"])
    n = c["T"] * c["N"] * c["V"]
    return dict(bytes=n * 2 * size[c["src"]] + 4 * c["T"] * c["N"] * (c["L"] + 1)
                + (4 * c["N"] * c["V"] if c["bias"] else 0) + (n // 8 if c["mask"] else 0), flops=6 * n)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    rand = lambda *shape: torch.rand(shape, generator=g, device=DEV)  # noqa: E731
    s = dict(case)
    c = case
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        # a residual stream whose rows differ in size, with a few columns far larger than the rest
        wide = torch.where(rand(d) < 0.004, 20.0, 1.0)
        s["h"] = (randn(T, d) * (0.3 + 3 * rand(T, 1)) * wide).to(TYPES[c["h"]])
        s["delta"] = (0.5 * randn(T, d)).to(TYPES[c["delta"]])
        s["gamma"] = 1 + 0.1 * randn(d)
        s["eps"] = 1e-6
        outs = dict(h=torch.empty_like(s["h"]), codes=torch.empty((T, d), dtype=torch.uint8, device=DEV),
                    scales=torch.empty((T, d // c["group"] if c["group"] else 1), device=DEV))
        if c["x"] != "none":
            outs["x"] = torch.empty((T, d), dtype=TYPES[c["x"]], device=DEV)
        s["outs"] = outs
    elif c["op"] == "append":
        D, Hq, Hkv, page, each = c["D"], c["Hq"], c["Hkv"], c["page"], c["each"]
        n, T = c["seqs"] * c["each"], c["seqs"] * c["each"] + c["pad"]
        qkv = (1.5 * randn(T, (Hq + 2 * Hkv) * D)).to(TYPES[c["src"]])
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        i = torch.arange(T, device=DEV)
        at = c["first"] + 3 * (i // each) + i % each
        s["seq"] = torch.where(i < n, i // each, -1).int()
        s["pos"] = torch.where(i < n, at, 0).int()
        # only the pages that get a token exist here; the earlier columns of the table point at page 0
        last = c["first"] + 3 * (c["seqs"] - 1) + each - 1
        cols, low = last // page + 1, c["first"] // page
        live = cols - low
        order = torch.randperm(c["seqs"] * live, generator=g, device=DEV).int()
        s["page_table"] = torch.zeros((c["seqs"], cols), dtype=torch.int32, device=DEV)
        s["page_table"][:, low:] = order.view(c["seqs"], live)
        shape = (c["seqs"] * live, Hkv, page, D)
        if c["kv"] == "e4m3":
            s["k_cache"], s["v_cache"] = (randn(*shape).mul_(64).to(E4M3).view(torch.uint8) for _ in range(2))
            s["k_scale"] = 0.01 + 0.01 * rand(Hkv)
            s["v_scale"] = 0.01 + 0.01 * rand(Hkv)
        else:
            s["k_cache"], s["v_cache"] = (randn(*shape).to(BF16) for _ in range(2))
            s["k_scale"] = s["v_scale"] = None
        r = c["rot"]
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
        s["q_gamma"], s["k_gamma"] = ((1 + 0.1 * randn(D)) if c["qknorm"] else None for _ in range(2))
        s["q_out"] = torch.zeros((T, Hq, D), dtype=BF16, device=DEV)
    elif c["op"] == "attn":
        B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
        lens = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
        need = (lens + page - 1) // page
        cols, total = int((c["longest"] + page - 1) // page), int(need.sum())
        order = torch.randperm(total, generator=g, device=DEV).int()
        s["page_table"] = torch.zeros((B, cols), dtype=torch.int32, device=DEV)
        s["page_table"][torch.arange(cols, device=DEV)[None] < need[:, None]] = order
        s["lens"] = lens
        shape = (total, Hkv, page, D)
        # keys that some tokens stand out of, as after training; values of unit size
        if c["kv"] == "e4m3":
            s["k_cache"] = randn(*shape).mul_(90).clamp_(-448, 448).to(E4M3).view(torch.uint8)
            s["v_cache"] = randn(*shape).mul_(90).clamp_(-448, 448).to(E4M3).view(torch.uint8)
            s["k_scale"] = (1.5 + rand(Hkv)) / 90
            s["v_scale"] = (0.5 + rand(Hkv)) / 90
        else:
            s["k_cache"] = randn(*shape).mul_(1.5).to(BF16)
            s["v_cache"] = randn(*shape).to(BF16)
            s["k_scale"] = s["v_scale"] = None
        s["q"] = (1.5 * randn(B, Hq, D)).to(BF16)
        s["scale"] = D ** -0.5
        s["gate"] = 2 * randn(B, Hq) if c["gate"] else None
        s["out"] = torch.empty((B, Hq, D), dtype=TYPES[c["out"]], device=DEV)
        s["lse"] = torch.empty((B, Hq), device=DEV)
    else:
        T, N, V, L = c["T"], c["N"], c["V"], c["L"]
        s["logits"] = (3 * randn(T, N, V)).to(TYPES[c["src"]])
        # a stream's history favours some ids; a frame that is not there yet is -1, behind the stream's length
        s["hist_lens"] = (L * rand(T)).int() if T > 1 else torch.full((1,), L, dtype=torch.int32, device=DEV)
        s["history"] = (V * rand(T, L, N) ** 3).int().clamp_(0, V - 1)
        s["history"][torch.arange(L, device=DEV)[None] >= s["hist_lens"][:, None]] = -1
        s["repetition"] = 1 + 0.5 * rand(T)
        s["presence"] = 0.4 * rand(T)
        s["frequency"] = 0.2 * rand(T)
        s["bias"] = 0.5 * randn(N, V) if c["bias"] else None
        words = (V + 31) // 32
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (T, N, words), generator=g, device=DEV).int() if c["mask"] else None
        s["out"] = torch.empty_like(s["logits"])
        s["ids"] = torch.empty((T, N), dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _RUN_OWN[state["op"]](state)
    return _RUN_PLAIN[state["op"]](state)


def _plain_norm(s):
    """h' = h + delta; x = h' / sqrt(mean h'^2 + eps) gamma; codes = E4M3(x / scale), scale = max|x| / 448."""
    T, d = s["h"].shape
    h = (s["h"].float() + s["delta"].float()).to(s["h"].dtype)
    hf = h.float()
    x = hf / torch.sqrt((hf * hf).mean(1, keepdim=True) + s["eps"]) * s["gamma"]
    xf = x.view(T, -1, s["group"] or d)
    top = xf.abs().amax(2)
    scales = torch.where(top > 0, top / 448, 1.0)
    codes = (xf * (1 / scales)[..., None]).clamp(-448, 448).to(E4M3).view(T, d)
    out = dict(h=h, codes=codes, scales=scales)
    if s["x"] != "none":
        out["x"] = x.to(TYPES[s["x"]])
    return out


def _rotate(x, cos, sin, pairs):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if pairs else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_append(s):
    """q, k normed and rotated by position, k and v stored in the pages of their sequences."""
    n, page = s["seqs"] * s["each"], s["page"]
    pos, seq = s["pos"][:n].long(), s["seq"][:n].long()
    angle = pos.double()[:, None, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q, k, v = s["q"][:n].float(), s["k"][:n].float(), s["v"][:n].float()
    if s["qknorm"]:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["q_gamma"]
        k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["k_gamma"]
    q, k = _rotate(q, cos, sin, s["pairs"]), _rotate(k, cos, sin, s["pairs"])
    pid, row = s["page_table"][seq, pos // page].long(), pos % page
    s["q_out"][:n] = q.to(BF16)
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        if s["kv"] == "e4m3":
            x = (x * (1 / scale)[:, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        cache[pid, :, row] = x.to(cache.dtype)
    return _caches(s)


def _caches(s):
    k, v = s["k_cache"], s["v_cache"]
    if s["kv"] == "e4m3":
        k, v = k.view(E4M3), v.view(E4M3)
    return dict(q=s["q_out"], k=k, v=v)


def _plain_attn(s):
    """softmax(scale q K^T) V over each sequence's pages, times the heads' gates."""
    B, Hq, D = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]

    def pages(cache, scale):
        x = cache[s["page_table"].long()]                                # [B, cols, Hkv, page, D]
        x = (x.view(E4M3) if s["kv"] == "e4m3" else x).float()
        x = x.transpose(1, 2).flatten(2, 3)                              # [B, Hkv, cols page, D]
        return x if scale is None else x * scale[:, None, None]

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    score = q @ pages(s["k_cache"], s["k_scale"]).transpose(2, 3) * s["scale"]
    dead = torch.arange(score.shape[-1], device=DEV) >= s["lens"][:, None]
    score = score.masked_fill(dead[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ pages(s["v_cache"], s["v_scale"]) / total).view(B, Hq, D)
    lse = (top + torch.log(total)).view(B, Hq)
    if s["gate"] is not None:
        out = out * (1 / (1 + torch.exp(-s["gate"])))[..., None]
    return dict(out=out.to(s["out"].dtype), lse=lse)


def _allowed(s):
    V = s["V"]
    if s["mask"] is None:
        return None
    bits = (s["mask"][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    return bits.flatten(2)[..., :V] != 0


def _plain_logits(s):
    """Repetition, frequency and presence penalties by the ids' counts, bias, mask; the largest's lowest id."""
    T, N, V = s["logits"].shape
    hist = s["history"].transpose(1, 2).long()
    seen = (hist >= 0) & (torch.arange(s["L"], device=DEV) < s["hist_lens"][:, None, None])
    counts = torch.zeros((T, N, V), device=DEV).scatter_add_(2, hist.clamp(min=0), seen.float())
    x = s["logits"].float()
    rep, col = s["repetition"][:, None, None], lambda name: s[name][:, None, None]
    hit = counts > 0
    x = torch.where(hit, torch.where(x > 0, x / rep, x * rep), x)
    x = x - col("frequency") * counts
    x = torch.where(hit, x - col("presence"), x)
    if s["bias"] is not None:
        x = x + s["bias"]
    ok = _allowed(s)
    if ok is not None:
        x = torch.where(ok, x, -math.inf)
    x = x.to(s["logits"].dtype)
    f = x.float()
    can = f == f if ok is None else ok & (f == f)
    best = torch.where(can, f, -math.inf).amax(2, keepdim=True)
    ids = torch.where(can & (f == best), torch.arange(V, device=DEV), V).amin(2)
    return dict(logits=x, ids=torch.where(ids < V, ids, -1).int())


_RUN_PLAIN = dict(norm=_plain_norm, append=_plain_append, attn=_plain_attn, logits=_plain_logits)


def _own_norm(s):
    from sparse_moe_decoder_b200 import zmoe_add_rmsnorm
    o = zmoe_add_rmsnorm(s["h"], s["gamma"], s["delta"], eps=s["eps"], group=s["group"],
                         out_dtype=F32 if s["x"] == "f32" else BF16, outs=s["outs"])
    out = dict(h=o["h"], codes=o["codes"].view(E4M3), scales=o["scales"])
    if s["x"] != "none":
        out["x"] = o["x"]
    return out


def _own_append(s):
    from sparse_moe_decoder_b200 import zmoe_kv_append
    zmoe_kv_append(s["k"], s["v"], s["pos"], s["k_cache"], s["v_cache"], s["page_table"], q=s["q"], seq=s["seq"],
                   inv_freq=s["inv_freq"], interleaved=s["pairs"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"],
                   eps=1e-6, k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"])
    return _caches(s)


def _own_attn(s):
    from sparse_moe_decoder_b200 import zmoe_paged_attention, zmoe_paged_attention_workspace_size
    if "workspace" not in s:
        n = zmoe_paged_attention_workspace_size(s["B"], s["Hq"], s["Hkv"], s["D"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    zmoe_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], scale=s["scale"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"], gate=s["gate"], out=s["out"], lse=s["lse"],
                         workspace=s["workspace"])
    return dict(out=s["out"], lse=s["lse"])


def _own_logits(s):
    from sparse_moe_decoder_b200 import zmoe_adjust_logits
    zmoe_adjust_logits(s["logits"], history=s["history"], hist_lens=s["hist_lens"], repetition=s["repetition"],
                       presence=s["presence"], frequency=s["frequency"], bias=s["bias"], mask=s["mask"],
                       out=s["out"], ids=s["ids"])
    return dict(logits=s["out"], ids=s["ids"])


_RUN_OWN = dict(norm=_own_norm, append=_own_append, attn=_own_attn, logits=_own_logits)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_norm(c, s):
    h = s["h"].double() + s["delta"].double()
    # the normalised row belongs to the stored, rounded sum
    kept = h.to(s["h"].dtype).double()
    x = kept * torch.rsqrt(kept.pow(2).sum(1, keepdim=True) / c["d"] + s["eps"]) * s["gamma"].double()
    width = c["group"] or c["d"]
    parts = x.reshape(c["T"], c["d"] // width, width)
    scales = parts.abs().max(2).values / 448.0
    codes = (parts / scales.clamp(min=1e-300)[:, :, None]).reshape(c["T"], c["d"])
    out = dict(h=h, codes=codes, scales=scales)
    if c["x"] != "none":
        out["x"] = x
    return out


def _exact_append(c, s):
    D, half, page = c["D"], c["rot"] // 2, c["page"]
    n = c["seqs"] * c["each"]
    pos = s["pos"][:n].double().cpu().numpy()
    freq = s["inv_freq"].cpu().numpy()
    turn = torch.from_numpy(np.exp(1j * np.outer(pos, freq))).to(DEV)[:, None, :]
    first = torch.arange(half, device=DEV) * (2 if c["pairs"] else 1)
    second = first + (1 if c["pairs"] else half)

    def head(x, gamma, rotate):
        x = x[:n].double()
        if gamma is not None:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * gamma.double()
        x = x.clone()
        if rotate:
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
        return x

    q_out = s["q_out"].double()
    q_out[:n] = head(s["q"], s["q_gamma"], True)
    where = s["pos"][:n].long()
    slot = s["page_table"].long()[s["seq"][:n].long(), where // page]
    out = dict(q=q_out)
    for name, x, scale in (("k", head(s["k"], s["k_gamma"], True), s["k_scale"]), ("v", head(s["v"], None, False), s["v_scale"])):
        cache = s[name + "_cache"]
        cache = (cache.view(E4M3) if c["kv"] == "e4m3" else cache).double()
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448, 448)
        cache[slot, :, where % page] = x
        out[name] = cache
    return out


def _exact_attn(c, s):
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lens(c)):
        ids = s["page_table"][b, :(n + page - 1) // page].long()
        for g in range(Hkv):
            k, v = (s[m][ids, g].reshape(-1, D)[:n] for m in ("k_cache", "v_cache"))
            if c["kv"] == "e4m3":
                k, v = k.view(E4M3).double() * s["k_scale"][g].double(), v.view(E4M3).double() * s["v_scale"][g].double()
            heads = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            logit = s["scale"] * (k.double() @ s["q"][b, heads].double().T)
            lse[b, heads] = torch.logsumexp(logit, 0)
            out[b, heads] = torch.exp(logit - lse[b, heads]).T @ v.double()
    if s["gate"] is not None:
        out *= torch.sigmoid(s["gate"].double())[..., None]
    return dict(out=out, lse=lse)


def _exact_logits(c, s):
    T, N, V = c["T"], c["N"], c["V"]
    x = s["logits"].double()
    for t in range(T):
        past = s["history"][t, :int(s["hist_lens"][t])].long()
        for n in range(N):
            times = torch.bincount(past[:, n], minlength=V).double()
            row, rep = x[t, n], s["repetition"][t].double()
            row = torch.where(times == 0, row, torch.where(row > 0, row / rep, row * rep))
            x[t, n] = row - s["frequency"][t].double() * times - s["presence"][t].double() * (times > 0)
    if s["bias"] is not None:
        x = x + s["bias"].double()
    if s["mask"] is not None:
        v = torch.arange(V, device=DEV)
        on = (s["mask"].long()[:, :, v // 32] >> (v % 32)) & 1
        x = x.masked_fill(on == 0, -math.inf)
    # the ids are the largest of the values as they are stored, so 64 bits say nothing about them
    return dict(logits=x, ids=None)


_EXACT = dict(norm=_exact_norm, append=_exact_append, attn=_exact_attn, logits=_exact_logits)
