"""The decoder's attention blocks at decode steps: a paged key-value cache, the block that reads and extends it, and
the rules on the codebook logits that choose the next frame.

ZONOS2 Technical Report digest, "method overview and architecture", item 5 (grouped-query attention with headwise
gating, rotary positions, pre-norm blocks).  Everything on the device is preallocated and a step leaves no decision
to the host but new pages (``PagedCache.reserve``), so a step may be captured into a CUDA graph once the pages are
reserved.  The projections are zmoe_speaker_prefix's product W e, which streams the weights once per 8 tokens.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional

import torch

from . import zmoe as Z


@dataclass
class AttentionWeights:
    """One attention block: h <- h + W_o (sigmoid(W_gate x) * attention(W_qkv x)), x = RMSNorm(h) * gamma.

    w_qkv [(Hq + 2 Hkv) D, d]: the queries', keys' and values' rows one after another; w_o [d, Hq D]; w_gate [Hq, d]
    or None (no gates); gamma f32 [d]; q_gamma, k_gamma f32 [D] or None (no query or key norm)."""

    w_qkv: torch.Tensor
    w_o: torch.Tensor
    gamma: torch.Tensor
    Hq: int
    Hkv: int
    w_gate: Optional[torch.Tensor] = None
    q_gamma: Optional[torch.Tensor] = None
    k_gamma: Optional[torch.Tensor] = None

    @property
    def D(self) -> int:
        return self.w_qkv.shape[0] // (self.Hq + 2 * self.Hkv)


class PagedCache:
    """Keys and values of ``n_seqs`` sequences in pages, for ``n_layers`` layers that share one page table.

    dtype torch.bfloat16, or torch.uint8 for E4M3 codes with k_scale, v_scale f32 [n_layers, Hkv].  Pages are handed
    out by ``reserve`` and taken back by ``release``; ``advance`` gives every sequence its next position.  ``lens`` counts
    cached tokens only: it never passes ``room``, the tokens that a sequence's pages hold.  A released sequence is idle
    until it gets pages again: its tokens are padding (``seq`` -1), it stays at position 0 and counts no errors.  A place
    that has had no sequence yet is made idle in the same way."""

    def __init__(self, n_layers: int, n_seqs: int, max_len: int, Hkv: int, D: int, page_size: int = 16,
                 n_pages: Optional[int] = None, dtype: torch.dtype = torch.bfloat16,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None, device="cuda"):
        if page_size < 16 or page_size % 16:
            raise ValueError("page_size must be a multiple of 16")
        if (dtype == torch.uint8) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("an E4M3 cache (uint8), and no other, has k_scale and v_scale")
        self.page_size, self.n_seqs, self.max_len = page_size, n_seqs, max_len
        cols = -(-max_len // page_size)
        self.n_pages = n_seqs * cols if n_pages is None else n_pages
        shape = (n_layers, self.n_pages, Hkv, page_size, D)
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        self.k_scale, self.v_scale = k_scale, v_scale
        self.table = torch.full((n_seqs, cols), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)   # cached tokens
        self.pos = torch.zeros(n_seqs, dtype=torch.int32, device=device)    # the step's positions
        self.room = torch.zeros(n_seqs, dtype=torch.int32, device=device)   # tokens that the reserved pages hold
        self.seq = torch.arange(n_seqs, dtype=torch.int32, device=device)   # the sequences' own numbers, -1: idle
        self.idle = torch.zeros(n_seqs, dtype=torch.int32, device=device)   # -1 where idle, 0 elsewhere
        self.rules: List["LogitRules"] = []   # whose streams these sequences are: they forget a sequence with its release
        self.free: List[int] = list(range(self.n_pages - 1, -1, -1))
        self.pages: List[List[int]] = [[] for _ in range(n_seqs)]

    def reserve(self, length: int, seq: Optional[int] = None, stream=None) -> None:
        """Pages for the first ``length`` tokens of sequence ``seq`` (None: of every sequence).  The device's side of it
        happens on ``stream`` (None: the current one): the stream of the steps, between which it belongs."""
        if length > self.max_len:
            raise ValueError(f"{length} tokens in a cache of {self.max_len}")
        need = -(-length // self.page_size)
        for s in range(self.n_seqs) if seq is None else (seq,):
            have = len(self.pages[s])
            if need <= have:
                continue
            if need - have > len(self.free):
                raise RuntimeError(f"the cache is out of pages: sequence {s} needs {need - have}, {len(self.free)} are free")
            new = [self.free.pop() for _ in range(need - have)]
            self.pages[s] += new
            with torch.cuda.stream(stream):
                self.table[s, have:need] = torch.tensor(new, dtype=torch.int32)
                self.room[s] = need * self.page_size
                self.seq[s] = s
                self.idle[s] = 0

    def release(self, seq: int, stream=None) -> None:
        """Takes a sequence's pages back; it is idle until ``reserve`` gives it pages, and starts again at position 0,
        with no frames in the history of ``rules``.  ``stream``: as for ``reserve``."""
        self.free += reversed(self.pages[seq])
        self.pages[seq] = []
        with torch.cuda.stream(stream):
            self.table[seq].fill_(-1)
            self.lens[seq].zero_()
            self.room[seq].zero_()
            self.seq[seq] = -1
            self.idle[seq] = -1
        for r in self.rules:
            r.release(seq, stream)

    def advance(self, stream=None) -> None:
        """One more token for every sequence: its position in ``pos``, its new length in ``lens``.  A position
        without a reserved page counts a device error when the token is stored, and the token is lost: the length
        stays, so that a page that comes later holds no row that was never stored."""
        with torch.cuda.stream(stream):
            self.pos.copy_(self.lens)
            self.lens.add_(1)
            torch.minimum(self.lens, self.room, out=self.lens)

    def layer(self, i: int) -> dict:
        """The cache arguments of zmoe_kv_append and zmoe_paged_attention for layer ``i``."""
        return dict(k_cache=self.k[i], v_cache=self.v[i], page_table=self.table,
                    k_scale=None if self.k_scale is None else self.k_scale[i],
                    v_scale=None if self.v_scale is None else self.v_scale[i])


class AttentionRunner:
    """Preallocated buffers of one attention block shape for T sequences."""

    def __init__(self, T: int, d: int, Hq: int, Hkv: int, D: int, inv_freq: Optional[torch.Tensor] = None,
                 interleaved: bool = False, device="cuda"):
        dev = torch.device(device)
        if D not in (64, 128) or d < 8 or d % 8 or max(d, Hq * D) > 6400:
            raise ValueError(f"heads of 64 or 128 columns, d a multiple of 8, d and Hq * D at most 6400 (the rows that the "
                             f"projections hold in shared memory): got D {D}, d {d}, Hq {Hq}")
        self.Hq, self.Hkv, self.D, self.inv_freq, self.interleaved = Hq, Hkv, D, inv_freq, interleaved
        f32 = dict(dtype=torch.float32, device=dev)
        self.x = torch.empty((T, d), **f32)
        qkv = self.qkv = torch.empty((T, (Hq + 2 * Hkv) * D), **f32)
        self.q_in = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        self.k_in = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        self.v_in = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        self.q = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=dev)   # a token that is not stored leaves its row
        self.gate = torch.empty((T, Hq), **f32)
        self.o = torch.empty((T, Hq, D), **f32)
        self.delta = torch.empty((T, d), **f32)
        n = Z.zmoe_paged_attention_workspace_size(T, Hq, Hkv, D)
        self.workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)

    def run(self, h: torch.Tensor, W: AttentionWeights, cache: PagedCache, layer: int, eps: float = 1e-6,
            gamma_next: Optional[torch.Tensor] = None, x_next: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """h <- h + the block's output for the token at cache.pos of each sequence, in place; h f32 [T, d].  An idle
        sequence has no cached tokens, so its row of h stays.

        With ``gamma_next``, x_next [T, d] receives RMSNorm(h) * gamma_next of the new h (the next block's input)."""
        c = cache.layer(layer)
        Z.zmoe_add_rmsnorm(h, W.gamma, eps=eps, outs=dict(x=self.x), stream=stream)
        Z.zmoe_speaker_prefix(self.x, W.w_qkv, out=self.qkv, stream=stream)
        if W.w_gate is not None:
            Z.zmoe_speaker_prefix(self.x, W.w_gate, out=self.gate, stream=stream)
        Z.zmoe_kv_append(self.k_in, self.v_in, cache.pos, q=self.q_in, seq=cache.seq, inv_freq=self.inv_freq,
                         interleaved=self.interleaved, q_gamma=W.q_gamma, k_gamma=W.k_gamma, eps=eps, q_out=self.q,
                         stream=stream, **c)
        Z.zmoe_paged_attention(self.q, lens=cache.lens, gate=self.gate if W.w_gate is not None else None, out=self.o,
                               workspace=self.workspace, stream=stream, **c)
        Z.zmoe_speaker_prefix(self.o.flatten(1), W.w_o, out=self.delta, stream=stream)
        outs = dict(h=h)
        if gamma_next is not None:
            outs["x"] = x_next
        Z.zmoe_add_rmsnorm(h, W.gamma if gamma_next is None else gamma_next, self.delta, eps=eps, outs=outs, stream=stream)
        return h


class LogitRules:
    """What zmoe_adjust_logits does to the heads' logits: penalties by the last ``window`` frames of each of T streams,
    bias f32 [N, V], mask int32 [T, N, ceil(V / 32)] of allowed ids (bits).  repetition, presence, frequency: f32 [T]."""

    def __init__(self, T: int, N: int, window: int, repetition: Optional[torch.Tensor] = None,
                 presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None, device="cuda"):
        if not 1 <= window <= 65535:
            raise ValueError("window must be at least 1 and at most 65535")
        self.repetition, self.presence, self.frequency, self.bias, self.mask = repetition, presence, frequency, bias, mask
        self.history = torch.full((T, window, N), -1, dtype=torch.int32, device=device)
        self.hist_lens = torch.zeros(T, dtype=torch.int32, device=device)
        self.frame = torch.empty((T, N), dtype=torch.int32, device=device)
        # where the next frame of every stream goes: the order is free, and -1 is no id
        self.slot = torch.zeros(1, dtype=torch.int64, device=device)

    def choose(self, logits: torch.Tensor, ids: torch.Tensor, stream=None) -> None:
        """Adjusts logits [T, N, V] in place and writes the greedy frame to ids int32 [T, N]."""
        Z.zmoe_adjust_logits(logits, self.history, self.hist_lens, self.repetition, self.presence, self.frequency,
                             self.bias, self.mask, out=logits, ids=ids, stream=stream)

    def release(self, t: int, stream=None) -> None:
        """Forgets the frames of stream ``t`` of the T, for the next request in its place."""
        with torch.cuda.stream(stream):
            self.history[t].fill_(-1)

    def remember(self, ids: torch.Tensor, stream=None, idle: Optional[torch.Tensor] = None) -> None:
        """Adds the frame ids [T, N] to the history, in place of the oldest when the window is full.  Of streams whose
        entry in idle int32 [T] is -1 (of the others it is 0) nothing is added."""
        window = self.history.shape[1]
        with torch.cuda.stream(stream):
            frame = ids if idle is None else torch.bitwise_or(ids, idle.unsqueeze(1), out=self.frame)   # -1 where idle
            self.history.index_copy_(1, self.slot, frame.unsqueeze(1))
            self.slot.add_(1).remainder_(window)
            self.hist_lens.add_(1).clamp_(max=window)
