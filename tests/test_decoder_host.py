"""The decoder's host side on the CPU: pages given out and taken back, positions, and the window of frames."""
import pytest
import torch

from sparse_moe_decoder_b200 import LogitRules, PagedCache


def test_pages_are_given_out_once_and_taken_back():
    c = PagedCache(2, 3, 50, 1, 64, 16, n_pages=7, device="cpu")
    assert c.table.shape == (3, 4) and bool((c.table == -1).all())
    c.reserve(17)
    c.reserve(16, seq=0)                       # no more than it has
    assert [len(p) for p in c.pages] == [2, 2, 2]
    used = c.table[c.table >= 0].tolist()
    assert len(used) == len(set(used)) == 6 and all(0 <= x < 7 for x in used)
    c.reserve(33, seq=1)
    assert c.free == [] and c.table[1, :3].tolist() == c.pages[1]
    with pytest.raises(RuntimeError, match="out of pages"):
        c.reserve(33, seq=2)
    assert [len(p) for p in c.pages] == [2, 3, 2]      # the refused call took nothing
    c.advance()
    c.advance()
    assert c.lens.tolist() == [2, 2, 2] and c.pos.tolist() == [1, 1, 1]
    mine = c.pages[1]
    c.release(1)
    assert sorted(c.free) == sorted(mine) and bool((c.table[1] == -1).all()) and c.lens.tolist() == [2, 0, 2]
    c.reserve(40, seq=2)
    assert c.table[2, 2].item() in mine


def test_a_layer_is_a_view_of_the_cache():
    s = torch.ones(2, 1)
    c = PagedCache(2, 1, 16, 1, 64, 16, dtype=torch.uint8, k_scale=s, v_scale=2 * s, device="cpu")
    a = c.layer(1)
    assert a["k_cache"].data_ptr() == c.k[1].data_ptr() and a["v_scale"].tolist() == [2.0] and a["page_table"] is c.table


def test_cache_refusals():
    for kw in (dict(page_size=8), dict(page_size=24), dict(dtype=torch.uint8), dict(k_scale=torch.ones(1, 1)),
               dict(dtype=torch.uint8, k_scale=torch.ones(1, 1))):
        with pytest.raises(ValueError):
            PagedCache(1, 1, 16, 1, 64, device="cpu", **kw)
    with pytest.raises(ValueError):
        PagedCache(1, 1, 16, 1, 64, device="cpu").reserve(17)


def test_the_window_keeps_the_last_frames():
    r = LogitRules(2, 3, 4, device="cpu")
    for i in range(6):
        r.remember(torch.full((2, 3), i, dtype=torch.int32))
        assert r.hist_lens.tolist() == [min(i + 1, 4)] * 2
    assert sorted(r.history[1, :, 2].tolist()) == [2, 3, 4, 5]
    with pytest.raises(ValueError):
        LogitRules(1, 1, 0, device="cpu")


def test_a_released_sequence_starts_again_though_others_went_on():
    c = PagedCache(1, 2, 32, 1, 64, 16, device="cpu")
    c.reserve(16)
    for _ in range(5):
        c.advance()
    c.release(0)
    for _ in range(5):
        c.advance()
    assert c.lens.tolist() == [0, 10] and c.pos.tolist() == [0, 9]
    c.reserve(16, 0)
    c.advance()
    assert c.pos.tolist() == [0, 10] and c.lens.tolist() == [1, 11]


def test_the_length_counts_no_token_without_a_page():
    c = PagedCache(1, 2, 64, 1, 64, 16, device="cpu")
    c.reserve(3, 0)                            # one page; sequence 1 has none
    for _ in range(20):
        c.advance()
    assert c.lens.tolist() == [16, 0] and c.pos.tolist() == [16, 0]
    c.reserve(17)
    c.advance()
    assert c.pos.tolist() == [16, 0] and c.lens.tolist() == [17, 1]


def test_a_released_sequence_is_padding_until_it_has_pages():
    c = PagedCache(1, 3, 32, 1, 64, 16, device="cpu")
    assert c.seq.tolist() == [0, 1, 2]         # without a page, but not released: its tokens count errors
    c.reserve(1, 0)
    c.release(1)
    c.release(0)
    assert c.seq.tolist() == [-1, -1, 2]
    c.reserve(0, 1)                            # no pages, so idle as before
    c.reserve(17, 0)
    assert c.seq.tolist() == [0, -1, 2] and c.room.tolist() == [32, 0, 0]


def test_a_released_stream_forgets_its_frames():
    c, r = PagedCache(1, 2, 64, 1, 64, 16, device="cpu"), LogitRules(2, 2, 8, device="cpu")
    c.rules.append(r)
    c.reserve(64)
    for i in range(5):
        c.advance()
        r.remember(torch.full((2, 2), i, dtype=torch.int32), idle=c.idle)
    c.release(0)
    kept = lambda t: sorted(x for x in r.history[t, :r.hist_lens[t], 0].tolist() if x >= 0)  # noqa: E731
    assert kept(0) == [] and kept(1) == [0, 1, 2, 3, 4]
    for i in range(5, 7):                      # nothing is added while it is idle
        c.advance()
        r.remember(torch.full((2, 2), i, dtype=torch.int32), idle=c.idle)
    c.reserve(16, 0)
    assert kept(0) == [] and kept(1) == [0, 1, 2, 3, 4, 5, 6]
    for i in range(7, 19):                     # from here on the window of the one before it
        c.advance()
        r.remember(torch.full((2, 2), i, dtype=torch.int32), idle=c.idle)
        assert kept(0) == list(range(max(7, i - 7), i + 1)) and kept(1) == list(range(max(0, i - 7), i + 1))


def test_attention_runner_refuses_sizes_that_no_step_can_have():
    from sparse_moe_decoder_b200 import AttentionRunner
    AttentionRunner(2, 6400, 50, 2, 128, device="cpu")
    for d, Hq, Hkv, D in ((6408, 16, 4, 128), (2048, 52, 4, 128), (2044, 16, 4, 128), (2048, 16, 4, 96), (0, 16, 4, 128)):
        with pytest.raises(ValueError, match="6400"):
            AttentionRunner(2, d, Hq, Hkv, D, device="cpu")


def test_a_window_has_no_more_frames_than_are_counted():
    assert LogitRules(1, 1, 65535, device="cpu").history.shape == (1, 65535, 1)
    with pytest.raises(ValueError, match="65535"):
        LogitRules(1, 1, 65536, device="cpu")
