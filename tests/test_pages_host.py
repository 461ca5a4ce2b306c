"""Refusals of Lfm3Pages and beam_search, on a state of CPU tensors (no kernel is called)."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch


def fake_state(slots, width, pages):
    return SimpleNamespace(model=SimpleNamespace(cfg=SimpleNamespace(n_pages=pages, max_streams=slots, max_batch=2), device="cpu"), h_page_table=np.zeros((slots, width), np.int32),
                           page_table=torch.zeros(slots, width, dtype=torch.int32), h_seq_len=np.zeros(slots, np.int32),
                           seq_len=torch.zeros(slots, dtype=torch.int32), conv=torch.zeros(1, slots, 6, 8))


def test_slots_and_lengths_outside_are_refused():
    from attention_decoder_b200 import Lfm3Error, Lfm3Pages
    st = fake_state(3, 4, 9)
    pool = Lfm3Pages(st)
    pool.lease(2, 130)
    st.h_seq_len[2] = 130
    before = pool.h.copy(), pool.refs.copy()
    for call in (lambda: pool.lease(-1, 200), lambda: pool.lease(3, 1), lambda: pool.release(-1), lambda: pool.release(3),
                 lambda: pool.lease(0, -100)):
        with pytest.raises(Lfm3Error) as e:
            call()
        assert e.value.status == -1
        assert np.array_equal(pool.h, before[0]) and np.array_equal(pool.refs, before[1]) and st.h_seq_len.tolist() == [0, 0, 130]
    pool.release(2)
    assert pool.free_pages == 9 and torch.equal(st.page_table, torch.full((3, 4), -1, dtype=torch.int32))


def test_beam_search_refuses_before_it_releases_a_slot():
    from attention_decoder_b200 import Lfm3Pages, beam_search
    st = fake_state(80, 4, 320)
    pool = Lfm3Pages(st)
    for s in range(80):
        pool.lease(s, 70)
    st.h_seq_len[:] = 70
    ids = torch.arange(9, dtype=torch.int32)
    for word, call in (("slots", lambda: beam_search(pool, ids, 2, 4, slots=[1, 1])), ("slots", lambda: beam_search(pool, ids, 2, 4, slots=[0, 80])),
                       ("slots", lambda: beam_search(pool, ids, 2, 4, slots=[0, -1])), ("max_batch", lambda: beam_search(pool, ids, 3, 4)),
                       ("64", lambda: beam_search(pool, ids, 65, 1)), ("prompt", lambda: beam_search(pool, ids.long(), 2, 4)),
                       ("prompt", lambda: beam_search(pool, ids[:0], 2, 4)), ("prompt", lambda: beam_search(pool, ids[::2], 2, 4)),
                       ("prompt", lambda: beam_search(pool, ids.view(3, 3), 2, 4)), ("prompt", lambda: beam_search(pool, ids.to("meta"), 2, 4))):
        with pytest.raises(ValueError, match=word):
            call()
        assert (pool.refs[:160] == 1).all() and (st.h_seq_len == 70).all()
