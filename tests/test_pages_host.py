"""Lfm3Pages' own refusals, on a state of CPU tensors (no kernel is called)."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch


def fake_state(slots, width, pages):
    return SimpleNamespace(model=SimpleNamespace(cfg=SimpleNamespace(n_pages=pages)), h_page_table=np.zeros((slots, width), np.int32),
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
