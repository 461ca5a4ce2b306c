"""Pages and slots: lfm3_copy_pages, lfm3_reorder and the host-side pool (Lfm3Pages).

The data movement is compared byte for byte with indexing in torch on a copy of the state (pools, rings, conv columns, tails,
table, lengths); the pool's bookkeeping with a count of every page's holders; and a forked, reordered and compacted
state goes on decoding exactly as an unshared copy of it does.
"""
import numpy as np
import pytest
import torch

from lfm3_inputs import lfm3_1p7b, make_tokens, make_weights

pytestmark = pytest.mark.gpu
NAMES = ("conv", "ring_k", "ring_v", "kv_k", "kv_v", "kv_k_scale", "kv_v_scale", "tail_k", "tail_v", "page_table", "seq_len")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_decoder_b200 import build
    build.build(verbose=False)
    from attention_decoder_b200.model import Lfm3Model
    return Lfm3Model


@pytest.fixture(scope="module")
def weights():
    return make_weights(lfm3_1p7b(layer_types=(0, 2, 1, 1)), 0)


def random_state(m, lens, seed, pages=None):
    """A state of random bytes whose slots hold shuffled pages of their own."""
    st = m.new_state()
    g = torch.Generator(device="cuda").manual_seed(seed)
    for n in NAMES[:-2]:
        t = getattr(st, n)
        if t is not None:
            t.copy_(torch.randint(-127, 128, t.shape, generator=g, device="cuda"))
    S, mpp = m.cfg.max_streams, m.cfg.max_pages_per_stream
    st.h_page_table[:] = np.random.default_rng(seed).permutation(m.cfg.n_pages)[: S * mpp].reshape(S, mpp)
    st.page_table.copy_(torch.from_numpy(st.h_page_table))
    st.h_seq_len[:] = lens
    st.seq_len.copy_(torch.from_numpy(st.h_seq_len))
    return st


def snapshot(st):
    return {n: None if getattr(st, n) is None else getattr(st, n).clone() for n in NAMES}


def same(st, want):
    torch.cuda.synchronize()
    for n in NAMES:
        if want[n] is not None:
            assert torch.equal(getattr(st, n), want[n]), n
    assert np.array_equal(st.h_page_table, want["page_table"].cpu().numpy())
    assert np.array_equal(st.h_seq_len, want["seq_len"].cpu().numpy())


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 3, 16, 17, 45])
def test_copy_pages(lib, weights, fmt, n):
    m = lib(weights, max_streams=2, max_pages_per_stream=50, max_chunk=64, kv_format=fmt)
    st = random_state(m, [5, 70], 1)
    perm = np.random.default_rng(n).permutation(100)
    src, dst = perm[:n], perm[50:50 + n]
    src[n // 2:] = src[0]  # one source for many
    want = snapshot(st)
    for name in NAMES[3:7]:
        if want[name] is not None:
            want[name][:, dst] = want[name][:, src]
    m.copy_pages(st, src, dst)
    same(st, want)


def test_copy_more_pages_than_one_launch_takes(lib, weights):
    m = lib(weights, max_streams=1, max_pages_per_stream=64, n_pages=4101, max_chunk=64, kv_format="int8")
    st = m.new_state()
    st.kv_k.copy_(torch.randint(-127, 128, st.kv_k.shape, device="cuda"))
    want = st.kv_k.clone()
    want[:, :2050] = want[:, 2051:]
    m.copy_pages(st, np.arange(2051, 4101), np.arange(2050))
    torch.cuda.synchronize()
    assert torch.equal(st.kv_k, want) and m.last_launch_count() == 2


def reordered(st, slots, parents, pages, int8):
    """The state after the reorder, by indexing."""
    want, old = snapshot(st), snapshot(st)
    for i, (s, p) in enumerate(zip(slots, parents)):
        if i == p:
            continue
        src = slots[p]
        n = int(old["seq_len"][src])
        for name in ("conv", "ring_k", "ring_v", "tail_k", "tail_v"):
            if old[name] is not None:
                want[name][:, s] = old[name][:, src]
        want["seq_len"][s] = n
        want["page_table"][s] = -1
        want["page_table"][s, : n // 64] = old["page_table"][src, : n // 64]
        if n // 64 < old["page_table"].shape[1]:
            want["page_table"][s, n // 64] = max(-1, pages[i])
        if n % 64:
            a, rows = int(old["page_table"][src, n // 64]), n % 64
            if int8:
                for name in ("kv_k_scale", "kv_v_scale"):
                    want[name][:, pages[i], :, : rows // 16] = old[name][:, a, :, : rows // 16]
                rows = rows // 16 * 16
            for name in ("kv_k", "kv_v"):
                want[name][:, pages[i], :, :rows] = old[name][:, a, :, :rows]
    return want


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("parents", [
    [0, 0],                              # a fork
    [1, 0],                              # a swap
    [1, 2, 0],                           # a cycle
    [1, 2, 3, 3],                        # a chain
    [0, 1, 2],                           # nothing moves
    list(np.random.default_rng(3).integers(0, 9, 9)),
    list(np.random.default_rng(4).permutation(33)),
    list(np.random.default_rng(5).integers(0, 64, 64)),
])
def test_reorder(lib, weights, fmt, parents):
    n, S, mpp = len(parents), 66, 4
    m = lib(weights, max_streams=S, max_pages_per_stream=mpp, n_pages=S * mpp + n, max_chunk=64, max_batch=1, kv_format=fmt)
    rng = np.random.default_rng(n)
    lens = rng.choice([0, 1, 15, 16, 63, 64, 65, 100, 128, 191, 255, 256], S)
    st = random_state(m, lens, 7)
    free = sorted(set(range(m.cfg.n_pages)) - set(st.h_page_table.reshape(-1).tolist()))
    slots = rng.permutation(S)[:n]
    want = reordered(st, slots, parents, free, fmt == "int8")
    m.reorder(st, slots, parents, free[:n])
    same(st, want)


def test_a_child_may_take_over_the_page_its_parent_gives_up(lib, weights):
    m = lib(weights, max_streams=3, max_pages_per_stream=2, max_chunk=64)
    st = random_state(m, [70, 100, 80], 3)
    a, b, c = (int(st.h_page_table[s, 1]) for s in range(3))
    want = reordered(st, [0, 1, 2], [1, 0, 2], [b, a, -1], False)
    m.reorder(st, [0, 1, 2], [1, 0, 2], [b, a, -1])
    same(st, want)


def test_refusals_change_nothing(lib, weights):
    from attention_decoder_b200 import Lfm3Error
    m = lib(weights, max_streams=4, max_pages_per_stream=3, n_pages=14, max_chunk=64)
    st = random_state(m, [70, 100, 0, 128], 5)
    free = sorted(set(range(14)) - set(st.h_page_table.reshape(-1).tolist()))
    t = st.h_page_table
    want = snapshot(st)
    bad = [
        (-1, lambda: m.copy_pages(st, [0], [14])), (-1, lambda: m.copy_pages(st, [-1], [0])), (-1, lambda: m.copy_pages(st, [], [])),
        (-1, lambda: m.copy_pages(st, [0, 1], [2, 2])), (-1, lambda: m.copy_pages(st, [0, 1], [1, 2])),
        (-1, lambda: m.reorder(st, [0, 4], [0, 0], [-1, free[0]])),           # a slot outside
        (-1, lambda: m.reorder(st, [0, 0], [0, 0], [-1, free[0]])),           # listed twice
        (-1, lambda: m.reorder(st, [0, 1], [0, 2], [-1, free[0]])),           # a parent outside
        (-1, lambda: m.reorder(st, [0, 1], [0, 0], [-1, -1])),                # no page for the partly filled one
        (-1, lambda: m.reorder(st, [0, 1], [0, 0], [-1, 14])),                # a page outside
        (-1, lambda: m.reorder(st, [0, 1, 2], [0, 0, 0], [-1, free[0], free[0]])),
        (-1, lambda: m.reorder(st, [0, 1], [0, 0], [-1, int(t[0, 1])])),      # the parent keeps that page
        (-1, lambda: m.reorder(st, [0, 1], [0, 0], [-1, int(t[3, 0])])),      # held by a slot that is not listed
        (-1, lambda: m.reorder(st, [0, 1, 2], [1, 0, 1], [int(t[0, 1]), free[0], free[1]])),  # also copied from
        (-1, lambda: m.reorder(st, [0, 1], [0, 0], None)),
    ]
    for status, call in bad:
        with pytest.raises(Lfm3Error) as e:
            call()
        assert e.value.status == status
    st.h_page_table[0, 0] = -1
    with pytest.raises(Lfm3Error) as e:
        m.reorder(st, [0, 1], [0, 0], [-1, free[0]])
    assert e.value.status == -3
    st.h_page_table[0, 0] = int(want["page_table"][0, 0])
    same(st, want)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_other_streams_and_captured_calls(lib, weights, fmt):
    m = lib(weights, max_streams=3, max_pages_per_stream=2, n_pages=10, max_chunk=64, kv_format=fmt)
    st = random_state(m, [70, 100, 20], 7)
    free = sorted(set(range(10)) - set(st.h_page_table.reshape(-1).tolist()))
    side = torch.cuda.Stream()
    before = {n: t if t is None else t.clone() for n, t in snapshot(st).items()}
    want = reordered(st, [0, 1, 2], [0, 0, 1], [-1, free[0], free[1]], fmt == "int8")
    side.wait_stream(torch.cuda.current_stream())
    m.reorder(st, [0, 1, 2], [0, 0, 1], [-1, free[0], free[1]], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same(st, want)
    src, dst = [int(st.h_page_table[0, 0])], [free[2]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.copy_pages(st, src, dst)
    for n in ("kv_k", "kv_v"):
        getattr(st, n).copy_(before[n].flip(1))               # the pages' bytes at the time of the replay
    graph.replay()
    torch.cuda.synchronize()
    for n in ("kv_k", "kv_v"):
        ref = before[n].flip(1)
        ref[:, dst] = ref[:, src]
        assert torch.equal(getattr(st, n).view(torch.uint8), ref.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_a_captured_reorder_moves_when_it_is_replayed(lib, weights, fmt):
    m = lib(weights, max_streams=3, max_pages_per_stream=2, n_pages=10, max_chunk=64, kv_format=fmt)
    st = random_state(m, [70, 100, 20], 8)
    free = sorted(set(range(10)) - set(st.h_page_table.reshape(-1).tolist()))
    before = snapshot(st)
    want = reordered(st, [0, 1, 2], [1, 0, 1], free, fmt == "int8")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.reorder(st, [0, 1, 2], [1, 0, 1], free[:3])
    torch.cuda.synchronize()
    for n in NAMES:
        assert before[n] is None or torch.equal(getattr(st, n), before[n]), n
    graph.replay()
    same(st, want)


def test_arrays_that_are_not_aligned_are_refused(lib, weights):
    from attention_decoder_b200 import Lfm3Error
    m = lib(weights, max_streams=2, max_pages_per_stream=1, max_chunk=64)
    st = random_state(m, [10, 10], 6)
    want = snapshot(st)
    for name, calls in (("kv_v", "cr"), ("conv_state", "r"), ("ring_k", "r")):
        at = getattr(st.struct, name)
        setattr(st.struct, name, at + 8)
        for call in calls:
            with pytest.raises(Lfm3Error) as e:
                m.copy_pages(st, [0], [1]) if call == "c" else m.reorder(st, [0, 1], [1, 1], [int(st.h_page_table[0, 0]), -1])
            assert e.value.status == -1 and "aligned" in str(e.value)
        setattr(st.struct, name, at)
    same(st, want)


def holders(pages):
    n = np.zeros_like(pages.refs)
    for v in pages.h.reshape(-1):
        if v >= 0:
            n[v] += 1
    assert np.array_equal(n, pages.refs)
    assert torch.equal(pages.state.page_table.cpu(), torch.from_numpy(pages.h))


def test_pool_bookkeeping(lib, weights):
    from attention_decoder_b200 import Lfm3Error, Lfm3Pages
    m = lib(weights, max_streams=6, max_pages_per_stream=4, n_pages=13, max_chunk=64)
    st = m.new_state()
    pool = Lfm3Pages(st)
    assert pool.free_pages == 13
    rng = np.random.default_rng(2)
    pool.lease(0, 130)
    st.h_seq_len[0] = 130
    st.seq_len[0] = 130
    pool.fork(0, [1, 2, 3])
    holders(pool)
    assert pool.free_pages == 13 - 2 - 4 and st.h_seq_len[:4].tolist() == [130] * 4
    for _ in range(20):
        pool.reorder(range(4), rng.integers(0, 4, 4))
        holders(pool)
        assert len({int(pool.h[s, 2]) for s in range(4)}) == 4      # partly filled pages are private
    pool.release(0)
    pool.release(2)
    holders(pool)
    assert pool.compact() > 0
    holders(pool)
    assert (pool.refs[: 13 - pool.free_pages] > 0).all() and pool.compact() == 0
    with pytest.raises(Lfm3Error) as e:
        pool.lease(4, 4 * 64 + 1)
    assert e.value.status == -3
    before = pool.h.copy()
    pool.lease(4, 256)
    pool.lease(5, 256)
    with pytest.raises(Lfm3Error) as e:
        pool.lease(0, 256)
    assert e.value.status == -3 and (pool.h[0] == -1).all() and np.array_equal(before[1], pool.h[1])
    holders(pool)


def test_forked_reordered_and_compacted_slots_decode_like_unshared_ones(lib):
    """Four beams forked from one prompt, reordered twice with steps between, compacted: every step's logits equal those
    of slots that were prefilled and decoded on their own."""
    from attention_decoder_b200 import Lfm3Pages
    g = lfm3_1p7b(layer_types=(0, 2, 1, 0))
    m = lib(make_weights(g, 0), max_streams=4, max_pages_per_stream=6, n_pages=40, max_batch=4)
    prompt = torch.from_numpy(make_tokens(1, "fork", 121, g.vocab)).cuda()
    tok = make_tokens(2, "fork.steps", 4 * 12, g.vocab).reshape(12, 4)
    st = m.new_state(poison=True)
    pool = Lfm3Pages(st)
    pool.lease(3, 121)
    m.prefill(st, 3, tokens=prompt)
    pool.fork(3, [0, 1, 2])
    history = [[] for _ in range(4)]
    maps = {4: [2, 0, 1, 1], 8: [0, 3, 3, 3], 10: [1, 0, 3, 2]}
    for i in range(12):
        if i in maps:
            pool.reorder(range(4), maps[i])
            history = [list(history[p]) for p in maps[i]]
        if i == 9:
            pool.compact()
        for s in range(4):
            pool.lease(s, int(st.h_seq_len[s]) + 1)
            history[s].append(int(tok[i, s]))
        out = m.decode(st, range(4), tokens=torch.from_numpy(tok[i]).cuda())
        holders(pool)
    plain = m.new_state(page_table=np.arange(24).reshape(4, 6))
    for s in range(4):
        m.prefill(plain, s, tokens=prompt)
    for i in range(12):
        ref = m.decode(plain, range(4), tokens=torch.tensor([h[i] for h in history], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out["logits"], ref["logits"])
    m.check_device_errors()


def test_forked_reordered_and_compacted_slots_with_an_8_bit_pool(lib):
    """The same over 8-bit codes: states of the same lengths split their keys alike, so the bits are the same too."""
    from attention_decoder_b200 import Lfm3Pages
    g = lfm3_1p7b(layer_types=(0, 2, 1, 1))
    m = lib(make_weights(g, 0), max_streams=4, max_pages_per_stream=6, n_pages=40, max_batch=4, kv_format="int8")
    prompt = torch.from_numpy(make_tokens(1, "fork8", 117, g.vocab)).cuda()
    tok = make_tokens(2, "fork8.steps", 4 * 30, g.vocab).reshape(30, 4)
    st = m.new_state(poison=True)
    pool = Lfm3Pages(st)
    pool.lease(1, 117)
    m.prefill(st, 1, tokens=prompt)
    pool.fork(1, [0, 2, 3])
    history = [[] for _ in range(4)]
    maps = {3: [2, 0, 1, 1], 11: [1, 2, 3, 0], 12: [0, 3, 3, 3], 20: [3, 3, 0, 2]}  # at 120, 128 (a block and a page full), 129, 137
    for i in range(30):
        if i in maps:
            pool.reorder(range(4), maps[i])
            history = [list(history[p]) for p in maps[i]]
        if i in (9, 21):
            pool.compact()
        for s in range(4):
            pool.lease(s, int(st.h_seq_len[s]) + 1)
            history[s].append(int(tok[i, s]))
        out = m.decode(st, range(4), tokens=torch.from_numpy(tok[i]).cuda())
        holders(pool)
    plain = m.new_state(page_table=np.arange(24).reshape(4, 6))
    for s in range(4):
        m.prefill(plain, s, tokens=prompt)
    for i in range(30):
        ref = m.decode(plain, range(4), tokens=torch.tensor([h[i] for h in history], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out["logits"], ref["logits"])
    m.check_device_errors()
