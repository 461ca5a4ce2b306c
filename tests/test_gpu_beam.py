"""Beam selection (lfm3_beam_select) and the beam search built on it.

The selection is compared with the definition in float64. Scores: the kernel's log-sum-exp sums 2^-22-accurate exponentials
in fp32 over at most 4096 / 256 = 16 terms a thread and 256 threads (relative error of a sum below 2^-22 + 13 * 2^-24 < 2^-20),
so a score is off by less than 2^-20 before its one rounding to fp32: |score| * 2^-24 + 2^-20.
"""
import numpy as np
import pytest
import torch

from lfm3_inputs import lfm3_1p7b, make_tokens, make_weights

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def select():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_decoder_b200 import beam_select, build
    build.build(verbose=False)
    return beam_select


def reference(x, s, n_out, done=None, end=0):
    """The definition, in float64 on the CPU; x [G, B, V]."""
    G, B, V = x.shape
    x, s = x.double().cpu().numpy(), s.double().cpu().numpy()
    score, parent, token = np.full((G, n_out), -np.inf), np.full((G, n_out), -1), np.full((G, n_out), -1)
    for g in range(G):
        c = np.full((B, V), -np.inf)
        for b in range(B):
            if not s[g, b] > -np.inf:
                continue
            if done is not None and done[g, b]:
                c[b, end] = s[g, b]
            elif not np.isnan(x[g, b]).any() and x[g, b].max() < np.inf and x[g, b].max() > -np.inf:
                m = x[g, b].max()
                c[b] = s[g, b] + (x[g, b] - m - np.log(np.exp(x[g, b] - m).sum()))  # m first: it may dwarf the log
        order = np.argsort(-c.reshape(-1), kind="stable")[:n_out]
        order = order[c.reshape(-1)[order] > -np.inf]
        score[g, : len(order)] = c.reshape(-1)[order]
        parent[g, : len(order)], token[g, : len(order)] = order // V, order % V
    return score, parent, token


def check(select, x, s, n_out, done=None, end=0, ties=False):
    out = select(x, s, n_out, done=done, end_token=end)
    torch.cuda.synchronize()
    score, parent, token = reference(x, s, n_out, None if done is None else done.cpu().numpy(), end)
    got = out["score"].double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), np.isfinite(score))
    f = np.isfinite(score)
    assert (np.abs(got[f] - score[f]) <= np.abs(score[f]) * 2.0**-24 + 2.0**-20).all()
    assert np.array_equal(out["parent"].cpu().numpy(), parent)
    assert np.array_equal(out["token"].cpu().numpy(), token)


def draw(G, B, V, seed, pitch=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(G * B * (V + pitch) + offset, generator=g, device="cuda") * 2.5
    x = buf[offset:].view(G, B, V + pitch)[:, :, :V]
    return x, -10 * torch.rand(G, B, generator=g, device="cuda")


@gpu
@pytest.mark.parametrize("G,B,V,n_out", [
    (1, 1, 1, 1), (1, 1, 7, 3), (1, 4, 128000, 8), (3, 5, 50001, 10), (2, 2, 1023, 64), (1, 64, 4099, 64), (7, 3, 33, 6),
    (1, 1, 1 << 20, 64), (64, 1, 1000, 1), (5, 8, 4096, 16), (1, 2, 2, 5),
])
def test_matches_the_definition(select, G, B, V, n_out):
    for offset, pitch in ((0, 0), (1, 0), (0, 1), (3, 5), (2, 64)):
        check(select, *draw(G, B, V, V + offset, pitch, offset), n_out)


@gpu
@pytest.mark.parametrize("V", [100, 5000])
def test_ties_go_to_the_lowest_beam_and_token(select, V):
    x = torch.zeros(2, 3, V, device="cuda")                     # all equal: 5000 candidates of one part above the threshold
    check(select, x, torch.zeros(2, 3, device="cuda"), 20)
    x[:, :, V // 2:] = 1.0
    check(select, x, torch.zeros(2, 3, device="cuda"), 64)
    x = torch.randint(-3, 4, (4, 2, V), device="cuda").float()
    x[:, 1] = x[:, 0]                                           # two beams with the same row: the first one's tokens first
    check(select, x, torch.full((4, 2), -1.5, device="cuda"), 24)


@gpu
def test_beams_far_apart(select):
    """Three poor beams hold all of one warp's lists, so that its bound lets 45 x 64 candidates through."""
    x, s = draw(1, 48, 700, 10)
    check(select, x, s, 64)
    s[0, ::16] -= 1000
    check(select, x, s, 64)
    check(select, x, s - 40.0 * torch.arange(48, device="cuda").view(1, 48), 64)


@gpu
def test_the_largest_group(select):
    x, s = draw(1, 64, 1 << 20, 11)
    out = select(x, s, 64)
    c = (s.double()[0, :, None] + (x[0].double() - torch.logsumexp(x[0].double(), 1, keepdim=True))).view(-1)
    top = torch.topk(c, 64).values
    at = out["parent"][0].long() * (1 << 20) + out["token"][0].long()
    assert len(set(at.tolist())) == 64 and ((c[at] - top).abs() <= 1e-9).all()
    assert ((out["score"][0].double() - top).abs() <= top.abs() * 2.0**-24 + 2.0**-20).all()


@gpu
def test_sorted_rows(select):
    x = torch.linspace(-8, 8, 20000, device="cuda").view(1, 1, -1)
    for row in (x, x.flip(2)):
        check(select, row.contiguous(), torch.zeros(1, 1, device="cuda"), 64)


@gpu
def test_banned_tokens_masked_rows_and_missing_candidates(select):
    x, s = draw(3, 4, 9001, 5)
    x[:, :, 100:] = float("-inf")
    check(select, x, s, 16)
    x[0] = float("-inf")                                        # a group without candidates
    x[1, :, 3:] = float("-inf")                                 # 12 candidates for 16 places
    x[2, 1] = torch.finfo(torch.float32).min                    # the lowest finite value is a logit like others
    check(select, x, s, 16)


@gpu
def test_rows_and_scores_that_are_not_finite(select):
    x, s = draw(2, 5, 3001, 6)
    x[0, 1, 77], x[0, 2, 2999], x[1, 0, 0] = float("nan"), float("inf"), float("nan")
    s[0, 3], s[1, 1] = float("-inf"), float("nan")
    check(select, x, s, 10)
    x[0] = float("nan")
    check(select, x, s, 10)


@gpu
def test_finished_beams_offer_one_token(select):
    x, s = draw(4, 6, 12345, 7)
    done = (torch.arange(24, device="cuda") % 3 == 0).to(torch.int32).view(4, 6)
    done[3] = 1                                                 # all finished: 6 candidates for 12 places
    x[0, 0] = float("nan")                                      # the logits of a finished beam do not count
    check(select, x, s, 12, done=done, end=2)
    check(select, x, s, 12, done=done, end=12344)


@gpu
def test_a_nan_among_masked_tokens_counts(select):
    """A NaN with nothing but -inf around it, one after the last whole part of a row, and a stretch of nothing else."""
    x, s = draw(3, 4, 5001, 21)
    x[0, 1, 100:] = float("-inf")
    x[0, 1, 3333] = float("nan")
    x[1, 2, 900:5000] = float("nan")
    x[2, :, 2000:] = float("-inf")
    x[2, 3, 5000] = float("nan")
    s[0, 1] = s[1, 2] = s[2, 3] = 0.0                           # (they would come first)
    check(select, x, s, 10)
    for offset in range(4):
        x, s = draw(1, 3, 1025 + offset, 22, 0, offset)
        x[0, 1, -1], s[0, 1] = float("nan"), 0.0
        check(select, x, s, 10)


@gpu
def test_zeros_of_either_sign_tie(select):
    x = torch.tensor([[[-0.0, 0.0]]], device="cuda")
    check(select, x, torch.zeros(1, 1, device="cuda"), 1)
    x, s = draw(2, 2, 700, 23)
    x = -x.abs() - 1
    x[:, :, 100:400] = 0.0
    x[:, :, 100:400:2] = -0.0                                   # 300 ties in a part: more than are ranked directly
    check(select, x, s, 24)
    x[:, :, 120:400] = -7.0
    check(select, x, s, 9)
    both = torch.ones(2, 2, dtype=torch.int32, device="cuda")
    check(select, x, torch.tensor([[-0.0, 0.0], [0.0, -0.0]], device="cuda"), 1, done=both)


@gpu
def test_outputs_on_another_stream_are_not_handed_out_early(select):
    """The memory of outputs on a side stream: what is dropped before the call has run is not another tensor's yet, and what a
    pending write on the current stream still has is not an output's."""
    x, s = draw(4, 4, 3000, 24)
    want = select(x, s, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    del_me = select(x, s, 64, stream=side)
    del del_me
    others = [torch.full((4, 64), 7, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in others)
    del others
    torch.cuda._sleep(50_000_000)
    others = [torch.full((4, 64), 7, dtype=torch.int32, device="cuda") for _ in range(2000)]  # all the free memory of that size
    del others
    got = select(x, s, 64, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)


@gpu
def test_a_workspace_that_is_not_scratch_is_refused(select):
    """(On the host: none of these reaches a kernel.)"""
    from attention_decoder_b200 import _lib as L
    x, s = draw(2, 4, 3000, 25)
    n = L.lfm3_beam_workspace(2, 4, 3000, 8)
    want = select(x, s, 8)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(n, device="cuda"), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            select(x, s, 8, workspace=ws)
    with pytest.raises(L.Lfm3Error, match="workspace") as e:
        select(x, s, 8, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -3
    got = select(x, s, 8, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(got[k], want[k]) for k in want)


@gpu
def test_two_streams_and_a_captured_graph(select):
    from attention_decoder_b200 import _lib as L
    (x1, s1), (x2, s2) = draw(4, 4, 30000, 8), draw(4, 4, 30000, 9)
    want = [select(x, s, 8) for x, s in ((x1, s1), (x2, s2))]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        got[0].append(select(x1, s1, 8, stream=a))
        got[1].append(select(x2, s2, 8, stream=b))
    torch.cuda.synchronize()
    for k in range(2):
        for o in got[k]:
            assert all(torch.equal(o[n], want[k][n]) for n in o)
    ws = torch.empty(L.lfm3_beam_workspace(4, 4, 30000, 8), dtype=torch.uint8, device="cuda")
    out = {n: torch.zeros_like(t) for n, t in want[0].items()}
    x, s = x1.clone(), s1.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        select(x, s, 8, out=out, workspace=ws)
    for k, (xs, ss) in enumerate(((x1, s1), (x2, s2), (x1, s1))):
        x.copy_(xs)
        s.copy_(ss)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[k % 2][n]) for n in out)


def test_refusals():
    from attention_decoder_b200 import build
    build.build(verbose=False)
    from attention_decoder_b200 import _lib as L
    p, odd = 0x10000, 0x10002  # never dereferenced

    def call(G=1, B=4, V=100, n=4, x=p, ld=100, s=p, done=None, end=0, o=p, par=p, t=p, ws=p, nws=1 << 20):
        return L.lfm3_beam_select(G, B, V, n, x, ld, s, done, end, o, par, t, ws, nws, None)

    for kw, word in ((dict(G=0), b"groups"), (dict(B=65), b"beams"), (dict(n=0), b"out"), (dict(n=65), b"out"), (dict(V=0), b"vocab"),
                     (dict(V=(1 << 20) + 1, ld=1 << 21), b"vocab"), (dict(G=65535, B=2), b"groups"), (dict(ld=99), b"pitch"),
                     (dict(x=None), b"NULL"), (dict(s=None), b"NULL"), (dict(ws=None), b"NULL"), (dict(t=None), b"NULL"),
                     (dict(x=odd), b"aligned"), (dict(par=odd), b"aligned"), (dict(ws=0x10008), b"aligned"),
                     (dict(done=p, end=100), b"end_token"), (dict(done=p, end=-1), b"end_token")):
        assert call(**kw) == -1, kw
        assert word in L.lfm3_last_error(None), kw
    assert call(nws=L.lfm3_beam_workspace(1, 4, 100, 4) - 1) == -3 and b"workspace" in L.lfm3_last_error(None)
    assert L.lfm3_beam_workspace(1, 65, 100, 4) == 0 and L.lfm3_beam_workspace(1, 4, 100, 4) > 0


@gpu
def test_beam_search_equals_a_search_without_shared_state(select):
    """beam_search against hypotheses that are each prefilled from scratch, selected by the definition in float64."""
    from attention_decoder_b200 import Lfm3Pages, beam_search
    from attention_decoder_b200.model import Lfm3Model
    g = lfm3_1p7b(layer_types=(0, 2, 1, 0))
    m = Lfm3Model(make_weights(g, 0), max_streams=5, max_pages_per_stream=4, n_pages=16, max_batch=5)
    st = m.new_state(poison=True)
    pool = Lfm3Pages(st)
    prompt = make_tokens(4, "beam", 60, g.vocab)
    one = m.new_state(page_table=np.arange(20).reshape(5, 4) % 16)

    def logits(ids):
        one.h_seq_len[:] = 0
        one.seq_len.zero_()
        one.conv.zero_()
        return m.prefill(one, 0, tokens=torch.from_numpy(np.array(ids, np.int32)).cuda())["logits"].clone()

    def search(B, steps, end):
        beams = [([], 0.0, False)]
        least = np.inf
        for _ in range(steps):
            cand = []
            for b, (ids, sc, fin) in enumerate(beams):
                if fin:
                    cand.append((sc, ids, True))
                    continue
                x = logits(list(prompt) + ids).double().cpu().numpy()
                lp = sc + x - (x.max() + np.log(np.exp(x - x.max()).sum()))
                cand += [(lp[v], ids + [int(v)], v == end) for v in np.argsort(-lp)[: B + 1]]
            cand.sort(key=lambda c: -c[0])
            least = min(least, min(a[0] - b[0] for a, b in zip(cand[:B], cand[1: B + 1])))
            beams = [(ids, sc, bool(fin)) for sc, ids, fin in cand[:B]]
        return beams, least

    end = None
    for B in (4, 3):
        want, margin = search(B, 8, end)
        tokens, scores = beam_search(pool, torch.from_numpy(prompt).cuda(), B, 8, end_token=end)
        # the decode and prefill paths agree to 0.1 in a logit at worst; the comparison stops at closer candidates
        np.testing.assert_allclose(scores.cpu().numpy(), [b[1] for b in want], atol=0.1)
        if margin > 1e-3:
            assert tokens == [b[0] for b in want]
        end = tokens[0][3]                                      # the second search ends beams at this token
    m.check_device_errors()


@gpu
def test_beam_search_with_fewer_candidates_than_beams(select):
    from attention_decoder_b200 import Lfm3Pages, beam_search
    from attention_decoder_b200.model import Lfm3Model
    from dataclasses import replace
    g = replace(lfm3_1p7b(layer_types=(0, 1)), vocab=16)
    w = make_weights(g, 0)
    prompt = torch.arange(9, dtype=torch.int32, device="cuda")
    m = Lfm3Model(w, max_streams=20, max_pages_per_stream=1, max_batch=20)
    tokens, scores = beam_search(Lfm3Pages(m.new_state()), prompt, 20, 1)
    assert sorted(t[0] for t in tokens[:16]) == list(range(16)) and tokens[16:] == [[]] * 4
    assert torch.isfinite(scores[:16]).all() and (scores[16:] == -float("inf")).all()
    tokens, scores = beam_search(Lfm3Pages(m.new_state()), prompt, 20, 3)    # 256 candidates from the second step on
    assert all(len(t) == 3 for t in tokens) and len({tuple(t) for t in tokens}) == 20
    assert torch.isfinite(scores).all() and (scores[:-1] >= scores[1:]).all()
    m.check_device_errors()
    state = m.new_state()
    state.kv_v.fill_(float("nan"))                                           # as a damaged cache would
    pool = Lfm3Pages(state)
    tokens, scores = beam_search(pool, prompt, 20, 2)
    assert torch.isfinite(scores).all()                                      # (rows never written are never read)
    nan = Lfm3Model({**w, "embed": np.full_like(w["embed"], 0x7fc0)}, max_streams=3, max_pages_per_stream=1, max_batch=3)
    tokens, scores = beam_search(Lfm3Pages(nan.new_state()), prompt, 3, 4)
    assert tokens == [[]] * 3 and (scores == -float("inf")).all()
