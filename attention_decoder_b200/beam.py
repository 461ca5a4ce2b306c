"""Beam search over the decoder: selection on the GPU (lfm3_beam_select), states reordered by sharing pages (lfm3_reorder)."""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L
from .model import outputs_for


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def beam_select(logits, scores, n_out, done=None, end_token=0, out=None, workspace=None, stream=None):
    """The n_out best continuations of each group of beams (see lfm3_beam_select).

    logits: fp32 [groups, beams, vocab], rows of any one pitch; scores: fp32 [groups, beams]; done: int32 [groups, beams]
    or None, all on one GPU. Returns {"score", "parent", "token"}, each [groups, n_out] (``out``: the same, to write
    into). ``workspace``: uint8 scratch of L.lfm3_beam_workspace bytes, for callers that keep one."""
    if logits.dim() != 3 or logits.dtype != torch.float32 or not logits.is_cuda:
        raise ValueError("logits must be fp32 [groups, beams, vocab] on the GPU")
    G, B, V = logits.shape
    if (V > 1 and logits.stride(2) != 1) or (G > 1 and B > 1 and logits.stride(0) != B * logits.stride(1)):
        raise ValueError("logits must have contiguous rows of one pitch")
    ld = logits.stride(1) if B > 1 else logits.stride(0) if G > 1 else V
    for t, kind in ((scores, torch.float32), (done, torch.int32)):
        if t is not None and (t.shape != (G, B) or t.dtype != kind or t.device != logits.device or not t.is_contiguous()):
            raise ValueError(f"scores and done must be contiguous [{G}, {B}], fp32 and int32, beside the logits")
    dev = logits.device
    if out is None:
        out = dict(zip(("score", "parent", "token"), outputs_for(stream, lambda: [
            torch.empty(G, n_out, dtype=kind, device=dev) for kind in (torch.float32, torch.int32, torch.int32)])))
    for n, kind in (("score", torch.float32), ("parent", torch.int32), ("token", torch.int32)):
        t = out[n]
        if t.shape != (G, n_out) or t.dtype != kind or t.device != dev or not t.is_contiguous():
            raise ValueError(f"out[{n!r}] must be contiguous [{G}, {n_out}] {kind} beside the logits")
    if workspace is None:
        (workspace,) = outputs_for(stream, lambda: (torch.empty(max(16, L.lfm3_beam_workspace(G, B, V, n_out)), dtype=torch.uint8,
                                                                device=dev),))
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8 beside the logits")
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream() if stream is None else stream
        L.check(L.lfm3_beam_select(G, B, V, n_out, _ptr(logits), ld, _ptr(scores), _ptr(done), int(end_token), _ptr(out["score"]),
                                   _ptr(out["parent"]), _ptr(out["token"]), _ptr(workspace), workspace.numel(),
                                   C.c_void_p(s.cuda_stream)))
        if stream is not None:
            workspace.record_stream(s)
    return out


def beam_search(pages, prompt, n_beams, max_new, end_token=None, slots=None):
    """Beam search from one prompt on the slots of ``pages`` (a ``Lfm3Pages``; its model has a head).

    prompt: device int32 [n]. Uses ``slots`` (default 0 .. n_beams - 1; what they held is released) and leaves them
    holding the beams' states, best first. A beam that chose ``end_token`` keeps its score. Returns (tokens: a list of
    max_new or fewer ids for each beam, scores: fp32 [n_beams]), best first; where there are fewer candidates than beams (or
    the logits are not finite) the last have no tokens and a score of -inf."""
    model = pages.model
    slots = list(range(n_beams)) if slots is None else [int(s) for s in slots]
    if len(slots) != n_beams or n_beams < 1 or max_new < 1:
        raise ValueError("beam_search needs n_beams slots, and n_beams and max_new of at least 1")
    # all of it before the slots lose what they hold
    cfg = model.cfg
    if len(set(slots)) != n_beams or not all(0 <= s < cfg.max_streams for s in slots):
        raise ValueError(f"slots must be different ones of 0..{cfg.max_streams - 1}")
    if n_beams > 64 or (max_new > 1 and n_beams > cfg.max_batch):
        raise ValueError(f"{n_beams} beams are more than 64 or than the model's max_batch of {cfg.max_batch}")
    if (prompt.dim() != 1 or len(prompt) < 1 or prompt.dtype != torch.int32 or prompt.device != pages.state.seq_len.device
            or not prompt.is_contiguous()):
        raise ValueError(f"prompt must be contiguous int32 [n] on {pages.state.seq_len.device}")
    with torch.cuda.device(model.device):
        return _search(pages, prompt, n_beams, max_new, end_token, slots)


def _search(pages, prompt, n_beams, max_new, end_token, slots):
    model, state = pages.model, pages.state
    dev, V = model.device, model.geom.vocab
    for s in slots:
        pages.release(s)
    pages.lease(slots[0], len(prompt))
    logits = model.prefill(state, slots[0], tokens=prompt, argmax=False)["logits"]
    pages.fork(slots[0], slots[1:])
    best = beam_select(logits.view(1, 1, V), torch.zeros(1, 1, device=dev), n_beams)
    history, done = [[]], [False]
    _extend(history, done, best, end_token)
    d_slots = torch.tensor(slots, dtype=torch.int32, device=dev)
    out = {"logits": torch.empty(n_beams, V, device=dev)}
    ws = torch.empty(L.lfm3_beam_workspace(1, n_beams, V, n_beams), dtype=torch.uint8, device=dev)
    for _ in range(max_new - 1):
        if all(done):
            break
        for s in slots:
            pages.lease(s, int(state.h_seq_len[s]) + 1)
        model.decode(state, slots, tokens=best["token"].view(-1).clamp_(min=0), argmax=False, d_slots=d_slots, out=out)
        flags = torch.tensor([done], dtype=torch.int32, device=dev) if any(done) else None
        best = beam_select(out["logits"].view(1, n_beams, V), best["score"].clone(), n_beams, done=flags, end_token=end_token or 0,
                           workspace=ws)
        pages.reorder(slots, _extend(history, done, best, end_token))
    return history, best["score"][0]


def _extend(history, done, best, end_token):
    """The chosen continuations enter ``history`` and ``done``, which are by beam; returns the parents (its own, where a
    place has no candidate: a beam without tokens that counts as finished)."""
    chosen = list(zip(best["parent"][0].tolist(), best["token"][0].tolist()))
    history[:] = [[] if p < 0 else history[p] + ([] if done[p] else [t]) for p, t in chosen]
    done[:] = [p < 0 or done[p] or t == end_token for p, t in chosen]
    return [i if p < 0 else p for i, (p, _) in enumerate(chosen)]
