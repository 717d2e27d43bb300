"""Multi-round decoding over the C ABI: each round drafts a block of gamma
positions from the requests' anchors, verifies it against the target logits
and emits the accepted prefix plus one corrective or bonus token; that last
token is the next round's anchor.  Summary page §요약 (a drafted block is
verified by rejection sampling, which keeps the target distribution), §3
(a round's accepted length tau counts the bonus token; per-token latency
L = (T_draft + T_verify) / tau) and §3.1 (a block is drafted from the anchor).

Round t draws its random numbers with the Philox key seed + t * 2^32 (the
round index in the key's high word), so round 0 is the single-round call and
different rounds use independent streams.  The anchors are handed from one
round to the next on the device (two alternating buffers, no host copy).

With a cache (cache.PagedCache, slot r for request r) a round also keeps the
target's keys and values: it reserves pages for the gamma + 1 tokens of each
request's chunk (the anchor and the drafts) before the target runs on them,
and commits the anchor and the accepted drafts after the verify step.  The
target's layers call cache.append and cache.attend with the loop's offsets.
Argument marshalling only: every step runs in the HIP library.
"""
from __future__ import annotations

import torch

from . import dspark

ROUND_KEY_STRIDE = 1 << 32


def round_seed(seed: int, t: int) -> int:
    """Philox key of round t: the round index added to the key's high word."""
    return (int(seed) + int(t) * ROUND_KEY_STRIDE) & ((1 << 64) - 1)


class DecodeLoop:
    """Rounds of draft + verify (+ Algorithm 1 on the round's c*, when an SPS
    table is given) with the anchors carried on the device.

    W1 [V, 256] and W2p (packed) stay fixed; each round takes its backbone
    logits U [R, gamma, V] and a callable that returns the target logits
    T [R, gamma + 1, V] for the drafted tokens (the target model's verify
    forward pass).  cache: the target's PagedCache, with as many slots as
    requests.  logprobs: None, or how many of the most likely tokens to report
    with every emitted token's log probability."""

    def __init__(self, W1, W2p, anchors, seed: int, gamma: int, sps=None, cache=None,
                 logprobs: int | None = None):
        R = anchors.numel()
        V = W1.shape[0]
        dev = W1.device
        self.W1, self.W2p, self.seed, self.gamma, self.sps = W1, W2p, int(seed), gamma, sps
        self.t = 0
        self._anchors = [anchors.clone(), torch.empty_like(anchors)]
        self.ws = dspark.workspace(dspark.problem(R, gamma, V, W1.dtype, seed), dev)
        self.d_out = (torch.empty((R, gamma), dtype=torch.int32, device=dev),
                      torch.empty((R, gamma), dtype=torch.float64, device=dev),
                      torch.empty((R, gamma), dtype=torch.float64, device=dev))
        self.v_out = {"cstar": torch.empty((R, gamma), dtype=torch.float32, device=dev),
                      "n_accept": torch.empty(R, dtype=torch.int32, device=dev),
                      "out_token": None,
                      "accept_mask": torch.empty((R, gamma), dtype=torch.uint8, device=dev),
                      "lse_t": None}
        self.s_out = {"a": torch.empty((R, gamma), dtype=torch.float32, device=dev),
                      "lengths": torch.empty(R, dtype=torch.int32, device=dev),
                      "stats": torch.empty(4, dtype=torch.float64, device=dev),
                      "theta_path": None}
        self.cache, self.logprobs = cache, logprobs
        if cache is not None:
            if cache.slots != R:
                raise ValueError(f"cache must have one slot per request ({R}), got {cache.slots}")
            if cache.device != dev:
                raise ValueError(f"cache must be on {dev}, got {cache.device}")
            self.offsets = torch.arange(R + 1, dtype=torch.int32, device=dev) * (gamma + 1)
            self._add = torch.full((R,), gamma + 1, dtype=torch.int32, device=dev)
            self.c_out = {n: torch.empty(R, dtype=torch.int32, device=dev)
                          for n in ("status", "cow_src", "cow_dst")}
            self._status = torch.empty(R, dtype=torch.int32, pin_memory=True)
            self._served = torch.cuda.Event()
        if logprobs is not None:
            if not 0 <= logprobs <= 64:
                raise ValueError(f"logprobs must be in [0, 64], got {logprobs}")
            lead = (R, gamma + 1)
            self.emitted = torch.empty(lead, dtype=torch.int32, device=dev)
            self.l_ws = dspark.logprobs_workspace(R * (gamma + 1), V, logprobs, dev)
            self.l_out = {"logprob": torch.empty(lead, dtype=torch.float32, device=dev),
                          "entropy": torch.empty(lead, dtype=torch.float32, device=dev),
                          "top_ids": torch.empty((*lead, logprobs), dtype=torch.int32, device=dev),
                          "top_logprobs": torch.empty((*lead, logprobs), dtype=torch.float32,
                                                      device=dev)}

    @property
    def anchors(self):
        """Anchors of the next round (device int32 [R])."""
        return self._anchors[self.t % 2]

    def round(self, U, target_fn):
        """One round; returns a dict of device tensors: tokens, lse, logq,
        cstar, n_accept, out_token (= the next anchors), accept_mask and, with
        an SPS table, the scheduler's a, lengths and stats; with logprobs,
        emitted (dspark_emitted_tokens) and its logprob, entropy, top_ids and
        top_logprobs under T.  The buffers are the loop's, written again by
        the next round.

        With a cache, a request that finds no pages ends the call with a
        RuntimeError before the target runs: no length has changed, and the
        round can be repeated once slots have been freed.  The host learns this
        while the draft step runs, so it waits for no work that follows; for
        this reason a round with a cache cannot be captured into a graph."""
        if self.cache is not None:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a round with a cache cannot be captured")
            self.cache.reserve(self._add, out=self.c_out)
            self._status.copy_(self.c_out["status"], non_blocking=True)
            self._served.record()
        seed_t = round_seed(self.seed, self.t)
        anchors = self._anchors[self.t % 2]
        nxt = self._anchors[(self.t + 1) % 2]
        tok, lse, logq = dspark.draft_step(U, self.W1, self.W2p, anchors, seed_t, ws=self.ws,
                                           out=self.d_out)
        if self.cache is not None:
            self._served.synchronize()
            if self._status.any():
                short = [r for r, st in enumerate(self._status.tolist()) if st]
                raise RuntimeError(f"no cache pages for requests {short}")
        T = target_fn(self.t, tok)
        self.v_out["out_token"] = nxt
        v = dspark.verify(U, self.W1, self.W2p, anchors, tok, lse, logq, T, None, seed_t,
                          ws=self.ws, out=self.v_out)
        res = {"tokens": tok, "lse": lse, "logq": logq, "cstar": v["cstar"],
               "n_accept": v["n_accept"], "out_token": nxt, "accept_mask": v["accept_mask"],
               "anchors": anchors, "seed": seed_t}
        if self.sps is not None:
            s = dspark.schedule(v["cstar"], self.sps, out=self.s_out, with_path=False)
            res.update({"a": s["a"], "lengths": s["lengths"], "stats": s["stats"]})
        if self.cache is not None:
            self.cache.commit(v["n_accept"], 1)
        if self.logprobs is not None:
            ids = dspark.emitted_tokens(tok, v["n_accept"], nxt, out=self.emitted)
            res.update(dspark.token_logprobs(T, ids, self.logprobs, ws=self.l_ws, out=self.l_out))
            res["emitted"] = ids
        self.t += 1
        return res
