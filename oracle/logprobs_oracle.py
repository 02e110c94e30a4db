"""fp64 CPU oracle of the output head's log probabilities -- TEST INFRASTRUCTURE ONLY.

Log probabilities of given tokens, entropies, the most likely alternatives and the
gradients with respect to H and W over the logits s = H W^T, straight from their
definitions in float64 numpy.  Shares no code with the HIP library.
"""

from __future__ import annotations

import numpy as np


def log_probs(hidden, weight, targets=None, ignore_index=-100, temperature=1.0, top_k=0, grad_logprobs=None,
              grad_entropy=None):
    """dict of live, s, logp (of every word), lse, entropy, logprobs, top_ids, top_logprobs and, for upstream
    gradients, ds (by s), dh, dw.  Every target of a row that counts is in the vocabulary."""
    hidden = np.asarray(hidden, dtype=np.float64)
    weight = np.asarray(weight, dtype=np.float64)
    t = len(hidden)
    live = np.ones(t, dtype=bool) if targets is None else np.asarray(targets) != ignore_index
    h = np.where(live[:, None], hidden, 0.0)
    s = h @ weight.T
    x = s / temperature
    m = x.max(axis=1, keepdims=True)
    lse = m + np.log(np.exp(x - m).sum(axis=1, keepdims=True))
    logp = x - lse
    p = np.exp(logp)
    entropy = -np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0).sum(axis=1)
    out = {"live": live, "s": s, "logp": logp, "lse": np.where(live, lse[:, 0], 0.0),
           "entropy": np.where(live, entropy, 0.0)}
    hot = np.zeros_like(s)
    if targets is not None:
        hot[np.nonzero(live)[0], np.asarray(targets)[live]] = 1.0
        out["logprobs"] = np.where(live, np.where(hot > 0, logp, 0.0).sum(axis=1), 0.0)
    if top_k:
        ids = np.argsort(-s, axis=1, kind="stable")[:, :top_k]
        out["top_ids"] = np.where(live[:, None], ids, -1)
        out["top_logprobs"] = np.where(live[:, None], np.take_along_axis(logp, ids, axis=1), 0.0)
    if grad_logprobs is not None or grad_entropy is not None:
        zero = np.zeros(t)
        g = np.where(live, zero if grad_logprobs is None else grad_logprobs, 0.0)[:, None]
        e = np.where(live, zero if grad_entropy is None else grad_entropy, 0.0)[:, None]
        ds = (g * (hot - p) - e * p * (np.where(p > 0, logp, 0.0) + entropy[:, None])) / temperature
        out.update(ds=ds, dh=ds @ weight, dw=ds.T @ h)
    return out
