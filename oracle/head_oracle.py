"""fp64 CPU oracle of the output-head losses -- TEST INFRASTRUCTURE ONLY.

Cross entropy and distillation from a teacher's top logits over the logits
s = H W^T, and the gradients with respect to H and W, straight from their
definitions in float64 numpy.  Shares no code with the HIP library.
"""

from __future__ import annotations

import numpy as np


def _logits(hidden, weight, live):
    # rows that carry no loss may hold anything: they are left out here
    h = np.where(live[:, None], np.asarray(hidden, dtype=np.float64), 0.0)
    return h, h @ np.asarray(weight, dtype=np.float64).T


def _log_sum_exp(x):
    m = x.max(axis=1, keepdims=True)
    return (m + np.log(np.exp(x - m).sum(axis=1, keepdims=True)))[:, 0]


def cross_entropy(hidden, weight, targets, ignore_index=-100, grad_losses=None, grad_lse=None):
    """dict of losses, lse, s, ds, dh, dw (the last three for grad_losses)."""
    targets = np.asarray(targets)
    live = targets != ignore_index
    h, s = _logits(hidden, weight, live)
    lse = _log_sum_exp(s)
    hot = np.zeros_like(s)
    hot[np.nonzero(live)[0], targets[live]] = 1.0
    out = {"live": live, "s": s, "lse": np.where(live, lse, 0.0),
           "losses": np.where(live, lse - (hot * s).sum(axis=1), 0.0)}
    if grad_losses is not None:
        g = np.where(live, np.asarray(grad_losses, dtype=np.float64), 0.0)[:, None]
        gl = 0.0 if grad_lse is None else np.where(live, np.asarray(grad_lse, dtype=np.float64), 0.0)[:, None]
        p = np.exp(s - lse[:, None])
        ds = (g + gl) * p - g * hot
        out.update(p=p, ds=ds, cp=np.abs(g + gl), ct=np.abs(g), hot=hot, dh=ds @ np.asarray(weight, np.float64),
                   dw=ds.T @ h)
    return out


def distill(hidden, weight, ids, teacher, temperature=1.0, grad_losses=None):
    """As cross_entropy; ids (tokens x K, negative: absent), teacher logits."""
    ids = np.asarray(ids)
    z = np.where(ids >= 0, np.asarray(teacher, dtype=np.float64), -np.inf) / temperature
    live = (z > -np.inf).any(axis=1)
    h, s = _logits(hidden, weight, live)
    lse = _log_sum_exp(s / temperature)
    q = np.zeros_like(z)
    loss = np.zeros(len(ids))
    mass = np.zeros_like(s)
    student = np.zeros_like(z)
    for t in np.nonzero(live)[0]:
        k = np.nonzero(z[t] > -np.inf)[0]
        e = np.exp(z[t, k] - z[t, k].max())
        q[t, k] = e / e.sum()
        logq = z[t, k] - z[t, k].max() - np.log(e.sum())
        loss[t] = temperature ** 2 * np.sum(q[t, k] * (logq - s[t, ids[t, k]] / temperature + lse[t]))
        np.add.at(mass[t], ids[t, k], q[t, k])
        held = ids[t] >= 0
        student[t, held] = s[t, ids[t, held]]
    out = {"live": live, "s": s, "lse": np.where(live, lse, 0.0), "losses": loss, "q": q, "student": student}
    if grad_losses is not None:
        g = np.where(live, np.asarray(grad_losses, dtype=np.float64), 0.0)[:, None] * temperature
        p = np.exp(s / temperature - lse[:, None])
        ds = g * (p - mass)
        out.update(p=p, ds=ds, cp=np.abs(g), ct=np.abs(g), hot=mass, dh=ds @ np.asarray(weight, np.float64),
                   dw=ds.T @ h)
    return out
