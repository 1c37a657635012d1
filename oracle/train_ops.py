"""FP64 statements of the training-step operators beside the loss: linear cross entropy,
scaled embedding and its gradient, gradient clipping.  Plain torch on any device, written
from the formulas of include/dspark.h; test infrastructure only, the library never calls
it.
"""

from __future__ import annotations

import torch


def linear_ce(hidden, weight, targets, row_weight=None, ignore_index=-100, z_alpha=0.0, grad_scale=1.0):
    """Loss, row outputs and gradients, and the magnitudes the error bounds need:
    ``reach`` = max over labelled rows and the vocabulary of sum_k |h_k w_k|, ``dh_mag`` and
    ``dw_mag`` = |dz| |weight| and |dz|^T |hidden|, ``dh_pmag`` and ``dw_pmag`` the same with
    the probabilities' part of dz alone."""
    V = weight.shape[0]
    live = (targets != ignore_index) & (targets >= 0) & (targets < V)
    h = torch.where(live[:, None], hidden, torch.zeros_like(hidden)).double()
    w = weight.double()
    t = torch.where(live, targets, torch.zeros_like(targets))
    a = live.double() if row_weight is None else torch.where(live, row_weight, torch.zeros_like(row_weight)).double()
    z = h @ w.T
    lse = torch.logsumexp(z, dim=1)
    ce = lse - z.gather(1, t[:, None])[:, 0]
    dz = torch.exp(z - lse[:, None]) * (1.0 + 2.0 * z_alpha * lse)[:, None]
    dp = dz * (grad_scale * a)[:, None].abs()
    dz.scatter_add_(1, t[:, None], torch.full_like(dz[:, :1], -1.0))
    dz *= (grad_scale * a)[:, None]
    zero = torch.zeros_like(lse)
    return dict(loss_num=(a * (ce + z_alpha * lse * lse)).sum(), num_tokens=int(live.sum()),
                ce_rows=torch.where(live, ce, zero), lse_rows=torch.where(live, lse, zero),
                dhidden=dz @ w, dweight=dz.T @ h, dh_mag=dz.abs() @ w.abs(), dw_mag=dz.abs().T @ h.abs(),
                dh_pmag=dp.abs() @ w.abs(), dw_pmag=dp.abs().T @ h.abs(),
                reach=float((h.abs() @ w.abs().T).max()) if bool(live.any()) else 0.0)


def embed(ids, table, scale=1.0, valid=None):
    Vt = table.shape[0]
    live = (ids >= 0) & (ids < Vt)
    if valid is not None:
        live &= valid.reshape(ids.shape) != 0
    rows = table.double()[torch.where(live, ids, torch.zeros_like(ids))] * scale
    return torch.where(live[..., None], rows, torch.zeros_like(rows))


def embed_grad(ids, dout, vocab, scale=1.0, valid=None):
    """(gradient, sum of the magnitudes added up, rows added up) per table row."""
    live = (ids >= 0) & (ids < vocab)
    if valid is not None:
        live &= valid != 0
    g = torch.zeros(vocab, dout.shape[1], dtype=torch.float64, device=dout.device)
    mag = torch.zeros_like(g)
    x = dout[live].double() * scale
    g.index_add_(0, ids[live], x)
    mag.index_add_(0, ids[live], x.abs())
    return g, mag, torch.bincount(ids[live], minlength=vocab)


def clip(grads, max_norm):
    norm = sum(float(g.double().pow(2).sum()) for g in grads) ** 0.5
    finite = norm == norm and norm not in (float("inf"), float("-inf"))
    coef = min(1.0, max_norm / (norm + 1e-6)) if finite else 1.0
    return norm, coef, [g.double() * coef for g in grads]
