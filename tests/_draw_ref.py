"""Probabilities and tokens from logits in 64 bits, row by row on the CPU."""
import torch


def weights(z, t=1.0, k=0, top_p=1.0, min_p=0.0):
    """exp((z - max) / t) of the entries that stand, 0 elsewhere; z one row."""
    z = z.double().cpu()
    z = torch.where(torch.isnan(z), torch.full_like(z, -float("inf")), z) + 0.0
    w = torch.zeros_like(z)
    if bool((z == -float("inf")).all()) or not t >= 0 or top_p != top_p or min_p != min_p:
        return w
    order = torch.sort(-z, stable=True).indices
    if t == 0 or top_p <= 0:
        order = order[:1]
    if k > 0:
        order = order[:k]
    top = float(z.max())
    if top == float("inf"):
        p = (z[order] == top).double()
    else:
        p = torch.exp((z[order] - top) / (t if t > 0 else 1.0))
    if 0 < top_p < 1:
        before = torch.cumsum(p, 0) - p
        n = max(1, int((before < top_p * p.sum()).sum()))
        order, p = order[:n], p[:n]
    keep = p >= min(max(min_p, 0.0), 1.0)
    w[order[keep]] = p[keep]
    return w


def token(z, noise, **params):
    w = weights(z, **params)
    score = torch.where(w > 0, w / noise.double().cpu(), torch.full_like(w, -1.0))
    return int(torch.argmax(score)) if bool((w > 0).any()) else -1
