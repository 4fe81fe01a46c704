"""The gated linear recurrence and its derivatives in 64 bits, token by token on the CPU, each value with a
bound of what fp32 arithmetic may do to it."""
import torch

BF, F32 = torch.bfloat16, torch.float32


def gates(x, r, i, a_log, dtype):
    """Everything per element, and ``unit``, the relative error of a product of the elementary functions:
    at |r| and |i| up to 8 a fast exponential is off by 8 log2(e) 2^-24 < 2^-20 (its argument's rounding) and
    2^-22, the reciprocal, the rate's exponential, the root and their products by 2^-23 each, of which no
    value below takes more than eight: 2^-18.  The accurate functions are off by 2^-23 each: 2^-20."""
    x, r, a_log = x.double().cpu(), r.double().cpu(), a_log.double().cpu()
    s = torch.sigmoid(r)
    g = -torch.exp(a_log) * s
    m = torch.sqrt(-torch.expm1(2 * g))
    gi = torch.ones_like(x) if i is None else torch.sigmoid(i.double().cpu())
    hi = torch.zeros_like(x) if i is None else torch.sigmoid(-i.double().cpu())
    return dict(x=x, s=s, c=torch.sigmoid(-r), g=g, a=torch.exp(g), m=m, gi=gi, hi=hi, u=gi * x,
                unit=2.0 ** -18 if dtype == BF else 2.0 ** -20)


def forward(x, r, i, a_log, lens, states, dtype=None):
    """y [T, Ch] (not rounded), the final states [N, Ch], the state before every token, and the bounds of y
    and of the states before.  A decay is off by a (|g| + 1/4) unit: what its exponent's relative error
    makes of it, and its own rounding; a product of n of them as one number by n 2^-24 more, which the
    2^-22 of every step's magnitude covers."""
    k = gates(x, r, i, a_log, dtype or x.dtype)
    T, ch = k["x"].shape
    b, a, g, unit = k["m"] * k["u"], k["a"], k["g"], k["unit"]
    y, before, err, err_before, size_before = (torch.zeros(T, ch, dtype=torch.float64) for _ in range(5))
    final, at = [], 0
    for n, h in zip(lens, states):
        h = h.double().cpu().clone()
        size, e = h.abs(), torch.zeros_like(h)
        for t in range(at, at + n):
            before[t], err_before[t], size_before[t] = h, e, size
            e = a[t] * e + unit * (a[t] * (g[t].abs() + 0.25) * size + b[t].abs())
            h = a[t] * h + b[t]
            size = a[t] * size + b[t].abs()
            e = e + 2.0 ** -22 * size
            y[t], err[t] = h, e
        at += n
        final.append(h)
    k.update(y=y, final=torch.stack(final) if final else torch.zeros(0, ch, dtype=torch.float64), before=before,
             err=err, err_before=err_before, size_before=size_before)
    return k


def backward(k, dy, dfinal, lens):
    """Derivatives from ``forward``'s answer: dx, dr, di, dA_log, dstate, and a bound of each."""
    dy = dy.double().cpu()
    T, ch = dy.shape
    a, g, unit = k["a"], k["g"], k["unit"]
    lam, size, err = (torch.zeros(T, ch, dtype=torch.float64) for _ in range(3))
    dstate, dstate_err, at = [], [], 0
    for i, n in enumerate(lens):
        e = torch.zeros(ch, dtype=torch.float64) if dfinal is None else dfinal[i].double().cpu().clone()
        es, eb = e.abs(), torch.zeros_like(e)
        for t in range(at + n - 1, at - 1, -1):
            lam[t], size[t] = dy[t] + e, dy[t].abs() + es
            err[t] = eb + 2.0 ** -22 * size[t]
            e, es = a[t] * lam[t], a[t] * size[t]
            eb = a[t] * err[t] + unit * a[t] * (g[t].abs() + 0.25) * size[t]
        at += n
        dstate.append(e)
        dstate_err.append(eb)
    ratio = torch.where(k["m"] > 0, g / torch.where(k["m"] > 0, k["m"], 1.0), 0.0)
    p = g * a * lam * k["before"] - a * a * ratio * k["u"] * lam
    p_size = a * size * (g.abs() * k["size_before"] + a * (ratio * k["u"]).abs())
    p_err = a * err * (g.abs() * k["size_before"] + a * (ratio * k["u"]).abs()) \
        + a * size * g.abs() * k["err_before"] + 4 * unit * p_size * (1 + g.abs())
    ml, ml_size = k["m"] * lam, k["m"] * size
    ml_err = k["m"] * err + unit * ml_size
    add = (8 + 16 + T / 48 / 32 + 32) * 2.0 ** -24   # roundings on the way of one term of the sum
    z = lambda rows: torch.stack(rows) if rows else torch.zeros(0, ch, dtype=torch.float64)
    return dict(dx=ml * k["gi"], dr=p * k["c"], di=ml * k["u"] * k["hi"], dA_log=p.sum(0), dstate=z(dstate)), \
        dict(dx=(ml_err + unit * ml_size) * k["gi"], dr=(p_err + unit * p_size) * k["c"],
             di=(ml_err + 2 * unit * ml_size) * k["u"].abs() * k["hi"],
             dA_log=p_err.sum(0) + add * p_size.sum(0), dstate=z(dstate_err))


def check(got, want, bound, dtype=F32, what=""):
    """Element by element: the bound of the arithmetic and one rounding to ``dtype``."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    limit = bound * 1.01 + torch.finfo(dtype).eps / 2 * (want.abs() + bound) + 1e-37
    off = (got - want).abs()
    assert torch.isfinite(got).all() and (off <= limit).all(), \
        (what, float((off - limit).max()), float((off / limit).max()))
