"""Plain 64-bit implementations of the operators around the recurrence, token by token on the CPU,
and the bounds that their tests use."""
import torch

BF, F32 = torch.bfloat16, torch.float32
EPS = {BF: 2.0 ** -8, F32: 2.0 ** -24}  # largest relative error of one rounding: 2^-p, p = 8 and 24 bits


def cu_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


def slots_of(idx, num_slots):
    return [num_slots - 1 if int(i) < 0 else int(i) for i in idx]


def conv(x, w, bias, silu, lens, states):
    """y [T, Ch], the final states, and the states after every token (lists per sequence); ``states``
    is a list of [W-1, Ch]."""
    x, w = x.double().cpu(), w.double().cpu()
    W = w.shape[1]
    y, final, steps, a = torch.zeros_like(x), [], [], 0
    for n, h in zip(lens, states):
        h, each = h.double().cpu().clone(), []
        for t in range(a, a + n):
            win = torch.cat([h, x[t:t + 1]])
            s = (win * w.T).sum(0) + (0 if bias is None else bias.double().cpu())
            y[t] = s / (1 + torch.exp(-s)) if silu else s
            h = win[1:]
            each.append(h.clone())
        a += n
        final.append(h)
        steps.append(each)
        assert h.shape[0] == W - 1
    return y, final, steps


def ssm(x, dt, a_log, b, c, d, dt_bias, lens, states):
    """y [T, H, V], the final states, and the states after every token; states a list of [H, K, V]."""
    x, dt, b, c = (t.double().cpu() for t in (x, dt, b, c))
    H = x.shape[1]
    rep = H // b.shape[1]
    z = dt + (0 if dt_bias is None else dt_bias.double().cpu())
    step = torch.logaddexp(z, torch.zeros_like(z))
    keep = torch.exp(-torch.exp(a_log.double().cpu()) * step)
    y, final, steps, a = torch.zeros_like(x), [], [], 0
    for n, S in zip(lens, states):
        S, each = S.double().cpu().clone(), []
        for t in range(a, a + n):
            bt = b[t].repeat_interleave(rep, 0) * step[t][:, None]
            ct = c[t].repeat_interleave(rep, 0)
            S = S * keep[t][:, None, None] + bt[:, :, None] * x[t][:, None, :]
            y[t] = torch.einsum("hk,hkv->hv", ct, S)
            if d is not None:
                y[t] += d.double().cpu()[:, None] * x[t]
            each.append(S.clone())
        a += n
        final.append(S)
        steps.append(each)
    return y, final, steps


def verify(tokens, p, q, u, noise, lens):
    tokens, lens = tokens.tolist(), list(lens)
    kept, out, a = [], [], 0
    for i, n in enumerate(lens):
        if n == 0:
            kept.append(0)
            out.append(-1)
            continue
        r = a
        while r < a + n - 1:
            dtok = tokens[r + 1]
            qd = 1.0 if q is None else float(q[r, dtok])
            if not float(u[r]) * qd < float(p[r, dtok]):
                break
            r += 1
        w = p[r].double().cpu().clone()
        if r < a + n - 1:
            if q is None:
                diff = w.clone()
                diff[tokens[r + 1]] -= 1.0
            else:
                diff = w - q[r].double().cpu()
            diff = torch.where(diff > 0, diff, torch.zeros_like(diff))
            w = diff if bool((diff > 0).any()) else w
        ok = w > 0
        score = torch.where(ok, w / noise[i].double().cpu(), torch.full_like(w, -1.0))
        kept.append(r - a + 1)
        out.append(int(torch.argmax(score)) if bool(ok.any()) else -1)
        a += n
    return kept, out


def rel(x, ref):
    x, ref = x.detach().double().cpu(), ref.double()
    assert torch.isfinite(x).all()
    return float((x - ref).norm() / ref.norm().clamp_min(1e-300))
