"""Plain fp64 forms of the selective scan, draft verification and block norm, one token, one
entry, one row at a time where that is the definition. They share no code with the library."""
import math

import numpy as np
import torch


def d(t):
    return None if t is None else t.detach().cpu().double()


def step_size(dt, bias, softplus):
    v = d(dt) + (0 if bias is None else d(bias))
    return torch.nn.functional.softplus(v, threshold=80.0) if softplus else v


def scan(x, dt, a, b, c, lens, h0=None, d_skip=None, dt_bias=None, softplus=True):
    """Returns y [T, H, P] and the final states [N, H, 128, P]."""
    x, b, c, a = d(x), d(b), d(c), d(a)
    h = step_size(dt, dt_bias, softplus)
    T, H, P = x.shape
    R = H // b.shape[1]
    b, c = b.repeat_interleave(R, 1), c.repeat_interleave(R, 1)
    skip = torch.zeros(H, dtype=torch.float64) if d_skip is None else d(d_skip)
    y, states, t = torch.empty_like(x), [], 0
    for i, n in enumerate(lens):
        S = torch.zeros(H, b.shape[2], P, dtype=torch.float64) if h0 is None else d(h0[i]).clone()
        for t in range(t, t + n) if n else ():
            S = S * torch.exp(h[t] * a)[:, None, None] + b[t][:, :, None] * (h[t][:, None] * x[t])[:, None, :]
            y[t] = torch.einsum("hk,hkp->hp", c[t], S) + skip[:, None] * x[t]
        t = sum(lens[:i + 1])
        states.append(S)
    return y, torch.stack(states) if states else None


def conv(line, weight, bias, act):
    """line [W - 1 + n, C] -> n outputs."""
    line, w = d(line), d(weight)
    W = w.shape[1]
    n = line.shape[0] - (W - 1)
    z = torch.stack([(line[t:t + W] * w.t()).sum(0) for t in range(n)]) if n else line[:0]
    z = z if bias is None else z + d(bias)
    return z * torch.sigmoid(z) if act == "silu" else z


def step(xbc, dt, a, weight, bias, conv_state, state, groups, accept=None, slots=None, first=None, d_skip=None,
         dt_bias=None, softplus=True, act="silu"):
    """Returns y (rows that are not written: None), and the two pools after the call."""
    N, L, Cc = xbc.shape
    _, H, D, P = state.shape
    W = weight.shape[1]
    pool, cpool = d(state).clone(), conv_state.detach().cpu().clone() if W > 1 else None
    ys = {}
    for i in range(N):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < state.shape[0]:
            continue
        f = 0 if first is None else min(max(int(first[i]), 0), L)
        acc = L if accept is None else min(max(int(accept[i]), 0), L)
        rows = xbc[i, f:].cpu()
        line = torch.cat([conv_state[s].cpu(), rows], 0) if W > 1 else rows
        z = conv(line, weight, bias, act)
        x, b, c = z[:, :H * P].reshape(-1, H, P), z[:, H * P:H * P + groups * D].reshape(-1, groups, D), \
            z[:, H * P + groups * D:].reshape(-1, groups, D)
        y, _ = scan(x, dt[i, f:], a, b, c, [L - f], state[s:s + 1], d_skip, dt_bias, softplus)
        for t in range(L - f):
            ys[(i, f + t)] = y[t]
        k = acc - f
        if k > 0:
            pool[s] = scan(x[:k], dt[i, f:f + k], a, b[:k], c[:k], [k], state[s:s + 1], d_skip, dt_bias, softplus)[1][0]
            if W > 1:
                cpool[s] = line[k:k + W - 1]
    return ys, pool, cpool


def verify(p, q, draft, u, noise, draft_len=None):
    """Per sequence, entry by entry; the comparisons and the race in fp32, as they are defined."""
    p, q = p.float().cpu().numpy(), None if q is None else q.float().cpu().numpy()
    draft, u, noise = draft.cpu().numpy(), u.cpu().numpy(), noise.cpu().numpy()
    N, L1, V = p.shape
    L = L1 - 1
    accept, tokens = np.zeros(N, np.int32), np.full((N, L1), -1, np.int32)

    def race(r, e):
        best, at = np.float32(0), -1
        with np.errstate(all="ignore"):
            s = r / e
        for v in range(V):
            if r[v] > 0 and s[v] > best:
                best, at = s[v], v
        return at

    for i in range(N):
        n = L if draft_len is None else min(max(int(draft_len[i]), 0), L)
        k = 0
        while k < n and 0 <= draft[i, k] < V:
            x = draft[i, k]
            if not np.float32(u[i, k]) * (np.float32(1) if q is None else q[i, k, x]) < p[i, k, x]:
                break
            k += 1
        r = p[i, k].copy()
        if k < n and 0 <= draft[i, k] < V:
            if q is None:
                r[draft[i, k]] -= np.float32(1)
            else:
                with np.errstate(all="ignore"):
                    r = r - q[i, k]
        nxt = race(r, noise[i])
        if nxt < 0:
            nxt = race(p[i, k], noise[i])
        accept[i] = k
        tokens[i, :k] = draft[i, :k]
        tokens[i, k] = nxt
    return accept, (L - accept).astype(np.int32), tokens


def block_norm(u, w_post, gate, act, residual, scale, w_pre, eps):
    """fp64 tensors in, (out, normed or None) out, differentiable."""
    m = u
    if w_post is not None:
        m = m / torch.sqrt((m * m).mean(-1, keepdim=True) + eps) * w_post
    if gate is not None:
        m = m * (torch.sigmoid(gate) if act == "sigmoid" else gate * torch.sigmoid(gate))
    if scale is not None:
        m = m * scale
    out = m if residual is None else residual + m
    normed = None if w_pre is None else out / torch.sqrt((out * out).mean(-1, keepdim=True) + eps) * w_pre
    return out, normed


def rel(got, ref):
    """Largest difference over the largest value of the reference."""
    got, ref = d(got), d(ref)
    if ref.numel() == 0:
        return 0.0
    e = (got - ref).abs().max().item()
    return math.inf if math.isnan(e) else e / max(ref.abs().max().item(), 1e-30)
