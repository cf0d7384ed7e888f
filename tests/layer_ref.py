"""Plain 64-bit definitions of the operators of include/talker_layer.h and talker_draft.h, and of the tests' inputs."""
import math

import numpy as np
import torch

F64 = torch.float64


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def uni(seed, *shape):
    return torch.rand(*shape, generator=torch.Generator().manual_seed(seed))


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ norm

def rms_norm(x, gain, eps, residual=None):
    s = x.to(F64) if residual is None else x.to(F64) + residual.to(F64)
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * gain.to(F64), s


def by_block(t, block, width):
    """Scales [..., blocks] spread over the width."""
    return t.repeat_interleave(block or width, -1)[..., :width]


# ------------------------------------------------------------------ rotary

def frequencies(rotary, theta, scaling):
    """Radians a position and amplitude, pair by pair."""
    s = scaling or {"type": "none"}
    kind, amp, out = s["type"], 1.0, []
    base = theta * s["factor"] ** (rotary / (rotary - 2)) if kind == "ntk" else theta
    if kind == "yarn":
        def pair(b):
            return rotary * math.log(s["original"] / (2 * math.pi * b)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(pair(s["beta_fast"]))), min(rotary - 1, math.ceil(pair(s["beta_slow"])))
        amp = s.get("amplitude") or 0.1 * math.log(s["factor"]) + 1
    for i in range(rotary // 2):
        f = base ** (-2 * i / rotary)
        k = 1.0
        if kind == "linear":
            k = 0.0
        elif kind == "smooth":
            k = min(1.0, max(0.0, (s["original"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])))
        elif kind == "yarn":
            k = 1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(f * k + f / s.get("factor", 1.0) * (1 - k))
    return np.array(out), amp


def rotate(x, positions, rotary, theta, scaling, interleaved):
    """x [..., heads, head_dim], positions [...]: the result, and |a| + |b| of each pair in its dims (0 where they stay)."""
    f, amp = frequencies(rotary, theta, scaling)
    ang = positions.double().numpy()[..., None, None] * f
    c, s = amp * np.cos(ang), amp * np.sin(ang)
    y = x.double().numpy().copy()
    size = np.zeros_like(y)
    i = np.arange(rotary // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = (np.abs(a) + np.abs(b)) * amp
    return torch.from_numpy(y), torch.from_numpy(size)


# ------------------------------------------------------------------ 4-bit weights

def w4_values(codes, scales, zeros, k, group):
    """[n, k] f64 and the scales spread over k."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :k].to(F64)
    d = scales.to(F64).repeat_interleave(group, -1)[:, :k]
    z = 8.0 if zeros is None else (zeros & 15).to(F64).repeat_interleave(group, -1)[:, :k]
    return (n - z) * d, d


def w4_matrix(seed, n, k, group, zeros):
    g = torch.Generator().manual_seed(seed)
    groups = -(-k // group)
    codes = torch.randint(0, 256, (n, (k + 1) // 2), generator=g, dtype=torch.uint8)
    scales = (0.01 * torch.randn(n, groups, generator=g)).to(torch.float16)
    z = torch.randint(0, 16, (n, groups), generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, z


# ------------------------------------------------------------------ drafts

def unmask(x):
    x = np.asarray(x, np.float64)
    return np.where(x > -1e30, x, -np.inf)


def probabilities(row, temp):
    """p [vocab]; zeros for a row without a distribution."""
    x = unmask(row)
    top = x.max()
    if not np.isfinite(top):
        return np.zeros_like(x)
    if not temp > 1e-20:
        p = np.zeros_like(x)
        p[int(np.argmax(x))] = 1.0
        return p
    with np.errstate(over="ignore"):
        e = np.exp((x - top) / temp)
    return e / e.sum()


def verify(target, tokens, u, draft=None, count=None, temp=1.0):
    """One sequence: (tokens [K + 1], taken, logprobs [K + 1])."""
    K, V = target.shape[0] - 1, target.shape[1]
    count = K if count is None else min(max(count, 0), K)
    u = np.clip(np.nan_to_num(np.asarray(u, np.float64), nan=0.0), 0.0, 1.0)
    greedy = not temp > 1e-20
    out, lps, n = [-1] * (K + 1), [0.0] * (K + 1), 0
    while True:
        p = probabilities(target[n], temp)
        w = p
        if n < count:
            x = int(tokens[n])
            q = np.zeros(V)
            inside = 0 <= x < V
            if draft is not None and not greedy:
                q = probabilities(draft[n], temp)
            elif inside:
                q[x] = 1.0
            good = inside and (p[x] > 0 if greedy else u[n] * q[x] < p[x])
            if good:
                out[n], lps[n] = x, float(np.log(p[x]))
                n += 1
                continue
            if not greedy:
                w = np.maximum(p - q, 0.0)
                if w.sum() == 0:
                    w = p
        c = np.cumsum(w)
        if c[-1] > 0:
            above = np.nonzero(c > u[K] * c[-1])[0]
            t = int(above[0]) if len(above) else int(np.nonzero(w)[0][-1])
            out[n], lps[n] = t, float(np.log(p[t]))
        return out, n, lps
