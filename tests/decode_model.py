"""Plain statements of the decode cycle's operators in 64 bits, for their tests.

Nothing here is shared with the library: rotary positions, norms, attention over a sequence's
keys (whoever shares them), and next tokens with their filters.
"""
import math

import numpy as np
import torch


# ---- rotary positions ------------------------------------------------------------------
def frequencies(rot, base=10000.0, kind="plain", factor=1.0, context=4096.0, low=None, high=None):
    """Angle per position of every pair, one pair at a time."""
    out = []
    for k in range(rot // 2):
        f = base ** (-2.0 * k / rot)
        if kind == "linear":
            f /= factor
        elif kind == "ntk":
            f = (base * factor ** (rot / max(1, rot - 2))) ** (-2.0 * k / rot)
        elif kind in ("yarn", "wavelength"):
            lo = 1.0 if low is None else low
            hi = (32.0 if kind == "yarn" else 4.0) if high is None else high
            if kind == "yarn":
                first, last = (rot * math.log(context / (2 * math.pi * n)) /
                               (2 * math.log(base)) for n in (hi, lo))
                first, last = max(0, math.floor(first)), min(rot - 1, math.ceil(last))
                stretch = min(1.0, max(0.0, (k - first) / max(last - first, 1e-3)))
            else:
                turns = context * f / (2 * math.pi)
                stretch = 1.0 - min(1.0, max(0.0, (turns - lo) / (hi - lo)))
            f = f * (1 - stretch) + f / factor * stretch
        out.append(f)
    return np.array(out)


def magnitude(kind, factor):
    return 0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0


def turn(x, angles, layout, mag=1.0):
    """x [T, H, rot] turned by angles [T, rot/2]."""
    x = np.asarray(x, np.float64)
    n = x.shape[-1] // 2
    a, b = (x[..., :n], x[..., n:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    z = (a + 1j * b) * (mag * np.exp(1j * angles))[:, None]
    y = np.empty_like(x)
    if layout == "half":
        y[..., :n], y[..., n:] = z.real, z.imag
    else:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    return y


def pair_size(x, layout):
    """|a| + |b| of every element's pair."""
    x = np.abs(np.asarray(x, np.float64))
    n = x.shape[-1] // 2
    y = np.empty_like(x)
    if layout == "half":
        y[..., :n] = y[..., n:] = x[..., :n] + x[..., n:]
    else:
        y[..., 0::2] = y[..., 1::2] = x[..., 0::2] + x[..., 1::2]
    return y


def norm(x, w, eps):
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


# ---- attention -------------------------------------------------------------------------
def attention(ql, qp, c, kp, visible, scale):
    """One sequence: ql [Q,H,512], qp [Q,H,64], keys c [n,512], kp [n,64], visible [Q,n].
    Returns out, lse, A = sum_j p_j |c_j| and S = the largest scale sum |q||k| of a row."""
    q = torch.cat([ql, qp], -1).double()
    k = torch.cat([c, kp], -1).double()
    s = torch.einsum("qhd,nd->qhn", q, k) * scale
    s = s.masked_fill(~visible[:, None], -math.inf)
    size = (torch.einsum("qhd,nd->qhn", q.abs(), k.abs()) * scale).amax(-1)
    lse = torch.logsumexp(s, -1)
    p = torch.where(torch.isinf(s), torch.zeros_like(s), torch.exp(s - lse[..., None]))
    cd = c.double()
    return p @ cd, lse, p @ cd.abs(), size


# ---- next tokens -----------------------------------------------------------------------
def next_token(x, u, temperature=1.0, k=0, p=1.0, m=0.0):
    """(token, kept) of one row of logits; kept tokens one after another."""
    x = np.asarray(x, np.float64)
    if not temperature >= 0 or np.isnan(x).any() or not np.isfinite(x.max()):
        return -1, 0
    if temperature == 0:
        return int(np.argmax(x)), 1
    if np.isnan(p) or np.isnan(m):
        return -1, 0
    w = np.exp((x - x.max()) / float(np.float32(temperature)))
    order = [int(v) for v in np.argsort(-x, kind="stable") if x[v] > -np.inf]
    if k > 0:
        order = order[:k]
    if p < 1:
        share = max(0.0, float(np.float32(p))) * math.fsum(w[order])
        run, kept = 0.0, []
        sums = np.cumsum(w[order])
        for i, v in enumerate(order):
            run = sums[i - 1] if i else 0.0
            if i and not run < share:
                break
            kept.append(v)
        order = kept
    if m > 0:
        least = min(1.0, float(np.float32(m)))
        order = [v for i, v in enumerate(order) if i == 0 or w[v] >= least]
    chosen = sorted(order)
    total = np.cumsum(w[chosen])
    i = int(np.searchsorted(total, float(np.float32(u)) * total[-1], side="right"))
    return chosen[min(i, len(chosen) - 1)], len(chosen)
