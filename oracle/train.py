"""Group norm with a gate, and AdamW with states in 32 or 8 bits, in fp64 -- TEST
INFRASTRUCTURE ONLY (plain numpy)."""
import numpy as np

from . import orf, q8


def group_norm(x, gamma, beta, groups, gate=None, eps=1e-5):
    rows, cols = x.shape
    g = x.reshape(rows, groups, -1)
    n = (g - g.mean(2, keepdims=True)) / np.sqrt(g.var(2, keepdims=True) + eps)
    y = n.reshape(rows, cols) * gamma + beta
    return y if gate is None else y * gate / (1 + np.exp(-gate))


def group_norm_bwd(dy, x, gamma, beta, groups, gate=None, eps=1e-5):
    """(dx, dgate, dgamma, dbeta), each from its definition."""
    rows, cols = x.shape
    g = x.reshape(rows, groups, -1)
    rstd = 1 / np.sqrt(g.var(2, keepdims=True) + eps)
    n = (g - g.mean(2, keepdims=True)) * rstd
    flat = n.reshape(rows, cols)
    d, dgate = dy, None
    if gate is not None:
        s = 1 / (1 + np.exp(-gate))
        dgate = dy * (flat * gamma + beta) * (s + gate * s * (1 - s))
        d = dy * gate * s
    h = (d * gamma).reshape(n.shape)
    dx = rstd * (h - h.mean(2, keepdims=True) - n * (h * n).mean(2, keepdims=True))
    return dx.reshape(rows, cols), dgate, (d * flat).sum(0), d.sum(0)


def moments(g, m, v, betas):
    return betas[0] * m + (1 - betas[0]) * g, betas[1] * v + (1 - betas[1]) * g * g


def weight(p, m, v, t, lr, betas, eps, weight_decay):
    """p after step t, from the moments of that step."""
    rate = (m / (1 - betas[0] ** t)) / (np.sqrt(v / (1 - betas[1] ** t)) + eps)
    return p - lr * (rate + weight_decay * p)


def random16(n, tensor, t, seed):
    """(bits for m, bits for the root of v) of elements 0 .. n - 1."""
    ctr = np.zeros((-(-n // 4), 4), np.uint64)
    ctr[:, 0], ctr[:, 1], ctr[:, 3] = np.arange(ctr.shape[0]), tensor, t
    key = np.broadcast_to(np.array([seed & 0xFFFFFFFF, seed >> 32], np.uint64), (ctr.shape[0], 2))
    words = orf.philox4x32_10(ctr, key).astype(np.int64)
    words = words.reshape(-1)[:n]
    return words & 0xFFFF, words >> 16


def held_at_random(x, bits16, never_zero=False):
    """(values, scale bytes): blocks of 128 under the smallest power of two, each magnitude rounded up where
    its place between two codes and bits16 / 2^16 add up to 1 or more."""
    out, scales = np.zeros(x.size), []
    for b in range(0, x.size, 128):
        part = x[b:b + 128]
        if not np.isfinite(part).all():
            out[b:b + 128] = np.nan
            scales.append(255)
            continue
        e = q8.exponent(np.abs(part).max())
        scales.append(e + 127)
        for i, value in enumerate(part):
            a = abs(value) * 2.0 ** -e
            lo = np.searchsorted(q8.E4M3, a, side="right") - 1
            if lo == 126:
                code = q8.E4M3[126]
            else:
                place = (a - q8.E4M3[lo]) / (q8.E4M3[lo + 1] - q8.E4M3[lo])
                code = q8.E4M3[lo + (place + bits16[b + i] / 65536 >= 1)]
            if never_zero and a > 0:
                code = max(code, q8.E4M3[1])
            out[b + i] = np.copysign(code, value) * 2.0 ** e
    return out, np.array(scales, np.uint8)
