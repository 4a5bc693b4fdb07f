"""Linear attention with a decay for each head in fp64 -- TEST INFRASTRUCTURE ONLY
(plain numpy): the recurrence row by row, and its gradients by the reverse
recurrence.

q [T, Hq, dk], k [T, Hk, dk], v [T, Hk, dv]; sequences are rows
[cu[i], cu[i + 1]); states [n, Hk, dk, dv].
"""
import numpy as np


def forward(q, k, v, log_decay, cu, scale=1.0, state0=None):
    """(o, states behind the last rows); rows outside every sequence are 0."""
    hq, hk, group = q.shape[1], k.shape[1], q.shape[1] // k.shape[1]
    lam = np.exp(np.minimum(log_decay, 0.0))[:, None, None]
    o = np.zeros((q.shape[0], hq, v.shape[2]))
    ends = np.zeros((len(cu) - 1, hk, k.shape[2], v.shape[2]))
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        s = np.zeros(ends.shape[1:]) if state0 is None else state0[i].astype(np.float64)
        for t in range(a, b):
            s = lam * s + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * (q[t].reshape(hk, group, -1) @ s).reshape(hq, -1)
        ends[i] = s
    return o, ends


def backward(q, k, v, log_decay, cu, do, scale=1.0, state0=None, g_in=None):
    """(dq, dk, dv, gradient of state0) of sum(do o) + sum(g_in ends)."""
    hq, hk, group = q.shape[1], k.shape[1], q.shape[1] // k.shape[1]
    lam = np.exp(np.minimum(log_decay, 0.0))[:, None, None]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    g0 = np.zeros((len(cu) - 1, hk, k.shape[2], v.shape[2]))
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        s = np.zeros(g0.shape[1:]) if state0 is None else state0[i].astype(np.float64)
        for t in range(a, b):
            s = lam * s + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (do[t].reshape(hk, group, -1) @ s.transpose(0, 2, 1)).reshape(hq, -1)
        g = np.zeros(s.shape) if g_in is None else g_in[i].astype(np.float64)
        for t in range(b - 1, a - 1, -1):
            # the state behind row t is read by row t
            g = g + scale * q[t].reshape(hk, group, -1).transpose(0, 2, 1) @ do[t].reshape(hk, group, -1)
            dk[t] = np.einsum("hij,hj->hi", g, v[t])
            dv[t] = np.einsum("hij,hi->hj", g, k[t])
            g = lam * g
        g0[i] = g
    return dq, dk, dv, g0
