"""The balance loss in 64 bits for whole batches at once, and bounds of its
fp32 sums that follow the kernels' own structure, so that a token lost or taken
twice shows in the loss, in the shares and in the penalty.

A row is held by L lanes, a block of 512 threads so has 512 / L rows at a time.
One launch (up to 8 rows a lane) sums a sequence in one block; of two launches
the first has up to 512 blocks of neighbouring tokens, whose sums the second
joins in 64 bits.  A value so goes through one addition per row of a lane, 4 at
most over the wavefront's lanes and 8 over the block's wavefronts."""
import numpy as np

import mx_refs as mx
import operator_refs as ref

EPS = mx.EPS


def row_lanes(E):
    return 4 if E <= 16 else 8 if E <= 32 else 16 if E <= 256 else \
        32 if E <= 512 else 64


def one_launch(T, E):
    return T <= 8 * 512 // row_lanes(E)


def additions(T, E):
    """In fp32, of a value that enters a sum."""
    slots = 512 // row_lanes(E)
    if one_launch(T, E):
        return 8 + 12
    blocks = min(512, -(-T // slots))
    return -(-(-(-T // blocks)) // slots) + 12


def shares(logits, scoring):
    """Shares, log-sum-exps and how far exponents reach, of all rows."""
    L = ref.clean_logits(logits)
    live = L > -np.inf
    any_ = live.any(1)
    m = np.where(any_, L.max(1), 0.0)[:, None]
    x = np.exp(np.where(live, L - m, -np.inf))
    total = x.sum(1, keepdims=True)
    lse = np.where(any_, m[:, 0] + np.log(np.where(any_, total[:, 0], 1.0)),
                   0.0)
    v = np.where(live, L, 0.0)
    X = (m - np.where(live, L, m)).max(1)
    if scoring == "sigmoid":
        tail = np.log1p(np.exp(-np.abs(v)))
        ls = np.where(live, np.where(v > 0, -tail, v - tail), -np.inf)
        top = np.where(any_, ls.max(1), 0.0)[:, None]
        x = np.exp(ls - top)
        total = x.sum(1, keepdims=True)
        X = X + np.abs(v).max(1)
    p = x / np.where(any_[:, None], total, 1.0)
    return p, lse, np.minimum(X, 104.0)


def forward(logits, ids, scoring, offsets=None, lens=None, S=1, drop=None):
    """loss, z, counts, probs, and bounds of what fp32 makes of loss, z and
    probs.  ``drop``: a token that the sums leave out, for the bounds' own
    test."""
    T, E = logits.shape
    p, lse, X = shares(logits, scoring)
    adds = additions(T, E) * EPS
    loss, z, lerr, zerr = (np.zeros(S) for _ in range(4))
    counts = np.zeros((S, E), np.int64)
    probs, perr = np.zeros((S, E)), np.zeros((S, E))
    for s, (a, b) in enumerate(mx.sequences(T, offsets, lens, S)):
        if b <= a:
            continue
        t = np.array([i for i in range(a, b) if i != drop])
        n = b - a
        rel = mx.share_error(X[t], scoring) + adds
        probs[s] = p[t].sum(0) / n
        perr[s] = (p[t] * rel[:, None]).sum(0) / n + EPS * probs[s]
        z[s] = (lse[t] ** 2).sum() / n
        # as mx.balance: the sum's relative error, the logarithm's two steps
        d = ((1.3 * X[t] + 68) + 2 * np.abs(lse[t])) * EPS
        zerr[s] = (2 * np.abs(lse[t]) * d + d * d +
                   lse[t] ** 2 * (adds + EPS)).sum() / n + EPS * z[s]
        k = np.asarray(ids)[a:b].reshape(-1)
        counts[s] = np.bincount(k[(k >= 0) & (k < E)], minlength=E)
        if counts[s].sum():
            f = E * counts[s] / counts[s].sum()
            loss[s] = (f * probs[s]).sum()
            lerr[s] = (f * perr[s]).sum() + EPS * loss[s]
    # fp32's smallest normal value: exponentials below it are 0
    return loss, z, counts, probs, lerr + 1e-36, zerr, perr + 1e-37
