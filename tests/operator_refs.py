"""Plain 64-bit references (numpy, one token or expert at a time) of the
router, of the gradients of the expert sort and of the combine, and of the
experts' products.  They share no code with the kernels."""
import numpy as np


def bf16(a) -> np.ndarray:
    """Nearest-even bf16 of a 64-bit array, as float64 (through the bits of
    the exact fp32 neighbours; the inputs here are far from fp32's limits)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(
        torch.bfloat16).double().numpy()


# -------------------------------------------------------------------- router

def clean_logits(logits) -> np.ndarray:
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l[l == np.inf] = np.finfo(np.float32).max
    return l


def scores(l, scoring) -> np.ndarray:
    """Scores of one cleaned row; 0 where the logit is -inf."""
    live = l > -np.inf
    s = np.zeros_like(l)
    if not live.any():
        return s
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
    else:
        x = np.exp(l[live] - l[live].max())
        s[live] = x / x.sum()
    return s


def route(logits, K, scoring="softmax", bias=None, groups=1, top_groups=1,
          renorm=True, scale=1.0):
    L = clean_logits(logits)
    T, E = L.shape
    ids = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    for t in range(T):
        l = L[t]
        s = scores(l, scoring)
        if scoring == "softmax" and bias is None and groups == 1:
            c = l.copy()
        else:
            c = s + (0 if bias is None else np.asarray(bias, np.float64))
        c = np.where((l > -np.inf) & (c > -np.inf), c, -np.inf)
        allowed = c > -np.inf
        if groups > 1:
            gs = E // groups
            value = np.full(groups, -np.inf)
            for g in range(groups):
                two = sorted((v for v in c[g * gs:(g + 1) * gs]
                              if v > -np.inf), reverse=True)[:2]
                if two:
                    value[g] = sum(two)
            keep = sorted(range(groups), key=lambda g: (-value[g], g))
            keep = [g for g in keep[:top_groups] if value[g] > -np.inf]
            allowed &= np.isin(np.arange(E) // gs, keep)
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e))
                 if allowed[e]][:K]
        ids[t, :len(order)] = order
        p = s[order]
        if renorm:
            p = p / p.sum() if p.sum() > 0 else np.zeros_like(p)
        w[t, :len(order)] = scale * p
    return ids, w


def route_backward(g, logits, ids, scoring, renorm, scale):
    """From d(w_j)/d(l_e), written out."""
    L = clean_logits(logits)
    T, E = L.shape
    out = np.zeros((T, E))
    for t in range(T):
        s = scores(L[t], scoring)
        J = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not J:
            continue
        e = ids[t, J]
        gj = np.asarray(g, np.float64)[t, J]
        p = s[e]
        ds = np.zeros(len(J))  # d loss / d s of each chosen
        if renorm:
            S = p.sum()
            if S > 0:
                ds = scale / S * (gj - (gj * p).sum() / S)
        else:
            ds = scale * gj
        full = np.zeros(E)
        for k, ek in enumerate(e):
            full[ek] += ds[k]
        if scoring == "sigmoid":
            out[t] = full * s * (1 - s)
        else:
            out[t] = s * (full - (full * s).sum())
    return out


# ----------------------------------------------------------------- gradients

def scatter_rows_backward(rows, src2dst):
    rows = np.asarray(rows, np.float64)
    out = np.zeros((src2dst.shape[0], rows.shape[1]))
    for t in range(src2dst.shape[0]):
        for d in src2dst[t]:
            if 0 <= d < rows.shape[0]:
                out[t] += rows[d]
    return out


def combine_backward(g, y, src2dst, w, grad_y):
    """(grad_y, grad_weights); rows of grad_y that are no destination stay."""
    g, y, w = (np.asarray(a, np.float64) for a in (g, y, w))
    gy = np.asarray(grad_y, np.float64).copy()
    gw = np.zeros(w.shape)
    for t in range(src2dst.shape[0]):
        for j, d in enumerate(src2dst[t]):
            if 0 <= d < y.shape[0]:
                gy[d] = w[t, j] * g[t]
                gw[t, j] = (g[t] * y[d]).sum()
    return gy, gw


# --------------------------------------------------------- experts' products

def e4m3_values() -> np.ndarray:
    """The 256 OCP e4m3fn values (0x7F and 0xFF are NaN)."""
    v = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if (b & 0x7F) == 0x7F:
            x = np.nan
        v[b] = -x if b >> 7 else x
    return v


E4M3 = e4m3_values()


def dequant_rows(q, scales, group):
    two = 2.0 ** (scales.astype(np.float64) - 127)
    return E4M3[q] * np.repeat(two, group, 1)[:, :q.shape[1]]


def dequant_weight(w, ws):
    two = 2.0 ** (ws.astype(np.float64) - 127)
    two = np.repeat(np.repeat(two, 128, 0), 128, 1)
    return E4M3[w] * two[:w.shape[0], :w.shape[1]]


def live_rows(offsets, counts, rows, e):
    """First row and number of live rows of expert e."""
    first = int(offsets[e])
    n = min(int(counts[e]), int(offsets[e + 1]) - first, rows - first)
    return first, max(n, 0) if first >= 0 else 0


def expert_matmul(q, scales, group, w, ws, offsets, counts, bias, act,
                  residual, cols):
    """fp64 rows [num_rows, cols] (NaN where not live) and how far the matrix
    unit's evaluation may be off, carried through the activation.

    The unit aligns the 32 products that a lane's registers hold to the
    largest one's exponent and drops what lies below 2^-13 of it (measured:
    2^13 below is kept, 2^14 is not), so each product is off by less than
    2^-13 of the largest, and a group by 32 * 2^-13 = 2^-8 of it.  A lane's
    registers hold two runs of 16 channels; whichever they are, the group's
    largest is at most the sum of both runs' largest, so all groups together
    are off by at most 2^-8 of the sum over runs of max|x| max|w|.  Each of
    the H additions after that is off by at most one fp32 step, 2^-23 of the
    sum of absolute products."""
    rows, H = q.shape
    out = np.full((rows, cols), np.nan)
    err = np.zeros((rows, cols))
    for e in range(w.shape[0]):
        a, n = live_rows(offsets, counts, rows, e)
        if n == 0:
            continue
        x = dequant_rows(q[a:a + n], scales[a:a + n], group)
        m = dequant_weight(w[e], ws[e])
        y = x @ m.T
        size = np.abs(x) @ np.abs(m).T
        if bias is not None:
            y = y + bias[e].astype(np.float64)
            size = size + np.abs(bias[e])
        run = [np.abs(v).reshape(v.shape[0], -1, 16).max(-1) for v in (x, m)]
        d = (H + 1) * 2.0 ** -23 * size + 2.0 ** -8 * (run[0] @ run[1].T)
        if act != "none":
            # |silu'| < 1.1.  exp(-x) of a product -x log2(e) rounded to fp32
            # (half a step: 2^-24 |x| log2(e), times ln(2) in the power) is
            # off by a factor 1 + |x| 2^-24, and so is the quotient at most;
            # the power, sum, quotient and product add up to 2^-21
            gate = y[:, :cols] if act == "silu_mul" else y
            dg = d[:, :cols] if act == "silu_mul" else d
            with np.errstate(over="ignore"):
                s = gate / (1 + np.exp(-gate))
            ds = 1.1 * dg + (2.0 ** -21 + 2.0 ** -24 * np.abs(gate)) * \
                np.abs(s)
            if act == "silu_mul":
                u, du = y[:, cols:], d[:, cols:]
                y, d = s * u, ds * np.abs(u) + (np.abs(s) + ds) * du
                d += 2.0 ** -23 * np.abs(y)
            else:
                y, d = s, ds
        if residual is not None:
            y = y + residual[a:a + n]
            d = d + 2.0 ** -23 * np.abs(y)
        out[a:a + n], err[a:a + n] = y, d
    return out, err


def check_quantized(y, err, q, scales, group, live):
    """Payload and scale bytes stand for y: the exponent is that of the
    group's largest value within its error, the payload within half a step
    (2^-4 of the value, 2^-10 below the smallest normal payload)."""
    y, err, q, scales = y[live], err[live], q[live], scales[live]
    n = y.shape[0]
    amax = np.abs(y).reshape(n, -1, group)
    at = amax.max(-1)
    slack = err.reshape(n, -1, group).max(-1)

    def exponent(v):
        with np.errstate(divide="ignore"):
            m, e = np.frexp(v)
        e = np.where(m > 0.875, e - 8, e - 9)
        return np.where(v > 0, np.clip(e, -127, 127), -127)

    e = scales.astype(np.int64) - 127
    lo = exponent(np.maximum(at - slack, 0))
    hi = exponent(at + slack)
    assert ((e >= lo) & (e <= hi)).all(), "scale exponents"
    two = np.repeat(2.0 ** e, group, 1)
    back = E4M3[q] * two
    off = np.abs(back - y)
    assert (off <= 2.0 ** -4 * 1.0001 * (np.abs(y) + err) + 2.0 ** -10 * two
            + err).all(), "payload"
