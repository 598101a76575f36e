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
