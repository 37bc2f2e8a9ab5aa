"""Plain float64 restatement of the training operators, for tests only (numpy, loops over
tokens and experts; shares no code with the CUDA path)."""
from __future__ import annotations

import numpy as np

SOFTMAX_ALL = (0,)
SOFTMAX_CHOSEN = (1, 4)
SIGMOID_EACH = (3,)
SIGMOID_SUM = (2, 5, 6, 16)


# ------------------------------------------------------------------ rows by expert and back

def sort_slots(ids: np.ndarray, E: int):
    """(inv [T, k], offsets [E + 1]): slots in the order (expert, flat index), those whose id is
    not an expert last and held as -1 - place."""
    flat = ids.reshape(-1)
    inv = np.empty(flat.size, np.int64)
    offsets = np.zeros(E + 1, np.int64)
    at = 0
    for e in range(E):
        offsets[e] = at
        for f in np.flatnonzero(flat == e):
            inv[f] = at
            at += 1
    offsets[E] = at
    for f in np.flatnonzero((flat < 0) | (flat >= E)):
        inv[f] = -1 - at
        at += 1
    return inv.reshape(ids.shape), offsets


def dispatch_rows(x: np.ndarray, inv: np.ndarray) -> np.ndarray:
    T, k = inv.shape
    out = np.zeros((T * k, x.shape[1]), x.dtype)
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                out[inv[t, j]] = x[t]
    return out


def combine(rows, inv, scales=None):
    """(y, sum of the magnitudes of its terms)."""
    T, k = inv.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                term = (1.0 if scales is None else scales[t, j]) * rows[inv[t, j]]
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def combine_backward(dy, rows, inv, scales=None):
    """(drows, dscales, the magnitudes summed in dscales)."""
    T, k = inv.shape
    drows = np.zeros(rows.shape)
    ds = np.zeros((T, k))
    mag = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = inv[t, j]
            if r >= 0:
                drows[r] = (1.0 if scales is None else scales[t, j]) * dy[t]
                ds[t, j] = float(dy[t] @ rows[r])
                mag[t, j] = float(np.abs(dy[t]) @ np.abs(rows[r]))
    return drows, ds, mag


# ----------------------------------------------------------------- SwiGLU and its checkpoint

# The non-negative e4m3 values in the order of their codes: exponent field 0 is m 2^-9, field f
# is (8 + m) 2^(f - 10); code 127 is NaN.
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (f - 10) for f in range(1, 16) for m in range(8)][:-1])


def e4m3_code(v: np.ndarray) -> np.ndarray:
    """Codes of values no larger than 448 in magnitude: the nearest, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 0, len(E4M3) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == 0, 0, code)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def scale_bytes(v: np.ndarray) -> np.ndarray:
    """Scale byte of each block of 32 of v [R, C]; 255 for a block that is not finite."""
    R, C = v.shape
    out = np.zeros((R, -(-C // 32)), np.uint8)
    for b in range(out.shape[1]):
        a = np.abs(v[:, 32 * b:32 * b + 32]).max(axis=1)
        for r in range(R):
            if not np.isfinite(a[r]):
                out[r, b] = 255
                continue
            e = -127
            while a[r] > 448.0 * 2.0 ** e:
                e += 1
            out[r, b] = e + 127
    return out


def scale_of(byte: np.ndarray) -> np.ndarray:
    return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))


def quantise(gu: np.ndarray):
    """(q, q_scales) of gu [R, 2I]."""
    I = gu.shape[1] // 2
    halves = [gu[:, :I], gu[:, I:]]
    qs = [scale_bytes(h) for h in halves]
    q = [e4m3_code(h / np.repeat(scale_of(s), 32, axis=1)[:, :I]) for h, s in zip(halves, qs)]
    return np.concatenate(q, 1), np.concatenate(qs, 1)


def kept(q: np.ndarray, qs: np.ndarray) -> np.ndarray:
    """The values a checkpoint stands for."""
    I, nb = q.shape[1] // 2, qs.shape[1] // 2
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    out = table[q]
    return np.concatenate([out[:, :I] * np.repeat(scale_of(qs[:, :nb]), 32, axis=1)[:, :I],
                           out[:, I:] * np.repeat(scale_of(qs[:, nb:]), 32, axis=1)[:, :I]], 1)


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-np.asarray(v, np.float64)))


def swiglu(gu):
    I = gu.shape[1] // 2
    return gu[:, :I] * sigmoid(gu[:, :I]) * gu[:, I:]


def swiglu_backward(dh, gu):
    I = dh.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    s = sigmoid(g)
    return np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)


# ------------------------------------------------------------------------ experts' products

def experts_matmul(x, w, offsets):
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        y[offsets[e]:offsets[e + 1]] = x[offsets[e]:offsets[e + 1]] @ w[e].T
    return y


def experts_matmul_dx(dy, w, offsets):
    dx = np.zeros((dy.shape[0], w.shape[2]))
    for e in range(w.shape[0]):
        dx[offsets[e]:offsets[e + 1]] = dy[offsets[e]:offsets[e + 1]] @ w[e]
    return dx


def experts_matmul_dw(dy, x, offsets):
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    for e in range(E):
        dw[e] = dy[offsets[e]:offsets[e + 1]].T @ x[offsets[e]:offsets[e + 1]]
    return dw


# ------------------------------------------------------------------------------ the router

def route_weights(logits, ids, method, rsf=1.0):
    """The weights of the chosen experts ids [T, k] (slots with an id outside [0, E) get 0),
    non-finite logits counting as -inf."""
    T, k = ids.shape
    E = logits.shape[1]
    l = np.where(np.isfinite(logits), logits, -np.inf).astype(np.float64)
    s = np.zeros((T, k))
    for t in range(T):
        live = [j for j in range(k) if 0 <= ids[t, j] < E and l[t, ids[t, j]] > -np.inf]
        if not live:
            continue
        lc = np.array([l[t, ids[t, j]] for j in live])
        if method in SOFTMAX_ALL:
            m = l[t].max()
            w = np.exp(lc - m) / np.exp(l[t] - m).sum()
        elif method in SOFTMAX_CHOSEN:
            w = np.exp(lc - lc.max())
            w = w / w.sum()
        elif method in SIGMOID_EACH:
            w = sigmoid(lc)
        else:
            a = sigmoid(lc)
            w = a / (a.sum() + (1e-20 if method == 2 else 0.0))
            if method in (2, 16):
                w = w * rsf
        for j, v in zip(live, w):
            s[t, j] = v
    return s


def route_backward(logits, ids, ds, method, rsf=1.0):
    """(dlogits, the magnitudes that meet in each): the Jacobian of route_weights, slot by slot."""
    T, k = ids.shape
    E = logits.shape[1]
    l = np.where(np.isfinite(logits), logits, -np.inf).astype(np.float64)
    dl = np.zeros((T, E))
    mag = np.zeros((T, E))
    for t in range(T):
        live = [j for j in range(k) if 0 <= ids[t, j] < E and l[t, ids[t, j]] > -np.inf]
        if not live:
            continue
        at = np.array([ids[t, j] for j in live])
        d = np.array([ds[t, j] for j in live], np.float64)
        lc = l[t, at]
        if method in SOFTMAX_ALL:
            m = l[t].max()
            p = np.exp(l[t] - m) / np.exp(l[t] - m).sum()
            jac = -np.outer(p[at], p)
            jac[np.arange(len(at)), at] += p[at]
            terms = d[:, None] * jac
            big = np.abs(d)[:, None] * np.outer(p[at], p)
            big[np.arange(len(at)), at] += np.abs(d) * p[at]
            dl[t] = terms.sum(0)
            mag[t] = big.sum(0)
            continue
        if method in SOFTMAX_CHOSEN:
            a = np.exp(lc - lc.max())
            slope, total, c = a, a.sum(), 1.0
        elif method in SIGMOID_EACH:
            a = sigmoid(lc)
            slope = a * sigmoid(-lc)
            for i, e in enumerate(at):
                dl[t, e] += d[i] * slope[i]
                mag[t, e] += abs(d[i] * slope[i])
            continue
        else:
            a = sigmoid(lc)
            slope = a * sigmoid(-lc)
            total = a.sum() + (1e-20 if method == 2 else 0.0)
            c = rsf if method in (2, 16) else 1.0
        for j, e in enumerate(at):
            for i in range(len(at)):
                own = 1.0 / total if i == j else 0.0
                dl[t, e] += d[i] * c * slope[j] * (own - a[i] / total ** 2)
                mag[t, e] += abs(d[i] * c * slope[j]) * (own + a[i] / total ** 2)
    return dl, mag
