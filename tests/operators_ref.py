"""Plain fp64 statements of the handle-free expert-layer operators (numpy, CPU),
written from their formulas, for tests/test_operators*.py.  Nothing here uses the
library."""
import numpy as np

BLK = 128
E4M3_MAX = 448.0
# The 127 finite non-negative E4M3 values in code order (code 0x7F is NaN).
GRID = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def code_values(codes):
    """Values of E4M3 codes (uint8)."""
    c = np.asarray(codes)
    v = np.append(GRID, np.nan)[c & 0x7F]
    return np.where(c & 0x80, -v, v)


def round_e4m3(q):
    """Codes of the nearest E4M3 values, ties to the even code, saturating."""
    q = np.asarray(q, dtype=np.float64)
    mag = np.abs(q)
    mid = (GRID[1:] + GRID[:-1]) / 2
    lo, hi = np.searchsorted(mid, mag, side="left"), np.searchsorted(mid, mag, side="right")
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)
    return code | np.where(np.signbit(q), 0x80, 0).astype(np.uint8)


def scale_of(amax):
    """fp32 scale of a block with this maximum magnitude."""
    s = np.maximum((np.asarray(amax, np.float64) / E4M3_MAX).astype(np.float32), np.float32(2.0 ** -126))
    return np.where(np.asarray(amax) > 0, s, np.float32(1)).astype(np.float32)


def quantize_rows(x):
    """x [R, K] fp64 -> codes [R, K], scales fp32 [ceil(K / 128), R]."""
    R, K = x.shape
    nb = -(-K // BLK)
    codes = np.zeros((R, K), np.uint8)
    scales = np.ones((nb, R), np.float32)
    for b in range(nb):
        v = x[:, b * BLK:(b + 1) * BLK]
        bad = ~np.isfinite(v).all(axis=1)
        s = scale_of(np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0)).max(axis=1)))
        c = round_e4m3(np.where(bad[:, None], 0.0, v) / s.astype(np.float64)[:, None])
        codes[:, b * BLK:(b + 1) * BLK] = np.where(bad[:, None], 0, c)
        scales[b] = np.where(bad, np.float32(np.nan), s)
    return codes, scales


def quantize_weights(w):
    """w [G, N, K] fp64 -> codes, scales fp32 [G, ceil(N/128), ceil(K/128)]."""
    G, N, K = w.shape
    codes = np.zeros(w.shape, np.uint8)
    scales = np.ones((G, -(-N // BLK), -(-K // BLK)), np.float32)
    for g in range(G):
        for i in range(scales.shape[1]):
            for j in range(scales.shape[2]):
                sl = (g, slice(i * BLK, (i + 1) * BLK), slice(j * BLK, (j + 1) * BLK))
                s = scale_of(np.abs(w[sl]).max())
                scales[g, i, j] = s
                codes[sl] = round_e4m3(w[sl] / np.float64(s))
    return codes, scales


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def scores_of(l, kind):
    """Scores of one row of logits; masked experts (NaN, -inf) score 0."""
    ok = l > -np.inf
    if kind == "sigmoid":
        return np.where(ok, sigmoid(np.where(ok, l, 0.0)), 0.0), ok
    if not ok.any():
        return np.zeros_like(l), ok
    e = np.where(ok, np.exp(np.where(ok, l, 0) - l[ok].max()), 0.0)
    return e / e.sum(), ok


def route(logits, k, scores="softmax", bias=None, n_groups=1, topk_groups=1, group_top=2, renormalize=False,
          routed_scale=1.0):
    T, E = logits.shape
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    n = E // n_groups
    for t in range(T):
        l = np.asarray(logits[t], np.float64)
        s, ok = scores_of(l, scores)
        key = s.copy() if bias is None else s + np.asarray(bias, np.float64)
        order_key = l.copy() if bias is None else key.copy()   # without a bias scores grow with the logits
        order_key[~ok] = -np.inf
        order_key[~(order_key > -np.inf)] = -np.inf
        if topk_groups < n_groups:
            sc = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                members = [e for e in range(g * n, (g + 1) * n) if order_key[e] > -np.inf]
                top = sorted((key[e] for e in members), reverse=True)[:group_top]
                if top:
                    sc[g] = order_key[members].max() if (group_top == 1 and bias is None) else sum(top)
            kept = sorted(range(n_groups), key=lambda g: (-sc[g], g))[:topk_groups]
            for g in range(n_groups):
                if g not in kept:
                    order_key[g * n:(g + 1) * n] = -np.inf
        best = [e for e in sorted(range(E), key=lambda e: (-order_key[e], e)) if order_key[e] > -np.inf][:k]
        if not best:
            continue
        idx[t, :len(best)] = best
        v = s[best]
        if renormalize:
            lb = l[best]
            if v.sum() < 1e-200:
                v = np.exp(lb - lb.max())
            v = v / v.sum()
        w[t, :len(best)] = v * routed_scale
    return idx, w


def weights_of(l, idx, scores, renormalize, routed_scale):
    """Weights of one row as a function of its logits, the choice held fixed."""
    s, _ = scores_of(l, scores)
    v = np.array([s[e] if 0 <= e < len(l) else 0.0 for e in idx])
    if renormalize and v.sum() > 0:
        v = v / v.sum()
    return v * routed_scale


def route_backward(logits, idx, dw, scores="softmax", renormalize=False, routed_scale=1.0):
    T, E = logits.shape
    dl = np.zeros((T, E))
    for t in range(T):
        l = np.asarray(logits[t], np.float64)
        s, ok = scores_of(l, scores)
        live = [(j, e) for j, e in enumerate(idx[t]) if 0 <= e < E and ok[e]]
        ds = np.zeros(E)
        if renormalize:
            S = sum(s[e] for _, e in live)
            if S == 0:
                continue
            mean = sum(dw[t, j] * s[e] for j, e in live) / S
            for j, e in live:
                ds[e] += (dw[t, j] - mean) / S
        else:
            for j, e in live:
                ds[e] += dw[t, j]
        ds *= routed_scale
        dl[t] = ds * s * (1 - s) if scores == "sigmoid" else s * (ds - (ds * s).sum())
    return dl


def group_rows(idx, E):
    T, k = idx.shape
    flat = idx.reshape(-1)
    rows = [i for e in range(E) for i in np.nonzero(flat == e)[0]]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    tok = np.full(T * k, -1, np.int32)
    slot = np.full(T * k, -1, np.int32)
    tok[:len(rows)] = [i // k for i in rows]
    slot[rows] = np.arange(len(rows))
    return offsets, tok, slot.reshape(T, k)


def glu(gu, act="swiglu", cg=np.inf, cu=np.inf, bg=4.0, bu=25.0):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    if act == "situ":
        return bg * np.tanh(g / bg) * sigmoid(g) * bu * np.tanh(u / bu)
    g = np.minimum(g, cg)
    return g * sigmoid(g) * np.clip(u, -cu, cu)


def glu_backward(gu, dh, act="swiglu", cg=np.inf, cu=np.inf, bg=4.0, bu=25.0):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    if act == "situ":
        tg, tu, sg = np.tanh(g / bg), np.tanh(u / bu), sigmoid(g)
        a, b = bg * tg * sg, bu * tu
        da, db = (1 - tg ** 2) * sg + bg * tg * sg * (1 - sg), 1 - tu ** 2
    else:
        gc, sg = np.minimum(g, cg), sigmoid(np.minimum(g, cg))
        a, b = gc * sg, np.clip(u, -cu, cu)
        da = np.where(g <= cg, sg * (1 + gc * (1 - sg)), 0.0)
        db = np.where(np.abs(u) <= cu, 1.0, 0.0)
    return np.concatenate([dh * b * da, dh * a * db], axis=1)


def wide_rows(codes, scales):
    K = codes.shape[-1]
    return code_values(codes) * np.repeat(scales.T.astype(np.float64), BLK, axis=1)[:, :K]


def wide_weights(codes, scales):
    N, K = codes.shape[-2:]
    s = np.repeat(np.repeat(scales.astype(np.float64), BLK, axis=-2)[..., :N, :], BLK, axis=-1)[..., :K]
    return code_values(codes) * s


def matmul(a, sa, w, sw, offsets=None, transposed=False):
    """(product, sum of the magnitudes of its terms); rows outside the groups are NaN."""
    x, m = wide_rows(a, sa), wide_weights(w, sw)
    offsets = [0, x.shape[0]] if offsets is None else offsets
    width = m.shape[2] if transposed else m.shape[1]
    out, mag = np.full((x.shape[0], width), np.nan), np.zeros((x.shape[0], width))
    for g in range(m.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        y = m[g] if transposed else m[g].T
        out[r] = x[r] @ y
        mag[r] = np.abs(x[r]) @ np.abs(y)
    return out, mag


def combine(y, row_of_slot, w=None, addend=None):
    T, k = row_of_slot.shape
    out = np.zeros((T, y.shape[1])) if addend is None else np.asarray(addend, np.float64).copy()
    for t in range(T):
        for j in range(k):
            r = row_of_slot[t, j]
            if 0 <= r < y.shape[0]:
                out[t] += (1.0 if w is None else float(w[t, j])) * y[r]
    return out
