"""Plain binary64 implementations of the expert-layer operators (numpy on the CPU), written from
their definitions and sharing no code with the library."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24          # half a step of f32, relative
BF16_HALF = 2.0 ** -8   # of bf16
E4M3_HALF = 2.0 ** -4   # of e4m3 normals


def e4m3_values(codes) -> np.ndarray:
    """Codes (uint8 tensor or array) as float64 values."""
    t = codes if isinstance(codes, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(codes))
    return t.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()


def bf16_round(a: np.ndarray) -> np.ndarray:
    """f32 values rounded to bf16 (nearest, ties to even), as f64."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).to(torch.float64).numpy()


def scores(logits: np.ndarray, kind: str) -> np.ndarray:
    """Scores in binary64; a logit that is not finite scores 0 and is no part of a softmax."""
    l = logits.astype(np.float64)
    ok = np.isfinite(l)
    out = np.zeros_like(l)
    with np.errstate(over="ignore"):
        if kind == "sigmoid":
            out[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
            return out
        for t in range(l.shape[0]):
            if ok[t].any():
                e = np.exp(l[t, ok[t]] - l[t, ok[t]].max())
                out[t, ok[t]] = e / e.sum()
    return out


def route(logits, bias, kind, k, groups, kept, best, renorm, scale, mask=None):
    """(topk_idx, topk_weights in f64), token by token, expert by expert."""
    T, E = logits.shape
    p = scores(logits, kind)
    idx = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        able = [e for e in range(E) if np.isfinite(logits[t, e]) and (bias is None or np.isfinite(bias[e]))]
        choice = {e: p[t, e] + (float(bias[e]) if bias is not None else 0.0) for e in able}
        key = {e: (choice[e] if bias is not None else float(logits[t, e])) for e in able}
        if groups > 1:
            size = E // groups
            rating = []
            for g in range(groups):
                of = [e for e in able if e // size == g]
                by = key if best == 1 else choice
                top = sorted((by[e] for e in of), reverse=True)[:best]
                rating.append((-sum(top) if top else np.inf, g))
            stay = {g for _, g in sorted(rating)[:kept]}
            able = [e for e in able if e // size in stay]
        order = sorted(able, key=lambda e: (-key[e], e))[:k]
        s = np.array([p[t, e] for e in order])
        v = s * scale
        if renorm:
            v = v / s.sum() if s.sum() > 0 else np.zeros_like(v)
        idx[t, :len(order)] = order
        w[t, :len(order)] = v
    return idx, w


def route_backward(logits, idx, grad, kind, renorm, scale):
    """(grad_logits, for each logit the size of what is added up in it, and the same of what the
    renormalising subtracts before) in f64."""
    T, E = logits.shape
    p = scores(logits, kind)
    out = np.zeros((T, E))
    size = np.zeros((T, E))
    before = np.zeros((T, E))
    with np.errstate(over="ignore"):
        rest = np.where(np.isfinite(logits), 1.0 / (1.0 + np.exp(np.where(np.isfinite(logits), logits, 0.0).astype(np.float64))), 0.0)
    for t in range(T):
        js = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        s = np.array([p[t, idx[t, j]] for j in js])
        g = np.array([float(grad[t, j]) for j in js])
        if renorm:
            total = s.sum()
            ds = scale * (g - (g * s).sum() / total) / total if total > 0 else np.zeros_like(g)
            whole = scale * (np.abs(g) + (np.abs(g) * s).sum() / total) / total if total > 0 else np.zeros_like(g)
        else:
            ds = scale * g
            whole = np.zeros_like(g)
        d, da, dw = np.zeros(E), np.zeros(E), np.zeros(E)
        for j, v, a in zip(js, ds, whole):
            d[idx[t, j]] += v
            da[idx[t, j]] += abs(v)
            dw[idx[t, j]] += a
        if kind == "sigmoid":
            out[t] = d * p[t] * rest[t]
            size[t] = da * p[t] * rest[t]
            before[t] = dw * p[t] * rest[t]
        else:
            mean = (ds * s).sum()
            out[t] = p[t] * (d - mean)
            size[t] = p[t] * (da + abs(ds * s).sum())
            before[t] = p[t] * (dw + (whole * s).sum())
        out[t][~np.isfinite(logits[t])] = 0.0
    return out, size, before


def product(x, xs, w, ws, rows, num_rows):
    """(sum, sum of magnitudes) [num_rows][N] f64 of the experts' products, NaN where no segment is.
    x, w: E4M3 codes; xs, ws: f32 scales."""
    xv = e4m3_values(x) * np.repeat(xs.astype(np.float64), 128, 1)
    E, N, K = w.shape
    out = np.full((num_rows, N), np.nan)
    mag = np.full((num_rows, N), np.nan)
    at = 0
    for e in range(E):
        n = max(int(rows[e]), 0)
        lo, hi = min(at, num_rows), min(at + n, num_rows)
        if hi > lo:
            wv = e4m3_values(w[e]) * np.repeat(np.repeat(ws[e].astype(np.float64), 128, 0)[:N], 128, 1)
            out[lo:hi] = xv[lo:hi] @ wv.T
            mag[lo:hi] = np.abs(xv[lo:hi]) @ np.abs(wv).T
        at += n
    return out, mag


def product_cut(x, xs, w, ws, rows, num_rows):
    """[num_rows][N]: sum over the groups of eight channels of the scaled largest product in each,
    what the E4M3 matrix instructions' cut is measured in."""
    xv = np.abs(e4m3_values(x))
    E, N, K = w.shape
    out = np.full((num_rows, N), np.nan)
    at = 0
    for e in range(E):
        n = max(int(rows[e]), 0)
        lo, hi = min(at, num_rows), min(at + n, num_rows)
        if hi > lo:
            wv = np.abs(e4m3_values(w[e]))
            acc = np.zeros((hi - lo, N))
            sw = np.repeat(ws[e].astype(np.float64), 128, 0)[:N]
            for g in range(0, K, 8):
                largest = (xv[lo:hi, None, g:g + 8] * wv[None, :, g:g + 8]).max(2)
                acc += largest * xs[lo:hi, g // 128, None].astype(np.float64) * sw[None, :, g // 128]
            out[lo:hi] = acc
        at += n
    return out


def swiglu(y):
    n = y.shape[1] // 2
    g, u = y[:, :n], y[:, n:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def positions(idx, send_slot, slot_pos, E, R, num_recv, num_rows):
    """Grouped row of each (token, slot), -1 without one."""
    T, K = idx.shape
    pos = np.full((T, K), -1, np.int64)
    for t in range(T):
        for j in range(K):
            e = idx[t, j]
            if not 0 <= e < E:
                continue
            s = send_slot[t, e // (E // R)]
            if 0 <= s < num_recv and 0 <= slot_pos[s, j] < num_rows:
                pos[t, j] = slot_pos[s, j]
    return pos


def combine(y, weights, pos):
    """(sum, sum of magnitudes) in f64."""
    T, K = pos.shape
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(K):
        on = pos[:, j] >= 0
        v = weights[on, j].astype(np.float64)[:, None] * y[pos[on, j]]
        out[on] += v
        mag[on] += np.abs(v)
    return out, mag
