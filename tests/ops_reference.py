"""Plain 64-bit forms of the routing rules, their gradients and the NVFP4 operands, for the tests: loops and numpy, apart from
the library's code."""
import numpy as np


def route(logits, k, bias=None, score="sigmoid", groups=1, top_groups=1, group_score="top2", renormalize=True, scale=1.0):
    """ids, weights and scores of logits [T][E] in fp64, expert by expert."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids, w, s = np.zeros((T, k), np.int32), np.zeros((T, k)), np.zeros((T, E))
    per = E // groups
    for t in range(T):
        served = [e for e in range(E) if l[t, e] > -np.inf]  # (false for NaN)
        x = np.minimum(l[t], 3.402823466e38)
        if served:
            if score == "sigmoid":
                with np.errstate(over="ignore"):
                    s[t, served] = 1.0 / (1.0 + np.exp(-x[served]))
            else:
                p = np.exp(x[served] - x[served].max())
                s[t, served] = p / p.sum()
        v = {e: (l[t, e] if bias is None else s[t, e] + float(bias[e])) for e in served}
        best = []
        for g in range(groups):
            vals = [(s[t, e] if bias is None and group_score == "top2" else v[e]) for e in served if e // per == g]
            vals.sort(reverse=True)
            best.append(-np.inf if not vals else vals[0] if group_score == "max" else sum(vals[:2]))
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        cand = [e for e in range(E) if e // per in kept]
        cand.sort(key=lambda e: (0, -v[e], e) if e in v else (1, 0.0, e))
        ids[t] = sorted(cand[:k])
        u = s[t, ids[t]]
        if renormalize:
            # in ratios, so that sums of scores below fp64's range keep them
            pl = x[ids[t]]
            live = np.array([e in v for e in ids[t]])
            if live.any():
                m = pl[live].max()
                if score == "softmax":
                    u = np.where(live, np.exp(np.where(live, pl, m) - m), 0.0)
                else:
                    m = min(m, 0.0)
                    q = np.where(live, pl, 0.0)
                    with np.errstate(over="ignore"):
                        u = np.where(live, np.where(q > 0, 1.0, np.exp(np.minimum(q, 0) - m)) / (1.0 + np.exp(-np.abs(q))), 0.0)
                        u = np.where(live & (q > 0), 1.0 / (1.0 + np.exp(-q)), u)
                u = u / u.sum()
        w[t] = scale * u
    return ids, w, s


def route_backward(logits, ids, dw, score="sigmoid", renormalize=True, scale=1.0, dscores=None):
    """dlogits in fp64 and, element by element, the sum of the magnitudes of the terms it is made of."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    dl, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        served = l[t] > -np.inf
        x = np.minimum(l[t], 3.402823466e38)
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s[served] = 1.0 / (1.0 + np.exp(-x[served]))
            elif served.any():
                p = np.exp(x[served] - x[served].max())
                s[served] = p / p.sum()
        ds, ms = np.zeros(E), np.zeros(E)
        u = s[ids[t]]
        S = u.sum()
        d = np.asarray(dw[t], np.float64) * scale
        if renormalize:
            if S > 0:
                ds[ids[t]] = d / S - (d * u).sum() / S ** 2
                ms[ids[t]] = np.abs(d) / S + np.abs(d * u).sum() / S ** 2
        else:
            ds[ids[t]], ms[ids[t]] = d, np.abs(d)
        if dscores is not None:
            ds = ds + dscores[t]
            ms = ms + np.abs(dscores[t])
        if score == "sigmoid":
            f = np.zeros(E)
            with np.errstate(over="ignore"):
                f[served] = s[served] / (1.0 + np.exp(x[served]))
            dl[t], mag[t] = ds * f, ms * f
        else:
            dl[t] = s * (ds - (ds * s).sum())
            mag[t] = s * (ms + (ms * s).sum())
    return dl, mag


def operand_bytes(codes, scales):
    """Codes [rows][K] (0..15) and scale bytes [rows][K/16] (K a multiple of 256) -> dicts of byte offset -> byte in the tensor-core
    layout, as two arrays with -1 where nothing was placed."""
    rows, K = codes.shape
    assert K % 256 == 0
    pr = -(-rows // 128) * 128
    q = np.full(pr * K // 2, -1, np.int64)
    s = np.full(pr * K // 16, -1, np.int64)
    for r in range(rows):
        for b in range(K // 2):
            tile, j = (r // 128) * (K // 256) + b // 128, (b % 128) // 16
            q[tile * 16384 + (r % 128) * 128 + ((j ^ (r % 8)) * 16) + b % 16] = codes[r, 2 * b] | (codes[r, 2 * b + 1] << 4)
        for c in range(K // 16):
            atom = (r // 128) * (K // 64) + c // 4
            s[atom * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + c % 4] = scales[r, c]
    return q, s
