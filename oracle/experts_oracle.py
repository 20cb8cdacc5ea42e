"""fp64 oracle of the routed layer around the expert fold: routing, grouping,
MXFP4 quantisation and product, combine.  Plain numpy, written from the
definitions; imports nothing of the package."""
import numpy as np

FLAG_BAD_OFFSETS = 32
FLAG_BAD_EXPERT = 128
FLAG_BAD_ROW = 256
FLAG_NONFINITE = 512

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def route(logits, bias, top_k, score="softmax", num_groups=1, top_groups=1, pair=False,
          renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k], flags), one token at a time."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.full((T, top_k), -1, dtype=np.int64)
    weights = np.zeros((T, top_k))
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    flags = 0
    b_bad = np.isnan(b) | (b == np.inf)
    for t in range(T):
        x = logits[t].copy()
        x_bad = np.isnan(x) | (x == np.inf)
        if T and (x_bad.any() or b_bad.any()):
            flags = FLAG_NONFINITE
        x[x_bad] = -np.inf
        if score == "softmax":
            top = x.max()
            s = np.exp(x - top) if top > -np.inf else np.zeros(E)
            s = s / s.sum() if s.sum() > 0 else s
        else:
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-x))
        open_ = (x > -np.inf) & ~b_bad & (b > -np.inf)
        # without a bias, or with one for all, the order of the scores is that of the
        # logits, also where scores underflow or saturate
        one = bias is None or (np.isfinite(b).all() and (b == b[0]).all())
        # (sums of two scores count where groups are left out by them)
        by_logit = one and not (top_groups < num_groups and pair)
        key = np.where(open_, x if by_logit else s + np.where(open_, b, 0.0), -np.inf)
        if num_groups > 1 and top_groups < num_groups:
            n = E // num_groups
            best = []
            for g in range(num_groups):
                k = np.sort(key[g * n:(g + 1) * n])[::-1]
                k = k[k > -np.inf]
                best.append(-np.inf if not len(k) else k[:2].sum() if pair else k[0])
            order = sorted(range(num_groups), key=lambda g: (-best[g], g))
            for g in order[top_groups:]:
                key[g * n:(g + 1) * n] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf]
        chosen = order[:top_k]
        ids[t, :len(chosen)] = chosen
        if chosen:
            if renormalize:
                # relative to the largest chosen score
                z = x[chosen]
                logs = z if score == "softmax" else -np.logaddexp(0.0, -z)
                w = np.exp(logs - logs.max())
                w = w / w.sum()
            else:
                w = s[chosen]
            weights[t, :len(chosen)] = w * scale
    return ids, weights, flags


def group(ids, token_slot, num_experts):
    """(offsets, row_token, pair_row, row_slot, flags): pairs by expert, in order."""
    T, k = ids.shape
    pair_row = np.full((T, k), -1, dtype=np.int64)
    offsets, row_token = [0], []
    for e in range(num_experts):
        for t in range(T):
            for j in range(k):
                if ids[t, j] == e:
                    pair_row[t, j] = len(row_token)
                    row_token.append(t)
        offsets.append(len(row_token))
    row_token = np.array(row_token, dtype=np.int64)
    row_slot = None if token_slot is None else np.asarray(token_slot)[row_token]
    bad = ((ids < -1) | (ids >= num_experts)).any()
    return np.array(offsets), row_token, pair_row, row_slot, FLAG_BAD_EXPERT if bad else 0


def mx_quantize(v):
    """(codes [rows, F] 0..15, scales [rows, F / 32] biased) of finite or other
    fp64 values, block by block; ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    rows, F = v.shape
    codes = np.zeros((rows, F), dtype=np.int64)
    scales = np.zeros((rows, F // 32), dtype=np.int64)
    mids = (E2M1[1:] + E2M1[:-1]) / 2
    for r in range(rows):
        for c in range(F // 32):
            b = v[r, 32 * c:32 * c + 32]
            if not np.isfinite(b).all():
                scales[r, c] = 255
                continue
            top = np.abs(b).max()
            e = -127 if top == 0 else max(np.frexp(top)[1] - 1 - 2, -127)
            scales[r, c] = e + 127
            a = np.abs(b) / 2.0 ** e
            code = np.zeros(32, dtype=np.int64)
            for i, m in enumerate(mids):
                # past the middle, or on it where the upper code is the even one
                code += (a > m) | ((a == m) & ((i + 1) % 2 == 0))
            codes[r, 32 * c:32 * c + 32] = code + 8 * np.signbit(b)
    return codes, scales


def mx_values(codes, scales):
    """Values of unpacked codes [..., F] and scales [..., F / 32]."""
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (np.asarray(scales, dtype=np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed):
    p = np.asarray(packed).astype(np.int64)
    return np.stack([p & 15, p >> 4], axis=-1).reshape(*p.shape[:-1], -1)


def silu_mul(x):
    """silu(first half) * second half, fp64."""
    F = x.shape[1] // 2
    g, u = x[:, :F], x[:, F:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def mx_linear(x, w):
    """(y, sum of |products|) of values x [rows, K], w [N, K]."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def mx_expert_linear(x, w, offsets):
    """(y, sum of |products|, touched rows, flags) with w [E, N, K]."""
    rows, N = x.shape[0], w.shape[1]
    y, mag = np.zeros((rows, N)), np.zeros((rows, N))
    touched = np.zeros(rows, dtype=bool)
    flags = 0
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < 0 or hi > rows or hi < lo:
            flags |= FLAG_BAD_OFFSETS
            continue
        y[lo:hi], mag[lo:hi] = mx_linear(x[lo:hi], w[e])
        touched[lo:hi] = True
    return y, mag, touched, flags


def combine(y, pair_row, weights, residual):
    """(out, sum of |terms|, flags)."""
    T, k = pair_row.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    mag = np.abs(out)
    flags = 0
    for t in range(T):
        for j in range(k):
            r = int(pair_row[t, j])
            if 0 <= r < y.shape[0]:
                out[t] += float(weights[t, j]) * y[r]
                mag[t] += abs(float(weights[t, j])) * np.abs(y[r])
            elif r != -1:
                flags |= FLAG_BAD_ROW
    return out, mag, flags
