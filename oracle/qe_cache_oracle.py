"""Plain definitions of the rotary positions, the paged cache, the attention over it and the verification of drafts
(numpy; test infrastructure only, sharing no code with the HIP path)."""

import numpy as np


def freqs(rot_dim, base, kind="plain", factor=1.0, trained_len=0.0, slow=1.0, fast=32.0):
    """Inverse frequencies and the factor of cosines and sines, one pair at a time."""
    out = []
    for i in range(rot_dim // 2):
        b = base * factor ** (rot_dim / (rot_dim - 2)) if kind == "ntk" else base
        f = 1.0 / b ** (2 * i / rot_dim)
        if kind == "linear":
            f = f / factor
        if kind == "yarn":
            wavelength = 2 * np.pi / f
            turns = trained_len / wavelength
            keep = 0.0 if turns < slow else 1.0 if turns > fast else (turns - slow) / (fast - slow)
            f = (1 - keep) * f / factor + keep * f
        out.append(f)
    return np.array(out), 0.1 * np.log(factor) + 1.0 if kind == "yarn" else 1.0


def rope(x, pos, inv_freq, pairs=False, sections=None, scale=1.0):
    """float64 rotation of x [T][heads][hd] at pos [rows][T] (cosines and sines not rounded)."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    y = x.copy()
    for i in range(half):
        row = 0 if sections is None else 0 if i < sections[0] else 1 if i < sections[0] + sections[1] else 2
        a = pos[row].astype(np.float64) * inv_freq[i]
        c, s = scale * np.cos(a)[:, None], scale * np.sin(a)[:, None]
        p, q = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        y[..., p] = x[..., p] * c - x[..., q] * s
        y[..., q] = x[..., q] * c + x[..., p] * s
    return y


def sees(n, ctx, length, tree=None):
    """Which of `length` keys the n new tokens see; ctx keys (may be negative) lie before the new ones; tree: [n][words]
    uint32 or None."""
    m = np.zeros((n, length), bool)
    for i in range(n):
        for j in range(length):
            r = j - ctx
            if r < 0:
                m[i, j] = True
            elif tree is None:
                m[i, j] = r <= i
            else:
                m[i, j] = r < 32 * tree.shape[1] and bool(int(tree[i, r // 32]) >> (r % 32) & 1)
    return m


def attention(q, K, V, seen, scale):
    """q [n][heads][hd], K and V [length][kv heads][hd], seen [n][length] or per key; float64.  Returns the rows and,
    for error bounds, sum_j p_j |v_j| and the largest sum_c |q_c k_jc| of a visible key."""
    q, K, V = (np.asarray(a, np.float64) for a in (q, K, V))
    n, heads, hd = q.shape
    group = heads // K.shape[1]
    o, spread = np.zeros((n, heads, hd)), np.zeros((n, heads, hd))
    reach = np.zeros((n, heads, 1))
    for h in range(heads):
        k, v = K[:, h // group], V[:, h // group]
        s = scale * (q[:, h] @ k.T)
        a = np.abs(q[:, h]) @ np.abs(k).T
        for i in range(n):
            at = np.nonzero(seen[i])[0]
            if len(at) == 0:
                continue
            e = np.exp(s[i, at] - s[i, at].max())
            p = e / e.sum()
            o[i, h] = p @ v[at]
            spread[i, h] = p @ np.abs(v[at])
            reach[i, h] = a[i, at].max()
    return o, spread, reach


def verify(p, token, u, draft_p=None, parent=None):
    """One sequence's accepted rows and next token, from the definition (float64)."""
    n, V = p.shape
    p = p.astype(np.float64)
    u = u.astype(np.float64)
    path, cur = [], 0
    if draft_p is not None:
        d = draft_p.astype(np.float64)
        w = None
        for i in range(1, n):
            x = int(token[i])
            if 0 <= x < V and u[i] * d[i, x] < p[i - 1, x]:
                path.append(i)
                cur = i
            else:
                w = np.maximum(p[cur] - d[i], 0.0)
                break
        w = p[cur] if w is None else w
    else:
        above = [-1] + [i - 1 if parent is None else int(parent[i]) for i in range(1, n)]
        moved = True
        while moved:
            moved, rest, gone = False, 1.0, []
            for i in range(cur + 1, n):
                x = int(token[i])
                if above[i] != cur or not 0 <= x < V or x in gone:
                    continue
                if u[i] * rest < p[cur, x]:
                    path.append(i)
                    cur, moved = i, True
                    break
                gone.append(x)
                rest -= p[cur, x]
        w = p[cur].copy()
        w[gone] = 0.0
    if not w.sum() > 0:
        w = p[cur]
    if not w.sum() > 0:
        return path, -1
    c = np.cumsum(w)
    return path, int(np.nonzero(c > u[0] * c[-1])[0][0])
