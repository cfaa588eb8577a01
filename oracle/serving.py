"""Plain fp64 NumPy forms of what stands beside the MoBA attention in a layer: the
per-head norm of queries and keys with the position rotation and its gradients, the
append to a paged cache and the attention of new tokens over it.

Test infrastructure: it shares no code with the CUDA path.  The formulas are those of
include/moba.h.  The attention also returns the sums that error bounds need."""
import numpy as np


def rotate(y, positions, inv_freq, interleaved=False, way=1.0):
    """y [T, h, d] turned by its tokens' angles (way = -1: back)."""
    y = np.array(y, np.float64)
    r = len(inv_freq)
    angle = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle), way * np.sin(angle)
    ia = np.arange(r) * 2 if interleaved else np.arange(r)
    ib = ia + 1 if interleaved else ia + r
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def norm(x, w, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def norm_rope(x, w, positions, inv_freq, eps, interleaved=False):
    return rotate(norm(x, w, eps), positions, inv_freq, interleaved)


def norm_rope_backward(x, w, positions, inv_freq, eps, dy, interleaved=False):
    """(dx, dw)"""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    z = rotate(dy, positions, inv_freq, interleaved, -1.0)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = z * w
    dx = r * g - x * r ** 3 * (x * g).mean(-1, keepdims=True)
    return dx, (z * x * r).sum((0, 1))


def new_tokens(cu_new, kv_len):
    """(row, sequence, position) of every new token."""
    got = []
    for b in range(len(kv_len)):
        n = int(cu_new[b + 1] - cu_new[b])
        got += [(int(cu_new[b]) + i, b, int(kv_len[b]) - n + i) for i in range(n)]
    return got


def paged_attention(q, k_pool, v_pool, cu_new, kv_len, table, scale, only=None):
    """out [T, hq, d], lse [hq, T], and the bounds' sums: the largest sum of |q_c k_c|
    of a row's keys and sum_u p_u |v_u|.  Rows of no sequence, and rows that see no
    key, are 0 and -inf.  `only`: the rows to compute (all)."""
    T, hq, d = q.shape
    hkv, page = k_pool.shape[1:3]
    G = hq // hkv
    out, absv = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, dots = np.full((hq, T), -np.inf), np.zeros((T, hq))
    for b in range(len(kv_len)):
        L, first, n = int(kv_len[b]), int(cu_new[b]), int(cu_new[b + 1] - cu_new[b])
        if n == 0 or L <= 0:
            continue
        at, slot = np.asarray(table[b])[np.arange(L) // page], np.arange(L) % page
        for h in range(hq):
            k, v = k_pool[at, h // G, slot], v_pool[at, h // G, slot]
            for i in range(n):
                see = L - n + i + 1
                if see <= 0 or (only is not None and first + i not in only):
                    continue
                z = k[:see] @ q[first + i, h] * scale
                m = z.max()
                p = np.exp(z - m)
                l = p.sum()
                out[first + i, h] = p @ v[:see] / l
                absv[first + i, h] = p @ np.abs(v[:see]) / l
                lse[h, first + i] = m + np.log(l)
                dots[first + i, h] = (np.abs(k[:see]) @ np.abs(q[first + i, h])).max()
    return out, lse, dots, absv
