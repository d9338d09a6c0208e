"""fp64 NumPy statements of the operators around the KL: norm and rotation of
heads with its gradients, the paged cache and the attention over it. Each
returns, beside the result, the same expression over absolute values, which
the tests' error bounds scale with."""
import numpy as np


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, cos, sin, interleaved, back=False):
    """Rotate the pairs of x's first rot = 2 * cos.shape[-1] elements."""
    a, b = _pairs(2 * cos.shape[-1], interleaved)
    s = -sin if back else sin
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * s
    y[..., b] = x[..., b] * cos + x[..., a] * s
    return y


def turn_abs(x, cos, sin, interleaved):
    """|a cos| + |b sin| of the same pairs, from x >= 0."""
    return np.maximum(turn(x, np.abs(cos), -np.abs(sin), interleaved, False),
                      turn(x, np.abs(cos), np.abs(sin), interleaved, False))


def norm_rope(x, w, cos, sin, eps, interleaved):
    """Rows x [..., d], cos, sin [..., rot / 2] of their positions; w may be None."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return turn(x, cos, sin, interleaved), turn_abs(np.abs(x), cos, sin, interleaved)


def norm_rope_bwd(x, w, dy, dy_abs, cos, sin, eps, interleaved):
    """dx, its absolute form, and per row dw, its absolute form. dy_abs: |dy|
    summed over the repeats that dy sums."""
    g = turn(dy, cos, sin, interleaved, back=True)
    ga = turn_abs(dy_abs, cos, sin, interleaved)
    if w is None:
        return g, ga, None, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, ua = g * w, ga * np.abs(w)
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdims=True))
    dxa = r * (ua + np.abs(x) * r * r * (ua * np.abs(x)).mean(-1, keepdims=True))
    return dx, dxa, g * x * r, ga * np.abs(x) * r


def gather(cache, table, length):
    """The first `length` rows of a sequence: [HK, length, d] from cache
    [pages, HK, page, d] and its row of page numbers."""
    page = cache.shape[2]
    n = -(-length // page)
    rows = cache[np.asarray(table[:n], dtype=np.int64)]  # [n, HK, page, d]
    return np.moveaxis(rows, 1, 0).reshape(cache.shape[1], n * page, -1)[:, :length]


def paged_attn(q, k, v, scale, causal):
    """One sequence: q [n, HQ, d] against k, v [HK, length, d]. Returns o, lse
    and sum_j p_j |v_j|. Rows that see no key: zeros and -inf."""
    n, HQ, d = q.shape
    HK, length, _ = k.shape
    group = HQ // HK
    o = np.zeros((n, HQ, d))
    oa = np.zeros((n, HQ, d))
    lse = np.full((n, HQ), -np.inf)
    for h in range(HQ):
        for i in range(n):
            lim = min(length, length - n + i + 1) if causal else length
            if lim <= 0:
                continue
            s = scale * (k[h // group, :lim] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            z = e.sum()
            o[i, h] = e @ v[h // group, :lim] / z
            oa[i, h] = e @ np.abs(v[h // group, :lim]) / z
            lse[i, h] = m + np.log(z)
    return o, lse, oa
