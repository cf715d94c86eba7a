"""Plain 64-bit forms of the norms with rotation, and bounds of what FP32 arithmetic may lose."""
import numpy as np

F32 = 2.0 ** -24          # half a step, relative
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def angles(pos, rope_dim, base=10000.0, inv_freq=None):
    f = np.array(inv_freq, np.float64) if inv_freq is not None else base ** (-np.arange(0, rope_dim, 2) / rope_dim)
    return np.asarray(pos, np.float64)[:, None] * f


def pairs(rope_dim, interleaved):
    i = np.arange(rope_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rope_dim // 2)


def rotate(x, ang, rope_dim, interleaved, sign=1.0):
    """x [T, H, D] turned by ang [T, rope_dim / 2]."""
    if rope_dim == 0:
        return x.copy()
    a, b = pairs(rope_dim, interleaved)
    c, s = np.cos(ang)[:, None], sign * np.sin(ang)[:, None]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def normed(x, norm, eps):
    if norm == "layer":
        x = x - x.mean(-1, keepdims=True)
    std = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x / std, std


def forward(x, w, b, pos, norm, eps, rope_dim, interleaved, base=10000.0, inv_freq=None):
    n, _ = normed(x, norm, eps)
    y = n * (1.0 if w is None else w) + (0.0 if b is None else b)
    return rotate(y, angles(pos, rope_dim, base, inv_freq), rope_dim, interleaved)


def backward(dy, x, w, pos, norm, eps, rope_dim, interleaved, base=10000.0, inv_freq=None):
    """dx, dw, db"""
    g = rotate(dy, angles(pos, rope_dim, base, inv_freq), rope_dim, interleaved, -1.0)
    n, std = normed(x, norm, eps)
    gw = g * (1.0 if w is None else w)
    dx = gw - n * (gw * n).mean(-1, keepdims=True)
    if norm == "layer":
        dx = dx - gw.mean(-1, keepdims=True)
    return dx / std, (g * n).sum((0, 1)), g.sum((0, 1))


def lost(x, norm, eps):
    """How far n may be from the exact one, absolutely, per row [T, H, 1]: x as given is exact.

    The mean of D values in a tree of at most 3 + log2(D / 8) levels after a chain of 8: each addition is off by F32
    of a partial sum, at most 12 F32 mean|x| in all; a difference, a square and the mean of squares 14 F32 relative
    together, the root, the division and the product 4 F32.  With m = max |x|: |dn| <= (12 + 2 + 18) F32 m / std."""
    _, std = normed(x, norm, eps)
    m = np.abs(x).max(-1, keepdims=True)
    return 32 * F32 * m / np.maximum(std, 1e-300)


TURN = 8 * F32      # cos and sin: the angle's 2^-32 of a turn (2 pi 2^-33 < F32), its rounding to 24 bits (pi F32), the function (2 F32)


def forward_tol(x, w, b, pos, norm, eps, rope_dim, interleaved, out, want):
    """|y - want| where y is formed in FP32 and rounded once to `out`."""
    n, _ = normed(x, norm, eps)
    aw = np.ones(x.shape[-1]) if w is None else np.abs(w)
    ab = np.zeros(x.shape[-1]) if b is None else np.abs(b)
    y, dy = np.abs(n) * aw + ab, lost(x, norm, eps) * aw + 2 * F32 * (np.abs(n) * aw + ab)
    if rope_dim:
        i, j = pairs(rope_dim, interleaved)
        yy, dd = y.copy(), dy.copy()
        for p, q in ((i, j), (j, i)):
            yy[..., p] = y[..., p] + y[..., q]
            dd[..., p] = dy[..., p] + dy[..., q] + (TURN + 2 * F32) * (y[..., p] + y[..., q])
        y, dy = yy, dd
    return dy * 1.01 + HALF[out] * (np.abs(want) + dy) + 1e-30


def backward_tol(dy, x, w, pos, norm, eps, rope_dim, interleaved, out, want):
    """Bounds of dx (rounded once to `out`), dw and db (FP32 sums over n rows in chains and trees of at most n additions)."""
    n, std = normed(x, norm, eps)
    aw = np.ones(x.shape[-1]) if w is None else np.abs(w)
    g = np.abs(dy)
    if rope_dim:
        i, j = pairs(rope_dim, interleaved)
        gg = g.copy()
        gg[..., i] = gg[..., j] = g[..., i] + g[..., j]
        g = gg
    dg = (TURN + 2 * F32) * g if rope_dim else 0.0 * g
    dn = lost(x, norm, eps)
    an = np.abs(n)
    gw, dgw = g * aw, dg * aw + F32 * g * aw
    dot = (gw * an).mean(-1, keepdims=True)
    ddot = (dgw * an + gw * dn).mean(-1, keepdims=True) + 16 * F32 * dot
    mean = gw.mean(-1, keepdims=True)
    dmean = dgw.mean(-1, keepdims=True) + 16 * F32 * mean
    inner = gw + an * dot + (mean if norm == "layer" else 0.0)
    err = dgw + an * ddot + dn * dot + (dmean if norm == "layer" else 0.0) + 6 * F32 * inner
    # 1 / std is off by as much as n is, relative to the largest element
    rel = 32 * F32 * np.abs(x).max(-1, keepdims=True) / np.maximum(std, 1e-300)
    tdx = (err + rel * inner) / std
    rows = x.shape[0] * x.shape[1]
    tdw = (dg * an + g * dn).sum((0, 1)) + (rows + 4) * F32 * (g * an).sum((0, 1))
    tdb = dg.sum((0, 1)) + (rows + 4) * F32 * g.sum((0, 1))
    return tdx * 1.01 + HALF[out] * (np.abs(want) + tdx) + 1e-30, tdw * 1.01 + 1e-30, tdb * 1.01 + 1e-30
