"""Plain 64-bit statements of the block norms and of the 8-bit floating-point
linears (numpy, no product code).

e4m3: sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent 0 is
subnormal (steps of 2^-9); the largest value is 448 (0x7e), 0x7f is NaN and
there are no infinities. A block of 128 features (of a row, or of 128 weight
rows) has the scale s = fp32(max|x| / 448) and the codes
e4m3(fp32(x / s)), rounded to nearest even; an all-zero block has scale 0 and
codes 0.
"""
import numpy as np

BLOCK = 128
MAX = 448.0
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2


def n_blocks(n):
    return -(-n // BLOCK)


def e4m3_values():
    """The value of every code, from its bit fields."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_encode(x):
    """Codes of x: the nearest value, ties to the even code, saturating."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()[:127]  # 0 .. 448, increasing
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=MAX, neginf=-MAX)), MAX)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(a == grid[hi], hi, code)
    code = np.where(np.isnan(x), 127, code)
    return (code + np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def fp8_pack(X, rows=1):
    """(codes uint8, scales fp32) of X over blocks of rows x 128."""
    X = np.asarray(X, np.float32)
    R, K = X.shape
    s = np.zeros((-(-R // rows), n_blocks(K)), np.float32)
    Q = np.zeros((R, K), np.uint8)
    with np.errstate(all="ignore"):
        for i in range(s.shape[0]):
            for j in range(s.shape[1]):
                b = X[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
                s[i, j] = np.max(np.abs(b)) / np.float32(MAX)
                q = np.zeros_like(b) if s[i, j] == 0 else b / s[i, j]
                Q[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK] = e4m3_encode(q)
    return Q, s


def widen(s, rows, cols, height=1):
    """Block scales as one factor per element."""
    return np.repeat(np.repeat(np.asarray(s, np.float64), height, 0)[:rows], BLOCK, 1)[:, :cols]


def fp8_linear(Qx, sx, Qw, sw, bias=None):
    """(Y, the sum of the products' magnitudes), 64 bits."""
    val = e4m3_values()
    X = val[Qx] * widen(sx, *Qx.shape)
    W = val[Qw] * widen(sw, *Qw.shape, BLOCK)
    Y, A = X @ W.T, np.abs(X) @ np.abs(W).T
    return (Y, A) if bias is None else (Y + np.asarray(bias, np.float64), A + np.abs(np.asarray(bias, np.float64)))


def norm(x, kind, eps):
    """(normalized rows, mean, 1 / deviation)."""
    x = np.asarray(x, np.float64)
    zero, one = np.zeros((x.shape[0], 1)), np.ones((x.shape[0], 1))
    if kind == NORM_NONE:
        return x, zero, one
    mean = x.mean(1, keepdims=True) if kind == NORM_LAYER else zero
    r = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    return (x - mean) * r, mean, r


def block_norm(H, Y=None, residual_scale=1.0, block_scale=1.0, post=NORM_NONE, post_eps=1e-6, post_weight=None,
               post_bias=None, gate=None, pre=NORM_RMS, pre_eps=1e-6, pre_weight=None, pre_bias=None, scale=None,
               shift=None, sample=None):
    """(h', u, magnitude of h''s terms, magnitude of u's terms), 64 bits. The
    magnitudes are what a rounding of relative size e in any step of fp32
    arithmetic moves the result by, divided by e (up to a small factor)."""
    f = lambda v: np.asarray(v, np.float64)  # noqa: E731
    H = f(H)
    sample = np.zeros(H.shape[0], np.int64) if sample is None else sample
    h, hm = residual_scale * H, np.abs(residual_scale * H)
    if Y is not None:
        n, mean, r = norm(Y, post, post_eps)
        nm = (np.abs(f(Y)) + np.abs(mean)) * r
        if post_weight is not None:
            n, nm = n * f(post_weight), nm * np.abs(f(post_weight))
        if post_bias is not None:
            n, nm = n + f(post_bias), nm + np.abs(f(post_bias))
        g = block_scale * (1.0 if gate is None else f(gate)[sample])
        h, hm = h + g * n, hm + np.abs(g) * nm
    u, mean, r = norm(h, pre, pre_eps)
    um = (hm + hm.mean(1, keepdims=True) * (pre == NORM_LAYER)) * r
    if pre_weight is not None:
        u, um = u * f(pre_weight), um * np.abs(f(pre_weight))
    if pre_bias is not None:
        u, um = u + f(pre_bias), um + np.abs(f(pre_bias))
    if scale is not None:
        u, um = u + u * f(scale)[sample], um * np.abs(1.0 + f(scale)[sample]) + um * 2.0 ** -24
    if shift is not None:
        u, um = u + f(shift)[sample], um + np.abs(f(shift)[sample])
    return h, u, hm, um
