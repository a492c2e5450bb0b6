"""Plain 64-bit forms of the operators of include/nhm_layer.h, and the tolerances of their 32-bit kernels (numpy).

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of f32 2^-24. The hardware's exp2 and reciprocal
are within 2^-22 of the value (one step of f32 and the rounding of the argument beside it)."""
import numpy as np

U = 2.0 ** -24          # half a step of f32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def half_step(ref, bf16):
    """Half a step of the output type at ref, and the smallest subnormal's half."""
    return np.abs(ref) * (2.0 ** -8 if bf16 else U) + (2.0 ** -134 if bf16 else 2.0 ** -150)


# ---- MXFP4

def mxfp4_quantize(x):
    """(codes [rows, cols], scale codes [rows, cols / 32]) of float rows: one code an entry, not packed."""
    x = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    amax = np.abs(x).max(axis=2)
    bad = ~np.isfinite(amax)
    e = np.frexp(np.where(bad | (amax == 0), 1.0, amax))[1] - 3            # floor(log2) - 2
    e = np.where(amax == 0, -127, np.clip(e, -127, 127))
    v = np.where(bad[:, :, None], 0.0, x) * 2.0 ** (-e[:, :, None].astype(float))
    d = np.abs(np.abs(v)[..., None] - GRID)
    best = d.min(axis=-1, keepdims=True)
    near = d == best                                                       # one code, or two at a tie: the even one
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(np.signbit(v) & ~bad[:, :, None], code + 8, code)
    return code.reshape(x.shape[0], -1).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mxfp4_pack(code):
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)


def mxfp4_values(code, scale):
    """float64 values of unpacked codes; those of scale code 255 are NaN."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(float) - 127))
    return v * np.repeat(s, 32, axis=1)


def mxfp4_linear(xv, wv):
    """(values, tolerance before the output's rounding) of float64 activations [m, k] and weights [n, k]: each matrix
    instruction's 128 products are summed within U of sum |a w|, and added to what came before them; sums of up to
    16 shares of k follow."""
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    return ref, U * (xv.shape[1] / 128 + 18) * mag


# ---- convolution

def _silu(y):
    return y / (1.0 + np.exp(-y))


def causal_conv(rows, w, b, silu):
    """rows [width - 1 + t, dim]: the window, then the tokens. (out [t, dim], tolerance before rounding)."""
    width, t = w.shape[1], rows.shape[0] - w.shape[1] + 1
    y, mag = np.zeros((t, w.shape[0])), np.zeros((t, w.shape[0]))
    for j in range(width):
        y += rows[j:j + t] * w[:, j]
        mag += np.abs(rows[j:j + t] * w[:, j])
    y, mag = y + b, mag + np.abs(b)
    tol = U * (width + 1) * mag
    if silu:      # its slope is at most 1.1; exp of an argument rounded once, reciprocal, two products
        return _silu(y), 1.1 * tol + (16 + 4 * np.abs(y)) * U * np.abs(_silu(y))
    return y, tol


# ---- selective scan

def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def selective_scan(u, dt, B, C, A_log, D, dt_bias, h, z=None):
    """One sequence from state h [dim, n]: (out [t, dim], tolerance before rounding, end state, its tolerance).

    The error of the state follows the state: each step takes the last one's with the decay, and adds the roundings of
    its own terms (exp2: its own 2 U and the argument's, (dt A) 16 U with softplus's and exp's; the new term 16 U; the
    sum's one)."""
    A = -np.exp(A_log)
    t, dim = u.shape
    out, tol = np.zeros((t, dim)), np.zeros((t, dim))
    h, mag, err = h.copy(), np.abs(h), np.zeros_like(h)
    for i in range(t):
        d = softplus(dt[i] + dt_bias)[:, None]
        decay, add = np.exp(d * A), d * u[i][:, None] * B[i]
        h = decay * h + add
        mag = decay * mag + np.abs(add)
        err = decay * err + U * (24 + 16 * np.abs(d * A)) * mag
        out[i] = (h * C[i]).sum(axis=1) + D * u[i]
        tol[i] = (err * np.abs(C[i])).sum(axis=1) + U * 16 * ((mag * np.abs(C[i])).sum(axis=1) + np.abs(D * u[i]))
    if z is not None:
        g = _silu(z)
        tol = tol * np.abs(g) + (16 + 4 * np.abs(z)) * U * np.abs(out * g)
        out = out * g
    return out, tol, h, err


# ---- scoring of tokens

def token_logprobs(x, token, n_top):
    """(logprob, rank, entropy, top logprobs, top tokens) of one row of logits (float64; NaN counts as -inf)."""
    x = np.where(np.isnan(x), -np.inf, x)
    top, n = x.max(), x.size
    if top == -np.inf:
        lp = np.full(n, -np.inf)
        entropy = 0.0
    else:
        d = np.where(x == top, 0.0, x - top) if np.isfinite(top) else np.where(x == top, 0.0, -np.inf)
        lp = d - np.log(np.exp(d).sum())
        p = np.exp(lp[lp > -np.inf])
        entropy = -(p * lp[lp > -np.inf]).sum()
    order = np.lexsort((np.arange(n), -x))
    best = order[:n_top]
    best = best[lp[best] > -np.inf]
    tl, tt = np.full(n_top, -np.inf), np.full(n_top, -1)
    tl[:best.size], tt[:best.size] = lp[best], best
    if not 0 <= token < n:
        return 0.0, 0, entropy, tl, tt
    return lp[token], int(np.flatnonzero(order == token)[0]) + 1, entropy, tl, tt


def logprob_tolerance(ref):
    """The sum's terms are within (2 + |log2 term|) 2 U of their values, which weighted by themselves is below 2^-19 for
    rows whose probability is spread over up to 2^24 entries; then the result's own rounding."""
    return 2.0 ** -19 + np.where(np.isfinite(ref), np.abs(ref), 0.0) * U
