"""Microscaled 4-bit matrices, fp64 CPU reference (the MXFP4 format of the OCP
Microscaling Formats specification v1.0).

A block of 32 consecutive elements of a row has the scale
2^(floor(log2 a) - 2), a its largest magnitude, at least 2^-127 (byte = exponent
+ 127); an element is the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (codes 0..7,
plus 8 for negative ones) to |x| / scale, an equal distance going to the even
code, anything above 6 to 6.  A block with a NaN or an infinity has the byte 255
and zero codes.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def _blocked(x):
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    p = np.zeros((rows, kb * BLOCK))
    p[:, :cols] = x
    return p.reshape(rows, kb, BLOCK)


def scale_bytes(amax):
    """Scale bytes of blocks with these largest magnitudes (finite)."""
    _, e = np.frexp(amax)  # amax = f 2^e, f in [0.5, 1)
    return np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0).astype(np.int64)


def nearest_codes(y):
    """Magnitude codes 0..7 of finite |y|."""
    d = np.abs(np.abs(y)[..., None] - LEVELS)
    # even codes win an equal distance
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    return order[np.argmin(d[..., order], axis=-1)]


def quantize(x):
    """(codes [rows, kb * 32] 0..15, scale bytes [rows, kb])"""
    b = _blocked(x)
    bad = ~np.all(np.isfinite(b), axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    s = scale_bytes(np.max(np.abs(b), axis=2))
    y = b * np.exp2(127.0 - s)[:, :, None]
    c = nearest_codes(y) + 8 * np.signbit(y)
    s = np.where(bad, 255, s)
    c = np.where(bad[:, :, None], 0, c)
    return c.reshape(c.shape[0], -1), s


def pack(codes):
    return (codes[:, 0::2] + 16 * codes[:, 1::2]).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.int64)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def values(codes, scales, cols):
    mag = LEVELS[codes & 7]
    v = np.where(codes & 8, -mag, mag).reshape(codes.shape[0], -1, BLOCK)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return (v * s[:, :, None]).reshape(codes.shape[0], -1)[:, :cols]


def round_trip(x):
    x = np.asarray(x)
    return values(*quantize(x), x.shape[1])


def round_trip_change(x, eps):
    """How far the value of each element can move when every element of x
    moves by at most eps (an array like x): the largest distance from
    round_trip(x) over both ends of each element's interval under every
    scale that the block's largest magnitude allows."""
    ref, cols = round_trip(x), x.shape[1]
    b, e = _blocked(x), _blocked(eps)
    lo = scale_bytes(np.max(np.maximum(np.abs(b) - e, 0.0), axis=2))
    hi = scale_bytes(np.max(np.abs(b) + e, axis=2))
    worst = np.zeros_like(b)
    refb = _blocked(ref)
    for s in (lo, hi):
        for end in (b - e, b + e):
            y = end * np.exp2(127.0 - s)[:, :, None]
            v = np.sign(end) * LEVELS[nearest_codes(y)] * np.exp2(s - 127.0)[:, :, None]
            worst = np.maximum(worst, np.abs(v - refb))
    return worst.reshape(b.shape[0], -1)[:, :cols]


def value_network(params, S, H1, H2, states, eps_scale=0.0):
    """V of fp32 parameters (flat w1, b1, w2, b2, w3, b3) with both hidden
    layers' operands in 4 bits; with eps_scale > 0 also a bound on V's change
    when every hidden sum is off by up to eps_scale times its terms' magnitudes."""
    p = np.asarray(params, dtype=np.float64)
    cut = np.cumsum([H1 * S, H1, H2 * H1, H2, H2])
    w1, b1, w2, b2, w3, b3 = np.split(p, cut)
    w1, w2 = round_trip(w1.reshape(H1, S)), round_trip(w2.reshape(H2, H1))
    x = round_trip(states)
    h1 = np.maximum(x @ w1.T + b1, 0.0)
    q1 = round_trip(h1)
    h2 = np.maximum(q1 @ w2.T + b2, 0.0)
    v = h2 @ w3 + b3[0]
    if not eps_scale:
        return v
    e1 = eps_scale * (np.abs(x) @ np.abs(w1).T + np.abs(b1))
    d1 = round_trip_change(h1, e1)
    e2 = d1 @ np.abs(w2).T + eps_scale * (np.abs(q1) @ np.abs(w2).T + np.abs(b2))
    return v, e2 @ np.abs(w3) + eps_scale * (h2 @ np.abs(w3) + abs(b3[0]))
