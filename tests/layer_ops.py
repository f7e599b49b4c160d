"""Plain definitions of the AdamW step and of a linear layer's forward and input
gradient, for their tests (numpy on the host; no code of the package).

AdamW's step is a chain of fp32 operations that each round once, so numpy's
float32 gives its one right result; the 8-bit moments are written from the
format's definition in 64 bits."""
import numpy as np

F = np.float32
TOP = 1.875 * 2.0 ** 127
M32 = 0xFFFFFFFF


def mix(x):
    x = np.asarray(x, np.uint64)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & np.uint64(M32)
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def dither(places, seed):
    """(16 bits for m, 16 bits for r) of the elements at these places of a list."""
    key = mix((seed & M32) ^ int(mix(((seed >> 32) + 0x9E3779B9) & M32)))
    p = np.asarray(places, np.uint64)
    with np.errstate(over="ignore"):
        k = (key + (p >> np.uint64(32)) * np.uint64(0x9E3779B9)) & np.uint64(M32)
    h = mix((p & np.uint64(M32)) ^ k)
    return h & np.uint64(0xFFFF), h >> np.uint64(16)


def _scale_exponent(a, top):
    """The smallest e >= -111 with a <= top * 2^e."""
    e = -111
    if a > 0:
        e = max(e, int(np.floor(np.log2(a / top))) - 1)
        while a > top * 2.0 ** e:
            e += 1
    return e


def _pick(x, d, least, bits, fine):
    """Codes of x >= 0 (in units of the scale): steps of 2^least / 2^bits up to 2^(least+1), then `bits` mantissa bits;
    below 2^least the remainder in units of 2^-fine of a step, to nearest even."""
    k = np.floor(np.log2(np.maximum(x, 2.0 ** least)))
    step = 2.0 ** (k - bits)
    q = x / step
    q = np.where(x < 2.0 ** least, np.rint(q * 2.0 ** fine) / 2.0 ** fine, q)
    n = np.floor(q + d.astype(np.float64) / 65536.0)
    return (n + (k - least) * 2.0 ** bits).astype(np.int64), n * step


def encode(m, r, places, seed):
    """(m codes, m scales, r codes, r scales) of one tensor's fp32 moments; blocks of 64 from its first element on."""
    n = len(m)
    dm, dr = dither(places, seed)
    out = [np.zeros(n, np.uint8), np.zeros((n + 63) // 64, np.uint8), np.zeros(n, np.uint8), np.zeros((n + 63) // 64, np.uint8)]
    for b in range((n + 63) // 64):
        at = slice(64 * b, min(64 * b + 64, n))
        for x, d, c, s, top, least, bits, fine in ((m[at], dm[at], out[0], out[1], 448.0, -6, 3, 20),
                                                   (r[at], dr[at], out[2], out[3], 31.0 * 2.0 ** 14, 4, 4, 19)):
            if not np.isfinite(x).all():
                s[b] = 255
                continue
            v = x.astype(np.float64)
            a = np.minimum(np.abs(v), TOP)
            e = _scale_exponent(a.max(), top)
            s[b] = e + 127
            code, _ = _pick(a / 2.0 ** e, d, least, bits, fine)
            if bits == 4:
                code = np.maximum(code, v > 0)
            else:
                code = code | (np.signbit(x).astype(np.int64) << 7)
            c[at] = code
    return out


def decode_m(codes, scales):
    c = codes.astype(np.int64)
    k, f = (c >> 3) & 15, c & 7
    x = np.where(k > 0, (8.0 + f) * 2.0 ** (k - 10.0), f * 2.0 ** -9)
    x = np.where(c >= 128, -x, x)
    return _scaled(x, scales)


def decode_r(codes, scales):
    c = codes.astype(np.int64)
    k, f = c >> 4, c & 15
    return _scaled(np.where(k > 0, (16.0 + f) * 2.0 ** (k - 1.0), f), scales)


def _scaled(x, scales):
    s = np.repeat(scales.astype(np.float64), 64)[: len(x)]
    with np.errstate(invalid="ignore"):
        return np.where(s == 255, np.nan, x * 2.0 ** (s - 127)).astype(F)


def adamw(grads, m, v, p, *, beta1, beta2, eps, lr, step, weight_decay=0.0, decay=1.0, grad_scale=None):
    """One tensor's step in fp32: grads [W][n] float32, m, v, p [n] float32; returns m, v, r, p."""
    with np.errstate(all="ignore"):
        g = np.zeros_like(m)
        for row in grads:
            g = g + row
        g = g / F(len(grads))
        if grad_scale is not None:
            g = g * F(grad_scale)
        m = F(beta1) * m + F(1.0 - beta1) * g
        v = F(beta2) * v + F(1.0 - beta2) * (g * g)
        r = np.sqrt(v)
        u = m / (r * F(1.0 / np.sqrt(1.0 - beta2 ** step)) + F(eps))
        p = (p - p * (F(lr * weight_decay) * F(decay))) - u * F(lr / (1.0 - beta1 ** step))
    assert p.dtype == F and m.dtype == F and v.dtype == F and r.dtype == F
    return m, v, r, p


def adamw64(grads, m, v, p, *, beta1, beta2, eps, lr, step, weight_decay=0.0, decay=1.0, grad_scale=None):
    """The same from the formula in 64 bits: m, v, p."""
    g = grads.astype(np.float64).mean(axis=0) * (1.0 if grad_scale is None else float(grad_scale))
    m = beta1 * m.astype(np.float64) + (1.0 - beta1) * g
    v = beta2 * v.astype(np.float64) + (1.0 - beta2) * g * g
    mh, vh = m / (1.0 - beta1 ** step), v / (1.0 - beta2 ** step)
    p = p.astype(np.float64)
    return m, v, p - lr * weight_decay * decay * p - lr * mh / (np.sqrt(vh) + eps)
