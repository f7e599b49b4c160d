"""Plain 64-bit definitions of the gradient-making operators, for their tests
(numpy on the host; no code of the package)."""
import math

import numpy as np
import torch

BLOCK = 32
TOP = 1.875 * 2.0 ** 127       # larger magnitudes count as this
U32 = 2.0 ** -24        # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step of each type, relative


def pitch(cols):
    return (cols + 63) // 64 * 64


def scale_bytes(x, fmt):
    """Scale bytes [blocks, cols] of x (float64): the smallest power of two, at
    least 2^-111, that keeps the block's largest magnitude within the format."""
    rows, cols = x.shape
    x = np.where(np.isfinite(x), np.clip(x, -TOP, TOP), x)
    top = 448.0 if fmt == "e4m3" else 127.0
    out = np.empty(((rows + BLOCK - 1) // BLOCK, cols), np.uint8)
    for b in range(out.shape[0]):
        blk = x[b * BLOCK:(b + 1) * BLOCK]
        for c in range(cols):
            a = np.abs(blk[:, c])
            if not np.isfinite(a).all():
                out[b, c] = 255
                continue
            e = -111
            if a.max() > 0:
                e = max(e, math.frexp(a.max())[1] - 10)
                while a.max() > top * 2.0 ** e:
                    e += 1
            out[b, c] = e + 127
    return out


def e4m3_values():
    """The value of each of the 256 codes, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = (-x if c & 128 else x) if (c & 127) != 127 else np.nan
    return v


E4M3 = e4m3_values()


def quantised(x, fmt):
    """The values a checkpoint of x (float64 [rows, cols]) stands for: each
    element rounded to the nearest multiple its format has there, ties to even."""
    s = np.repeat(2.0 ** (scale_bytes(x, fmt).astype(np.float64) - 127), BLOCK, axis=0)[: len(x)]
    nan = np.repeat(scale_bytes(x, fmt) == 255, BLOCK, axis=0)[: len(x)]
    with np.errstate(all="ignore"):
        q = np.where(nan, 0.0, np.clip(x, -TOP, TOP)) / s
        if fmt == "int8":
            q = np.rint(q)
        else:
            step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6))) - 3)
            q = np.rint(q / step) * step
    return np.where(nan, np.nan, q * s)


def decoded(codes, scales, cols, fmt):
    """Values of stored codes [rows, pitch] and scales [blocks, pitch] (uint8 arrays)."""
    c = codes[:, :cols]
    q = E4M3[c] if fmt == "e4m3" else c.view(np.int8).astype(np.float64)
    s = np.where(scales[:, :cols] == 255, np.nan, 2.0 ** (scales[:, :cols].astype(np.float64) - 127))
    return q * np.repeat(s, BLOCK, axis=0)[: len(c)]


def _phi(x):
    return 0.5 * torch.special.erfc(torch.from_numpy(-x / math.sqrt(2.0))).numpy()


def _sigmoid(v):
    return torch.sigmoid(torch.from_numpy(np.asarray(v))).numpy()


C, K = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def act(x, fn):
    if fn == "gelu":
        return x * _phi(x)
    return x * _sigmoid(C * (x + K * x ** 3) if fn == "gelu_tanh" else x)


def act_slope(x, fn):
    if fn == "gelu":
        return _phi(x) + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if fn == "gelu_tanh":
        s = _sigmoid(C * (x + K * x ** 3))
        return s + s * (1.0 - s) * x * C * (1.0 + 3 * K * x * x)
    s = _sigmoid(x)
    return s + s * (1.0 - s) * x


def act_error(x, fn):
    """Relative error allowed to fp32 arithmetic of Phi or sigma at x.

    The exponential's argument a carries 4 roundings, so its result a relative
    error of 4*|a|*2^-24; it, the reciprocal and some dozen products and sums
    are off by 2^-23 each at most; gelu's polynomial by 2^-22 (1.5e-7 rounded
    up).  a = x^2/2 for gelu, 2*sqrt(2/pi)*(x + 0.044715 x^3) for gelu_tanh, x for silu."""
    a = {"gelu": 0.5 * x * x, "gelu_tanh": C * np.abs(x + K * x ** 3), "silu": np.abs(x)}[fn]
    return 4 * a * U32 + 32 * U32 + 2.0 ** -22


def linear(dy, xhat):
    """(dW, db, sums of magnitudes for the error bound)."""
    return dy.T @ xhat, dy.sum(axis=0), np.abs(dy).T @ np.abs(xhat), np.abs(dy).sum(axis=0)


def embedding_grad(ids, dy, vocab):
    """(per-row sums, sums of magnitudes, tokens per row)."""
    keep = (ids >= 0) & (ids < vocab)
    out, mag = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(out, ids[keep], dy[keep])
    np.add.at(mag, ids[keep], np.abs(dy[keep]))
    return out, mag, np.bincount(ids[keep], minlength=vocab)
