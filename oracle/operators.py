"""Float64 reference of the adapter and optimizer operators (numpy only).

Shares no code with the GPU path: written from the formulas and the state
format that include/poetx.h states.
"""

import numpy as np

BLOCK = 256
ALPHA_POS, ALPHA_STEP = 0xC13FA9A9, 0x91E10DA5


# ---- low-rank adapters beside a shared projection

def segments(seg_start, seg_adapter, count):
    for lo, hi, a in zip(seg_start[:-1], seg_start[1:], seg_adapter):
        if 0 <= a < count and hi > lo:
            yield int(lo), int(hi), int(a)


def adapters_forward(X, Y, A, B, scale, seg_start, seg_adapter):
    """Y + s B (A x) for the tokens of each segment."""
    out = np.array(Y, dtype=np.float64)
    for lo, hi, a in segments(seg_start, seg_adapter, len(A)):
        out[lo:hi] += scale[a] * (X[lo:hi] @ A[a].T) @ B[a].T
    return out


def adapters_backward(X, dY, dX, A, B, scale, seg_start, seg_adapter):
    """(dX + its share, [dA], [dB]) of sum(dY * adapters_forward)."""
    dX = np.array(dX, dtype=np.float64)
    dA, dB = [np.zeros(a.shape) for a in A], [np.zeros(b.shape) for b in B]
    for lo, hi, a in segments(seg_start, seg_adapter, len(A)):
        u = scale[a] * dY[lo:hi] @ B[a]
        dX[lo:hi] += u @ A[a]
        dA[a] += u.T @ X[lo:hi]
        dB[a] += scale[a] * dY[lo:hi].T @ (X[lo:hi] @ A[a].T)
    return dX, dA, dB


# ---- gradient norm and AdamW

def grad_norm(grads, max_norm):
    norm = float(np.sqrt(sum(np.sum(np.square(g)) for g in grads)))
    return norm, (min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else float("nan"))


def dither(pos, step, shift, bits):
    """Fractional part of pos alpha + step beta, `bits` bits of it from bit `shift` on."""
    h = (np.asarray(pos, dtype=np.uint64) * np.uint64(ALPHA_POS) + np.uint64((step * ALPHA_STEP) & (2 ** 32 - 1)))
    h &= np.uint64(2 ** 32 - 1)
    return ((h >> np.uint64(shift)) & np.uint64(2 ** bits - 1)).astype(np.float64) / 2 ** bits


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, lr_mul=1.0, weight_decay=0.0):
    """(p, m, v) after one step, nothing rounded."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    up = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p - lr * lr_mul * (weight_decay * p + up), m, v


def decode8(codes, exps, signed):
    """Values of 8-bit codes [blocks * 256] with exponent bytes [blocks]."""
    c = np.asarray(codes).astype(np.int64).reshape(-1, BLOCK)
    E = np.maximum(np.asarray(exps).astype(np.int64), 40)[:, None]
    fields = 16 if signed else 32
    e, f = (c >> 3) % fields, c & 7
    x = np.where(e > 0, (8 + f) * 2.0 ** (e - 1), f * 1.0) * 2.0 ** (E - 127 - (fields + 1))
    if signed:
        x = np.where(c >= 128, -x, x)
    return np.where(E == 255, np.nan, x).reshape(-1)


def round8(x, pos, step, signed):
    """(value each element is stored as, its rounding step) for whole blocks of finite x."""
    a = np.abs(x).reshape(-1, BLOCK)
    top = a.max(1)
    # the octave of the largest value, the next one where rounding up could reach it
    E = np.floor(np.log2(np.maximum(top, 1e-300)))
    E = np.where(top + (2.0 ** 20 - 1) / 2 ** 23 * 2.0 ** E >= 2.0 ** (E + 1), E + 1, E)
    E = np.clip(np.where(top > 0, E, -200), 40 - 127, 127)[:, None]
    low = E - (14 if signed else 30)
    octave = np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))), low)
    unit = 2.0 ** (octave - 3)
    u = dither(pos, step, 12 if signed else 5, 20).reshape(-1, BLOCK)
    r = np.floor(a / unit + u) * unit
    if not signed:
        r = np.where((a > 0) & (r == 0), 2.0 ** (low - 3), r)
    r = np.sign(x) * r.reshape(-1)
    return r, unit.reshape(-1)


def round_bf16_dither(x, pos, step):
    """(value, rounding step) of a bf16 parameter."""
    a = np.abs(x)
    unit = 2.0 ** (np.floor(np.log2(np.maximum(a, 1e-300))) - 7)
    return np.sign(x) * np.floor(a / unit + dither(pos, step, 16, 16)) * unit, unit
