"""Plain numpy forms of the MXFP4 rows and of the norm, for the tests: each element by search among the
eight magnitudes, each scale from the exponent, in 64 bits."""
import numpy as np

F32, F64 = np.float32, np.float64
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], F64)


def quantise(v32):
    """codes uint8 [R, 16 B], scales uint8 [ceil(B / 4), R rounded up to 4, 4] of fp32 rows; entries that
    are not written are 0 here."""
    R, K = v32.shape
    B = (K + 31) // 32
    v = np.zeros((R, 32 * B), F64)
    v[:, :K] = v32
    v = v.reshape(R, B, 32)
    top = np.abs(v).max(-1, initial=0.0)
    bad = ~np.isfinite(v).all(-1)
    _, e = np.frexp(np.where(bad, 1.0, top))                  # top = m 2^e, 1/2 <= m < 1
    byte = np.where(top == 0, 0, np.maximum(e - 1 - 2 + 127, 0))
    a = np.where(bad[..., None], 0, np.abs(v)) * np.ldexp(1.0, 127 - byte)[..., None]
    d = np.abs(a[..., None] - VALUES)
    code = d.argmin(-1)                                       # of two equally near the lower ...
    up = np.minimum(code + 1, 7)
    tie = (up > code) & (np.take_along_axis(d, up[..., None], -1) == np.take_along_axis(d, code[..., None], -1))[..., 0]
    code = np.where(tie & (code % 2 == 1), up, code)          # ... unless its code is odd
    code = np.where(np.signbit(v), code + 8, code)
    code[bad] = 0
    byte = np.where(bad, 255, byte)
    code = code.reshape(R, -1).astype(np.uint8)
    scales = np.zeros(((B + 3) // 4, (R + 3) // 4 * 4, 4), np.uint8)
    for b in range(B):
        scales[b // 4, :R, b % 4] = byte[:, b]
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(codes, scales, K):
    """fp64 rows [R, K] that codes and scales stand for."""
    R = codes.shape[0]
    code = np.stack((codes & 15, codes >> 4), -1).reshape(R, -1)[:, :K]
    mag = VALUES[code & 7]
    byte = scales.transpose(1, 0, 2).reshape(scales.shape[1], -1)[:R]
    byte = np.repeat(byte, 32, axis=1)[:, :K].astype(np.int64)
    v = np.where(code >= 8, -mag, mag) * np.ldexp(1.0, byte - 127)
    return np.where(byte == 255, np.nan, v)


def norm(x, r, w, eps, dt):
    """h (fp64 of the type's values) and v (fp32) of 16-bit torch tensors x, r (or None), w (or None), and
    where v is sure: its fp64 value further than 2^-46 of itself from a tie between two fp32 numbers, so that no
    order of the fp64 sum decides it."""
    h = x if r is None else (x.float() + r.float()).to(dt)
    h = h.double().cpu().numpy()
    w = np.ones(h.shape[1]) if w is None else w.double().cpu().numpy()
    with np.errstate(all="ignore"):
        d = h * w / np.sqrt((h * h).sum(1, keepdims=True) / h.shape[1] + eps)
        d[~np.isfinite(h).all(1)] = np.nan
        v = d.astype(F32)
        other = np.nextafter(v, np.where(d > v, np.inf, -np.inf).astype(F32))
        tie = (v.astype(F64) + other.astype(F64)) / 2
        sure = ~(np.abs(d - tie) <= 2.0 ** -46 * np.abs(d))
    return h, v, sure


def int8_rows(v32):
    """codes, steps of fp32 rows as awq_int8_quantize makes them."""
    amax = np.max(np.abs(v32), axis=1, initial=0.0).astype(F32)
    finite = np.all(np.isfinite(v32), axis=1)
    step = (amax / F32(127)).astype(F32)
    step[step == 0] = 1
    with np.errstate(all="ignore"):
        q = np.clip(np.rint((v32 / step[:, None]).astype(F32)), -127, 127)
    q[~finite] = 0
    step[~finite] = np.nan
    return q.astype(np.int8), step
