"""Plain numpy forms of cached rows' encodings and of the turning of keys, for
skv_move_rows; written from include/sparsekv.h, used by the tests only."""
from __future__ import annotations

import numpy as np

GROUP = 64


def decode(kind, x, scale):
    """bf16 values as fp32, int8 codes [..][d] with fp16 scales [..], int4 codes [..][d] with scales [..][d/64]: the
    values, exact in fp32."""
    if kind == "bf16":
        return np.asarray(x, np.float32)
    s = np.asarray(scale, np.float32)
    s = np.where(np.isfinite(s), s, 0)
    s = np.repeat(s, GROUP, -1) if kind == "int4" else s[..., None]
    return np.asarray(x, np.float32) * s


def turn(x, angle, interleaved):
    """fp64 x [n][H][d], angle [n][rot/2] -> (z, mag): turned pairs, and for each value |x_a| + |x_b| (0 outside)."""
    x = np.asarray(x, np.float64)
    rot = 2 * angle.shape[1]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z, mag = x.copy(), np.zeros_like(x)
    z[..., a] = x[..., a] * c - x[..., b] * s
    z[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return z, mag


def encode(kind, x):
    """fp32 x [..][d] -> (codes [..][d], scales): int8 one scale per row, int4 one per 64 values."""
    x = np.asarray(x, np.float32)
    top, lowest = (127, -127) if kind == "int8" else (7, -8)
    if kind == "int4":
        x = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        largest = np.fmax.reduce(np.abs(x), -1, initial=np.float32(0))
        scale = (largest / np.float32(top)).astype(np.float16)
        s = scale.astype(np.float32)
        ok = (s != 0) & np.isfinite(s)
        q = np.rint(x / np.where(ok, s, 1)[..., None])
    q = np.clip(np.where(np.isnan(q), lowest, q), lowest, top) * ok[..., None]
    q = q.astype(np.int8)
    return (q.reshape(*q.shape[:-2], -1) if kind == "int4" else q), scale


def pack_int4(codes, scale):
    """Codes [..][d] and fp16 scales [..][d/64] -> bytes [..][d/2 + d/32]."""
    c = codes.astype(np.uint8) & 15
    return np.concatenate([c[..., 0::2] | c[..., 1::2] << 4, np.ascontiguousarray(scale).view(np.uint8)], -1)


def unpack_int4(b):
    d = b.shape[-1] * 32 // 17
    c = np.ascontiguousarray(b[..., :d // 2]).view(np.int8)
    codes = np.stack([(c << 4).astype(np.int8) >> 4, c >> 4], -1).reshape(*c.shape[:-1], d)
    return codes, np.ascontiguousarray(b[..., d // 2:]).view(np.float16)
