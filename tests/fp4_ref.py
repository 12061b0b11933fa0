"""MXFP4 and token dispatch in numpy doubles, for the tests of those operators."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([GRID, -GRID])


def half_step(dtype, v):
    """Most that rounding v to `dtype` can be off: half a step relative to the value, and where the value is below
    the smallest normal number (fp16: 2^-14) half of the constant step there (fp16: 2^-24 / 2)."""
    f = torch.finfo(dtype)
    return np.maximum(f.eps / 2 * np.abs(v), f.smallest_normal * f.eps / 2)


def within(got, want, tol):
    """Every |got - want| <= tol, compared in doubles (a hair of slack for the comparison's own rounding)."""
    return bool((np.abs(got - want) <= tol * (1 + 1e-9)).all())


def scale_bytes(x):
    """Scale byte of every block of 32 of x [..., K]; 255 where a block holds a NaN or an infinity."""
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    top = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    exp = np.frexp(top)[1] - 3                      # frexp: top = m 2^e, 0.5 <= m < 1
    byte = np.where(top > 0, np.maximum(exp + 127, 0), 0)
    return np.where(bad, 255, byte)


def quantize(x):
    """(code numbers 0..15, scale bytes) of x [..., K]: the nearest number, a tie to the even code."""
    byte = scale_bytes(x)
    scale = np.ldexp(1.0, np.where(byte == 255, 0, byte - 127)).repeat(32, -1)
    nan = (byte == 255).repeat(32, -1)
    v = np.where(nan, 0.0, np.asarray(x, dtype=np.float64)) / scale
    d = np.abs(np.abs(v)[..., None] - GRID)
    near = d.argmin(-1)                             # the lower of two at the same distance
    tie = np.take_along_axis(d, np.minimum(near + 1, 7)[..., None], -1)[..., 0] == d.min(-1)
    code = np.where(tie & (near < 7) & (near % 2 == 1), near + 1, near)
    return np.where(nan, 0, code + 8 * (np.signbit(v) & ~nan)), byte


def unpack(codes):
    """uint8 [..., K/2] -> code numbers [..., K]."""
    c = np.asarray(codes)
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,))


def rows_of_scales(scales, K):
    """uint8 [G, chunks, rows, 4] -> scale bytes [G, rows, K/32]."""
    s = np.asarray(scales).transpose(0, 2, 1, 3)
    return s.reshape(s.shape[0], s.shape[1], -1)[..., :K // 32].astype(np.int64)


def dequantize(codes, scales):
    """float64 [G, rows, K] of (codes, scales) in the library's layout."""
    n = unpack(codes)
    byte = rows_of_scales(scales, n.shape[-1])
    scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return VALUES[n] * scale.repeat(32, -1)


def pack(code, byte):
    """Code numbers [G, rows, K] and scale bytes [G, rows, K/32] -> (codes, scales) in the library's layout."""
    G, rows, K = code.shape
    pairs = code.reshape(G, rows, K // 2, 2).astype(np.uint8)
    full = np.zeros((G, rows, (K + 127) // 128 * 4), dtype=np.uint8)
    full[..., :K // 32] = byte
    return pairs[..., 0] | (pairs[..., 1] << 4), np.ascontiguousarray(
        full.reshape(G, rows, -1, 4).transpose(0, 2, 1, 3))


def sort_tokens(idx, E):
    """(offsets, slot_row) by walking the slots expert by expert."""
    flat = np.asarray(idx).reshape(-1)
    rows = np.full(flat.shape, -1, dtype=np.int32)
    offsets, at = [0], 0
    for e in range(E):
        for i in np.flatnonzero(flat == e):
            rows[i] = at
            at += 1
        offsets.append(at)
    return np.array(offsets, dtype=np.int32), rows.reshape(np.asarray(idx).shape)


def routing(rng, T, k, E, drop=0.0, skew=0.0):
    """topk_idx [T, k] int32: distinct experts a token (k <= E), some tokens and some slots without one."""
    p = (1.0 / np.arange(1, E + 1) ** skew)
    p /= p.sum()
    idx = np.stack([rng.choice(E, size=k, replace=k > E, p=p) for _ in range(T)]).astype(np.int32)
    if drop:
        idx[rng.random(T) < drop] = -1
        idx[rng.random((T, k)) < drop / 2] = -1
    return idx
