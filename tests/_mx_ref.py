"""64-bit NumPy forms of the MXFP4 tensors and the expert dispatch, written from
their definitions for the tests: brute force over the e2m1 values, Python sorts."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x float64 [R][C] -> (codes uint8 [R][C/2], scales uint8 [C/128][R][4])."""
    R, C = x.shape
    v = x.reshape(R, C // 32, 32)
    with np.errstate(invalid="ignore"):
        m = np.abs(v).max(-1)
    bad = ~np.isfinite(m)
    # frexp: m = f 2^e with f in [0.5, 1), so floor(log2 m) = e - 1
    e = np.frexp(np.where(bad | (m == 0), 1.0, m))[1] - 1 - 2
    e = np.where(m == 0, -127, np.clip(e, -127, 125))
    u = np.where(bad[..., None], 0.0, v) * np.exp2(-e.astype(np.float64))[..., None]
    d = np.abs(np.abs(u)[..., None] - GRID)
    # nearest; of two equally near the even code
    best = d.min(-1, keepdims=True)
    code = np.where(d == best, np.where(np.arange(8) % 2 == 0, np.arange(8), np.arange(8) + 100), 1000).min(-1) % 100
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(u)).astype(np.uint8).reshape(R, C)
    scales = np.where(bad, 255, e + 127).astype(np.uint8).reshape(R, C // 128, 4).transpose(1, 0, 2)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.ascontiguousarray(scales)


def values(codes, scales):
    """The float64 values [R][C]."""
    R = codes.shape[0]
    n = np.stack([codes & 15, codes >> 4], -1).reshape(R, -1)
    v = GRID[n & 7] * np.where(n & 8, -1.0, 1.0)
    b = scales.transpose(1, 0, 2).reshape(R, -1).astype(np.int64)
    s = np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def transposed(x):
    """x^T with its columns padded with zeros to a multiple of 128."""
    pad = -x.shape[0] % 128
    return np.concatenate([x, np.zeros((pad, x.shape[1]))]).T.copy()


def sort(ids, E):
    """(counts, offsets, perm, pos) of ids [M][k]."""
    flat = ids.reshape(-1).tolist()
    kept = sorted((a for a, e in enumerate(flat) if 0 <= e < E), key=lambda a: flat[a])
    counts = np.zeros(E, np.int32)
    for a in kept:
        counts[flat[a]] += 1
    perm = np.full(len(flat), -1, np.int32)
    perm[:len(kept)] = kept
    pos = np.full(len(flat), -1, np.int32)
    pos[kept] = np.arange(len(kept))
    return counts, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), perm, pos.reshape(ids.shape)
