"""Plain fp64 numpy forms of MXFP4 (include/qat_mx.h): quantisation, values, product.

OCP Microscaling Formats specification 1.0: blocks of 32, E8M0 scales, E2M1
elements. Test infrastructure only; shares no code with the kernels.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [rows, cols] float -> (codes [rows, cols] uint8, scale bytes [rows, cols / 32] uint8)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    a = np.abs(b).max(-1)
    odd = ~np.isfinite(b).all(-1)
    a = np.where(odd, 0.0, a)
    e = np.where(a > 0, np.frexp(a)[1] - 1 - 2, -127)      # frexp: a = m 2^ex, m in [0.5, 1)
    e = np.maximum(e, -127)
    y = np.ldexp(np.where(odd[..., None], 0.0, b), -e[..., None])
    mag = np.minimum(np.abs(y), 6.0)
    dist = np.abs(mag[..., None] - GRID)
    # nearest; of two equally near codes the even one
    best = dist.min(-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    codes = pick.astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 3)
    codes = np.where(odd[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(rows, cols), np.where(odd, 255, e + 127).astype(np.uint8)


def pack(codes):
    return (codes[:, ::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, ::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def values(codes, scales):
    """fp64 values of codes [rows, cols] and scale bytes [rows, cols / 32]."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    e = scales.astype(np.int64) - 127
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, np.minimum(e, 127)))
    return v * np.repeat(s, 32, axis=1)


def gemm(xv, wv):
    """(product, sum of |products|) of values [M, in] and [out, in]."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T
