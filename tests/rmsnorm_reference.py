"""Reference of the norm with quantised output: the residual's addition and the
statistic in numpy (64 bits where the definition has 64), the scales and codes
by the oracle's element functions."""
import math

import numpy as np

import oracle
from precision_activation_quantization_b200 import inputs

FMAX = {"e4m3": 448.0, "int8": 127.0, "e2m1": 6.0}


def add(x_bits, r_bits, in_dtype):
    """h = x + r, one fp32 addition rounded to the 16-bit type, as bits."""
    if r_bits is None:
        return np.ascontiguousarray(x_bits)
    s = oracle.decode(x_bits, in_dtype) + oracle.decode(r_bits, in_dtype)
    return inputs.to_bits(s.astype(np.float32), in_dtype)


def normed(h_bits, w_bits, eps, in_dtype):
    """y [M, K] fp32: (h * inv) * w with inv rounded once from 64 bits.  The sum
    of squares is the exactly rounded one."""
    h = oracle.decode(h_bits, in_dtype)
    w = oracle.decode(w_bits, in_dtype)
    sq = h.astype(np.float64) ** 2
    ss = np.array([math.fsum(row) for row in sq])
    inv = (1.0 / np.sqrt(ss / h.shape[1] + eps)).astype(np.float32)
    return (h * inv[:, None]) * w[None, :]


def quantise(y, group, out_dtype, scale_fmt, global_scale=None):
    """(code bytes [M, K] unpacked, scales [M, K / group]: fp32 values or bytes)."""
    M, K = y.shape
    v = y.reshape(M, K // group, group)
    amax = np.maximum(np.abs(v).max(-1), np.float32(1e-10)).astype(np.float32)
    if scale_fmt == "e4m3":
        scales = oracle.nvfp4_block_scale(amax, global_scale)
        t = v * oracle.nvfp4_multiplier(scales, global_scale)[..., None]
    elif scale_fmt == "ue8m0":
        scales = oracle.ue8m0_exponent_fmax(amax, FMAX[out_dtype])
        t = v * np.exp2(127.0 - scales.astype(np.float64)).astype(np.float32)[..., None]
    else:
        # the norm's own rule: one multiplication by the constant nearest 1 / FMAX
        scales = amax * np.float32(1.0 / FMAX[out_dtype])
        t = (v / scales[..., None]).astype(np.float32)
    t = t.reshape(M, K)
    encode = {"e4m3": oracle.e4m3_encode, "int8": oracle.int8_encode, "e2m1": oracle.e2m1_encode}
    return encode[out_dtype](t).view(np.uint8), scales


def pack_nibbles(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def place(scales, layout, fill):
    """The bytes of one scale plane holding the table ``scales`` [M, ng]."""
    M, ng = scales.shape
    mpad = (M + 3) // 4 * 4
    if layout == "row":
        return np.ascontiguousarray(scales).view(np.uint8).reshape(-1)
    if layout == "col":
        plane = np.full(ng * mpad * scales.itemsize, fill, np.uint8).view(scales.dtype)
        plane.reshape(ng, mpad)[:, :M] = scales.T
        return plane.view(np.uint8)
    if layout == "packed":
        plane = np.full(((ng + 3) // 4, mpad, 4), fill, np.uint8)
        plane[:, :M] = 0
        for g in range(ng):
            plane[g // 4, :M, g % 4] = scales[:, g]
        return plane.reshape(-1)
    plane = np.full((M + 127) // 128 * ((ng + 3) // 4) * 512, fill, np.uint8)
    m = np.arange(M)
    for g in range((ng + 3) // 4 * 4):
        at = ((m // 128) * ((ng + 3) // 4) + g // 4) * 512 + (m % 32) * 16 + (m // 32 % 4) * 4 + g % 4
        plane[at] = scales[:, g] if g < ng else 0
    return plane
