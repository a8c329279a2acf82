"""Reference of the paged 4-bit cache: a row's codes and scale bytes are the
oracle's for a one-group-per-G quantization of it; positions, values and the
attention over them are spelled out in numpy in 64 bits."""
import numpy as np

import oracle

GROUP = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def quantise(bits, fmt, g, in_dtype):
    """Codes [N, D / 2] and scale bytes [N, D / G] of 16-bit rows [N, D]."""
    N, D = bits.shape
    q, s = oracle.quant(bits, M=N, K=D, group=GROUP[fmt], in_dtype=in_dtype, out_dtype="e2m1",
                        scale_fmt="ue8m0" if fmt == "mxfp4" else "e4m3", layout="row",
                        global_scale=None if fmt == "mxfp4" else g)
    return q.reshape(N, D // 2), s.reshape(N, -1)


def scale_values(scales, fmt):
    if fmt == "mxfp4":
        return np.exp2(scales.astype(np.float64) - 127)
    return oracle.e4m3_decode(scales & 0x7F).astype(np.float64)


def held(codes, scales, fmt, g):
    """float64 values of code rows [..., D / 2] with scale bytes [..., D / G]."""
    v = np.stack((E2M1[codes & 15], E2M1[codes >> 4]), -1).reshape(*codes.shape[:-1], -1)
    s = np.repeat(scale_values(scales, fmt), GROUP[fmt], -1)
    return v * s / (1.0 if fmt == "mxfp4" else float(np.float32(g)))


def read_back(codes, scales, fmt, g):
    """The fp32 values that kv_read rounds once: code * scale, times fp32(1 / g)."""
    v = held(codes, scales, fmt, 1.0).astype(np.float32)
    return v if fmt == "mxfp4" else v * (np.float32(1) / np.float32(g))


def row(plane, page, off, head):
    """Codes or scale bytes of (page, head, offset): codes [..., P, D/2], scales [..., D/G, P]."""
    return plane[page, head, off]


def attention(q, k, v, sm_scale):
    """q [n, H * g, D], k and v [len, H, D], all float64: (out, lse); token t of
    the n newest sees the keys before position len - (n - 1 - t)."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    g = Hq // H
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    for t in range(n):
        seen = L - (n - 1 - t)
        if seen <= 0:
            continue
        for h in range(Hq):
            s = k[:seen, h // g] @ q[t, h] * sm_scale
            m = s.max()
            p = np.exp(s - m)
            out[t, h] = p @ v[:seen, h // g] / p.sum()
            lse[t, h] = m + np.log(p.sum())
    return out, lse
