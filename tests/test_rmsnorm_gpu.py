"""The norm with quantised output against its reference, bit for bit: codes,
scales, h and every byte the call must not touch."""
import ctypes

import numpy as np
import pytest
import torch

import rmsnorm_reference as ref
from gpu_parity import GUARD, SENTINEL, assert_same
from precision_activation_quantization_b200 import inputs, pqg

pytestmark = pytest.mark.gpu

KINDS = [("e4m3", "fp32", "row", 128), ("e4m3", "fp32", "col", 64), ("int8", "fp32", "row", 32),
         ("int8", "fp32", "col", "K"), ("e4m3", "fp32", "row", "K"), ("e4m3", "ue8m0", "row", 128),
         ("e4m3", "ue8m0", "col", 64), ("e4m3", "ue8m0", "packed", 128),
         ("e4m3", "ue8m0", "packed", 32), ("e4m3", "ue8m0", "packed", "K"),
         ("e4m3", "ue8m0", "tile128x4", 32), ("e4m3", "ue8m0", "tile128x4", "K"),
         ("e2m1", "ue8m0", "tile128x4", 32), ("e2m1", "ue8m0", "packed", 64),
         ("e2m1", "e4m3", "tile128x4", 16), ("e2m1", "e4m3", "col", 16)]


DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rows(M, K, seed, in_dtype):
    """Rows of unequal magnitude with outliers, zeros and an all-zero row."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x *= np.exp2(rng.uniform(-8, 6, (M, 1))).astype(np.float32)
    x[rng.random((M, K)) < 0.01] *= np.float32(40.0)
    x[rng.random((M, K)) < 0.02] = 0.0
    x[:, : min(K, 32)] = 0.0
    if M > 2:
        x[2] = 0.0
    return inputs.to_bits(np.clip(x, -60000, 60000), in_dtype)


def dev(bits, in_dtype):
    dt = torch.float16 if in_dtype == "fp16" else torch.bfloat16
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(dt).cuda()


def host(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def check(M, K, kind, in_dtype="bf16", residual=True, in_place=False, eps=1e-6, seed=0,
          stream=None, gscale=2.625):
    out_dtype, fmt, layout, group = kind
    group = K if group == "K" else group
    x, r, w = rows(M, K, seed, in_dtype), rows(M, K, seed + 1, in_dtype), None
    if residual and M > 2:
        r[2] = x[2] = 0
    w = inputs.to_bits((1 + 0.3 * np.random.default_rng(seed + 2).standard_normal(K)).astype(np.float32),
                       in_dtype)
    nbytes = pqg.pqg_scales_bytes(1, M, K, group, pqg.SCALE_FMTS[fmt], pqg.LAYOUTS[layout])
    n_out = M * (K // 2 if out_dtype == "e2m1" else K)
    full = lambda n: torch.full((n + GUARD,), SENTINEL, dtype=torch.uint8, device="cuda")  # noqa: E731
    out, sc, hb = full(n_out), full(nbytes), full(2 * M * K)
    xd, wd = dev(x, in_dtype), dev(w, in_dtype)
    rd = dev(r, in_dtype) if residual else None
    ho = rd if in_place else hb[:2 * M * K].view(xd.dtype).view(M, K)
    g = torch.tensor([gscale], device="cuda") if fmt == "e4m3" else None
    got = pqg.rmsnorm_quant(xd, wd, rd, out[:n_out], sc[:nbytes], residual_out=ho if residual else None,
                            eps=eps, group=group, out_dtype=out_dtype, scale_fmt=fmt, layout=layout,
                            global_scale=g, stream=stream)
    torch.cuda.synchronize()
    h = ref.add(x, r if residual else None, in_dtype)
    y = ref.normed(h, w, eps, in_dtype)
    codes, scales = ref.quantise(y, group, out_dtype, fmt, gscale)
    if out_dtype == "e2m1":
        codes = ref.pack_nibbles(codes)
    name = f"M{M} K{K} {kind} {in_dtype}"
    assert_same(host(got[2]), h, f"{name} h")
    o, s, b = out.cpu().numpy(), sc.cpu().numpy(), hb.cpu().numpy()
    assert_same(s[:nbytes], ref.place(scales, layout, SENTINEL), f"{name} scales")
    assert_same(o[:n_out], codes, f"{name} codes")
    assert (o[n_out:] == SENTINEL).all() and (s[nbytes:] == SENTINEL).all()
    assert (b[2 * M * K if residual and not in_place else 0:] == SENTINEL).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "_".join(map(str, k)))
@pytest.mark.parametrize("in_dtype", ["bf16", "fp16"])
def test_every_kind_bit_exact(kind, in_dtype):
    for M, K in [(1, 128), (3, 640), (37, 2048), (5, 7168)]:
        if kind[3] == "K" and K > 16384:
            continue
        check(M, K, kind, in_dtype, seed=M + K)


@pytest.mark.parametrize("M,K", [(1, 16), (2, 32), (9, 48), (130, 80), (1, 16384), (7, 16368),
                                 (4, 8192), (3, 4112), (600, 512), (2500, 1024)])
def test_sizes_per_token(M, K):
    check(M, K, ("e4m3", "fp32", "row", "K"), seed=K)
    check(M, K, ("int8", "fp32", "row", "K"), "fp16", residual=False, seed=K)


@pytest.mark.parametrize("M,K,residual", [(767, 4096, False), (768, 4096, True), (2047, 3840, True), (2048, 3840, True),
                                          (2047, 2048, False), (2048, 2064, False), (2100, 2048, True)])
def test_per_token_around_the_choices_of_warps(M, K, residual):
    check(M, K, ("int8", "fp32", "row", "K"), residual=residual, seed=K)


@pytest.mark.parametrize("M,K", [(1, 32), (4, 96), (131, 416), (1, 16384), (3, 8224), (1600, 544)])
def test_sizes_groups(M, K):
    check(M, K, ("e4m3", "ue8m0", "packed", 32), seed=K)
    check(M, K, ("e2m1", "e4m3", "row", 16), "fp16", seed=K)


@pytest.mark.parametrize("residual,in_place", [(False, False), (True, True)])
def test_without_residual_and_in_place(residual, in_place):
    for M, K in [(1, 4096), (67, 1536), (300, 7168)]:
        check(M, K, ("e4m3", "fp32", "row", 128), residual=residual, in_place=in_place, seed=5)


def test_x_may_be_the_output_of_the_sum():
    """residual_out = x: the sum replaces the input."""
    M, K = 33, 1024
    x, r = dev(rows(M, K, 1, "bf16"), "bf16"), dev(rows(M, K, 2, "bf16"), "bf16")
    w = torch.ones(K, dtype=x.dtype, device="cuda")
    want = pqg.rmsnorm_quant(x, w, r)
    got = pqg.rmsnorm_quant(x, w, r, residual_out=x)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert got[2] is x


def test_leading_dimensions_are_rows():
    x, r = (dev(rows(24, 512, s, "bf16"), "bf16") for s in (1, 2))
    w = torch.ones(512, dtype=x.dtype, device="cuda")
    want = pqg.rmsnorm_quant(x, w, r)
    got = pqg.rmsnorm_quant(x.view(2, 12, 512), w, r.view(2, 12, 512))
    assert got[0].shape == (24, 512) and got[2].shape == (2, 12, 512)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.reshape(a.shape).view(torch.uint8))


@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-5, 3.0])
def test_eps(eps):
    # eps = 0 with an all-zero row is outside the contract: M = 2 has none
    check(2, 896, ("e4m3", "ue8m0", "col", 128), eps=eps, seed=9)


def test_zero_rows_launch_nothing():
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    before = pqg.pqg_launch_count()
    out, scales, h = pqg.rmsnorm_quant(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w)
    assert out.shape == (0, 256) and scales.numel() == 0 and pqg.pqg_launch_count() == before


def test_rows_do_not_depend_on_the_batch():
    """A row's bytes are the same alone, among others and in a large call."""
    K = 7168
    x, r = dev(rows(4000, K, 3, "bf16"), "bf16"), dev(rows(4000, K, 4, "bf16"), "bf16")
    w = dev(rows(1, K, 5, "bf16")[0], "bf16")
    many = pqg.rmsnorm_quant(x, w, r)
    for at, n in ((0, 1), (17, 5), (1000, 160), (3999, 1)):
        few = pqg.rmsnorm_quant(x[at:at + n], w, r[at:at + n])
        for a, b in zip(few, many):
            assert torch.equal(a.view(torch.uint8), b[at:at + n].contiguous().view(torch.uint8))


def test_rows_past_4_gb():
    """Rows, codes and scales whose offsets pass 32 bits: as the same rows alone."""
    M, K = 620_000, 7168                                  # 8.9 GB of rows, 4.4 GB of codes
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    w = dev(rows(1, K, 5, "bf16")[0], "bf16")
    at = [0, 299_593, 299_594, 599_186, 599_187, M - 1]   # also around 2^32 bytes of each
    x[at] = dev(rows(len(at), K, 3, "bf16"), "bf16")
    got = pqg.rmsnorm_quant(x, w, x, residual_out=x)
    few = dev(rows(len(at), K, 3, "bf16"), "bf16")
    want = pqg.rmsnorm_quant(few, w, few)
    for a, b in zip(got, want):
        assert torch.equal(a[at].view(torch.uint8), b.view(torch.uint8))
    assert int((got[0][1:299_593].view(torch.uint8) & 0x7F).amax()) == 0   # a zero has its weight's sign


def test_other_stream_graph_and_pdl_off():
    K, M = 2048, 24
    x, r = dev(rows(M, K, 6, "fp16"), "fp16"), dev(rows(M, K, 7, "fp16"), "fp16")
    w = torch.ones(K, dtype=x.dtype, device="cuda")
    want = [t.clone() for t in pqg.rmsnorm_quant(x, w, r, out_dtype="int8")]
    same = lambda got: all(torch.equal(a, b) for a, b in zip(want, got))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pqg.rmsnorm_quant(x, w, r, out_dtype="int8", stream=side)
    side.synchronize()
    assert same(got)
    prev = pqg.pqg_set_pdl(False)
    try:
        assert same(pqg.rmsnorm_quant(x, w, r, out_dtype="int8"))
    finally:
        pqg.pqg_set_pdl(prev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = pqg.rmsnorm_quant(x, w, r, out_dtype="int8")
        second = pqg.rmsnorm_quant(x, w, first[2], out_dtype="int8")   # chained, reads the sum
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert same(first)
    again = pqg.rmsnorm_quant(x, w, first[2], out_dtype="int8")
    assert all(torch.equal(a, b) for a, b in zip(again, second))


def test_against_a_float64_norm():
    """The dequantised output lies within half a step of the norm in 64 bits:
    |code * s - y| <= 2^-4 |y| + 2^-10 s for E4M3, plus 3 fp32 roundings of y
    and one of the scale (each at most 2^-24 relative)."""
    M, K, G = 64, 7168, 128
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    r = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(K, device="cuda", dtype=torch.bfloat16) + 0.5
    q, s, h = pqg.rmsnorm_quant(x, w, r, eps=1e-5, group=G)
    hd = (x.float() + r.float()).to(torch.bfloat16)
    assert torch.equal(h, hd)
    hd = hd.double()
    y = hd / (hd.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w.double()
    step = s.double().repeat_interleave(G, -1)
    err = (q.double() * step - y).abs()
    assert (err <= (2 ** -4 + 2 ** -21) * y.abs() + 2 ** -10 * step).all()


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    bad = [dict(x=x.float()), dict(x=x.t()), dict(x=x[0]), dict(weight=w[:128]), dict(weight=w.half()),
           dict(weight=w.cpu()), dict(residual=x[:2]), dict(residual=x.half()),
           dict(residual_out=x), dict(residual=x, residual_out=x[:, :128]),
           dict(out=torch.empty(4, 128, dtype=torch.uint8, device="cuda")),
           dict(scales=torch.empty(4, 4, device="cuda")), dict(group=96), dict(eps=-1.0),
           dict(eps=float("nan")), dict(out_dtype="int8", scale_fmt="ue8m0"),
           dict(out_dtype="e2m1", scale_fmt="e4m3", group=16),
           dict(residual=x.clone(), residual_out=w.new_empty(5 * 256)[:1024].view(4, 256), scales=x)]
    for kw in bad:
        args = dict(x=x, weight=w)
        args.update(kw)
        before = pqg.pqg_launch_count()
        with pytest.raises((ValueError, TypeError, pqg.PqgError)):
            pqg.rmsnorm_quant(**args)
        assert pqg.pqg_launch_count() == before
    wide = torch.zeros(1, 32768, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pqg.PqgError):
        pqg.rmsnorm_quant(wide, wide[0])


@pytest.mark.parametrize("scale_fmt", ["fp32", "ue8m0"])
@pytest.mark.parametrize("K", [256, 1024, 7168])
def test_infinities_and_nans_stay_in_their_rows(K, scale_fmt):
    x = torch.randn(6, K, device="cuda", dtype=torch.float16)
    w = torch.randn(K, device="cuda", dtype=torch.float16)
    w[w == 0] = 1
    want, ws, _ = pqg.rmsnorm_quant(x, w, scale_fmt=scale_fmt)
    x[1, 5], x[3, K - 1], x[4, 7] = torch.inf, torch.nan, -torch.inf
    got, gs, _ = pqg.rmsnorm_quant(x, w, scale_fmt=scale_fmt)
    g, keep = got.view(torch.uint8), [0, 2, 5]
    assert torch.equal(g[keep], want.view(torch.uint8)[keep]) and torch.equal(gs[keep], ws[keep])
    assert ((g[3] & 0x7F) == 0x7F).all()
    zero = torch.zeros(K, dtype=torch.uint8, device="cuda")
    for row, at in ((1, 5), (4, 7)):
        zero[at] = 0x7F
        assert torch.equal(g[row] & 0x7F, zero)
        zero[at] = 0


@pytest.mark.parametrize("in_dtype,bits", [("bf16", 0x7FC0), ("bf16", 0xFFC0), ("bf16", 0x7F81), ("bf16", 0xFF81),
                                           ("fp16", 0x7E00), ("fp16", 0xFE00)])
@pytest.mark.parametrize("residual", [False, True])
def test_a_nan_of_either_sign_spoils_its_row(in_dtype, bits, residual):
    """Also NaNs with the sign bit set (0xFFC0 is what a host's 0 / 0 leaves) and signalling
    ones; with groups and per token, where few and where many rows split a row differently."""
    for M, K in ((4, 256), (3, 7168), (1100, 1024)):
        x = torch.randn(M, K, device="cuda").to(DT[in_dtype])
        r = torch.randn(M, K, device="cuda").to(DT[in_dtype]) if residual else None
        w = torch.rand(K, device="cuda").to(DT[in_dtype]) + 0.5
        for scale_fmt in ("fp32", "ue8m0"):
            for group in (128, K):
                kw = dict(scale_fmt=scale_fmt, group=group)
                want, ws, _ = pqg.rmsnorm_quant(x, w, r, **kw)
                bad = x.clone()
                bad.view(torch.int16)[1, K - 3] = bits - (1 << 16) if bits >> 15 else bits
                got, gs, _ = pqg.rmsnorm_quant(bad, w, r, **kw)
                g, keep = got.view(torch.uint8), [i for i in range(M) if i != 1]
                assert ((g[1] & 0x7F) == 0x7F).all(), (M, K, kw)
                assert torch.equal(g[keep], want.view(torch.uint8)[keep]) and torch.equal(gs[keep], ws[keep])
