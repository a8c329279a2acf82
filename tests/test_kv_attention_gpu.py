"""Attention over the paged 4-bit cache against attention in 64 bits over the
values the cache holds.

Tolerances, for a row with weights p_j (their sum is 1) over L keys: the score
of key j is off by at most e_j = (D + 8) 2^-24 sm_scale sum_d |q_d K_jd| (D
products and sums in fp32, then a few factors) in natural units, with e = max_j
e_j; a weight is rounded to 11 bits (2^-11 relative), its exponential is off by
2^-21, and the sums over L keys lose at most L 2^-24 each.  So out is off by at
most (2^-11 + 2^-20 + 2 e + 2 L 2^-24) sum_j p_j |V_j|, plus half a step of its
type; lse by e + L 2^-24 + 2^-21 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import cache_reference as ref
from precision_activation_quantization_b200 import pqg

pytestmark = pytest.mark.gpu

G_SCALE = (84.0, 42.0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = torch.tensor(ref.E2M1)


def build(lens, P, H, D, fmt, seed=0, spread=(118, 127), table_pad=2, extra=3):
    """A cache whose used slots hold random codes and scales, with every other
    slot (also the rest of a last page) at the largest code and a scale byte of
    0xFF, which is no number; and its page table."""
    rng = np.random.default_rng(seed)
    used = [-(-n // P) for n in lens]
    pages = sum(used) + extra
    width = max(1, max(used, default=1)) + table_pad
    table = np.full((len(lens), width), -1, np.int32)
    order = rng.permutation(pages)[:sum(used)]
    live = np.zeros((pages, P), bool)
    for b, n in enumerate(used):
        table[b, :n] = order[sum(used[:b]):sum(used[:b + 1])]
        for i in range(n):
            live[table[b, i], :min(P, lens[b] - i * P)] = True
    g = torch.Generator(device="cuda").manual_seed(seed)
    live = torch.from_numpy(live).cuda()
    args = []
    for _ in range(2):
        codes = torch.randint(0, 256, (pages, H, P, D // 2), generator=g, device="cuda", dtype=torch.uint8)
        args.append(torch.where(live[:, None, :, None], codes, 0x77).contiguous())
    lo, hi = spread if fmt == "mxfp4" else (24, 100)      # E4M3 2^-4 .. 24 over g
    for _ in range(2):
        sc = torch.randint(lo, hi, (pages, H, D // ref.GROUP[fmt], P), generator=g, device="cuda", dtype=torch.uint8)
        args.append(torch.where(live[:, None, None, :], sc, 0xFF).contiguous())
    gs = torch.tensor(G_SCALE, device="cuda") if fmt == "nvfp4" else None
    return pqg.kv_cache(*args, fmt=fmt, global_scale=gs), torch.from_numpy(table).cuda()


def values(codes, scales, fmt, g):
    """float64 [.., P, D] of codes [.., P, D/2] and scales [.., D/G, P]."""
    t = E2M1.to(codes.device)
    v = torch.stack((t[(codes & 15).long()], t[(codes >> 4).long()]), -1).flatten(-2)
    s = scales.transpose(-1, -2)
    s = torch.exp2(s.double() - 127) if fmt == "mxfp4" else s.view(torch.float8_e4m3fn).double() / float(np.float32(g))
    return v * s.repeat_interleave(ref.GROUP[fmt], -1)


def reference(q, c, table, lens, q_len, sm_scale):
    """(out, lse, weighted |V|, score error bound) in float64."""
    T, Hq, D = q.shape
    H, P = c.kv_heads, c.page_size
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    absv, lse = torch.zeros_like(out), torch.full((T, Hq), -torch.inf, dtype=torch.float64, device="cuda")
    err = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = table[b, :-(-n // P)].long()
        good = ((pages >= 0) & (pages < c.num_pages)).repeat_interleave(P)[:n]
        pg = pages.clamp(0, c.num_pages - 1)
        k, v = (values(x[pg], s[pg], c.fmt, g).transpose(0, 1).flatten(1, 2)[:, :n] for x, s, g in
                ((c.k_codes, c.k_scales, G_SCALE[0]), (c.v_codes, c.v_scales, G_SCALE[1])))
        for t in range(q_len):
            seen = good & (torch.arange(n, device="cuda") < n - (q_len - 1 - t))
            if not bool(seen.any()):
                continue
            x = q[b * q_len + t].double().view(H, Hq // H, D)
            kk, vv = k[:, seen], v[:, seen]
            s = x @ kk.transpose(1, 2) * sm_scale
            l = torch.logsumexp(s, -1)
            p = (s - l[..., None]).exp()
            i = b * q_len + t
            out[i], lse[i] = (p @ vv).flatten(0, 1), l.flatten()
            absv[i] = (p @ vv.abs()).flatten(0, 1)
            err[i] = (x.abs() @ kk.abs().transpose(1, 2)).amax(-1).flatten() * abs(sm_scale) * (D + 8) * 2.0 ** -24
    return out, lse, absv, err


def compare(got, lse, want, in_dtype, lens, what=""):
    out, wl, absv, err = want
    L = max(list(lens) + [1])
    half = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[in_dtype]
    tol = (2.0 ** -11 + 2.0 ** -20 + 2 * err[..., None] + 2 * L * 2.0 ** -24) * absv
    tol = tol + half * (out.abs() + tol) + 2.0 ** -25
    d = (got.double() - out).abs()
    assert torch.isfinite(got).all(), what
    assert (d <= tol).all(), f"{what}: {int((d > tol).sum())} off, worst {float((d / tol).max()):.2f} of the bound"
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty), what
    assert (got[empty] == 0).all(), what
    e = (lse.double() - wl)[~empty].abs()
    assert (e <= (err + L * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * wl.abs())[~empty]).all(), what


def check(lens, q_len, Hq, H, D, P, fmt, in_dtype, seed=0, sm_scale=None, max_len=0, strided=False,
          spread=(118, 127), q_size=1.0, table_pad=2):
    c, table = build(lens, P, H, D, fmt, seed, spread, table_pad)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    T = len(lens) * q_len
    wide = torch.randn(T, (Hq + 2 * H) * D, generator=g, device="cuda").mul_(q_size).to(DT[in_dtype])
    q = wide[:, :Hq * D].unflatten(1, (Hq, D))
    q = q if strided else q.contiguous()
    sm_scale = D ** -0.5 if sm_scale is None else sm_scale
    out = torch.full((T + 1, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T + 1, Hq), 7.0, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pqg.kv_attention(q, c, table, n, sm_scale=sm_scale, max_len=max_len, out=out[:T], lse=lse[:T])
    torch.cuda.synchronize()
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    compare(out[:T], lse[:T], reference(q, c, table, lens, q_len, sm_scale), in_dtype, lens,
            f"{lens} q_len {q_len} heads {Hq}/{H} D {D} P {P} {fmt} {in_dtype}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("in_dtype", ["bf16", "fp16"])
def test_types_and_head_dims(D, fmt, in_dtype):
    check([1], 1, 4, 1, D, 16, fmt, in_dtype)
    check([70, 0, 33, 16, 1], 1, 8, 2, D, 16, fmt, in_dtype, seed=1)
    check([300, 517], 1, 12, 3, D, 64, fmt, in_dtype, seed=2, strided=True)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("in_dtype", ["bf16", "fp16"])
def test_written_rows_against_the_oracle(fmt, in_dtype):
    """Keys and values written by kv_write: the cache holds the oracle's codes, and three tokens'
    attention over it is that of the oracle's values in numpy, within compare()'s bound."""
    from test_rmsnorm_gpu import dev, host
    lens, q_len, P, H, D = [37, 5], 3, 16, 2, 64
    gs = torch.tensor(G_SCALE, device="cuda") if fmt == "nvfp4" else None
    c = pqg.kv_allocate(6, P, H, D, fmt=fmt, global_scale=gs)
    table = np.array([[4, 0, 2], [5, -1, -1]], np.int32)
    rng = np.random.default_rng(3)
    kv = [host(torch.from_numpy(rng.standard_normal((sum(lens), H, D)).astype(np.float32)).to(DT[in_dtype])) for _ in range(2)]
    at = [(int(table[b, j // P]), j % P) for b, n in enumerate(lens) for j in range(n)]
    slots = torch.tensor([p * P + o for p, o in at], dtype=torch.int32, device="cuda")
    pqg.kv_write(c, dev(kv[0], in_dtype), dev(kv[1], in_dtype), slots)
    q = torch.from_numpy(rng.standard_normal((len(lens) * q_len, 2 * H, D)).astype(np.float32)).to(DT[in_dtype])
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = pqg.kv_attention(q.cuda(), c, torch.from_numpy(table).cuda(), n, return_lse=True)
    held = []
    for bits, codes, g in zip(kv, (c.k_codes, c.v_codes), G_SCALE):
        got, scales = ref.quantise(bits.reshape(-1, D), fmt, g, in_dtype)
        rows = [ref.row(codes.cpu().numpy(), p, o, h) for p, o in at for h in range(H)]
        assert (np.stack(rows) == got).all()
        held.append(ref.held(got, scales, fmt, g).reshape(-1, H, D))
    first = 0
    for b, length in enumerate(lens):
        k, v = (x[first:first + length] for x in held)
        qb = q[b * q_len:(b + 1) * q_len].double().numpy()
        wo, wl = ref.attention(qb, k, v, D ** -0.5)
        big = np.abs(v).max(0).repeat(2, 0)[None]              # at least sum p |V|
        err = np.abs(qb).sum(-1) * np.abs(k).max() * D ** -0.5 * (D + 8) * 2.0 ** -24
        want = [torch.from_numpy(x).cuda() for x in (wo, wl, np.broadcast_to(big, wo.shape).copy(), err)]
        compare(out[b * q_len:(b + 1) * q_len], lse[b * q_len:(b + 1) * q_len], want, in_dtype, [length])
        first += length


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16, 33])
def test_head_groups(group):
    check([65, 130], 1, 2 * group, 2, 128, 32, "mxfp4", "bf16", seed=group)
    check([40], 2, group, 1, 64, 16, "nvfp4", "bf16", seed=group)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_every_tail(P):
    """Lengths around the edges of tiles and pages."""
    for lens in ([15, 16, 17, 31, 32, 33], [47, 48, 49, 63, 64, 65, 127, 128, 129], [255, 256, 257, 511, 513]):
        check(lens, 1, 8, 2, 64, P, "mxfp4", "bf16", seed=P)
        check(lens, 1, 4, 1, 128, P, "nvfp4", "fp16", seed=P + 1)


@pytest.mark.parametrize("q_len", [2, 3, 4, 7, 16])
def test_several_tokens(q_len):
    """Also sequences shorter than their new tokens: the first rows see no key."""
    check([100, 1, 0, 33, q_len - 1, q_len, 600], q_len, 8, 2, 128, 32, "nvfp4", "bf16", seed=q_len)
    check([64, 2], q_len, 5, 5, 64, 16, "mxfp4", "fp16", seed=q_len)


def test_long_sequences_are_split_and_joined():
    check([20000], 1, 8, 1, 128, 64, "mxfp4", "bf16")
    check([9000, 40, 5000, 0, 12345], 1, 16, 4, 128, 64, "nvfp4", "fp16", seed=1)
    check([7000], 3, 40, 2, 64, 16, "mxfp4", "bf16", seed=2)
    check([5000], 1, 3, 1, 256, 128, "nvfp4", "bf16", seed=3)


@pytest.mark.parametrize("max_len", [1, 100, 1000, 5000, 1 << 20])
def test_the_length_hint_changes_nothing_but_the_split(max_len):
    check([3000, 17, 999], 1, 8, 2, 128, 16, "mxfp4", "bf16", seed=3, max_len=max_len, table_pad=400)


def test_sharp_and_flat_softmax():
    check([700, 90], 1, 8, 2, 128, 32, "mxfp4", "bf16", q_size=40.0)          # one key takes all
    check([700, 90], 1, 8, 2, 128, 32, "nvfp4", "fp16", q_size=0.0)           # all keys alike
    check([700], 1, 8, 2, 128, 32, "nvfp4", "bf16", sm_scale=-0.3, seed=1)
    check([700], 1, 8, 2, 128, 32, "mxfp4", "bf16", sm_scale=0.0, seed=1)


def test_scales_far_apart():
    """Groups whose scales span 2^40, and queries far from one in size."""
    check([400, 31], 1, 8, 2, 128, 16, "mxfp4", "bf16", spread=(90, 131), sm_scale=1e-2)
    check([400, 31], 2, 8, 2, 64, 16, "mxfp4", "fp16", spread=(96, 128), sm_scale=1e-2)
    check([200], 1, 4, 1, 128, 16, "mxfp4", "bf16", spread=(20, 30), sm_scale=1.0, q_size=2.0 ** 90)
    check([200], 1, 4, 1, 64, 16, "mxfp4", "bf16", spread=(200, 206), sm_scale=1.0, q_size=2.0 ** -80)
    check([200], 1, 4, 1, 128, 16, "mxfp4", "fp16", spread=(118, 127), q_size=20000.0, sm_scale=1e-6)


@pytest.mark.parametrize("in_dtype,fmt,wide", [("bf16", "mxfp4", 24), ("bf16", "mxfp4", 30), ("fp16", "mxfp4", 20),
                                               ("bf16", "nvfp4", 12), ("fp16", "nvfp4", 12)])
def test_queries_of_unequal_elements(in_dtype, fmt, wide):
    """The first group's query elements are 2^wide times the others', its keys' scales as much
    smaller, so that all groups weigh alike.  An element is off by 2^-39 of the row's largest, so a
    score by sm_scale 2^-39 max |q| sum_d |K_d| more than compare()'s bound has."""
    D, G, lens = 64, ref.GROUP[fmt], [300, 31]
    c, table = build(lens, 32, 2, D, fmt, spread=(125, 128))
    if fmt == "mxfp4":
        c.k_scales[:, :, 0] -= torch.where(c.k_scales[:, :, 0] < 0xFF, wide, 0).to(torch.uint8)
    else:                                                  # 2^-6, against 2^6 and more
        c.k_scales[:, :, 0], c.k_scales[:, :, 1:] = 0x08, 0x68
    q = torch.randn(2, 8, D, device="cuda")
    q[..., :G] *= 2.0 ** wide
    q = (q * (2.0 ** -8 if in_dtype == "fp16" else 1.0)).to(DT[in_dtype])
    sm = 2.0 ** 5 if in_dtype == "fp16" and fmt == "mxfp4" else 0.125
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = pqg.kv_attention(q, c, table, n, sm_scale=sm, return_lse=True)
    want = list(reference(q, c, table, lens, 1, sm))
    for b, length in enumerate(lens):
        pg = table[b, :-(-length // 32)].long()
        k = values(c.k_codes[pg], c.k_scales[pg], fmt, G_SCALE[0]).transpose(0, 1).flatten(1, 2)[:, :length]
        size = k.abs().sum(-1).amax(-1).repeat_interleave(4)
        want[3][b] += sm * 2.0 ** -39 * q[b].double().abs().amax(-1) * size
    assert want[3].max() < 0.2
    compare(out, lse, want, in_dtype, lens)


def test_scales_near_the_ends():
    """MXFP4 keys' scales up to 2^117 (with codes and queries: sums of 2^124), and down to 2^-126."""
    check([200], 1, 4, 1, 64, 32, "mxfp4", "bf16", spread=(238, 245), sm_scale=1.0, q_size=2.0 ** -116)
    check([200], 1, 9, 1, 256, 16, "mxfp4", "bf16", spread=(1, 8), sm_scale=1.0, q_size=2.0 ** 112)


def sink(B, L, H, fmt, at, gap, v_byte, D=64, P=64):
    """Sequences of L keys: key ``at`` has a score 2^gap above all the others, which are alike,
    and values of zero; the others' values are all 1 under the scale v_byte.  Returns (cache, table,
    sm_scale) for queries of one 1 and zeros."""
    c, table = build([L] * B, P, H, D, fmt)
    c.k_codes.zero_()
    c.k_scales.fill_(127 if fmt == "mxfp4" else 0x38)     # 1 (under g for nvfp4)
    c.v_scales.fill_(v_byte)
    c.v_codes.fill_(0x22)
    pages, off = table[:, at // P].long(), at % P
    c.v_codes[pages, :, off] = 0
    c.k_codes[pages, :, off, 0] = 0x02
    return c, table, gap * np.log(2.0) * (1.0 if fmt == "mxfp4" else G_SCALE[0])


@pytest.mark.parametrize("fmt,v_byte", [("mxfp4", 160), ("nvfp4", 0x7E)])
@pytest.mark.parametrize("gap", [20.0, 30.4, 33.0])
@pytest.mark.parametrize("B,L,H,at", [(1, 131072, 1, 0), (1, 131072, 1, 131071), (1, 500, 1, 40),
                                      (100, 1024, 8, 0), (100, 1024, 8, 700)])
def test_a_tail_far_below_one_key_keeps_its_weight(fmt, v_byte, gap, B, L, H, at):
    """One key takes nearly all weight and has values of zero: the result is the tail's, whose
    weights are 2^-20 to 2^-33.  Each is off by 2^-36 of the largest, whose weight is below 1, and all
    values of the tail are alike: 2^-36 (L - 1) v is added to compare()'s bound.  Few units, cut into
    pieces, and many, where the warp that has met the large key takes a quarter of the tail too."""
    c, table, sm = sink(B, L, H, fmt, at, gap, v_byte)
    n = torch.full((B,), L, dtype=torch.int32, device="cuda")
    v = float(values(c.v_codes[:1], c.v_scales[:1], fmt, G_SCALE[1]).max())
    for group in (1, 12):
        q = torch.zeros(B, group * H, 64, device="cuda", dtype=torch.bfloat16)
        q[..., 0] = 1.0
        out, lse = pqg.kv_attention(q, c, table, n, sm_scale=sm, return_lse=True)
        wo, wl, absv, err = reference(q, c, table, [L] * B, 1, sm)
        tol = (2.0 ** -11 + 2.0 ** -20 + 2 * err[..., None] + 2 * L * 2.0 ** -24) * absv + 2.0 ** -36 * (L - 1) * v
        tol = tol + 2.0 ** -8 * (wo + tol)
        assert ((out.double() - wo).abs() <= tol).all(), (float(out[0, 0, 0]), float(wo[0, 0, 0]))
        assert (wo > 0.8 * (L - 1) * v * 2.0 ** -gap).all() and (tol < 0.2 * wo).all()
        assert ((lse.double() - wl).abs() <= err + L * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * wl.abs()).all()


@pytest.mark.parametrize("e", [22, 24, 25, 26, 27, 28, 30])
def test_scores_as_coarse_as_the_weights_range(e):
    """Scores of about 2^e in log2 units, whose fp32 neighbours are 2^(e - 23) apart: the later keys
    are one, two or three of those above the earlier ones, and no weight leaves binary16.

    Every score is exact, so compare()'s error of the scores is 0: of an element's product 4 q_0 or
    q_32 each is the only one of its group, a power of two (times 1, 2 or 3) within 24 bits of
    the other; and fp32(ln 2) times log2(e), rounded to fp32, is 1."""
    L, B, H = 1024, 100, 8                                # a block takes several pieces of a unit
    c, table = build([L] * B, 64, H, 64, "mxfp4")
    c.k_scales.fill_(127)
    c.k_codes.zero_()
    c.k_codes[..., 0] = 0x06                              # 4
    for b in range(B):
        c.k_codes[table[b, 8:16].long(), :, :, 16] = 0x02     # 1, of keys 512 and on
    q = torch.zeros(B, 2 * H, 64, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** (e - 2)
    q[..., 32] = (2.0 ** (e - 23) * (1 + torch.arange(B, device="cuda") % 3))[:, None].bfloat16()
    n = torch.full((B,), L, dtype=torch.int32, device="cuda")
    sm = float(np.float32(np.log(2.0)))
    out, lse = pqg.kv_attention(q, c, table, n, sm_scale=sm, return_lse=True)
    want = reference(q, c, table, [L] * B, 1, sm)
    compare(out, lse, want[:3] + (torch.zeros_like(want[3]),), "bf16", [L])


@pytest.mark.parametrize("lens", [[128, 100, 1], [5000, 30000], [2000] * 700])
def test_huge_values_of_many_keys(lens):
    """All keys alike and values up to 2^118: their sum is no fp32 number, their mean is.  In
    whole units, in few and in many units that are split.  Values of one sign, so that the
    mean is as large as they are."""
    c, table = build(lens, 64, 1, 64, "mxfp4", spread=(240, 243))
    c.v_codes.bitwise_and_(0x77)
    c.k_scales.fill_(127)
    q = torch.zeros(len(lens), 2, 64, device="cuda", dtype=torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = pqg.kv_attention(q, c, table, n, return_lse=True)
    want = reference(q, c, table, lens, 1, 0.125)
    assert want[0].amax() > 2.0 ** 114
    compare(out, lse, want, "bf16", lens)


@pytest.mark.parametrize("lens", [[100, 40], [700, 5000], [900] * 300])
@pytest.mark.parametrize("low,high", [(170, 177), (165, 185), (230, 250)])
def test_large_values_beside_larger_ones(lens, low, high):
    """Warps and parts that have met scales of 2^50 and more, which move a power of two to their
    reference, joined with others that have not."""
    c, table = build(lens, 32, 1, 128, "mxfp4", spread=(low, low + 2))
    c.k_scales.fill_(120)
    for b, n in enumerate(lens):                          # every third page
        pages = table[b, :n // 32:3].long()
        c.v_scales[pages] += high - low
    q = torch.randn(len(lens), 4, 128, device="cuda").bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = pqg.kv_attention(q, c, table, n, return_lse=True)
    compare(out, lse, reference(q, c, table, lens, 1, 128 ** -0.5), "bf16", lens)


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_huge_scores(fmt, sign):
    """Every score beyond 1e30 in size, below or above zero: rows see their keys all the same."""
    lens = [70, 30000]
    c, table = build(lens, 32, 2, 128, fmt)
    c.k_codes.bitwise_and_(0x77).bitwise_or_(0x11)                 # no key element is below 0.5 scales
    q = torch.randn(2, 6, 128, device="cuda").abs_().add_(1.0).mul_(1e32).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = pqg.kv_attention(q, c, table, n, sm_scale=sign, return_lse=True)
    want = reference(q, c, table, lens, 1, sign)
    assert (want[1] * sign > 1e30).all()
    compare(out, lse, want, "bf16", lens)
    assert (out != 0).any(-1).all()


def test_bad_pages_are_not_seen():
    lens, P = [100, 64, 40], 16
    c, table = build(lens, P, 2, 64, "mxfp4")
    table[0, 2], table[1, 0], table[2, :] = -5, c.num_pages, 2 ** 30
    q = torch.randn(3, 4, 64, device="cuda", dtype=torch.bfloat16)
    out, lse = pqg.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    compare(out, lse, reference(q, c, table, lens, 1, 64 ** -0.5), "bf16", lens)
    assert (out[2] == 0).all()


def test_sequences_may_share_pages():
    """A common prefix held once, and one sequence listed twice."""
    lens, P = [100, 70], 16
    c, table = build(lens, P, 2, 64, "nvfp4")
    table[1, :4] = table[0, :4]
    table = torch.cat((table, table[:1]))
    lens = [100, 70, 100]
    q = torch.randn(3, 4, 64, device="cuda", dtype=torch.bfloat16)
    q[2] = q[0]
    out, lse = pqg.kv_attention(q, c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    compare(out, lse, reference(q, c, table, lens, 1, 64 ** -0.5), "bf16", lens)
    indptr = torch.tensor([0, 100, 170, 270], dtype=torch.int32, device="cuda")
    k, v = pqg.kv_read(c, table, indptr, 270)
    assert torch.equal(k[:64], k[100:164]) and torch.equal(v[:100], v[170:])


def test_many_sequences():
    """More sequences than a block has threads, and more rows than one wave takes."""
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(0, 200, 300)]
    check(lens, 1, 8, 2, 64, 16, "mxfp4", "bf16", seed=11)
    check([5000] + lens, 1, 4, 1, 128, 16, "nvfp4", "fp16", seed=12)


def test_lengths_outside_the_table_are_clamped():
    c, table = build([48, 48], 16, 1, 64, "nvfp4", table_pad=0)
    q = torch.randn(2, 2, 64, device="cuda", dtype=torch.float16)
    out, lse = pqg.kv_attention(q, c, table, torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32, device="cuda"), return_lse=True)
    compare(out, lse, reference(q, c, table, [48, 0], 1, 64 ** -0.5), "fp16", [48])


def test_masked_queries_are_not_read_into_others():
    """A row that sees nothing, of infinities and not-numbers, leaves the others alone."""
    lens = [2, 300]
    c, table = build(lens, 32, 2, 128, "mxfp4")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(2 * 4, 6, 128, device="cuda", dtype=torch.bfloat16)
    want = pqg.kv_attention(q, c, table, n)
    q2 = q.clone()
    q2[0], q2[1] = torch.inf, torch.nan           # tokens 0 and 1 of the first sequence see no key
    got = pqg.kv_attention(q2, c, table, n)
    assert (got[:2] == 0).all() and torch.equal(got[2:], want[2:])


@pytest.mark.parametrize("D,Hq", [(64, 2), (64, 24), (128, 8), (128, 24), (256, 8)])
@pytest.mark.parametrize("q_len,newest,before", [(2, 90, 40), (5, 90, 40), (40, 90, 40), (3, 27, 26), (4, 125, 121), (150, 60, 30)])
def test_hidden_values_do_not_touch_a_row(D, Hq, q_len, newest, before):
    """The newest token's values are up to 2^125 times the others', and the one's before them
    too: the rows of older tokens, which do not see them, are those of their own keys."""
    H, P = 2, 16
    lens = [q_len, 33 + q_len, 64, 100, 700, 3000]
    c, table = build(lens, P, H, D, "mxfp4", seed=q_len)
    for b, n in enumerate(lens):
        for at, up in ((n - 1, newest), (n - 2, before)):
            c.v_scales[int(table[b, at // P]), :, :, at % P] += up
    q = torch.randn(len(lens) * q_len, Hq, D, device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = pqg.kv_attention(q, c, table, n, return_lse=True)
    compare(out, lse, reference(q, c, table, lens, q_len, D ** -0.5), "bf16", lens)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("byte", [227, 255])
def test_hidden_keys_do_not_touch_a_row(D, byte):
    """The newest token's key has scales of 2^100, or the byte of no scale: rows of the tokens before
    it are those of their own keys, to the bit."""
    lens, q_len, P = [7, 64, 129, 700], 4, 32
    c, table = build(lens, P, 2, D, "mxfp4")
    q = torch.randn(len(lens) * q_len, 6, D, device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = pqg.kv_attention(q, c, table, n, return_lse=True)
    for b, length in enumerate(lens):
        c.k_scales[int(table[b, (length - 1) // P]), :, :, (length - 1) % P] = byte
    got = pqg.kv_attention(q, c, table, n, return_lse=True)
    older = torch.arange(len(q), device="cuda") % q_len < q_len - 1
    assert all(torch.equal(a[older], b[older]) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_nan_query_spoils_its_own_row(fmt):
    """One head's row, in a whole unit and in one that is split; other rows keep their bits."""
    lens = [40, 30000]
    c, table = build(lens, 32, 2, 128, fmt)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 6, 128, device="cuda", dtype=torch.bfloat16)
    want, wl = pqg.kv_attention(q, c, table, n, return_lse=True)
    bad = torch.zeros(2, 6, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 4] = True
    q[0, 1], q[1, 4, 77] = torch.nan, torch.nan
    got, lse = pqg.kv_attention(q, c, table, n, return_lse=True)
    assert got[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(got[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])


def test_deterministic_other_stream_graph_and_two_at_once():
    lens = [5000, 300, 2500]
    c, table = build(lens, 64, 4, 128, "nvfp4")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = [torch.randn(3, 16, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = [pqg.kv_attention(x, c, table, n) for x in q]
    side = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(10):                           # two calls in flight, each with its own scratch
        got = [pqg.kv_attention(x, c, table, n, stream=s) for x, s in zip(q, side)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = [torch.cuda.CUDAGraph() for _ in q]
    outs = []
    for x, g in zip(q, graphs):
        with torch.cuda.graph(g):
            outs.append(pqg.kv_attention(x, c, table, n))
    for _ in range(5):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # lengths are read when the graph runs
    n.copy_(torch.tensor([70, 0, 1], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], pqg.kv_attention(q[0], c, table, n))
    prev = pqg.pqg_set_pdl(False)
    try:
        assert torch.equal(outs[0], pqg.kv_attention(q[0], c, table, n))
    finally:
        pqg.pqg_set_pdl(prev)


def test_a_cache_past_4_gb():
    P, H, D = 256, 8, 256
    pages = (5 << 30) // (P * H * D // 2)
    big = pqg.kv_allocate(pages, P, H, D, fmt="mxfp4")
    c, table = build([300, 511], P, H, D, "mxfp4", table_pad=0, extra=0)
    far = torch.tensor([pages - 1, pages - 2, 2 ** 32 // (P * H * D // 2) + 1, 7], device="cuda")
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        getattr(big, name)[far] = getattr(c, name)
    n = torch.tensor([300, 511], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 16, D, device="cuda", dtype=torch.bfloat16)
    got = pqg.kv_attention(q, big, far[table.long()].to(torch.int32), n)
    assert torch.equal(got, pqg.kv_attention(q, c, table, n))


def test_nothing_to_do():
    c, _ = build([5], 16, 1, 64, "mxfp4")
    before = pqg.pqg_launch_count()
    out = pqg.kv_attention(torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda"), c,
                           torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
                           torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 64) and pqg.pqg_launch_count() == before


def test_refusals():
    c, table = build([40, 20], 16, 2, 64, "mxfp4")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
    bad = [dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q[0]), dict(q=q.cpu()),
           dict(q=torch.zeros(3, 4, 64, dtype=q.dtype, device="cuda")), dict(q=q[:0]),
           dict(seq_lens=n.long()), dict(seq_lens=n[:1]), dict(page_table=table.long()),
           dict(page_table=table[0]), dict(sm_scale=float("inf")), dict(sm_scale=float("nan")),
           dict(out=q.half()), dict(out=q[:1]), dict(lse=torch.zeros(2, 4, device="cuda").half()),
           dict(lse=torch.zeros(4, 2, device="cuda")), dict(out=q), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(q=torch.zeros(2 * 260 + 8, dtype=q.dtype, device="cuda")[4:].as_strided((2, 4, 64), (260, 64, 1)))]
    for kw in bad:
        args = dict(q=q, cache=c, page_table=table, seq_lens=n)
        args.update(kw)
        before = pqg.pqg_launch_count()
        with pytest.raises((ValueError, TypeError, pqg.PqgError)):
            pqg.kv_attention(**args)
        assert pqg.pqg_launch_count() == before
