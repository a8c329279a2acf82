"""The paged 4-bit cache: written bytes and read-back values against the
reference, bit for bit, and every byte that must stay as it was."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from gpu_parity import SENTINEL
from precision_activation_quantization_b200 import inputs, pqg

pytestmark = pytest.mark.gpu

G_SCALE = (84.0, 42.0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def rows(n, D, seed, in_dtype):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, D)).astype(np.float32)
    x *= np.exp2(rng.uniform(-9, 4, (n, 1))).astype(np.float32)
    x[rng.random((n, D)) < 0.02] *= np.float32(30.0)
    x[rng.random((n, D)) < 0.02] = -0.0
    x[: n // 7, :32] = 0.0
    return inputs.to_bits(np.clip(x, -60000, 60000), in_dtype)


def dev(bits, in_dtype):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(DT[in_dtype]).cuda()


def filled(pages, P, H, D, fmt, byte=SENTINEL):
    """A cache whose every byte is `byte`, inside larger guarded buffers."""
    g = torch.tensor(G_SCALE, device="cuda") if fmt == "nvfp4" else None
    sizes = [(pages, H, P, D // 2)] * 2 + [(pages, H, D // ref.GROUP[fmt], P)] * 2
    whole = [torch.full((int(np.prod(n)) + 4096,), byte, dtype=torch.uint8, device="cuda") for n in sizes]
    c = pqg.kv_cache(*(w[:-4096].view(n) for w, n in zip(whole, sizes)), fmt=fmt, global_scale=g)
    return c, whole


def expect(planes, k, v, slots, P, H, D, fmt, in_dtype):
    """Place the reference bytes of every live token into copies of the planes."""
    for n, x in enumerate((k, v)):
        codes, scales = ref.quantise(x.reshape(-1, D), fmt, G_SCALE[n], in_dtype)
        codes, scales = codes.reshape(-1, H, D // 2), scales.reshape(len(slots), H, -1)
        for t, s in enumerate(slots):
            if 0 <= s < planes[n].shape[0] * P:
                planes[n][s // P, :, s % P] = codes[t]
                planes[2 + n][s // P, :, :, s % P] = scales[t]
    return planes


def planes(c):
    return [getattr(c, n).cpu().numpy() for n in ("k_codes", "v_codes", "k_scales", "v_scales")]


def check_write(T, pages, P, H, D, fmt, in_dtype, strided, seed=0):
    rng = np.random.default_rng(seed)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    if T > 4:
        slots[[1, T - 1]] = -1
        slots[2] = pages * P                      # just past the cache
        slots[3] = 2 ** 31 - 1
    k, v = rows(T * H, D, seed + 1, in_dtype).reshape(T, H * D), rows(T * H, D, seed + 2, in_dtype).reshape(T, H * D)
    c, whole = filled(pages, P, H, D, fmt)
    if strided:                                   # slices of [q | k | v] rows
        qkv = np.concatenate((np.full((T, 2 * D), 0x7F80, np.uint16), k, v), 1)
        x = dev(qkv, in_dtype)
        kd, vd = (x[:, a:a + H * D].unflatten(1, (H, D)) for a in (2 * D, 2 * D + H * D))
    else:
        kd, vd = dev(k, in_dtype).view(T, H, D), dev(v, in_dtype).view(T, H, D)
    before = planes(c)
    pqg.kv_write(c, kd, vd, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    want = expect(before, k, v, slots, P, H, D, fmt, in_dtype)
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), planes(c), want):
        assert np.array_equal(a, b), f"{name}: {np.argwhere(a != b)[:4].tolist()}"
    assert all((w[-4096:] == SENTINEL).all() for w in whole)
    return c


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("in_dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 64, 8), (256, 32, 1), (128, 128, 5), (64, 256, 2)])
def test_written_bytes(fmt, in_dtype, D, P, H):
    for T, strided in [(1, False), (1, True), (5, True), (16, False), (131, True)]:
        check_write(T, -(-150 // P) + 1, P, H, D, fmt, in_dtype, strided, seed=T)


def check_read(lens, P, H, D, fmt, out_dtype, lead=0, seed=0, bad=False, table_pad=0):
    """Random bytes as the cache's contents (every code; scales of the written range)."""
    rng = np.random.default_rng(seed)
    used = [-(-n // P) for n in lens]
    pages = sum(used) + 2
    c, whole = filled(pages, P, H, D, fmt)
    for n in range(2):
        (c.k_codes, c.v_codes)[n].copy_(torch.from_numpy(rng.integers(0, 256, c.k_codes.shape).astype(np.uint8)))
        lo, hi = (100, 135) if fmt == "mxfp4" else (0, 127)
        (c.k_scales, c.v_scales)[n].copy_(torch.from_numpy(rng.integers(lo, hi, c.k_scales.shape).astype(np.uint8)))
    width = max(1, max(used))
    table = np.full((len(lens), width + table_pad), -1, np.int32)
    order = rng.permutation(pages)[:sum(used)]
    for b, n in enumerate(used):
        table[b, :n] = order[sum(used[:b]):sum(used[:b + 1])]
    if bad:                                       # pages outside the cache
        table[0, 0], table[-1, 0] = -7, pages
    indptr = (np.concatenate(([0], np.cumsum(lens))) + lead).astype(np.int32)
    M = int(indptr[-1]) + 5                       # rows behind the last sequence
    outs = [torch.full((M, H, D), -3.0, dtype=DT[out_dtype], device="cuda") for _ in range(2)]
    tab = torch.from_numpy(table).cuda()[:, :width]
    got = pqg.kv_read(c, tab, torch.from_numpy(indptr).cuda(), M, k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    p = planes(c)
    for n in range(2):
        want = np.full((M, H, D), -3.0, np.float32)
        for b, L in enumerate(lens):
            for j in range(L):
                page = table[b, j // P]
                want[indptr[b] + j] = (0.0 if not 0 <= page < pages else
                                       ref.read_back(p[n][page, :, j % P], p[2 + n][page, :, :, j % P],
                                                     fmt, G_SCALE[n]))
        want = torch.from_numpy(want).to(DT[out_dtype])
        assert torch.equal(got[n].cpu().view(torch.int16), want.view(torch.int16))
    return c


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 64, 2), (256, 32, 1), (128, 256, 1)])
def test_read_back_values(fmt, out_dtype, D, P, H):
    check_read([1], P, H, D, fmt, out_dtype)
    check_read([P, 3 * P + 1, 0, 2 * P - 1, 0], P, H, D, fmt, out_dtype, lead=3, seed=1, table_pad=3)


@pytest.mark.parametrize("fmt,out_dtype", [("mxfp4", "fp16"), ("nvfp4", "bf16")])
@pytest.mark.parametrize("D,P,H", [(64, 16, 8), (128, 32, 5), (256, 64, 3)])
def test_read_many_rows(fmt, out_dtype, D, P, H):
    """Calls large enough to take several rows a thread: sequences of every length
    from 0, starting anywhere, sharing pages; a page outside the cache; a gap before
    the first row and rows behind the last."""
    g = torch.Generator(device="cuda").manual_seed(D)
    pages, rows_wanted = 64, 2 * 4 * 148 * 2048 * 16 // (H * D) + 1000
    c, _ = filled(pages, P, H, D, fmt)
    lo, hi = (100, 135) if fmt == "mxfp4" else (0, 127)
    for n in ("k", "v"):
        codes, scales = getattr(c, n + "_codes"), getattr(c, n + "_scales")
        codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
        scales.copy_(torch.randint(lo, hi, scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    lens = np.random.default_rng(D).integers(0, 9, 1000).tolist() + [0, 1, 2, 3]
    lens += [700] * ((rows_wanted - sum(lens)) // 700 + 1)
    table = torch.randint(0, pages, (len(lens), 700 // P + 1), generator=g, device="cuda", dtype=torch.int32)
    table[5, 0] = pages
    indptr = np.concatenate(([0], np.cumsum(lens))) + 7
    M = int(indptr[-1]) + 9
    ip = torch.from_numpy(indptr.astype(np.int32)).cuda()
    out = [torch.full((M, H, D), -3.0, dtype=DT[out_dtype], device="cuda") for _ in range(2)]
    pqg.kv_read(c, table, ip, M, k_out=out[0], v_out=out[1])
    row = torch.arange(7, M - 9, device="cuda")
    b = torch.bucketize(row, ip[1:].long(), right=True)
    j = row - ip.long()[b]
    page, off = table[b, j // P].long(), j % P
    bad = page >= pages
    page = page.clamp(max=pages - 1)
    e2m1 = torch.tensor(ref.E2M1, dtype=torch.float32, device="cuda")
    for n, (codes, scales) in enumerate(((c.k_codes, c.k_scales), (c.v_codes, c.v_scales))):
        assert (out[n][:7] == -3).all() and (out[n][M - 9:] == -3).all()
        s = scales.transpose(-1, -2)
        s = torch.exp2(s.float() - 127) if fmt == "mxfp4" else s.view(torch.float8_e4m3fn).float()
        x = torch.stack((e2m1[(codes & 15).long()], e2m1[(codes >> 4).long()]), -1).flatten(-2)
        x = x * s.repeat_interleave(ref.GROUP[fmt], -1)
        if fmt == "nvfp4":
            x = x * (torch.ones((), device="cuda") / torch.tensor(G_SCALE[n], device="cuda"))
        want = x.to(DT[out_dtype])[page, :, off]
        want[bad] = 0
        assert torch.equal(out[n][7:M - 9].view(torch.int16), want.view(torch.int16))


def test_read_bad_pages_are_zeros():
    check_read([40, 100, 17], 16, 2, 64, "mxfp4", "bf16", bad=True)


def test_read_rows_past_the_table_are_left():
    """A sequence longer than its table's pages: the rest of its rows stay."""
    c, _ = filled(4, 16, 1, 64, "mxfp4", byte=0x22)
    table = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")
    out = [torch.full((50, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pqg.kv_read(c, table, torch.tensor([0, 50], dtype=torch.int32, device="cuda"), 50, k_out=out[0], v_out=out[1])
    assert (out[0][32:] == 9).all() and (out[0][:32] != 9).all()


def test_read_zero_sequences_and_rows():
    c, _ = filled(2, 16, 1, 64, "mxfp4")
    before = pqg.pqg_launch_count()
    k, v = pqg.kv_read(c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                       torch.zeros(1, dtype=torch.int32, device="cuda"), 0)
    assert k.shape == (0, 1, 64) and pqg.pqg_launch_count() == before
    pqg.kv_write(c, k, v, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert pqg.pqg_launch_count() == before


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_write_then_read_is_quant_then_dequant(fmt):
    """What is read back is within half a code's step of what was written:
    |v' - v| <= step / 2 * scale + roundings, step <= 1/3 of the largest code 6
    times the group's scale; a group's largest magnitude is at most 6 scales."""
    T, H, D, P = 300, 4, 128, 32
    c = pqg.kv_allocate(12, P, H, D, fmt=fmt,
                        global_scale=torch.tensor(G_SCALE, device="cuda") if fmt == "nvfp4" else None)
    k = torch.randn(T, H, D, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(T, H, D, device="cuda", dtype=torch.bfloat16) * 3
    slots = torch.randperm(12 * P, device="cuda")[:T].to(torch.int32)
    pqg.kv_write(c, k, v, slots)
    table = torch.arange(12, dtype=torch.int32, device="cuda")[None]
    got = pqg.kv_read(c, table, torch.tensor([0, 12 * P], dtype=torch.int32, device="cuda"), 12 * P)
    for x, y in zip((k, v), got):
        y = y[slots.long()].double().unflatten(-1, (-1, ref.GROUP[fmt]))
        x = x.double().unflatten(-1, (-1, ref.GROUP[fmt]))
        amax = x.abs().amax(-1, keepdim=True)
        # scale <= 2 amax / 6 (UE8M0 rounds up to a power of two), <= (1 + 2^-4) amax / 6 (E4M3);
        # half of the coarsest step (2) of a code is 1; saturation of a scale rounded down adds 6 * 2^-4
        bound = amax * ((2 / 6) if fmt == "mxfp4" else (1 + 2 ** -4) / 6 + 2 ** -4) + amax * 2 ** -8
        assert ((x - y).abs() <= bound).all()


def test_other_stream_and_graph():
    T, H, D, P = 40, 2, 64, 16
    c, _ = filled(8, P, H, D, "nvfp4")
    k, v = dev(rows(T * H, D, 1, "bf16"), "bf16").view(T, H, D), dev(rows(T * H, D, 2, "bf16"), "bf16").view(T, H, D)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    indptr = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    pqg.kv_write(c, k, v, slots)
    want = pqg.kv_read(c, table, indptr, T)
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pqg.kv_write(c, k, v, slots, stream=side)
    got = pqg.kv_read(c, table, indptr, T, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    raw = pqg.kv_read(c, table, indptr, T, stream=side.cuda_stream)      # a raw handle
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, raw))
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pqg.kv_write(c, k, v, slots)
        got = pqg.kv_read(c, table, indptr, T)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_cache_past_4_gb():
    """Pages whose byte offsets pass 32 bits."""
    P, H, D = 256, 8, 256
    pages = (5 << 30) // (P * H * D // 2)
    c = pqg.kv_allocate(pages, P, H, D, fmt="mxfp4")
    far = [pages - 1, 2 ** 32 // (P * H * D // 2) + 3, 5]
    slots = torch.tensor([f * P + 9 for f in far], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(3, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pqg.kv_write(c, k, v, slots)
    small = pqg.kv_allocate(1, P, H, D, fmt="mxfp4")
    pqg.kv_write(small, k, v, torch.arange(3, dtype=torch.int32, device="cuda"))
    for name in ("k_codes", "v_codes"):
        for i, f in enumerate(far):
            assert torch.equal(getattr(c, name)[f, :, 9], getattr(small, name)[0, :, i])
    assert int(c.k_codes[0].max()) == 0 and int(c.k_codes[6].max()) == 0
    table = torch.tensor([far], dtype=torch.int32, device="cuda")
    got = pqg.kv_read(c, table, torch.tensor([0, 3 * P], dtype=torch.int32, device="cuda"), 3 * P)
    want = pqg.kv_read(small, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                       torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 3)
    assert torch.equal(got[0][9::P], want[0]) and torch.equal(got[1][9::P], want[1])


def test_refusals():
    c, _ = filled(4, 16, 2, 64, "mxfp4")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [dict(k=k.float()), dict(v=k.half()), dict(k=k[:, :1]), dict(v=k[:2]), dict(k=k.cpu()),
           dict(slots=slots.long()), dict(slots=slots[:2]), dict(slots=slots.cpu()),
           dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(k=torch.zeros(3, 2, 72, dtype=torch.bfloat16, device="cuda")[..., 8:]),
           dict(k=torch.zeros(3 * 130 + 64, dtype=torch.bfloat16, device="cuda").as_strided((3, 2, 64), (130, 64, 1)))]
    for kw in bad:
        args = dict(k=k, v=k.clone(), slots=slots)
        args.update(kw)
        before = pqg.pqg_launch_count()
        with pytest.raises((ValueError, TypeError, pqg.PqgError)):
            pqg.kv_write(c, **args)
        assert pqg.pqg_launch_count() == before
    table, ip = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in [dict(page_table=table.long()), dict(page_table=table.t()), dict(page_table=table[0]),
               dict(indptr=ip[:2]), dict(indptr=ip.float()), dict(dtype=torch.float32),
               dict(k_out=k[:2]), dict(v_out=k.half(), dtype=torch.bfloat16), dict(num_tokens=4, k_out=k)]:
        args = dict(page_table=table, indptr=ip, num_tokens=3)
        args.update(kw)
        with pytest.raises((ValueError, TypeError, pqg.PqgError)):
            pqg.kv_read(c, **args)
    cc, sc = torch.zeros(4, 2, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, 2, 16, dtype=torch.uint8, device="cuda")
    for args, kw in [((cc, cc.clone(), sc, sc[:2]), {}), ((cc, cc.clone(), sc, sc.clone()), dict(fmt="nvfp4")),
                     ((cc, cc.clone(), sc, sc.clone()), dict(global_scale=torch.ones(2, device="cuda"))),
                     ((cc, cc.clone(), sc, sc.clone()), dict(fmt="int4")), ((cc.cpu(), cc, sc, sc), {}),
                     ((cc.float(), cc.clone(), sc, sc.clone()), {})]:
        with pytest.raises(ValueError):
            pqg.kv_cache(*args, **kw)
    same = pqg.kv_cache(cc, cc, sc, sc.clone())              # keys and values in one buffer
    with pytest.raises(pqg.PqgError):
        pqg.kv_write(same, k, k.clone(), slots)
    odd = pqg.kv_allocate(2, 24, 1, 64)                      # page sizes are powers of two
    with pytest.raises(pqg.PqgError):
        pqg.kv_write(odd, k[:, :1].contiguous(), k[:, :1].contiguous(), slots)
