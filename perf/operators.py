"""Measured cases of the operators around the GEMMs of a quantised decoder layer.

``rmsnorm``   residual addition, root-mean-square norm and quantised output
``cache``     keys and values quantised into a paged 4-bit cache and read back
``read``      a 4-bit cache read back into 16-bit keys and values
``attention`` queries of one or a few new tokens against a paged 4-bit cache

With ``own`` false each runs in its plain form (elementary torch operations in
32 bits); with ``own`` true through the library's public entry points.
"""
import math
import random

import torch

own = False

EPS = 1e-10          # floor of a group's absolute maximum
NORM_EPS = 1e-6
GROUP = {"mxfp4": 32, "nvfp4": 16}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token entering a layer: its norm feeds an FP8 GEMM that reads packed exponents
        dict(name="norm_token", op="rmsnorm", M=1, K=7168, dtype="bf16", out="e4m3", fmt="ue8m0",
             layout="packed", group=128, residual=True),
        # a decode batch, one INT8 scale per token
        dict(name="norm_decode", op="rmsnorm", M=96, K=4096, dtype="fp16", out="int8", fmt="fp32",
             layout="row", group=4096, residual=True),
        # the first norm of a short prompt: nothing to add yet, column-major scales, an odd row count
        dict(name="norm_prompt", op="rmsnorm", M=1531, K=2048, dtype="bf16", out="e4m3",
             fmt="fp32", layout="col", group=64, residual=False),
        # prefill of a long prompt at the hidden size of the library's own workloads
        dict(name="norm_prefill", op="rmsnorm", M=8192, K=7168, dtype="bf16", out="e4m3",
             fmt="fp32", layout="row", group=128, residual=True),
        # a decode step's new tokens: 48 live sequences in a batch padded to 64 rows
        dict(name="cache_decode", op="cache", B=48, L=1, pad=16, heads=8, D=128, page=64,
             dtype="bf16", fmt="mxfp4"),
        # long prompts written and read back for their prefill attention
        dict(name="cache_prefill", op="cache", B=4, L=8192, pad=0, heads=8, D=128, page=64,
             dtype="bf16", fmt="nvfp4"),
        # short ragged prefixes, small heads, small pages
        dict(name="read_short", op="read", B=7, L=300, pad=0, heads=4, D=64, page=16,
             dtype="fp16", fmt="nvfp4"),
        # shared prefixes read back before a batch of chunked prefills
        dict(name="read_prefixes", op="read", B=16, L=8192, pad=0, heads=8, D=128, page=64,
             dtype="bf16", fmt="mxfp4"),
        # one user, a short context
        dict(name="attention_short", op="attention", B=1, L=517, q_len=1, q_heads=32, heads=8,
             D=128, page=64, dtype="bf16", fmt="mxfp4"),
        # four drafted tokens of each sequence verified at once, small heads; one sequence is empty
        dict(name="attention_verify", op="attention", B=17, L=2000, q_len=4, q_heads=16, heads=4,
             D=64, page=16, dtype="fp16", fmt="nvfp4"),
        # one user, a long context: few rows over a long axis
        dict(name="attention_long", op="attention", B=1, L=131072, q_len=1, q_heads=64, heads=8,
             D=128, page=64, dtype="bf16", fmt="nvfp4"),
        # a full decode batch of ragged lengths
        dict(name="attention_batch", op="attention", B=64, L=8192, q_len=1, q_heads=32, heads=8,
             D=128, page=64, dtype="bf16", fmt="mxfp4"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rmsnorm", "cache", "read", "attention"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rmsnorm":
        K = 128 * _between(rng, 4, 64)
        out, fmt, layout = rng.choice([("e4m3", "fp32", "row"), ("e4m3", "fp32", "col"),
                                       ("e4m3", "ue8m0", "packed"), ("int8", "fp32", "row")])
        return dict(op=op, M=_between(rng, 1, 8192 * 7168 // K if K > 7168 else 8192), K=K,
                    dtype=dtype, out=out, fmt=fmt, layout=layout,
                    group=rng.choice([32, 64, 128, K]), residual=rng.random() < 0.75)
    fmt = rng.choice(["mxfp4", "nvfp4"])
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("cache", "read"):
        L = _between(rng, 1, 8192)
        B = _between(rng, 1, max(1, min(64, (4 if op == "cache" else 16) * 8192 // L)))
        return dict(op=op, B=B, L=L, pad=rng.choice([0, 0, 5, 32]), heads=heads, D=D, page=page,
                    dtype=dtype, fmt=fmt)
    L = _between(rng, 1, 131072)
    return dict(op=op, B=_between(rng, 1, max(1, min(64, 64 * 8192 // L))), L=L,
                q_len=rng.choice([1, 1, 1, 2, 4]), q_heads=heads * rng.choice([1, 2, 4, 5, 8, 16]),
                heads=heads, D=D, page=page, dtype=dtype, fmt=fmt)


def _lengths(c):
    """Tokens of each sequence: the first has all L, the others are spread
    below; a batch of attention over ten sequences has an empty one."""
    r = random.Random(c["B"] * 1000003 + c["L"])
    n = [c["L"]] + [r.randint(max(1, c["L"] // 8), c["L"]) for _ in range(c["B"] - 1)]
    if c["op"] == "attention" and c["B"] > 10 and c["q_len"] > 1:
        n[3] = 0
    return n


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _activations(shape, g, dtype, spread):
    """Normal values whose last axis has channels of unequal size, as a model's
    hidden states and keys have."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    channel = torch.randn(shape[-1], generator=g, device="cuda").mul_(spread).exp_()
    return x.mul_(channel).to(dtype)


def _pages(c, g):
    """A page table of shuffled pages (entries past a sequence's end: -1) and
    the page count, with a few pages that no sequence uses."""
    used = [-(-n // c["page"]) for n in _lengths(c)]
    total, width = sum(used), max(1, max(used))
    order = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    col = torch.arange(width, device="cuda")
    need = torch.tensor(used, device="cuda")
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device="cuda")
    table[col < need[:, None]] = order
    return table, total + 3


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPE[c["dtype"]]
    s = {"case": c}
    if c["op"] == "rmsnorm":
        s["x"] = _activations((c["M"], c["K"]), g, dt, 0.7)
        s["residual"] = _activations((c["M"], c["K"]), g, dt, 0.7) if c["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(c["K"], generator=g, device="cuda")).to(dt)
        return s
    lens, heads, D, G = _lengths(c), c["heads"], c["D"], GROUP[c["fmt"]]
    s["table"], pages = _pages(c, g)
    P = c["page"]
    cache = {n: torch.zeros((pages, heads, P, D // 2) if "codes" in n else (pages, heads, D // G, P),
                            dtype=torch.uint8, device="cuda")
             for n in ("k_codes", "v_codes", "k_scales", "v_scales")}
    s["cache"] = cache
    # NVFP4: the global scales put magnitudes of 32 (keys) and 64 (values) on 448 * 6
    s["gscale"] = (torch.tensor([448 * 6 / 32.0, 448 * 6 / 64.0], device="cuda")
                   if c["fmt"] == "nvfp4" else None)
    indptr = torch.tensor([0] + lens, device="cuda").cumsum(0)
    s["indptr"], total = indptr.to(torch.int32), sum(lens)
    if c["op"] == "cache":
        # keys and values are slices of one projection's rows, as a layer has them
        T = total + c["pad"]
        qkv = _activations((T, 2 * heads * D), g, dt, 0.5)
        s["k"] = qkv[:, :heads * D].unflatten(1, (heads, D))
        s["v"] = qkv[:, heads * D:].unflatten(1, (heads, D))
        row = torch.arange(T, device="cuda")
        b = torch.bucketize(row, indptr[1:], right=True).clamp(max=c["B"] - 1)
        j = row - indptr[b]
        slot = s["table"][b, (j // P).clamp(max=s["table"].shape[1] - 1)] * P + j % P
        s["slots"] = torch.where(row < total, slot, -1).to(torch.int32)
        s["total"] = total
        return s
    for n, spread, gi in (("k", 0.5, 0), ("v", 0.2, 1)):     # filled a few hundred pages at a time
        for at in range(0, pages, 512):
            x = _activations((min(512, pages - at), heads, P, D), g, dt, spread)
            codes, scales = _quantise(x, c["fmt"], s["gscale"][gi] if s["gscale"] is not None else None)
            cache[n + "_codes"][at:at + 512] = codes
            cache[n + "_scales"][at:at + 512] = scales.transpose(-1, -2)
    s["total"] = total
    if c["op"] == "attention":
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _activations((c["B"] * c["q_len"], c["q_heads"], D), g, dt, 0.3)
        s["sm_scale"] = 1 / math.sqrt(D)
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _exponent(amax, fmax):
    """The byte e of the smallest power of two 2^(e - 127) >= amax / fmax."""
    bits = (amax / fmax).view(torch.int32)
    return ((bits >> 23) & 255) + ((bits & 0x7FFFFF) != 0)


def _power(e):
    return (e.to(torch.int32) << 23).view(torch.float32)


def _e2m1(t):
    """The nearest FP4 value of each t (ties to the even code, at most 6), and its code."""
    a = t.abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(a / step) * step
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    return code | (torch.signbit(t).to(torch.uint8) << 3)


def _quantise(x, fmt, g):
    """4-bit codes (two to a byte) and scale bytes of the last axis' groups."""
    v = x.float().unflatten(-1, (-1, GROUP[fmt]))
    amax = v.abs().amax(-1).clamp(min=EPS)
    if fmt == "mxfp4":
        e = _exponent(amax, 6.0)
        mult, scales = _power(254 - e), e.to(torch.uint8)
    else:
        sf = (amax / 6 * g).clamp(max=448).to(torch.float8_e4m3fn)
        mult = torch.where(sf.float() == 0, 0.0, g / sf.float())
        scales = sf.view(torch.uint8)
    code = _e2m1(v * mult[..., None]).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _dequantise(codes, scales, fmt, g):
    """fp32 values of codes [..., D/2] with scale bytes [..., D/G]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    s = _power(scales) if fmt == "mxfp4" else scales.view(torch.float8_e4m3fn).float()
    v = (v.unflatten(-1, (-1, GROUP[fmt])) * s[..., None]).flatten(-2)
    return v if g is None else v * (1 / g)


def _plain_rmsnorm(s):
    c, x = s["case"], s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    # the statistic in 64 bits: a last-place difference of it would move codes at rounding borders
    inv = (1 / (h.double().square().mean(-1, keepdim=True) + NORM_EPS).sqrt()).float()
    y = ((h.float() * inv) * s["weight"].float()).unflatten(-1, (-1, c["group"]))
    amax = y.abs().amax(-1).clamp(min=EPS)
    fmax = 448.0 if c["out"] == "e4m3" else 127.0
    if c["fmt"] == "ue8m0":
        e = _exponent(amax, fmax)
        t, scales = y * _power(254 - e)[..., None], e
    else:
        scales = amax / fmax
        t = y / scales[..., None]
    if c["out"] == "e4m3":
        q = t.clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        q = torch.round(t).clamp(-128, 127).to(torch.int8)
    if c["layout"] == "packed":      # four exponents to a word, a column of words per row
        w = torch.nn.functional.pad(scales, (0, -scales.shape[-1] % 4)).unflatten(-1, (-1, 4))
        shift = torch.tensor([0, 8, 16, 24], device=w.device)
        scales = (w.long() << shift).sum(-1).to(torch.int32)
    if c["layout"] != "row":
        scales = scales.t()
    return {"codes": q.flatten(-2), "scales": scales, "h": h}


def _plain_write(s):
    c, n = s["case"], s["total"]
    slot = s["slots"][:n].long()
    page, at = slot // c["page"], slot % c["page"]
    for name, gi in (("k", 0), ("v", 1)):
        codes, scales = _quantise(s[name][:n], c["fmt"], s["gscale"][gi] if s["gscale"] is not None else None)
        s["cache"][name + "_codes"][page, :, at] = codes
        s["cache"][name + "_scales"][page, :, :, at] = scales


def _plain_read(s):
    c, got = s["case"], {}
    P, width = c["page"], s["table"].shape[1]
    row = torch.arange(s["total"], device="cuda")
    ends = s["indptr"][1:].long()
    b = torch.bucketize(row, ends, right=True)
    j = row - s["indptr"].long()[b]
    page, at = s["table"][b, j // P].long(), j % P
    for name, gi in (("k", 0), ("v", 1)):
        v = _dequantise(s["cache"][name + "_codes"][page, :, at], s["cache"][name + "_scales"][page, :, :, at],
                        c["fmt"], s["gscale"][gi] if s["gscale"] is not None else None)
        got[name] = v.to(DTYPE[c["dtype"]])
    return got


def _plain_attention(s):
    c, D = s["case"], s["case"]["D"]
    B, H, n = c["B"], c["heads"], c["q_len"]
    page = s["table"].clamp(min=0).long()
    kv = []
    for name, gi in (("k", 0), ("v", 1)):
        codes = s["cache"][name + "_codes"][page].transpose(1, 2).flatten(2, 3)
        scales = s["cache"][name + "_scales"][page].permute(0, 2, 1, 4, 3).flatten(2, 3)
        kv.append(_dequantise(codes, scales, c["fmt"], s["gscale"][gi] if s["gscale"] is not None else None))
    k, v = kv                                                    # [B, H, keys, D]
    q = s["q"].float().view(B, n, H, -1, D).transpose(1, 2).flatten(2, 3)   # rows: (token, head)
    w = torch.matmul(q, k.transpose(-1, -2)) * s["sm_scale"]
    reach = s["lens"].long()[:, None] - torch.arange(n - 1, -1, -1, device="cuda")
    reach = reach.repeat_interleave(q.shape[2] // n, 1)[:, None, :, None]
    w = w.masked_fill(torch.arange(k.shape[2], device="cuda") >= reach, -math.inf)
    m = w.amax(-1, keepdim=True)
    p = (w - m.clamp(min=-1e30)).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (m + total.log())[..., 0]
    out = out.unflatten(2, (n, -1)).transpose(1, 2).reshape(B * n, -1, D)
    return {"out": out.to(s["q"].dtype), "lse": lse.unflatten(2, (n, -1)).transpose(1, 2).reshape(B * n, -1)}


# --------------------------------------------------------------------------
# the library's entry points
# --------------------------------------------------------------------------

def _handle(s):
    """The cache's handle, which a program makes once with its buffers."""
    if "handle" not in s:
        from precision_activation_quantization_b200 import pqg
        s["handle"] = pqg.kv_cache(**s["cache"], fmt=s["case"]["fmt"], global_scale=s["gscale"])
    return s["handle"]


def _own(s):
    from precision_activation_quantization_b200 import pqg
    c = s["case"]
    if c["op"] == "rmsnorm":
        codes, scales, h = pqg.rmsnorm_quant(
            s["x"], s["weight"], s["residual"], eps=NORM_EPS, group=c["group"], out_dtype=c["out"],
            scale_fmt=c["fmt"], layout=c["layout"])
        if c["layout"] != "row":     # rows of a column-major plane are padded to a multiple of 4
            scales = scales[:, :c["M"]]
        return {"codes": codes, "scales": scales, "h": h}
    if c["op"] == "attention":
        out, lse = pqg.kv_attention(s["q"], _handle(s), s["table"], s["lens"],
                                    sm_scale=s["sm_scale"], return_lse=True)
        return {"out": out, "lse": lse}
    if c["op"] == "cache":
        pqg.kv_write(_handle(s), s["k"], s["v"], s["slots"])
    k, v = pqg.kv_read(_handle(s), s["table"], s["indptr"], s["total"], dtype=DTYPE[c["dtype"]])
    return {"k": k, "v": v}


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "rmsnorm":
        return _plain_rmsnorm(s)
    if op == "attention":
        return _plain_attention(s)
    if op == "cache":
        _plain_write(s)
    return _plain_read(s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(c):
    if c["op"] == "rmsnorm":
        n = c["M"] * c["K"]
        scale = n // c["group"] * (4 if c["fmt"] == "fp32" else 1)
        moved = n * (2 + 1 + (4 if c["residual"] else 0)) + scale + 2 * c["K"]
        return {"bytes": moved, "flops": 15 * n}
    tokens, D, G = sum(_lengths(c)), c["D"], GROUP[c["fmt"]]
    held = 2 * tokens * c["heads"] * (D // 2 + D // G)             # 4-bit keys and values
    wide = 2 * tokens * c["heads"] * 2 * D                         # 16-bit keys and values
    if c["op"] == "cache":
        return {"bytes": 2 * (held + wide) + 4 * tokens, "flops": 10 * 2 * tokens * c["heads"] * D}
    if c["op"] == "read":
        return {"bytes": held + wide, "flops": 2 * 2 * tokens * c["heads"] * D}
    rows = c["B"] * c["q_len"] * c["q_heads"]
    return {"bytes": held + rows * (4 * D + 4),
            "flops": 4 * c["q_len"] * c["q_heads"] * D * tokens}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_power(r):
    """The smallest power of two >= r > 0."""
    m, e = torch.frexp(r)
    return torch.ldexp(torch.ones_like(r), e - (m == 0.5).to(e.dtype))


def _exact_e4m3(t):
    """The nearest value of 4 significant bits from 2^-6 up (steps of 2^-9 below), at most 448."""
    a = t.abs().clamp(max=448)
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a)[1] - 1).clamp(min=-6) - 3)
    return torch.round(a / step) * step * torch.sign(t)


def _exact_e2m1(t):
    a = t.abs()
    rank = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=t.device)
    return grid[rank] * torch.sign(t)


def _exact_held(x, fmt, g):
    """What a 4-bit cache holds of x."""
    v = x.double().unflatten(-1, (-1, GROUP[fmt]))
    amax = v.abs().amax(-1, keepdim=True).clamp(min=EPS)
    if fmt == "mxfp4":
        scale = _exact_power(amax / 6)
        return (_exact_e2m1(v / scale) * scale).flatten(-2)
    sf = _exact_e4m3(amax / 6 * g)
    return torch.where(sf == 0, 0.0, _exact_e2m1(v * g / sf) * sf / g).flatten(-2)


def _exact_values(codes, scales, fmt, g):
    """The values of stored codes [..., P, D/2] with scales [..., D/G, P]."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    low = n % 8
    mag = torch.where(low < 2, low * 0.5, (2 + low % 2) * torch.exp2((low // 2 - 2).double()))
    s = scales.transpose(-1, -2).long()
    if fmt == "mxfp4":
        scale = torch.exp2((s - 127).double())
    else:
        e, m = s // 8, s % 8
        scale = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double())) / g
    return torch.where(n >= 8, -mag, mag) * scale.repeat_interleave(GROUP[fmt], -1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rmsnorm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        # the norm is that of the stored, rounded sum
        kept = h.to(s["x"].dtype).double()
        y = kept / (kept.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * s["weight"].double()
        y = y.unflatten(-1, (-1, c["group"]))
        amax = y.abs().amax(-1, keepdim=True).clamp(min=EPS)
        scale = _exact_power(amax / 448) if c["fmt"] == "ue8m0" else amax / (448 if c["out"] == "e4m3" else 127)
        codes = _exact_e4m3(y / scale).flatten(-2) if c["out"] == "e4m3" else None
        scales = None if c["layout"] == "packed" else scale[..., 0].t() if c["layout"] == "col" else scale[..., 0]
        return {"codes": codes, "scales": scales, "h": h}
    G = [None, None] if s["gscale"] is None else [float(v) for v in s["gscale"]]
    lens = _lengths(c)
    if c["op"] == "cache":
        return {n: _exact_held(s[n][:s["total"]], c["fmt"], g) for n, g in (("k", G[0]), ("v", G[1]))}
    out = {"k": [], "v": []} if c["op"] == "read" else {"out": [], "lse": []}
    for b, n in enumerate(lens):
        page = s["table"][b, :-(-n // c["page"])].long()
        k, v = (_exact_values(s["cache"][name + "_codes"][page], s["cache"][name + "_scales"][page], c["fmt"], g)
                .transpose(0, 1).flatten(1, 2)[:, :n] for name, g in (("k", G[0]), ("v", G[1])))
        if c["op"] == "read":
            out["k"].append(k.transpose(0, 1))
            out["v"].append(v.transpose(0, 1))
            continue
        q = s["q"][b * c["q_len"]:(b + 1) * c["q_len"]].double().unflatten(1, (c["heads"], -1))
        w = torch.einsum("thgd,hjd->thgj", q, k) * s["sm_scale"]
        seen = n - c["q_len"] + 1 + torch.arange(c["q_len"], device="cuda")
        hidden = torch.arange(n, device="cuda") >= seen[:, None]
        lse = torch.logsumexp(w.masked_fill(hidden[:, None, None], -math.inf), -1)
        p = torch.where(hidden[:, None, None], 0.0, (w - lse[..., None]).exp()) if n else w
        out["out"].append(torch.einsum("thgj,hjd->thgd", p, v).flatten(1, 2))
        out["lse"].append(lse.flatten(1, 2))
    return {name: torch.cat(parts) for name, parts in out.items()}
