"""The operators together, as a decoder layer runs them: norm with FP8 output, QKV
product, keys and values into the 4-bit cache, attention over it, FP8 quantization
of its output, output product, norm of the sum.  The products are torch's.  Prefill
and decode steps, the decode step captured once and replayed."""
import numpy as np
import pytest
import torch

import rmsnorm_reference as norm_ref
from gpu_parity import assert_same
from precision_activation_quantization_b200 import pqg
from test_kv_attention_gpu import compare, reference
from test_rmsnorm_gpu import host

pytestmark = pytest.mark.gpu

K, H, HQ, D, P, G = 512, 2, 8, 64, 16, 128


def fp8_matmul(codes, scales, w):
    x = codes.float().unflatten(-1, (-1, G)) * scales[..., None]
    return (x.flatten(-2) @ w).to(torch.bfloat16)


class Layer:
    def __init__(self, fmt, pages, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
        self.wqkv, self.wo = r(K, (HQ + 2 * H) * D) / K ** 0.5, r(HQ * D, K) / (HQ * D) ** 0.5
        self.n1, self.n2 = (1 + 0.1 * r(K)).to(torch.bfloat16), (1 + 0.1 * r(K)).to(torch.bfloat16)
        gs = torch.tensor([448 * 6 / 16.0, 448 * 6 / 16.0], device="cuda") if fmt == "nvfp4" else None
        self.cache = pqg.kv_allocate(pages, P, H, D, fmt=fmt, global_scale=gs)

    def __call__(self, x, residual, slots, table, lens):
        """One layer over the newest tokens; everything a stage read and made."""
        q1, s1, h1 = pqg.rmsnorm_quant(x, self.n1, residual, group=G)
        qkv = fp8_matmul(q1, s1, self.wqkv)
        q = qkv[:, :HQ * D].unflatten(1, (HQ, D))
        k = qkv[:, HQ * D:(HQ + H) * D].unflatten(1, (H, D))
        v = qkv[:, (HQ + H) * D:].unflatten(1, (H, D))
        pqg.kv_write(self.cache, k, v, slots)
        o, lse = pqg.kv_attention(q, self.cache, table, lens, return_lse=True)
        qo, so = pqg.quant(o.view(-1, HQ * D), group=G)
        y = fp8_matmul(qo[0], so[0], self.wo)
        q2, s2, h2 = pqg.rmsnorm_quant(y, self.n2, h1, group=G, scale_fmt="ue8m0", layout="row")
        return dict(q1=q1, s1=s1, h1=h1, q=q, o=o, lse=lse, y=y, q2=q2, s2=s2, h2=h2)


def check_norm(x, residual, weight, q, s, h, fmt):
    hb = norm_ref.add(host(x), host(residual), "bf16")
    codes, scales = norm_ref.quantise(norm_ref.normed(hb, host(weight), 1e-6, "bf16"), G, "e4m3", fmt)
    assert_same(host(h), hb, "h")
    assert_same(q.view(torch.uint8).cpu().numpy(), codes, "norm codes")
    assert_same(s.cpu().numpy().view(np.uint8), scales.view(np.uint8), "norm scales")


def check(layer, got, x, residual, table, lens, q_len):
    check_norm(x, residual, layer.n1, got["q1"], got["s1"], got["h1"], "fp32")
    check_norm(got["y"], got["h1"], layer.n2, got["q2"], got["s2"], got["h2"], "ue8m0")
    c = layer.cache
    import test_kv_attention_gpu as t
    scale, t.G_SCALE = t.G_SCALE, (448 * 6 / 16.0, 448 * 6 / 16.0)
    try:
        want = reference(got["q"].contiguous(), c, table, lens, q_len, D ** -0.5)
    finally:
        t.G_SCALE = scale
    compare(got["o"], got["lse"], want, "bf16", lens)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_prefill_then_captured_decode_steps(fmt):
    prompt, steps = [37, 16, 3], 20
    B, width = len(prompt), 4
    layer = Layer(fmt, B * width + 1)
    table = torch.randperm(B * width, device="cuda").view(B, width).to(torch.int32)
    slot = lambda b, j: int(table[b, j // P]) * P + j % P  # noqa: E731
    rand = lambda n, s: torch.randn(n, K, generator=torch.Generator(device="cuda").manual_seed(s),  # noqa: E731
                                    device="cuda").to(torch.bfloat16)
    # prompts, one sequence at a time: all their tokens attend to the cache at once
    for b, n in enumerate(prompt):
        x, r = rand(n, b), rand(n, 10 + b)
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        slots = torch.tensor([slot(b, j) for j in range(n)], dtype=torch.int32, device="cuda")
        got = layer(x, r, slots, table[b:b + 1], lens)
        torch.cuda.synchronize()
        check(layer, got, x, r, table[b:b + 1], [n], n)
    # decode: a batch padded by one token (no slot, an empty sequence), captured once
    x, r = rand(B + 1, 50), rand(B + 1, 51)
    slots = torch.full((B + 1,), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    full = torch.cat((table, torch.full((1, width), -1, dtype=torch.int32, device="cuda")))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, r, slots, full, lens)                # warm-up: writes nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, r, slots, full, lens)
    for step in range(steps):
        now = [n + step + 1 for n in prompt]
        x.copy_(rand(B + 1, 100 + step))
        r.copy_(rand(B + 1, 200 + step))
        slots[:B].copy_(torch.tensor([slot(b, n - 1) for b, n in enumerate(now)], dtype=torch.int32))
        lens[:B].copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        if step % 5 == 0 or step == steps - 1:
            check(layer, got, x, r, full, now + [0], 1)
    # what the cache holds reads back in order, and the spare page was never written
    indptr = torch.tensor(np.concatenate(([0], np.cumsum([n + steps for n in prompt]))), dtype=torch.int32,
                          device="cuda")
    k, v = pqg.kv_read(layer.cache, table, indptr, int(indptr[-1]))
    assert torch.isfinite(k).all() and (k.abs().amax(-1) > 0).all() and (v.abs().amax(-1) > 0).all()
    assert int(layer.cache.k_codes[-1].max()) == 0 and int(layer.cache.v_scales[-1].max()) == 0


def test_a_stream_may_be_a_handle():
    """Calls on streams given as numbers run there and allocate from their pools, the default stream's 0 included."""
    side = torch.cuda.Stream()
    dev = torch.device("cuda", torch.cuda.current_device())
    for stream in (0, side.cuda_stream, side):
        for current in (torch.cuda.default_stream(), torch.cuda.Stream()):
            with torch.cuda.stream(current), pqg._allocating_on(stream, dev):
                assert torch.cuda.current_stream().cuda_stream == getattr(stream, "cuda_stream", stream)
    layer = Layer("mxfp4", 4)
    x, r = (torch.randn(5, K, device="cuda").to(torch.bfloat16) for _ in range(2))
    k = torch.randn(5, H, D, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, HQ, D, device="cuda").to(torch.bfloat16)
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    n = torch.tensor([5], dtype=torch.int32, device="cuda")
    indptr = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = []
    for stream in (None, 0, side.cuda_stream, side):
        pqg.kv_write(layer.cache, k, k, slots, stream=stream)
        got.append([*pqg.rmsnorm_quant(x, layer.n1, r, stream=stream),
                    *pqg.kv_read(layer.cache, table, indptr, 5, stream=stream),
                    pqg.kv_attention(q, layer.cache, table, n, stream=stream)])
        torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got[0], other))
