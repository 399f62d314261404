"""The decoder layer's operators together (examples/decoder_layer.py)."""

import math
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    import importlib.util
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"), "--hidden", "512",
                        "--prompts", "9", "70", "--steps", "2"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "step 1: lengths [11, 72]" in r.stdout and "training step" in r.stdout


def test_a_token_decoded_equals_the_token_in_its_prompt():
    """The last token behind a cached prompt, against the whole prompt at once.
    Both read the same cache but for the scale of the last block, whose amax
    meets the tokens in two parts: the same power of two, so the same codes.  What
    differs is the order of FP32 sums: under one step of BF16 in nearly all."""
    import torch
    m = _example()
    layer = m.Layer(512, heads=2, group=2, dim=128, experts=4, expert_hidden=256, top_k=2)
    n = 150
    x = torch.randn((n, 512), device="cuda").to(torch.bfloat16)
    at_once, apart = (m.Cache(8, 2, 32, 128, 1, 8) for _ in range(2))
    at_once.grow([n])
    y, _ = layer.forward(None, x, at_once)
    apart.grow([n - 1])
    layer.forward(None, x[:n - 1], apart)
    apart.grow([1])
    z, _ = layer.forward(None, x[n - 1:], apart)
    err = (z[0].float() - y[-1].float()).norm() / y[-1].float().norm()
    assert float(err) < 0.05  # one step of e4m3 in a few of an operand's codes


def test_layer_against_32_bits():
    """The layer's output against the same layer in FP32 with the dequantised
    weights: the activations' e4m3 (2^-4 relative, random) through four products
    leaves the result within a tenth."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as fp8
    m = _example()
    H, heads, group, dim, E, I, k = 512, 2, 4, 128, 4, 256, 2
    layer = m.Layer(H, heads, group, dim, E, I, k)
    n = 40
    x = torch.randn((n, H), device="cuda").to(torch.bfloat16)
    cache = m.Cache(4, heads, 32, dim, 1, 4)
    cache.grow([n])
    y, stream = layer.forward(None, x, cache)

    def deq(w):
        q, s = w
        f = q.view(torch.float8_e4m3fn).float()
        return f * s.repeat_interleave(128, -2)[..., :f.shape[-2], :].repeat_interleave(128, -1)[..., :f.shape[-1]]

    def norm(t):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6)

    h = x.float()
    qkv = norm(h) @ deq(layer.qkv).t()
    q, kk, v = qkv.split([group * heads * dim, heads * dim, heads * dim], 1)
    q = q.view(n, heads * group, dim).transpose(0, 1)
    kk, v = (t.view(n, heads, dim).transpose(0, 1).repeat_interleave(group, 0) for t in (kk, v))
    s = (q @ kk.transpose(1, 2)) / math.sqrt(dim)
    s = s.masked_fill(torch.ones((n, n), device="cuda").triu(1).bool(), -math.inf)
    o = (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, -1)
    h = h + o @ deq(layer.out).t()
    a = norm(h)
    logits = a @ layer.router.t()
    ids = logits.topk(k, 1).indices
    w = torch.softmax(logits.gather(1, ids), 1)
    out = torch.zeros_like(h)
    w1, w2 = deq(layer.w1), deq(layer.w2)
    for e in range(E):
        u = a @ w1[e].t()
        f = (torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ w2[e].t()
        out += f * (w * (ids == e)).sum(1, keepdim=True)
    assert float((stream.float() - h).norm() / h.norm()) < 0.03
    # tokens whose second and third expert nearly tie may be routed apart: compare the others
    top = logits.sort(1, descending=True).values
    clear = top[:, k - 1] - top[:, k] > 0.2
    assert int(clear.sum()) > n // 2
    assert float((y.float() - out)[clear].norm() / out[clear].norm()) < 0.1
    assert fp8.fp8gemm_get_device_status() == fp8.OK


def test_training_step_against_autograd():
    """norm -> linear and back against autograd in FP32, within the FP8 of the
    product's operands (e5m2 gradient 2^-3, e4m3 weight 2^-4, relative and random)."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as fp8
    m = _example()
    T, K, N = 100, 512, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, s, dy, dh, w, gain = r(T, K), r(T, K), r(T, N), r(T, K), r(N, K) / 20, 1 + 0.1 * r(K)
    x, s, dy, dh = (t.to(torch.bfloat16) for t in (x, s, dy, dh))
    out, saved = m.norm_linear(x, s, gain, *fp8.fp8_quant_128x128(w))
    dx, dgain = m.norm_linear_backward(dy, dh, saved, gain, *fp8.fp8_quant_128x128(w.t().contiguous()))
    h = saved[0].float().requires_grad_()
    gg = gain.clone().requires_grad_()
    y = (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gg) @ w.t()
    ((y * dy.float()).sum() + (h * dh.float()).sum()).backward()
    assert float((out.float() - y).norm() / y.norm()) < 0.06
    assert float((dx.float() - h.grad).norm() / h.grad.norm()) < 0.08
    assert float((dgain - gg.grad).norm() / gg.grad.norm()) < 0.08


def test_a_captured_graph_outlives_larger_calls():
    """Calls captured on a stream, then larger ones made there, which need more
    of the same workspaces: replays of the graph still equal the direct calls, and the
    workspaces have not grown."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def codes(*shape):
        return torch.randint(0, 112, shape, generator=g, dtype=torch.uint8, device="cuda")

    def norm(M, K):
        dy, h, rstd, gain = bf16(M, K), bf16(M, K), torch.ones(M, device="cuda"), torch.ones(K, device="cuda")
        return lambda: b.fp8_rmsnorm_backward(dy, h, rstd, gain)

    def attend(B, group, tokens):
        k, v = codes(B * tokens // 64, 2, 64, 128), codes(B * tokens // 64, 2, 64, 128)
        s = torch.full(k.shape[:2], 2.0 ** -7, device="cuda")
        table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda").view(B, -1)
        lens, q = torch.full((B,), tokens - 5, dtype=torch.int32, device="cuda"), bf16(B, 2 * group, 128)
        return lambda: (b.fp8_kv_attention(q, k, s, v, s, table, lens),)

    def moe(T, E, k, H=512, I=256):
        A, W1, W2 = codes(T, H), codes(E, 2 * I, H), codes(E, H, I)
        one = [torch.full(n, 2.0 ** -6, device="cuda") for n in ((T, H // 128), (E, 2 * I // 128, H // 128),
                                                                (E, H // 128, I // 128))]
        logits = torch.randn((T, E), generator=g, device="cuda")
        return lambda: b.fp8_moe_few(A, one[0], logits, W1, one[1], W2, one[2], k)

    s = torch.cuda.Stream()
    for small, large in ((norm(3, 64), norm(700, 16384)), (attend(1, 1, 1024), attend(40, 16, 4096)),
                         (moe(1, 4, 2), moe(64, 32, 16))):
        want = small()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            small()
            s.synchronize()
            held = b.workspace_bytes()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = small()
            large()
            s.synchronize()
            assert b.workspace_bytes() == held
            graph.replay()
            s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert b.fp8gemm_get_device_status() == b.OK
    b.fp8gemm_release_workspaces(s)
