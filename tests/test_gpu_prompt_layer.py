"""Rotary positions, append, chunk attention and the gated feed-forward block as they are used together:
prompts and single tokens of a layer against a plain one, a training step against autograd, and calls that share
streams, workspaces and graphs."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("decoder_layer_prompt", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_prompts_then_single_tokens_against_plain_attention():
    """Two prompts, a second chunk of each and then single tokens, with rotary positions: each output within the cache's
    FP8 (2^-4 of a key or value, random over 100 tokens and more) of attention over the unrounded keys."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as fp8
    from fp8_fine_grained_e4m3_gb300 import rotary
    m = _example()
    heads, group, dim = 2, 4, 128
    freq, amplitude = rotary.frequencies(dim, scaling="parts", factor=4.0, trained=64)
    cache = m.Cache(32, heads, 64, dim, 2, 8)
    g = _gen(1)
    w = (group + 2) * heads * dim
    seen = [torch.empty((0, w), device="cuda") for _ in range(2)]

    def rotated(rows, h):  # FP64, half layout
        x = rows.double().view(rows.shape[0], h, dim)
        t = torch.arange(rows.shape[0], device="cuda").double()[:, None] * freq.double()
        c, s = (amplitude * f(t)[:, None] for f in (torch.cos, torch.sin))
        a, b = x[..., :dim // 2], x[..., dim // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    for counts in ([130, 70], [45, 64], [1, 1], [1, 1]):
        T = sum(counts)
        qkv = torch.randn((T, w), generator=g, device="cuda").to(torch.bfloat16)
        raw = qkv.clone()
        cache.grow(counts)
        q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([group * heads * dim, heads * dim, heads * dim], 1))
        ones = counts == [1, 1]
        cu = None if ones else torch.tensor([0, counts[0], T], dtype=torch.int32, device="cuda")
        fp8.fp8_rope(q, k, freq, seq_lens=cache.lens, cu=cu, amplitude=amplitude, Qo=q, Ko=k)
        fp8.fp8_kv_append(k, v, *cache.tensors(), cu_new=cu, max_new=max(counts))
        attend = fp8.fp8_kv_attention if ones else fp8.fp8_kv_attention_chunk
        o = attend(q, *cache.tensors(), cu_q=cu, max_q=max(counts))
        at = 0
        for b, n in enumerate(counts):
            seen[b] = torch.cat((seen[b], raw[at:at + n].float()))
            L = seen[b].shape[0]
            qs, ks, vs = seen[b].split([group * heads * dim, heads * dim, heads * dim], 1)
            Q = rotated(qs, heads * group)[L - n:].transpose(0, 1)
            K = rotated(ks, heads).repeat_interleave(group, 1).transpose(0, 1)
            V = vs.double().view(L, heads, dim).repeat_interleave(group, 1).transpose(0, 1)
            x = Q @ K.transpose(1, 2) / math.sqrt(dim)
            hidden = torch.arange(L, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None]
            ref = (torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ V).transpose(0, 1)
            err = float((o[at:at + n].double() - ref).norm() / ref.norm())
            assert err < 0.08, (counts, b, err)
            at += n
    assert fp8.fp8gemm_get_device_status() == fp8.OK


def test_feed_forward_block_against_autograd():
    """Forward and backward within the FP8 of their operands (e4m3 2^-4, e5m2 2^-3, relative and random), and the gate's
    and up's gradients that the weights' gradient is formed from."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as fp8
    m = _example()
    T, H, I = 200, 512, 384
    g = _gen(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, up, down, dy = r(T, H), r(2 * I, H) / math.sqrt(H), r(H, I) / math.sqrt(I), r(T, H).to(torch.bfloat16)
    w1, w2, w1t, w2t = (fp8.fp8_quant_128x128(w.contiguous()) for w in (up, down, up.t(), down.t()))
    y, GU = m.gated_ffn(*fp8.fp8_quant_1x128(x), w1, w2)
    dx, dGU = m.gated_ffn_backward(dy, GU, w1t, w2t)
    x.requires_grad_()
    u = x @ up.t()
    u.retain_grad()
    ref = (torch.nn.functional.silu(u[:, :I]) * u[:, I:]) @ down.t()
    ref.backward(dy.float())
    near = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    assert near(GU, u.detach()) < 0.05 and near(y, ref.detach()) < 0.08
    assert near(dGU, u.grad) < 0.12 and near(dx, x.grad) < 0.12
    assert fp8.fp8gemm_get_device_status() == fp8.OK


def _attention(B, n, L, seed, heads=2, group=4, dim=128, block=64):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = _gen(seed)
    blocks = B * L // block
    k, v = (torch.randint(0, 112, (blocks, heads, block, dim), generator=g, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.full((blocks, heads), 2.0 ** -7, device="cuda")
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), L - 5, dtype=torch.int32, device="cuda")
    q = torch.randn((B * n, heads * group, dim), generator=g, device="cuda").to(torch.bfloat16)
    return lambda: b.fp8_kv_attention_chunk(q, k, s, v, s, table, lens)


def _gated(M, K, I, seed):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = _gen(seed)
    A, W = (torch.randint(0, 112, s, generator=g, dtype=torch.uint8, device="cuda") for s in ((M, K), (2 * I, K)))
    sA, sW = (torch.full((n, K // 128), 2.0 ** -9, device="cuda") for n in (M, 2 * I // 128))
    return lambda: b.fp8gemm_gated(A, sA, W, sW)[0]


def _gated_back(M, K, I, seed):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = _gen(seed)
    A, W = (torch.randint(0, 112, s, generator=g, dtype=torch.uint8, device="cuda") for s in ((M, K), (I, K)))
    sA, sW = (torch.full((n, K // 128), 2.0 ** -9, device="cuda") for n in (M, I // 128))
    GU = torch.randn((M, 2 * I), generator=g, device="cuda").to(torch.bfloat16)
    return lambda: b.fp8gemm_gated_backward(A, sA, W, sW, GU)[0]


CALLS = {"chunk, parts": lambda i: _attention(1, 20, 8192, i), "chunk, units": lambda i: _attention(3, 300, 512, i),
         "gated, split": lambda i: _gated(5, 2048, 256, i), "gated, whole": lambda i: _gated(2600, 256, 2048, i),
         "gradient, split": lambda i: _gated_back(5, 2048, 256, i), "gradient, whole": lambda i: _gated_back(2600, 256, 2048, i)}


@pytest.mark.parametrize("name", CALLS)
def test_two_streams_at_once(name):
    """The same call with other inputs on two streams, without order between them."""
    import torch
    one, two = CALLS[name](1), CALLS[name](2)
    want = one(), two()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, call) in enumerate(zip(streams, (one, two))):
            with torch.cuda.stream(s):
                got[i].append(call())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("name", CALLS)
def test_two_graphs_of_one_stream(name):
    """Two graphs captured on one stream share its workspace: replayed in turn, with direct calls between."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    calls = CALLS[name](1), CALLS[name](2)
    want = [c() for c in calls]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        calls[0]()
        s.synchronize()
        graphs, got = [], []
        for c in calls:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                got.append(c())
        for _ in range(3):
            for x in got:
                x.zero_()
            graphs[1].replay()
            direct = calls[0]()
            graphs[0].replay()
            graphs[1].replay()
            s.synchronize()
            assert torch.equal(direct, want[0]) and all(torch.equal(x, y) for x, y in zip(got, want))
    b.fp8gemm_release_workspaces(s)
    assert b.fp8gemm_get_device_status() == b.OK


def test_from_several_threads_on_one_stream():
    import threading
    import torch
    calls = [CALLS[n](i) for i, n in enumerate(("chunk, parts", "chunk, units", "gated, split", "gradient, split"))]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(20):
            if not torch.equal(calls[i](), want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
