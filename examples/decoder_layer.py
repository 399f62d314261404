"""One decoder layer in FP8, as a server and a trainer would run it.

    python examples/decoder_layer.py            # prompts, then decode steps, then a training step

Serving, for a batch of sequences with a paged FP8 cache:

    norm (8-bit output) -> QKV product -> rotary positions -> append to the cache -> attention ->
    output product -> residual + norm (8-bit output) -> router -> mixture of experts

(prompts attend a chunk of tokens at a time, single tokens by the other call).

Training, for the norm and the linear layer behind it: the output's gradient in
e5m2 -> product with the transposed weight -> the norm's gradient; and for a gated
feed-forward block: gate and up products with SwiGLU -> down product, and back
through both.

Weights are random.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp8_fine_grained_e4m3_gb300 import binding as fp8  # noqa: E402
from fp8_fine_grained_e4m3_gb300 import rotary  # noqa: E402

BF16 = torch.bfloat16


class Cache:
    """Blocks of `block` tokens for `heads` cached heads; a sequence takes the
    next free ones as it grows."""

    def __init__(self, num_blocks, heads, block, dim, sequences, table_width):
        shape = (num_blocks, heads, block, dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(shape[:2], device="cuda") for _ in range(2))
        self.table = torch.zeros((sequences, table_width), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.block, self.free, self.host_lens = block, list(range(num_blocks)), [0] * sequences
        self.blocks = [[] for _ in range(sequences)]

    def grow(self, counts):
        """Room for counts[b] more tokens of each sequence."""
        for b, n in enumerate(counts):
            self.host_lens[b] += n
            while len(self.blocks[b]) * self.block < self.host_lens[b]:
                self.blocks[b].append(self.free.pop())
                self.table[b, len(self.blocks[b]) - 1] = self.blocks[b][-1]
        self.lens.copy_(torch.tensor(self.host_lens, dtype=torch.int32))

    def tensors(self):
        return self.k, self.ks, self.v, self.vs, self.table, self.lens


class Layer:
    def __init__(self, hidden, heads, group, dim, experts, expert_hidden, top_k, seed=0, positions=None):
        """positions: rotary.frequencies' result, or None for none."""
        self.positions = positions
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape):
            return fp8.fp8_quant_128x128(
                torch.randn(shape, generator=g, device="cuda") / math.sqrt(shape[-1]))

        self.heads, self.group, self.dim, self.top_k = heads, group, dim, top_k
        self.gain1, self.gain2 = (torch.ones(hidden, device="cuda") for _ in range(2))
        self.qkv = weight((group + 2) * heads * dim, hidden)
        self.out = weight(hidden, group * heads * dim)
        self.router = torch.randn((experts, hidden), generator=g, device="cuda") / math.sqrt(hidden)
        self.w1 = weight(experts, 2 * expert_hidden, hidden)
        self.w2 = weight(experts, hidden, expert_hidden)

    def moe(self, A, sA, h, rstd):
        """The mixture of experts of any number of tokens, 64 at a time."""
        logits = (h.float() * rstd[:, None] * self.gain2) @ self.router.t()
        parts = [fp8.fp8_moe_few(A[i:i + 64], sA[i:i + 64], logits[i:i + 64], *self.w1, *self.w2,
                                 self.top_k)[0] for i in range(0, A.shape[0], 64)]
        return torch.cat(parts) if len(parts) > 1 else parts[0]

    def forward(self, x, stream, cache, cu=None, most=None):
        """x: what the layer before adds to the residual stream (None: nothing
        yet), bf16 [T, hidden]; the tokens of sequence b at cu[b] .. cu[b + 1] - 1
        (None: one each).  Returns what this layer adds and the stream."""
        T = stream.shape[0]
        if x is None:
            A, sA, stream, _ = fp8.fp8_rmsnorm_quant(stream, self.gain1)
        else:
            A, sA, stream, _ = fp8.fp8_rmsnorm_quant(x, self.gain1, residual=stream)
        qkv = fp8.fp8gemm_dense(A, sA, *self.qkv)
        nq, nk = self.group * self.heads, self.heads
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in qkv.split(
            [nq * self.dim, nk * self.dim, nk * self.dim], dim=1))
        if self.positions is not None:  # in place: parts of the product's rows
            freq, amplitude = self.positions
            fp8.fp8_rope(q, k, freq, seq_lens=cache.lens, cu=cu, amplitude=amplitude, Qo=q, Ko=k)
        fp8.fp8_kv_append(k, v, *cache.tensors(), cu_new=cu, max_new=most)
        attend = fp8.fp8_kv_attention if cu is None else fp8.fp8_kv_attention_chunk
        o = attend(q, *cache.tensors(), cu_q=cu, max_q=most)
        o8, so = fp8.fp8_quant_1x128(o.view(T, -1).float())
        y = fp8.fp8gemm_dense(o8, so, *self.out)
        A, sA, stream, rstd = fp8.fp8_rmsnorm_quant(y, self.gain2, residual=stream)
        return self.moe(A, sA, stream, rstd), stream


def norm_linear(x, stream, gain, w8, sw):
    """y = norm(x + stream) W^T and what its gradient needs."""
    A, sA, h, rstd = fp8.fp8_rmsnorm_quant(x, gain, residual=stream)
    return fp8.fp8gemm_dense(A, sA, w8, sw), (h, rstd)


def norm_linear_backward(dy, dh, saved, gain, wt8, swt):
    """Gradients of x (and of the stream) and of the gain: dy [T, N] in e5m2
    against W^T (quantised as [K, N]), then the norm's; dh reaches the stream past it."""
    h, rstd = saved
    g8, sg = fp8.fp8_quant_1x128_fmt(dy.float(), "e5m2")
    dnorm = fp8.fp8gemm_dense_fmt(g8, sg, "e5m2", wt8, swt, "e4m3")
    return fp8.fp8_rmsnorm_backward(dnorm, h, rstd, gain, dH=dh)


def gated_ffn(A, sA, w1, w2):
    """y = (silu(gate) up) W2^T of A's rows in FP8, w1 and w2 (codes, scales) of [gate; up] and
    W2 -> y bf16 and what the gradient needs."""
    GU = torch.empty((A.shape[0], w1[0].shape[0]), dtype=BF16, device=A.device)
    h, sh = fp8.fp8gemm_gated(A, sA, *w1, GU=GU)
    return fp8.fp8gemm_dense(h, sh, *w2), GU


def gated_ffn_backward(dy, GU, w1t, w2t):
    """Gradients of A's rows (bf16) and of gate and up values (bf16) from dy: w2t is W2
    transposed, w1t [hidden, 2 Ip] is [gate; up] transposed, each half in columns of its own
    (Ip: its width up to a multiple of 128)."""
    g8, sg = fp8.fp8_quant_1x128_fmt(dy.float(), "e5m2")
    dGU = torch.empty_like(GU)
    d8, sd = fp8.fp8gemm_gated_backward(g8, sg, *w2t, GU, dGU=dGU)
    return fp8.fp8gemm_dense_fmt(d8, sd, "e5m2", *w1t, "e4m3"), dGU


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--prompts", type=int, nargs="+", default=[37, 5, 130, 64])
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    layer = Layer(a.hidden, heads=4, group=4, dim=128, experts=16, expert_hidden=1024, top_k=2,
                  positions=rotary.frequencies(128, scaling="parts", factor=4.0, trained=8192))
    B = len(a.prompts)
    cache = Cache(64, 4, 64, 128, B, 16)
    T = sum(a.prompts)
    cu = torch.tensor([sum(a.prompts[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    cache.grow(a.prompts)
    y, stream = layer.forward(None, torch.randn((T, a.hidden), device="cuda").to(BF16), cache, cu,
                              max(a.prompts))
    print(f"prompts: {T} tokens of {B} sequences, output rms {y.float().square().mean().sqrt():.3f}")
    token = stream[cu[1:].long() - 1] + y[cu[1:].long() - 1]
    for i in range(a.steps):
        cache.grow([1] * B)
        y, stream = layer.forward(None, token, cache)
        token = stream + y
        print(f"step {i}: lengths {cache.host_lens}, output rms {y.float().square().mean().sqrt():.3f}")
    w = torch.randn((512, a.hidden), device="cuda") / math.sqrt(a.hidden)
    x, s, dy, dh = (torch.randn((T, n), device="cuda").to(BF16) for n in (a.hidden, a.hidden, 512, a.hidden))
    out, saved = norm_linear(x, s, layer.gain1, *fp8.fp8_quant_128x128(w))
    dx, dgain = norm_linear_backward(dy, dh, saved, layer.gain1, *fp8.fp8_quant_128x128(w.t().contiguous()))
    print(f"training step: output {tuple(out.shape)}, input gradient {tuple(dx.shape)}, gain gradient "
          f"rms {dgain.square().mean().sqrt():.3f}")
    up = torch.randn((2 * 640, a.hidden), device="cuda") / math.sqrt(a.hidden)
    down = torch.randn((a.hidden, 640), device="cuda") / math.sqrt(640)
    w1, w2, w1t, w2t = (fp8.fp8_quant_128x128(w.contiguous()) for w in (up, down, up.t(), down.t()))
    y, GU = gated_ffn(*fp8.fp8_quant_1x128(x.float()), w1, w2)
    dx, dGU = gated_ffn_backward(dh, GU, w1t, w2t)
    print(f"feed-forward block: output {tuple(y.shape)}, input gradient {tuple(dx.shape)}, gate and up gradients rms "
          f"{dGU.float().square().mean().sqrt():.3f}")
    assert fp8.fp8gemm_get_device_status() == fp8.OK


if __name__ == "__main__":
    main()
