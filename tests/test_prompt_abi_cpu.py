"""Rotary positions, chunk attention and the gated products refuse what they cannot take on the host, before any
CUDA call, and tensors of another device before any address is passed on.  CPU only."""

import ctypes
import math

import pytest
import torch

from tests.test_layer_devices_cpu import BF, I32, U8, on

P = ctypes.c_void_p
GOOD = P(1 << 20)  # never dereferenced
ODD8, ODD2 = P((1 << 20) + 8), P((1 << 20) + 2)
S = P(0)


@pytest.fixture(scope="module")
def lib():
    from fp8_fine_grained_e4m3_gb300 import build, binding
    build.build()
    return binding.lib()


def _rope(lib, **kw):
    a = dict(Q=GOOD, ld_q=256, K=GOOD, ld_k=128, t=0, Qo=GOOD, ld_qo=256, Ko=GOOD, ld_ko=128, freq=GOOD, pos=None,
             lens=GOOD, cu=GOOD, amp=1.0, T=8, B=4, hq=4, hk=2, dim=64, rot=64, inter=0, back=0, s=S)
    a.update(kw)
    return lib.fp8_rope(*a.values())


def _chunk(lib, **kw):
    a = dict(Q=GOOD, ld_q=1024, kc=GOOD, ks=GOOD, vc=GOOD, vs=GOOD, table=GOOD, lens=GOOD, cu=GOOD, scale=1.0, causal=1,
             O=GOOD, T=8, B=4, heads=2, group=4, dim=128, block=64, width=3, n=12, most=4, fmt=0, s=S)
    a.update(kw)
    return lib.fp8_kv_attention_chunk(*a.values())


def _gated(lib, **kw):
    a = dict(A=GOOD, sA=GOOD, af=0, W1=GOOD, s1=GOOD, bf=0, Q=GOOD, sQ=GOOD, qf=0, GU=GOOD, M=4, I=128, K=256, s=S)
    a.update(kw)
    return lib.fp8gemm_gated(*a.values())


def _back(lib, **kw):
    a = dict(dY=GOOD, sdY=GOOD, af=1, W=GOOD, sW=GOOD, bf=0, GU=GOOD, Q=GOOD, sQ=GOOD, qf=1, dGU=GOOD, M=4, I=128, K=256,
             s=S)
    a.update(kw)
    return lib.fp8gemm_gated_backward(*a.values())


@pytest.mark.parametrize("call,kw,code", [
    (_rope, dict(T=-1), "SHAPE"), (_rope, dict(B=-1), "SHAPE"), (_rope, dict(dim=72), "SHAPE"),
    (_rope, dict(dim=528), "SHAPE"), (_rope, dict(dim=0), "SHAPE"), (_rope, dict(rot=8), "SHAPE"),
    (_rope, dict(rot=0), "SHAPE"), (_rope, dict(rot=80), "SHAPE"), (_rope, dict(hq=65536), "SHAPE"),
    (_rope, dict(ld_q=252), "SHAPE"), (_rope, dict(ld_ko=120), "SHAPE"), (_rope, dict(ld_k=132), "SHAPE"),
    (_rope, dict(t=2), "FORMAT"), (_rope, dict(cu=None, T=7), "SHAPE"), (_rope, dict(freq=None), "NULL"),
    (_rope, dict(Q=None), "NULL"), (_rope, dict(Ko=None), "NULL"), (_rope, dict(lens=None), "NULL"),
    (_rope, dict(K=ODD8), "ALIGN"), (_rope, dict(Qo=ODD8), "ALIGN"), (_rope, dict(freq=ODD2), "ALIGN"),
    (_rope, dict(pos=ODD2), "ALIGN"), (_rope, dict(cu=ODD2), "ALIGN"), (_rope, dict(T=0, Q=None), "OK"),
    (_rope, dict(hq=0, hk=0), "OK"), (_rope, dict(B=0, T=0, cu=None), "OK"),
    (_chunk, dict(group=-1), "SHAPE"), (_chunk, dict(dim=96), "SHAPE"), (_chunk, dict(block=8), "SHAPE"),
    (_chunk, dict(ld_q=1016), "SHAPE"), (_chunk, dict(ld_q=1028), "SHAPE"), (_chunk, dict(cu=None, T=6), "SHAPE"),
    (_chunk, dict(cu=None, most=1), "SHAPE"), (_chunk, dict(group=40000), "SHAPE"),
    (_chunk, dict(width=1 << 25), "SHAPE"), (_chunk, dict(T=1 << 30), "SHAPE"), (_chunk, dict(B=32768), "SHAPE"),
    (_chunk, dict(fmt=2), "FORMAT"), (_chunk, dict(O=None), "NULL"), (_chunk, dict(vs=None), "NULL"),
    (_chunk, dict(Q=ODD8), "ALIGN"), (_chunk, dict(vc=ODD8), "ALIGN"), (_chunk, dict(table=ODD2), "ALIGN"),
    (_chunk, dict(T=0), "OK"), (_chunk, dict(most=0, Q=None), "OK"), (_chunk, dict(group=0), "OK"),
    (_gated, dict(M=-1), "SHAPE"), (_gated, dict(I=0), "SHAPE"), (_gated, dict(I=24), "SHAPE"),
    (_gated, dict(I=(1 << 29) + 16), "SHAPE"), (_gated, dict(K=0), "SHAPE"), (_gated, dict(K=200), "SHAPE"),
    (_gated, dict(M=1 << 30, I=1 << 20), "SHAPE"), (_gated, dict(af=2), "FORMAT"), (_gated, dict(bf=-1), "FORMAT"),
    (_gated, dict(qf=3), "FORMAT"), (_gated, dict(W1=None), "NULL"), (_gated, dict(sQ=None), "NULL"),
    (_gated, dict(Q=ODD8), "ALIGN"), (_gated, dict(GU=ODD8), "ALIGN"), (_gated, dict(s1=ODD8), "ALIGN"),
    (_gated, dict(M=0, A=None), "OK"),
    (_back, dict(M=-1), "SHAPE"), (_back, dict(I=8), "SHAPE"), (_back, dict(K=24), "SHAPE"), (_back, dict(af=5), "FORMAT"),
    (_back, dict(GU=None), "NULL"), (_back, dict(dY=None), "NULL"), (_back, dict(sQ=ODD8), "ALIGN"),
    (_back, dict(dGU=ODD8), "ALIGN"), (_back, dict(M=0, GU=None), "OK")])
def test_host_validation(lib, call, kw, code):
    from fp8_fine_grained_e4m3_gb300 import binding as b
    assert call(lib, **kw) == (b.OK if code == "OK" else getattr(b, "ERR_" + code))


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_on_host():
    from fp8_fine_grained_e4m3_gb300 import binding as b
    q, k, f, pos = _t(6, 4, 64, dtype=BF), _t(6, 2, 64, dtype=BF), _t(32), _t(6, dtype=I32)

    def rope(Q=q, K=k, f=f, **kw):
        b.fp8_rope(Q, K, f, **(kw or {"positions": pos}))

    for match, error, call in [
            ("bfloat16 or float32", TypeError, lambda: rope(Q=q.half())), ("K must be", TypeError, lambda: rope(K=k.float())),
            ("T, heads, dim", ValueError, lambda: rope(Q=q[0])), ("K has shape", ValueError, lambda: rope(K=k[:5])),
            ("freq", TypeError, lambda: rope(f=f.double())), ("either", ValueError, lambda: b.fp8_rope(q, k, f)),
            ("either", ValueError, lambda: rope(positions=pos, seq_lens=pos)),
            ("positions", ValueError, lambda: rope(positions=pos[:5])), ("positions", TypeError, lambda: rope(positions=pos.long())),
            ("cu goes with", ValueError, lambda: rope(positions=pos, cu=pos)),
            ("give the offsets", ValueError, lambda: rope(seq_lens=pos[:4])),
            ("offsets", ValueError, lambda: rope(seq_lens=pos[:4], cu=pos[:4])),
            ("Qo", ValueError, lambda: rope(positions=pos, Qo=q[:, :2])), ("Qo must be", TypeError, lambda: rope(positions=pos, Qo=q.float())),
            ("without K", ValueError, lambda: rope(K=None, positions=pos, Ko=k)),
            ("contiguously", ValueError, lambda: rope(Q=_t(6, 64, 4, dtype=BF).transpose(1, 2))),
            ("CUDA", ValueError, lambda: rope())]:
        with pytest.raises(error, match=match):
            call()

    kc, ks, tab, lens = _t(6, 2, 16, 64, dtype=U8), _t(6, 2), _t(3, 2, dtype=I32), _t(3, dtype=I32)

    def chunk(Q=_t(6, 4, 64, dtype=BF), kc=kc, tab=tab, lens=lens, **kw):
        b.fp8_kv_attention_chunk(Q, kc, ks, kc, ks, tab, lens, **kw)

    for match, error, call in [
            ("num_blocks", ValueError, lambda: chunk(kc=kc[0])), ("block_table", TypeError, lambda: chunk(tab=tab.long())),
            ("seq_lens", ValueError, lambda: chunk(lens=lens[:2])), ("float8", TypeError, lambda: chunk(kc=kc.view(torch.float8_e5m2))),
            ("cached heads", ValueError, lambda: chunk(Q=_t(6, 3, 64, dtype=BF))),
            ("give the offsets", ValueError, lambda: chunk(Q=_t(5, 4, 64, dtype=BF))),
            ("O must be", TypeError, lambda: chunk(O=_t(6, 4, 64))), ("O has", ValueError, lambda: chunk(O=_t(6, 2, 64, dtype=BF))),
            ("format", ValueError, lambda: chunk(fmt="fp8")), ("CUDA", ValueError, lambda: chunk())]:
        with pytest.raises(error, match=match):
            call()

    A, sA, W1, s1 = _t(4, 256, dtype=U8), _t(4, 2), _t(64, 256, dtype=U8), _t(1, 2)

    def gated(A=A, sA=sA, W1=W1, s1=s1, **kw):
        b.fp8gemm_gated(A, sA, W1, s1, **kw)

    def back(dY=A, s=sA, W=W1[:32], sW=s1, GU=_t(4, 64, dtype=BF), **kw):
        b.fp8gemm_gated_backward(dY, s, W, sW, GU, **kw)

    for match, error, call in [
            ("W1", ValueError, lambda: gated(W1=W1[:63])), ("W1", ValueError, lambda: gated(W1=W1[:, :128])),
            ("sA", ValueError, lambda: gated(sA=sA[:3])), ("s1", ValueError, lambda: gated(s1=_t(2, 2))),
            ("Q has", ValueError, lambda: gated(Q=_t(4, 64, dtype=U8))), ("sQ", ValueError, lambda: gated(sQ=_t(4, 2))),
            ("GU must", TypeError, lambda: gated(GU=_t(4, 64))), ("GU has", ValueError, lambda: gated(GU=_t(4, 32, dtype=BF))),
            ("format", ValueError, lambda: gated(fmt="bf16")), ("Q is torch", TypeError, lambda: gated(Q=_t(4, 32, dtype=U8).view(torch.float8_e5m2))),
            ("CUDA", ValueError, lambda: gated()),
            ("GU has", ValueError, lambda: back(GU=_t(4, 128, dtype=BF))), ("Q has", ValueError, lambda: back(Q=_t(4, 64, dtype=U8))),
            ("W2T", ValueError, lambda: back(W=W1[:32, :128])), ("dGU", ValueError, lambda: back(dGU=_t(4, 32, dtype=BF))),
            ("CUDA", ValueError, lambda: back())]:
        with pytest.raises(error, match=match):
            call()


def _calls():
    from fp8_fine_grained_e4m3_gb300 import binding as b

    def at(d):
        return lambda n, *s, dtype=torch.float32: on(d.get(n, 0), *s, dtype=dtype)

    def rope(d):
        x = at(d)
        return lambda: b.fp8_rope(x("Q", 6, 4, 64, dtype=BF), x("K", 6, 2, 64, dtype=BF), x("freq", 32),
                                  seq_lens=x("seq_lens", 3, dtype=I32), cu=x("cu", 4, dtype=I32),
                                  Qo=x("Qo", 6, 4, 64, dtype=BF), Ko=x("Ko", 6, 2, 64, dtype=BF))

    def packed(d):
        x = at(d)
        return lambda: b.fp8_rope(x("Q", 6, 4, 64, dtype=BF), None, x("freq", 32), positions=x("positions", 6, dtype=I32),
                                  Qo=x("Qo", 6, 4, 64, dtype=BF))

    def chunk(d):
        x = at(d)
        return lambda: b.fp8_kv_attention_chunk(
            x("Q", 6, 4, 64, dtype=BF), x("k_cache", 6, 2, 16, 64, dtype=U8), x("k_scale", 6, 2),
            x("v_cache", 6, 2, 16, 64, dtype=U8), x("v_scale", 6, 2), x("block_table", 3, 2, dtype=I32),
            x("seq_lens", 3, dtype=I32), cu_q=x("cu_q", 4, dtype=I32), O=x("O", 6, 4, 64, dtype=BF))

    def gated(d):
        x = at(d)
        return lambda: b.fp8gemm_gated(x("A", 4, 256, dtype=U8), x("sA", 4, 2), x("W1", 64, 256, dtype=U8), x("s1", 1, 2),
                                       GU=x("GU", 4, 64, dtype=BF), Q=x("Q", 4, 32, dtype=U8), sQ=x("sQ", 4, 1))

    def back(d):
        x = at(d)
        return lambda: b.fp8gemm_gated_backward(
            x("dY", 4, 256, dtype=U8), x("sdY", 4, 2), x("W2T", 32, 256, dtype=U8), x("s2T", 1, 2), x("GU", 4, 64, dtype=BF),
            dGU=x("dGU", 4, 64, dtype=BF), Q=x("Q", 4, 256, dtype=U8), sQ=x("sQ", 4, 2))

    return [(rope, ["Q", "K", "freq", "seq_lens", "cu", "Qo", "Ko"]), (packed, ["Q", "freq", "positions", "Qo"]),
            (chunk, ["Q", "k_cache", "k_scale", "v_cache", "v_scale", "block_table", "seq_lens", "cu_q", "O"]),
            (gated, ["A", "sA", "W1", "s1", "GU", "Q", "sQ"]),
            (back, ["dY", "sdY", "W2T", "s2T", "GU", "dGU", "Q", "sQ"])]


@pytest.mark.parametrize("i", range(5))
def test_tensors_of_another_device(lib, monkeypatch, i):
    from fp8_fine_grained_e4m3_gb300 import binding as b
    f, made = b._lookup(), []
    monkeypatch.setattr(f, "device", lambda: 0)
    monkeypatch.setattr(f, "current", lambda device: made.append(device) or 0)
    for name in ("rope", "kv_attention_chunk", "gated", "gated_backward"):
        monkeypatch.setattr(f, name, lambda *a: 0)
    make, tensors = _calls()[i]
    make({})()
    assert made == [0]
    for t in tensors:
        with pytest.raises(ValueError, match="cuda:"):
            make({t: 1})()
    with pytest.raises(ValueError, match="current device is cuda:0"):
        make({t: 1 for t in tensors})()
    assert made == [0]


@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_frequencies(scaling):
    from fp8_fine_grained_e4m3_gb300 import rotary
    f, amplitude = rotary.frequencies(128, base=10000.0, scaling=scaling, factor=8.0, trained=4096, device="cpu")
    plain = torch.tensor([10000.0 ** (-2 * i / 128) for i in range(64)], dtype=torch.float64)
    assert f.dtype == torch.float32 and f.shape == (64,)
    ratio = f.double() / plain
    assert amplitude == (0.1 * math.log(8.0) + 1 if scaling == "parts" else 1.0)
    if scaling is None:
        assert torch.allclose(ratio, torch.ones_like(ratio), rtol=1e-6)
    elif scaling == "linear":
        assert torch.allclose(ratio, torch.full_like(ratio, 1 / 8), rtol=1e-6)
    else:  # from all of it to an eighth, falling
        assert math.isclose(float(ratio[0]), 1.0, rel_tol=1e-6) and math.isclose(float(ratio[-1]), 1 / 8, rel_tol=1e-6)
        assert bool((ratio[1:] <= ratio[:-1] * (1 + 1e-6)).all())
    if scaling == "parts":
        turns = 4096 * plain / (2 * math.pi)
        assert torch.allclose(ratio[turns >= 32], torch.ones(()).double(), rtol=1e-6)
        assert torch.allclose(ratio[turns <= 1], torch.full((), 1 / 8).double(), rtol=1e-6)


def test_frequencies_refuses():
    from fp8_fine_grained_e4m3_gb300 import rotary
    for kw in (dict(rot=0), dict(rot=7), dict(rot=8, scaling="other"), dict(rot=8, factor=0.5), dict(rot=8, base=0.0),
               dict(rot=2, scaling="base"), dict(rot=8, scaling="parts"), dict(rot=8, scaling="parts", trained=9, fast=1.0)):
        with pytest.raises(ValueError):
            rotary.frequencies(device="cpu", **kw)


MOST = 0x7fffff00


@pytest.mark.parametrize("call,kw,code", [
    # counts that would pass 2^31 when they are rounded up to tiles
    (_rope, dict(T=MOST + 1, pos=GOOD), "SHAPE"), (_rope, dict(B=(1 << 30) + 1), "SHAPE"),
    (_gated, dict(M=MOST + 1, I=16, K=16), "SHAPE"), (_back, dict(M=MOST + 1, I=16, K=16), "SHAPE"),
    (_chunk, dict(T=MOST // 4 + 1), "SHAPE"), (_chunk, dict(most=MOST // 4 + 1), "SHAPE"),
    (_chunk, dict(width=MOST // 64 + 1), "SHAPE"),
    # in place, but rows of the output elsewhere than the input's
    (_rope, dict(ld_qo=264), "SHAPE"), (_rope, dict(ld_k=136), "SHAPE"),
    (_rope, dict(ld_k=136, hk=0, T=0), "OK"),
])
def test_limits_of_counts_and_turning_in_place(lib, call, kw, code):
    from fp8_fine_grained_e4m3_gb300 import binding
    assert call(lib, **kw) == getattr(binding, "OK" if code == "OK" else f"ERR_{code}")
