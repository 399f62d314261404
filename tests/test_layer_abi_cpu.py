"""The decoder-layer calls refuse what they cannot take on the host, before
any CUDA call.  CPU only."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p
GOOD = P(1 << 20)  # never dereferenced
S = P(0)


@pytest.fixture(scope="module")
def lib():
    from fp8_fine_grained_e4m3_gb300 import build, binding
    build.build()
    return binding.lib()


def _norm(lib, **kw):
    a = dict(X=GOOD, R=GOOD, t=0, G=GOOD, eps=1e-6, H=GOOD, Q=GOOD, sQ=GOOD, rstd=GOOD, M=4, K=256, fmt=0, s=S)
    a.update(kw)
    return lib.fp8_rmsnorm_quant(*a.values())


def _back(lib, **kw):
    a = dict(dY=GOOD, H=GOOD, t=0, rstd=GOOD, G=GOOD, dH=GOOD, dX=GOOD, dG=GOOD, M=4, K=256, s=S)
    a.update(kw)
    return lib.fp8_rmsnorm_backward(*a.values())


def _append(lib, **kw):
    a = dict(K=GOOD, V=GOOD, ld_k=256, ld_v=256, kc=GOOD, ks=GOOD, vc=GOOD, vs=GOOD, table=GOOD, lens=GOOD, cu=GOOD,
             T=8, B=4, heads=2, dim=128, block=64, width=3, n=12, most=4, fmt=0, s=S)
    a.update(kw)
    return lib.fp8_kv_append(*a.values())


def _attend(lib, **kw):
    a = dict(Q=GOOD, ld_q=1024, kc=GOOD, ks=GOOD, vc=GOOD, vs=GOOD, table=GOOD, lens=GOOD, cu=GOOD, scale=1.0, O=GOOD,
             T=8, B=4, heads=2, group=4, dim=128, block=64, width=3, n=12, most=4, fmt=0, s=S)
    a.update(kw)
    return lib.fp8_kv_attention(*a.values())


def _moe(lib, **kw):
    a = dict(A=GOOD, sA=GOOD, logits=GOOD, W1=GOOD, s1=GOOD, W2=GOOD, s2=GOOD, D=GOOD, ids=GOOD, w=GOOD, T=4, H=256,
             I=128, E=8, k=2, renorm=1, s=S)
    a.update(kw)
    return lib.fp8_moe_few(*a.values())


ODD8, ODD2 = P((1 << 20) + 8), P((1 << 20) + 2)


@pytest.mark.parametrize("call,kw,code", [
    (_norm, dict(M=-1), "SHAPE"), (_norm, dict(K=0), "SHAPE"), (_norm, dict(K=200), "SHAPE"),
    (_norm, dict(K=16400), "SHAPE"), (_norm, dict(fmt=2), "FORMAT"), (_norm, dict(t=2), "FORMAT"),
    (_norm, dict(X=None), "NULL"), (_norm, dict(R=None), "NULL"), (_norm, dict(H=None), "NULL"),
    (_norm, dict(Q=ODD8), "ALIGN"), (_norm, dict(R=ODD8), "ALIGN"), (_norm, dict(rstd=ODD2), "ALIGN"),
    (_norm, dict(M=0, X=None), "OK"),
    (_back, dict(M=-1), "SHAPE"), (_back, dict(K=24), "SHAPE"), (_back, dict(t=-1), "FORMAT"),
    (_back, dict(dG=None), "NULL"), (_back, dict(dY=None), "NULL"), (_back, dict(rstd=None), "NULL"),
    (_back, dict(dH=ODD8), "ALIGN"), (_back, dict(dX=ODD8), "ALIGN"), (_back, dict(G=ODD8), "ALIGN"),
    (_append, dict(T=-1), "SHAPE"), (_append, dict(dim=96), "SHAPE"), (_append, dict(block=48), "SHAPE"),
    (_append, dict(block=256), "SHAPE"), (_append, dict(ld_k=255), "SHAPE"), (_append, dict(ld_v=260), "SHAPE"),
    (_append, dict(cu=None, T=7), "SHAPE"), (_append, dict(cu=None, most=1), "SHAPE"), (_append, dict(fmt=7), "FORMAT"),
    (_append, dict(width=-1), "SHAPE"), (_append, dict(B=32768), "SHAPE"), (_append, dict(heads=65536), "SHAPE"),
    (_append, dict(V=None), "NULL"), (_append, dict(lens=None), "NULL"), (_append, dict(K=ODD8), "ALIGN"),
    (_append, dict(vc=ODD8), "ALIGN"), (_append, dict(table=ODD2), "ALIGN"), (_append, dict(cu=ODD2), "ALIGN"),
    (_append, dict(T=0), "OK"), (_append, dict(most=0, K=None), "OK"),
    (_attend, dict(group=-1), "SHAPE"), (_attend, dict(dim=256), "SHAPE"), (_attend, dict(ld_q=1016), "SHAPE"),
    (_attend, dict(ld_q=1028), "SHAPE"), (_attend, dict(cu=None, T=6), "SHAPE"),
    (_attend, dict(group=40000), "SHAPE"), (_attend, dict(fmt=-1), "FORMAT"), (_attend, dict(O=None), "NULL"),
    (_attend, dict(ks=None), "NULL"), (_attend, dict(O=ODD8), "ALIGN"), (_attend, dict(ks=ODD2), "ALIGN"),
    (_attend, dict(B=0, cu=None, T=0), "OK"), (_attend, dict(group=0), "OK"),
    (_moe, dict(T=65), "SHAPE"), (_moe, dict(T=-1), "SHAPE"), (_moe, dict(H=100), "SHAPE"), (_moe, dict(I=0), "SHAPE"),
    (_moe, dict(I=24), "SHAPE"), (_moe, dict(k=0), "SHAPE"), (_moe, dict(k=9), "SHAPE"), (_moe, dict(E=513), "SHAPE"),
    (_moe, dict(E=64, k=17), "SHAPE"), (_moe, dict(W2=None), "NULL"), (_moe, dict(ids=None), "NULL"),
    (_moe, dict(W1=ODD8), "ALIGN"), (_moe, dict(sA=ODD8), "ALIGN"), (_moe, dict(logits=ODD2), "ALIGN"),
    (_moe, dict(T=0, A=None), "OK")])
def test_host_validation(lib, call, kw, code):
    from fp8_fine_grained_e4m3_gb300 import binding as b
    want = b.OK if code == "OK" else getattr(b, "ERR_" + code)
    assert call(lib, **kw) == want


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_on_host():
    from fp8_fine_grained_e4m3_gb300 import binding as b
    x, g = _t(4, 256, dtype=torch.bfloat16), _t(256)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        b.fp8_rmsnorm_quant(x.half(), g)
    with pytest.raises(ValueError, match="gain"):
        b.fp8_rmsnorm_quant(x, _t(255))
    with pytest.raises(TypeError, match="residual"):
        b.fp8_rmsnorm_quant(x, g, residual=x.float())
    with pytest.raises(ValueError, match="residual"):
        b.fp8_rmsnorm_quant(x, g, residual=x[:2])
    with pytest.raises(ValueError, match="give residual"):
        b.fp8_rmsnorm_quant(x, g, H=x)
    with pytest.raises(ValueError, match="sQ"):
        b.fp8_rmsnorm_quant(x, g, sQ=_t(4, 3))
    with pytest.raises(ValueError, match="format"):
        b.fp8_rmsnorm_quant(x, g, fmt="fp8")
    with pytest.raises(ValueError, match="CUDA"):
        b.fp8_rmsnorm_quant(x, g)
    with pytest.raises(TypeError, match="dY"):
        b.fp8_rmsnorm_backward(x.float(), x, _t(4), g)
    with pytest.raises(ValueError, match="rstd"):
        b.fp8_rmsnorm_backward(x, x, _t(3), g)

    i32, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    kc, ks, tab, lens = _t(6, 2, 16, 64, dtype=u8), _t(6, 2), _t(3, 2, dtype=i32), _t(3, dtype=i32)
    k = _t(3, 2, 64, dtype=bf)

    def append(K=k, V=k, kc=kc, ks=ks, vc=kc, vs=ks, tab=tab, lens=lens, **kw):
        b.fp8_kv_append(K, V, kc, ks, vc, vs, tab, lens, **kw)

    def attend(Q=_t(3, 4, 64, dtype=bf), kc=kc, tab=tab, lens=lens, **kw):
        b.fp8_kv_attention(Q, kc, ks, kc, ks, tab, lens, **kw)

    for call in (append, attend):
        with pytest.raises(ValueError, match="num_blocks"):
            call(kc=kc[0])
        with pytest.raises(TypeError, match="block_table"):
            call(tab=tab.long())
        with pytest.raises(ValueError, match="block_table"):
            call(tab=tab[0])
        with pytest.raises(ValueError, match="seq_lens"):
            call(lens=lens[:2])
        with pytest.raises(TypeError, match="float8"):
            call(kc=kc.view(torch.float8_e5m2))
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="k_scale"):
        append(ks=ks[:5])
    with pytest.raises(ValueError, match="offsets"):
        append(cu_new=_t(3, dtype=i32))
    with pytest.raises(ValueError, match="give the offsets"):
        append(K=k[:2], V=k[:2])
    with pytest.raises(TypeError, match="bfloat16"):
        append(K=k.float())
    with pytest.raises(ValueError, match="cached heads"):
        attend(Q=_t(3, 3, 64, dtype=bf))

    A, lg = _t(2, 256, dtype=u8), _t(2, 4)
    W1, W2 = _t(4, 256, 256, dtype=u8), _t(4, 256, 128, dtype=u8)

    def moe(A=A, sA=_t(2, 2), lg=lg, W1=W1, s1=_t(4, 2, 2), W2=W2, s2=_t(4, 2, 1), k=2, **kw):
        b.fp8_moe_few(A, sA, lg, W1, s1, W2, s2, k, **kw)

    with pytest.raises(ValueError, match="W1"):
        moe(W1=W1[0])
    with pytest.raises(ValueError, match="W2"):
        moe(W2=W2[:, :, :64])
    with pytest.raises(ValueError, match="logits"):
        moe(lg=lg[:, :3])
    with pytest.raises(ValueError, match="s2"):
        moe(s2=_t(4, 2, 2))
    with pytest.raises(ValueError, match="ids"):
        moe(ids=_t(2, 3, dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        moe()
