"""The decoder-layer calls refuse tensors of another device than the current one, or
than their first tensor's, before any address is passed on.  CPU only: tensors that
say that they lie on a GPU, and a library that counts its calls."""

import pytest
import torch

from fp8_fine_grained_e4m3_gb300 import binding as b


class On(torch.Tensor):
    """A tensor that says that it lies on GPU `at`."""
    at = 0

    def get_device(self):
        return self.at

    is_cuda = True


def on(device, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.at = device
    return t


BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def _norm(d):
    x = lambda n: on(d.get(n, 0), 4, 256, dtype=BF)  # noqa: E731
    f = lambda n, *s: on(d.get(n, 0), *s)  # noqa: E731
    return lambda: b.fp8_rmsnorm_quant(x("X"), f("gain", 256), residual=x("residual"), H=x("H"),
                                       Q=on(d.get("Q", 0), 4, 256, dtype=U8), sQ=f("sQ", 4, 2), rstd=f("rstd", 4))


def _back(d):
    x = lambda n: on(d.get(n, 0), 4, 256, dtype=BF)  # noqa: E731
    f = lambda n, *s: on(d.get(n, 0), *s)  # noqa: E731
    return lambda: b.fp8_rmsnorm_backward(x("dY"), x("H"), f("rstd", 4), f("gain", 256), dH=x("dH"), dX=x("dX"),
                                          dgain=f("dgain", 256))


def _cache(d):
    return (on(d.get("k_cache", 0), 6, 2, 16, 64, dtype=U8), on(d.get("k_scale", 0), 6, 2),
            on(d.get("v_cache", 0), 6, 2, 16, 64, dtype=U8), on(d.get("v_scale", 0), 6, 2),
            on(d.get("block_table", 0), 3, 2, dtype=I32), on(d.get("seq_lens", 0), 3, dtype=I32))


def _append(d):
    x = lambda n: on(d.get(n, 0), 3, 2, 64, dtype=BF)  # noqa: E731
    return lambda: b.fp8_kv_append(x("K"), x("V"), *_cache(d), cu_new=on(d.get("cu_new", 0), 4, dtype=I32))


def _attend(d):
    x = lambda n: on(d.get(n, 0), 3, 4, 64, dtype=BF)  # noqa: E731
    return lambda: b.fp8_kv_attention(x("Q"), *_cache(d), cu_q=on(d.get("cu_q", 0), 4, dtype=I32), O=x("O"))


def _moe(d):
    u = lambda n, *s: on(d.get(n, 0), *s, dtype=U8)  # noqa: E731
    f = lambda n, *s: on(d.get(n, 0), *s)  # noqa: E731
    return lambda: b.fp8_moe_few(u("A", 2, 256), f("sA", 2, 2), f("logits", 2, 4), u("W1", 4, 256, 256), f("s1", 4, 2, 2),
                                 u("W2", 4, 256, 128), f("s2", 4, 2, 1), 2, D=on(d.get("D", 0), 2, 256, dtype=BF),
                                 ids=on(d.get("ids", 0), 2, 2, dtype=I32), weights=f("weights", 2, 2))


CACHE = ["k_cache", "k_scale", "v_cache", "v_scale", "block_table", "seq_lens"]
CALLS = [(_norm, "rmsnorm_quant", ["X", "gain", "residual", "H", "Q", "sQ", "rstd"]),
         (_back, "rmsnorm_backward", ["dY", "H", "rstd", "gain", "dH", "dX", "dgain"]),
         (_append, "kv_append", ["K", "V", *CACHE, "cu_new"]), (_attend, "kv_attention", ["Q", *CACHE, "cu_q", "O"]),
         (_moe, "moe_few", ["A", "sA", "logits", "W1", "s1", "W2", "s2", "D", "ids", "weights"])]


@pytest.fixture
def calls(monkeypatch):
    from fp8_fine_grained_e4m3_gb300 import build
    build.build()
    f, made = b._lookup(), []
    monkeypatch.setattr(f, "device", lambda: 0)
    monkeypatch.setattr(f, "current", lambda device: made.append(device) or 0)
    for _, name, _ in CALLS:
        monkeypatch.setattr(f, name, lambda *a: 0)
    return made


@pytest.mark.parametrize("make,name,tensors", CALLS)
def test_one_tensor_elsewhere(calls, make, name, tensors):
    make({})()
    assert calls == [0]
    for t in tensors:
        with pytest.raises(ValueError, match="cuda:"):
            make({t: 1})()
    assert calls == [0]


@pytest.mark.parametrize("make,name,tensors", CALLS)
def test_all_of_them_elsewhere(calls, make, name, tensors):
    with pytest.raises(ValueError, match="current device is cuda:0"):
        make({t: 1 for t in tensors})()
    assert calls == []
