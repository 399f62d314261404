"""Host threads that share a stream: a call of several kernels, which hand data on
through the stream's workspace, is enqueued as a whole."""

import sys
import threading

import pytest

pytestmark = pytest.mark.gpu


def _moe(T, k, I, seed):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H, E = 512, 8
    A, W1, W2 = (torch.randint(0, 112, s, generator=g, dtype=torch.uint8, device="cuda")
                 for s in ((T, H), (E, 2 * I, H), (E, H, I)))
    sA, s1, s2 = (torch.full(s, 2.0 ** -7, device="cuda")
                  for s in ((T, H // 128), (E, -(-2 * I // 128), H // 128), (E, H // 128, -(-I // 128))))
    logits = torch.randn((T, E), generator=g, device="cuda")
    return lambda: b.fp8_moe_few(A, sA, logits, W1, s1, W2, s2, k)


def _norm_gradient(M, K, seed):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dy, h = (torch.randn((M, K), generator=g, device="cuda") for _ in range(2))
    rstd, gain = torch.ones(M, device="cuda"), torch.ones(K, device="cuda")
    return lambda: b.fp8_rmsnorm_backward(dy, h, rstd, gain)


def _quant_a(M, seed):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, sB = b.fp8_quant_128x128(torch.randn((256, 512), generator=g, device="cuda"))
    X = torch.randn((M, 512), generator=g, device="cuda")
    return lambda: (b.fp8gemm_dense_quant_a(X, B, sB),)


CALLS = {"moe": lambda: [_moe(3, 2, 256, 1), _moe(40, 2, 256, 2), _moe(64, 3, 256, 3)],
         "moe, a growing workspace": lambda: [_moe(3, 2, 128, 4), _moe(40, 2, 2048, 5), _moe(64, 3, 4096, 6)],
         "norm gradient": lambda: [_norm_gradient(900, 1024, 7), _norm_gradient(77, 4096, 8), _norm_gradient(500, 256, 9)],
         "quantise and multiply": lambda: [_quant_a(100, 10), _quant_a(2000, 11), _quant_a(300, 12)]}


@pytest.mark.parametrize("name", CALLS)
def test_threads_share_a_stream(name):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    calls = CALLS[name]()
    want = []
    for c in calls:
        want.append([t.clone() for t in c()])
    torch.cuda.synchronize()
    b.fp8gemm_release_workspaces()
    bad, rounds = [], 60
    start = threading.Barrier(len(calls))

    def work(i):
        start.wait()
        got = [calls[i]() for _ in range(rounds)]
        torch.cuda.synchronize()
        bad.extend(i for r in got if not all(torch.equal(x, y) for x, y in zip(r, want[i])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not bad
    assert b.fp8gemm_get_device_status() == b.OK
