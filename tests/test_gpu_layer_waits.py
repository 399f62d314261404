"""Waits that run out in the cache attention and the MoE layer: whatever the
limit, every warp of the launch ends, and no copy outlives its CTA."""

import pytest

pytestmark = pytest.mark.gpu


def _attention(B, length, heads=8, dim=128, block=64, group=2, seed=0):
    """A call over a cache of more than the L2, as a function of nothing."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = B * length // block
    k, v = (torch.randint(0, 120, (n, heads, block, dim), generator=g, dtype=torch.uint8, device="cuda")
            for _ in range(2))
    ks, vs = (torch.full((n, heads), 2.0 ** -7, device="cuda") for _ in range(2))
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(B, -1)
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    q = torch.randn((B, heads * group, dim), generator=g, device="cuda").to(torch.bfloat16)
    return lambda **kw: b.fp8_kv_attention(q, k, ks, v, vs, table, lens, **kw)


def _moe(T, k, H=4096, I=2048, E=16, seed=0):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    W1, W2, A = (torch.randint(0, 100, s, generator=g, dtype=torch.uint8, device="cuda")
                 for s in ((E, 2 * I, H), (E, H, I), (T, H)))
    s1, s2, sA = (torch.full(s, 2.0 ** -8, device="cuda")
                  for s in ((E, 2 * I // 128, H // 128), (E, H // 128, I // 128), (T, H // 128)))
    logits = torch.randn((T, E), generator=g, device="cuda")
    return lambda **kw: b.fp8_moe_few(A, sA, logits, W1, s1, W2, s2, k, **kw)[0]


CALLS = {"attention, parts of items": lambda: _attention(1, 262144), "attention, runs": lambda: _attention(64, 4096),
         "moe, 8 tokens a pass": lambda: _moe(2, 8), "moe, 16 tokens a pass": lambda: _moe(40, 2),
         "moe, 32 tokens a pass": lambda: _moe(64, 10)}


@pytest.mark.parametrize("name", CALLS)
def test_limits_from_no_time_to_enough(name):
    """Limits that pass at the first wait, somewhere on the way, and never: the
    call always ends, says whether it gave up, and the next one is right."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    call = CALLS[name]()
    want = call()
    torch.cuda.synchronize()
    seen = set()
    for ns in (1, 100, 500, 1000, 2000, 4000, 8000, 16000, 10 ** 9):
        b.set_wait_limit_ns(ns)
        try:
            got = call()
            status = b.fp8gemm_get_device_status()
        finally:
            b.set_wait_limit_ns(0)
        seen.add(status)
        assert status in (b.OK, b.ERR_TIMEOUT)
        if status == b.OK:
            assert torch.equal(got, want)
        assert torch.equal(call(), want)
        assert b.fp8gemm_get_device_status() == b.OK
    assert b.OK in seen


@pytest.mark.parametrize("gives_up", CALLS)
@pytest.mark.parametrize("beside", ["attention, runs", "moe, 8 tokens a pass"])
def test_calls_beside_and_behind_one_that_gave_up(gives_up, beside):
    """Shared memory that the CTAs of a call which gave up leave is taken at once by
    the CTAs of the next call on the stream and of a call on another one: a copy
    that landed after its CTA had gone would fall into theirs."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    bad, good = CALLS[gives_up](), CALLS[beside]()
    want = good()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()  # the inputs were made on the first stream
    with torch.cuda.stream(other):
        assert torch.equal(good(), want)
    torch.cuda.synchronize()
    behind = []
    for _ in range(6):
        b.set_wait_limit_ns(1)
        try:
            bad()
        finally:
            b.set_wait_limit_ns(0)
        with torch.cuda.stream(other):
            behind.append(good())
        # the bad call leaves its own counters mid-count: only calls with other buffers follow it
        if gives_up.split(",")[0] != beside.split(",")[0]:
            behind.append(good())
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in behind)
    assert b.fp8gemm_get_device_status() in (b.OK, b.ERR_TIMEOUT)
    assert torch.equal(good(), want)
    b.fp8gemm_release_workspaces(other)
