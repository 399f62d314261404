"""Waits that run out in the chunk attention and the gated products: whatever the limit, every warp of the launch
ends, no copy outlives its CTA, and the next calls are right."""

import pytest

from tests.test_gpu_prompt_layer import CALLS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", CALLS)
def test_limits_from_no_time_to_enough(name):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    call = CALLS[name](1)
    want = call()
    torch.cuda.synchronize()
    seen = set()
    for ns in (1, 500, 2000, 8000, 32000, 10 ** 9):
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
def test_calls_beside_and_behind_one_that_gave_up(gives_up):
    """The shared memory and the TMEM of CTAs that gave up are taken at once by the next call's and by another
    stream's."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    bad, good = CALLS[gives_up](1), CALLS["chunk, units"](2)
    want = good()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        assert torch.equal(good(), want)
    torch.cuda.synchronize()
    behind = []
    for _ in range(4):
        b.set_wait_limit_ns(1)
        try:
            bad()
        finally:
            b.set_wait_limit_ns(0)
        with torch.cuda.stream(other):
            behind.append(good())
        behind.append(good())
    torch.cuda.synchronize()
    assert b.fp8gemm_get_device_status() in (b.OK, b.ERR_TIMEOUT)
    assert all(torch.equal(x, want) for x in behind)
    assert torch.equal(good(), want) and b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("name", [n for n in CALLS if not n.startswith("chunk")])
def test_limits_that_run_out_somewhere_in_a_product(name):
    """Limits in small steps, so that waits run out at the first K block, in the middle and behind the last one: every
    warp goes on to its matrix instructions and shuffles as a whole."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    call = CALLS[name](1)
    want = call()
    torch.cuda.synchronize()
    for i in range(60):
        b.set_wait_limit_ns(int(1.2 ** i))
        try:
            got = call()
            status = b.fp8gemm_get_device_status()
        finally:
            b.set_wait_limit_ns(0)
        assert status in (b.OK, b.ERR_TIMEOUT)
        if status == b.OK:
            assert torch.equal(got, want)
    assert torch.equal(call(), want)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("name", CALLS)
def test_no_time_is_not_enough(name):
    """A limit of 1 ns runs out, and the status says so: in one of a few calls at the least, since a wait may find that
    what it waits for is there."""
    from fp8_fine_grained_e4m3_gb300 import binding as b
    call = CALLS[name](1)
    call()
    assert b.fp8gemm_get_device_status() == b.OK
    seen = set()
    for _ in range(4):
        b.set_wait_limit_ns(1)
        try:
            call()
            seen.add(b.fp8gemm_get_device_status())
        finally:
            b.set_wait_limit_ns(0)
    assert b.ERR_TIMEOUT in seen and seen <= {b.OK, b.ERR_TIMEOUT}
