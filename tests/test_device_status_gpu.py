"""The device status word: what several kernels leave in it before it is read."""
import pytest
import torch

from attention_forward_gb300 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def timeout():
    """A call whose bounded waits run out (20 ms)."""
    q = torch.zeros((1, 2, 256, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 2, 512, 128), dtype=torch.bfloat16, device="cuda")
    fa.fa_set_watchdog_ns(20_000_000)
    try:
        fa.fa_fwd_ex(q, k, k, flags=fa.FA_FLAG_TEST_STALL)
    finally:
        fa.fa_set_watchdog_ns(0)


def cache_calls(per):
    """Calls that meet a page or a length that does not exist (per * 16 keys)."""
    cache = fa.fa_cache_empty(per, 1, 16, 64)
    good = torch.arange(per, dtype=torch.int32, device="cuda")[None].contiguous()
    bad = good.clone()
    bad[0, 0] = per
    row = torch.ones((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    out = [torch.empty_like(row), torch.empty_like(row)]
    return {"write": lambda: fa.fa_cache_write(row, row, cache, bad),
            "read": lambda: fa.fa_cache_read(cache, bad, out=out),
            "page": lambda: fa.fa_fwd_cache(row, cache, bad, ints([3])),
            "length": lambda: fa.fa_fwd_cache(row, cache, good, ints([16 * per + 1]))}


@pytest.mark.parametrize("per", [2, 80], ids=["short table", "long table"])
@pytest.mark.parametrize("which", ["write", "read", "page", "length"])
def test_a_place_that_does_not_exist_hides_no_timeout(which, per):
    call = cache_calls(per)[which]
    assert fa.fa_get_device_status() == fa.FA_OK
    call()
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    timeout()
    call()
    assert fa.fa_get_device_status() == fa.FA_ERR_TIMEOUT
    call()
    timeout()
    assert fa.fa_get_device_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_get_device_status() == fa.FA_OK
