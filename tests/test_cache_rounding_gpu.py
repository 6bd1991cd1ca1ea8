"""Values read back from the 4-bit cache are the stored ones, rounded once."""
import numpy as np
import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def rounded(values, bits, least):
    """Numbers in 64 bits (exact: a code of 4 bits times a scale of 11, plus a
    minimum of 11, whose exponents are 40 apart at most) to the nearest of `bits`
    significant ones, ties to even; `least`: the smallest normal number's exponent."""
    v = values.cpu().numpy()
    _, e = np.frexp(v)
    e = np.maximum(e, least + 1)
    return np.ldexp(np.rint(np.ldexp(v, bits - e)), e - bits)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_every_value_is_rounded_once(dt, D):
    """Scales and minima over all of fp16's exponents, so that sums lie on and
    beside every tie; the largest kept within fp16."""
    pages, Hkv, page = 64, 2, 64
    g = torch.Generator("cuda").manual_seed(1)
    cache = list(fa.fa_cache_empty(pages, Hkv, page, D))
    rows = (pages, Hkv, page)
    for n in (0, 2):
        cache[n] = torch.randint(0, 256, rows + (D // 2,), generator=g, device="cuda", dtype=torch.uint8)
        par = torch.randint(0, 1 << 16, rows + (D // 32, 2), generator=g, device="cuda")
        # scale: at most 2^11, positive; minimum: at most 2^14 in magnitude
        scale = par[..., 0] & 0x7FFF
        scale = torch.where(scale >= (26 << 10), scale & 0x3FFF, scale)
        least = torch.where((par[..., 1] & 0x7FFF) >= (29 << 10), par[..., 1] & 0xBFFF, par[..., 1])
        # and codes of one significant bit beside round minima, where ties are
        tie = torch.randint(0, 2, scale.shape, generator=g, device="cuda").bool()
        scale = torch.where(tie, scale & 0x7C00, scale)
        least = torch.where(tie, least & 0xFFFC, least)
        both = torch.stack([scale, least], -1)
        cache[n + 1] = both.to(torch.int32).to(torch.int16).view(torch.float16).contiguous()
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    out = [torch.empty((1, Hkv, pages * page, D), dtype=dt, device="cuda") for _ in range(2)]
    fa.fa_cache_read(cache, table, out=out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    for n in range(2):
        assert cache[2 * n + 1].isfinite().all()
        exact = ops_ref.unpack(cache[2 * n], cache[2 * n + 1])  # [pages, Hkv, page, D]
        exact = exact.transpose(0, 1).reshape(1, Hkv, pages * page, D)
        want = rounded(exact, 8, -126) if dt is torch.bfloat16 else rounded(exact, 11, -14)
        got = out[n].double().cpu().numpy()
        assert (got == want).all(), int((got != want).sum())


def test_a_sum_beside_a_tie():
    """1 + 2^-8 is a tie of bf16; 2^-24 more goes up."""
    cache = list(fa.fa_cache_empty(1, 1, 16, 64))
    cache[0].fill_(0x11)
    cache[1][..., 0], cache[1][..., 1] = 2.0 ** -24, 1 + 2.0 ** -8
    out = [torch.empty((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.fa_cache_read(cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), out=out)
    assert (out[0] == 1 + 2.0 ** -7).all()
