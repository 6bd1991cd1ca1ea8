"""The accuracy that fa_paged_write states for its angles: 2^-23 radian at n up to 2^24.

Channels (1, 0) turn to (cos a, sin a).  Where a is within 2^-12 of a multiple of pi, fp16
holds sin a in steps of 2^-24 to 2^-22, and shows errors of that size.  Bound, for any a:
2^-23 of the angle, 2^-22 of the value for sine and cosine (1 ulp) and the product with 1,
then one rounding to fp16: eps / 2 of the value and half its smallest step, 2^-25."""
import math

import pytest
import torch

from attention_forward_gb300 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def near_multiples_of_pi(freqs, each):
    """`each` positions below 2^24 for each frequency, whose angles are nearest to one."""
    n = torch.randint(0, 1 << 24, (400000,), generator=torch.Generator().manual_seed(3))
    picked = [torch.tensor([0, 1, (1 << 24) - 1])]
    for f in freqs.double().tolist():
        off = (n.double() * f / math.pi)
        picked.append(n[(off - off.round()).abs().argsort()[:each]])
    return torch.cat(picked)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_angles_are_off_by_2_to_the_minus_23_at_most(pairs, sign):
    page, per, half = 1024, 1 << 14, 32
    g = torch.Generator().manual_seed(5)
    freqs = torch.cat([torch.rand(24, generator=g), torch.tensor([1.0, 1.5, 3.0, 6.5, 1e-3, 1e-6, 255.0, 0.0])])
    at = near_multiples_of_pi(freqs, 12)
    B = len(at)
    table = torch.full((B, per), -1, dtype=torch.int32)
    table[torch.arange(B), at // page] = torch.arange(B, dtype=torch.int32)
    table = table.cuda()
    start = at.int().cuda()
    cache = fa.fa_paged_empty(B, 1, page, 2 * half, torch.float16)
    x = torch.zeros((B, 1, 1, 2 * half), dtype=torch.float16)
    x[..., (torch.arange(half) * 2) if pairs else torch.arange(half)] = 1.0
    x = x.cuda()
    out = [torch.empty_like(x) for _ in range(2)]
    fa.fa_paged_write(x, x, cache, table, start, freqs=(sign * freqs).cuda(), interleaved=pairs)
    fa.fa_paged_read(cache, table, start, out=out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    got = out[0][:, 0, 0].double().cpu()
    one, two = (got[:, 0::2], got[:, 1::2]) if pairs else (got[:, :half], got[:, half:])
    a = at.double()[:, None] * (sign * freqs).double()
    assert (a.sin().abs() < 2.0 ** -12).sum() > 100
    for y, want in ((one, a.cos()), (two, a.sin())):
        room = 2.0 ** -23 + (2.0 ** -22 + 2.0 ** -11) * want.abs() + 2.0 ** -25
        over = (y - want).abs() - room
        assert over.max().item() <= 0, f"off by {over.max().item():.3g} more"
