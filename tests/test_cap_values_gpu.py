"""What values V may have under a cap that bounds the scores (bf16, up to 50), with
every score at the cap's ends, and without that limit where slopes are given.
Bounds: ops_ref.py."""
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


def at_the_cap(sign, Sq, Skv, D=64):
    """Scores far past the cap, all of one sign."""
    g = torch.Generator("cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q = ((n(1, 4, Sq, D).abs() + 1) * 6).bfloat16()
    k = ((n(1, 2, Skv, D).abs() + 1) * 2 * sign).bfloat16()
    return q, k, n(1, 2, Skv, D).clamp(-4, 4)


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("Sq,Skv", [(1, 1), (200, 300), (300, 9000)])
@pytest.mark.parametrize("power,slopes", [(28, False), (-50, False), (56, True), (100, True), (-100, True)])
def test_values_at_their_limits(power, slopes, Sq, Skv, sign):
    """|V| up to 2^30 (4 * 2^28)."""
    q, k, v = at_the_cap(sign, Sq, Skv)
    v = v.double() * 2.0 ** power
    if power == -50:
        v = v + torch.where(v < 0, -1.0, 1.0) * 2.0 ** -50
    v = v.float().bfloat16()
    s = torch.zeros(4, device="cuda") if slopes else None
    o, lse = fa.fa_fwd_score(q, k, v, softcap=50.0, slopes=s)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    seen, dist = ops_ref.score_seen(Sq, Skv, False)
    ops_ref.check(o, lse, ops_ref.attention(q, k, v, seen, 0.125, 50.0, p_step=2.0 ** -8))
