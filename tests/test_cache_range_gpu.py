"""The 4-bit cache's attention with queries at the ends of their type's range,
against the 64-bit form.  Bounds: ops_ref.py."""
import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref
from test_cache_gpu import cache_of, expect, ints, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top,scale", [(2.0 ** 112, 1e-34), (2.0 ** 113, 1e-34), (2.0 ** 120, 1e-36),
                                       (3e38, 1e-38), (3e38, 5e-37), (1e-36, 1e36), (2.0 ** -133, 3e38)])
def test_queries_at_the_ends_of_their_range(top, scale, D, cap):
    """Rows of every size up to `top` in one block, whose scores are ordinary."""
    B, H, Hkv, L = 1, 16, 2, 300
    cache, table, _, _ = cache_of(B, L, Hkv, 16, D, "bf16", 1)
    q = torch.rand((B, H, 1, D), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    q = (2 * q - 1).double() * top
    q[:, 3::4] *= 2.0 ** -20  # zeros among them
    q = q.to(torch.float32).bfloat16()
    assert q.isfinite().all() and q.abs().amax() > 0
    scale = torch.tensor(scale).item()
    o, lse = fa.fa_fwd_cache(q, cache, table, ints([L]), scale=scale, softcap=cap)
    ok()
    ops_ref.check(o, lse, expect(q, cache, table, ints([L]), scale, cap))
