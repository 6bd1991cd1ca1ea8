"""bf16 values up to the magnitude that the calls on 16-bit pages, latent rows and
expanded heads are stated for, 2^88: the sums of unnormalised probabilities (up to 2^15
each, 2^8 in the expanded form) times values stay in fp32."""
import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref
import paged_ref

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def normal(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def large(seed, *shape):
    """2^87 to 2^88 in magnitude, of either sign."""
    x = normal(seed, *shape)
    return ((1.0 + x.abs().fmod(0.96)) * 2.0 ** 87 * x.sign()).bfloat16()


def risen(L, by):
    """Scores in log2 units by key: every tenth tile of 64 low, which sets a reference that
    the others stay `by` above."""
    return torch.where(torch.arange(L, device="cuda") // 64 % 10 == 0, 0.0, by)


def ok():
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


@pytest.mark.parametrize("H", [2, 40])
@pytest.mark.parametrize("D,L", [(64, 16384), (128, 700)])
def test_pages(D, L, H):
    page = 64
    per = -(-L // page)
    cache = fa.fa_paged_empty(per, 1, page, D)
    table = torch.arange(per, dtype=torch.int32, device="cuda").view(1, per)
    k = torch.zeros((1, 1, L, D), device="cuda")
    k[..., 0] = risen(L, 6.9) / LOG2E
    fa.fa_paged_write(k.bfloat16(), large(1, 1, 1, L, D), cache, table)
    q = torch.zeros((1, H, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    length = torch.tensor([L], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_paged(q, cache, table, length, scale=1.0)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, *cache, table, length, 1.0))


@pytest.mark.parametrize("H", [4, 24, 64, 128])
@pytest.mark.parametrize("L", [200, 9000])
def test_latent_rows(L, H):
    page = 64
    per = -(-L // page)
    cache = fa.fa_latent_empty(per, page)
    table = torch.arange(per, dtype=torch.int32, device="cuda").view(1, per)
    rope = torch.zeros((1, L, 64), device="cuda")
    rope[..., 0] = risen(L, 6.9) / LOG2E
    fa.fa_latent_write(large(2, 1, L, 512), rope.bfloat16(), cache, table)
    q = torch.zeros((1, H, 1, 576), dtype=torch.bfloat16, device="cuda")
    q[..., 512] = 1.0  # the scores come from the rotated part alone
    length = torch.tensor([L], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_latent(q, cache, table, length, scale=1.0)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, cache, None, table, length, 1.0))


@pytest.mark.parametrize("Sq,Skv", [(300, 300), (100, 3000)])
def test_expanded(Sq, Skv):
    kv = torch.zeros((1, 2, Skv, 256), device="cuda")
    kv[..., 0] = (torch.arange(Skv, device="cuda") // 128 % 10 != 0) * 7.9 / LOG2E
    kv = kv.bfloat16()
    kv[..., 128:] = large(3, 1, 2, Skv, 128)
    q = torch.zeros((1, 2, Sq, 192), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    rope = torch.zeros((1, Skv, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_fwd_expanded(q, kv, rope, causal=True, scale=1.0)
    ok()
    i = torch.arange(Sq, device="cuda")[:, None] + (Skv - Sq)
    seen = torch.arange(Skv, device="cuda")[None] <= i
    ops_ref.check(o, lse, paged_ref.attention(q[..., :128], kv[..., :128], kv[..., 128:],
                                              seen[None, None], 1.0))
