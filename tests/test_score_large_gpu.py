"""fa_fwd_score on tensors past 2^31 elements: sampled rows against the 64-bit
form.  Bounds: ops_ref.py."""
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


def test_queries_past_2_to_31_elements():
    """Documents of 700 tokens under a cap and a bias: a row's keys are few."""
    B, H, Hkv, S, D, doc, cap = 2, 130, 2, 65536, 128, 700, 30.0
    assert B * H * S * D > 2 ** 31
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.randn((B, H, S, D), generator=g, device="cuda", dtype=torch.bfloat16)
    k = torch.randn((B, Hkv, S, D), generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn((B, Hkv, S, D), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.arange(S, device="cuda").div(doc, rounding_mode="floor").int().expand(B, S).contiguous()
    slopes = torch.logspace(-2, -9, H, 2.0, device="cuda")
    o, lse = fa.fa_fwd_score(q, k, v, causal=True, softcap=cap, slopes=slopes, doc_q=ids, doc_k=ids)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    for b, h in ((0, 0), (0, 129), (1, 0), (1, 64), (1, 128), (1, 129)):
        for first in (0, doc * 46, doc * ((S - 1) // doc)):
            last = min(first + doc, S)
            n = last - first
            i = torch.arange(n, device="cuda")
            seen, dist = (i[None] <= i[:, None])[None, None], (i[:, None] - i[None]).abs()
            kv = h // (H // Hkv)
            ref = ops_ref.attention(q[b:b + 1, h:h + 1, first:last], k[b:b + 1, kv:kv + 1, first:last],
                                    v[b:b + 1, kv:kv + 1, first:last], seen, D ** -0.5, cap,
                                    slopes[h:h + 1], dist, p_step=2.0 ** -8)
            ops_ref.check(o[b:b + 1, h:h + 1, first:last], lse[b:b + 1, h:h + 1, first:last], ref)


def test_cache_rows_past_2_to_31_elements():
    """A chunk of that size into the cache and back: its ends."""
    B, Hkv, S, D, page = 2, 130, 65536, 128, 1024
    assert B * Hkv * S * D > 2 ** 31
    per = S // page
    g = torch.Generator("cuda").manual_seed(2)
    k = torch.randn((B, Hkv, S, D), generator=g, device="cuda", dtype=torch.bfloat16)
    cache = fa.fa_cache_empty(B * per, Hkv, page, D)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(3)).view(B, per).int().cuda()
    fa.fa_cache_write(k, k, cache, table)
    out = [torch.empty_like(k), torch.empty_like(k)]
    fa.fa_cache_read(cache, table, out=out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    for b, h in ((0, 0), (0, 129), (1, 0), (1, 63), (1, 129)):
        for rows in (slice(0, 40), slice(S // 2 - 20, S // 2 + 20), slice(S - 40, S)):
            x = k[b, h, rows]
            codes, params = ops_ref.quantise(x)
            at = torch.arange(S, device="cuda")[rows]
            pg = table[b, at // page].long()
            for n in (0, 2):
                assert torch.equal(cache[n][pg, h, at % page], ops_ref.pack(codes))
                assert torch.equal(cache[n + 1][pg, h, at % page], params)
            val = ops_ref.unpack(ops_ref.pack(codes), params)
            for t in out:
                assert ((t[b, h, rows].double() - val).abs() <= 2.0 ** -8 * val.abs()).all()
