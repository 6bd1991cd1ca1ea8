"""Latent attention: its paged cache and the absorbed form, within the bounds of
paged_ref.py."""
import math
import random

import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref
import paged_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def table_of(B, per, pages, seed=0):
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    return ints(order[:B * per]).view(B, per)


def ok():
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


def normal(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def freqs_of():
    j = torch.arange(32, dtype=torch.float64, device="cuda")
    return (10000.0 ** (-j / 32)).float()


def cache_of(B, L, page, dt, seed=0):
    """A cache of B sequences of L random rows and its table; slots past L hold NaN."""
    per = -(-L // page)
    cache = fa.fa_latent_empty(B * per + 2, page, DT[dt]).fill_(math.nan)
    table = table_of(B, per, B * per + 2, seed)
    c, r = normal(seed, B, L, 512).to(DT[dt]), normal(seed + 1, B, L, 64).to(DT[dt])
    fa.fa_latent_write(c, r, cache, table)
    ok()
    return cache, table, c, r


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("B,H,S,page,width", [(1, 1, 1, 16, 64), (2, 5, 17, 16, 192),
                                              (3, 16, 130, 64, 576), (1, 128, 40, 128, 200)])
def test_write_rotates_and_reads_back(B, H, S, page, width, pairs, dt):
    per = -(-(S + 40) // page)
    cache = fa.fa_latent_empty(B * per + 2, page, DT[dt]).fill_(7.0)
    table = table_of(B, per, B * per + 2, 1)
    c, r = normal(1, B, S, 512).to(DT[dt]), normal(2, B, S, 64).to(DT[dt])
    qr, q = normal(3, B, H, S, 64).to(DT[dt]), normal(4, B, H, S, width).to(DT[dt])
    kept = q[..., :width - 64].clone()
    start = ints([(37 * b) % 41 for b in range(B)])
    count = ints([S] + [S - S // 3] * (B - 1))
    last = q[..., width - 64:].clone()
    got = fa.fa_latent_write(c, r, cache, table, start, count, freqs_of(), pairs, q_rope=qr, q=q)
    out = [torch.full_like(x, 5.0) for x in (c, r)]
    fa.fa_latent_read(cache, table, start, count, out=out)
    ok()
    assert got is q and torch.equal(q[..., :width - 64], kept)
    mine = torch.zeros(cache.shape[:2], dtype=torch.bool, device="cuda")
    for b in range(B):
        n = int(count[b])
        at = int(start[b]) + torch.arange(n, device="cuda")
        paged_ref.close(q[b, :, :n, width - 64:], *paged_ref.rotate(qr[b, :, :n], at, freqs_of(), pairs))
        paged_ref.close(out[1][b, :n], *paged_ref.rotate(r[b, :n], at, freqs_of(), pairs))
        assert torch.equal(out[0][b, :n], c[b, :n])
        assert torch.equal(q[b, :, n:, width - 64:], last[b, :, n:])
        assert (out[0][b, n:] == 5.0).all() and (out[1][b, n:] == 5.0).all()
        pg = table[b][at // page].long()
        assert torch.equal(cache[pg, at % page], torch.cat([out[0][b, :n], out[1][b, :n]], -1))
        mine[pg, at % page] = True
    assert (cache[~mine] == 7.0).all()


def test_places_that_do_not_exist_are_skipped_and_reported():
    cache, table, c, r = cache_of(2, 64, 16, "bf16", 3)
    before = cache.clone()
    bad = table.clone()
    bad[0, 1], bad[1, 0] = -1, cache.shape[0]
    fa.fa_latent_write(c[:, :16].contiguous(), r[:, :16].contiguous(), cache, bad, ints([16, 0]))
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    assert torch.equal(cache.view(torch.int16), before.view(torch.int16))
    out = [torch.full_like(x, 7.0) for x in (c, r)]
    fa.fa_latent_read(cache, bad, None, ints([40, 20]), out=out)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    for o, x in zip(out, (c, r)):
        assert torch.equal(o[0, :16], x[0, :16]) and (o[0, 16:32] == 0).all()
        assert torch.equal(o[0, 32:40], x[0, 32:40]) and (o[0, 40:] == 7.0).all()
        assert (o[1, :16] == 0).all() and torch.equal(o[1, 16:20], x[1, 16:20])


# ------------------------------------------------------------ absorbed

@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("B,H,Sq,L,page", [
    (1, 1, 1, 1, 16), (2, 16, 1, 17, 16), (1, 16, 1, 300, 32), (3, 8, 2, 129, 128),
    (2, 5, 3, 1000, 64), (1, 20, 1, 700, 16), (1, 32, 1, 1100, 64), (2, 24, 2, 90, 16),
    (1, 64, 1, 5000, 1024), (2, 128, 1, 2000, 64), (1, 128, 3, 65, 16), (1, 40, 5, 33, 16),
    (1, 3, 40, 8, 16)])
def test_attention(B, H, Sq, L, page, dt):
    cache, table, _, _ = cache_of(B, L, page, dt, 5)
    length = ints([L, max(0, L - 1), L // 2][:B])
    q = normal(6, B, H, Sq, 576).to(DT[dt])
    o, lse = fa.fa_fwd_latent(q, cache, table, length)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, cache, None, table, length, SCALE))


@pytest.mark.parametrize("H", [4, 32, 64])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rise", [1.0, 40.0])
def test_scores_that_rise_and_fall_along_the_keys(rise, dt, H):
    L = 900
    cache, table, c, r = cache_of(1, L, 16, dt, 7)
    at = torch.arange(L, device="cuda")
    c = c.clone()
    c[..., 0] = (at / L * rise).to(DT[dt])
    c[..., 1] = (-at / L * rise).to(DT[dt])
    c[..., 2] = ((at % 97) / 97 * rise).to(DT[dt])
    fa.fa_latent_write(c, r, cache, table)
    q = normal(8, 1, H, 1, 576) * 0.3
    for h in range(H):
        q[:, h, :, h % 3] = 8.0 if h % 2 else -8.0
    q = q.to(DT[dt])
    o, lse = fa.fa_fwd_latent(q, cache, table, ints([L]), scale=0.4)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, cache, None, table, ints([L]), 0.4))


@pytest.mark.parametrize("H", [8, 24, 100])
def test_lengths_of_zero_and_garbage_behind_the_last_token(H):
    """Slots past the length hold NaN and infinities; unused table entries anything."""
    B, L = 6, 90
    cache, table, _, _ = cache_of(B, L, 16, "bf16", 9)
    length = ints([0, 1, 3, 81, 64, 72])
    wide = torch.full((B, 20), -7, dtype=torch.int32, device="cuda")
    wide[:, 15:] = 2 ** 31 - 1
    for b in range(B):
        n = -(-int(length[b]) // 16)
        wide[b, :n] = table[b, :n]
        for pos in range(int(length[b]), 16 * n):
            cache[int(table[b, pos // 16]), pos % 16] = math.inf if pos % 2 else math.nan
    for Sq in (1, 2):
        q = normal(10, B, H, Sq, 576).bfloat16()
        ref = paged_ref.newest(q, cache, None, table, length, SCALE)
        for t in (wide, torch.cat([wide, wide[:, -1:].repeat(1, 100)], 1).contiguous()):
            o, lse = fa.fa_fwd_latent(q, cache, t, length)
            ok()
            ops_ref.check(o, lse, ref)


def test_a_nan_row_reaches_its_sequence_and_bad_pages_are_reported():
    cache, table, c, r = cache_of(2, 1300, 16, "fp16", 11)
    q = normal(12, 2, 6, 1, 576).half()
    bad = table.clone()
    bad[0, 1], bad[0, 7], bad[1, 80] = 10 ** 6, -1, cache.shape[0]
    length = ints([1300, 1300])
    o, lse = fa.fa_fwd_latent(q, cache, bad, length)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    page = torch.arange(1300, device="cuda") // 16
    rows = torch.cat([c, r], -1)[:, None]
    for b, gone in ((0, (page == 1) | (page == 7)), (1, page == 80)):
        ref = paged_ref.attention(q[b:b + 1], rows[b:b + 1], c[b:b + 1, None],
                                  (~gone).view(1, 1, 1, -1), SCALE)
        ops_ref.check(o[b:b + 1], lse[b:b + 1], ref)
    c[0, 5, 3] = math.nan
    fa.fa_latent_write(c, r, cache, table)
    o, lse = fa.fa_fwd_latent(q, cache, table, length)
    ok()
    assert o[0].isnan().all() and lse[0].isnan().all() and o[1].isfinite().all()


@pytest.mark.parametrize("B,L", [(1, 20000), (2, 3000), (7, 900), (300, 70)])
@pytest.mark.parametrize("H", [4, 24, 128])
def test_ragged_batches_and_wide_tables(B, L, H):
    """The keys are dealt by the lengths found, not by the table's room."""
    cache, table, _, _ = cache_of(B, L, 64, "bf16", 13)
    q = normal(14, B, H, 1, 576).bfloat16()
    rng = random.Random(B)
    length = ints([rng.choice([0, 1, 63, 64, 65, L // 2, L]) for _ in range(B - 1)] + [L])
    wide = torch.cat([table, torch.full((B, 4000), -1, dtype=torch.int32, device="cuda")],
                     1).contiguous()
    ref = paged_ref.newest(q, cache, None, table, length, SCALE)
    for t in (table, wide):
        o, lse = fa.fa_fwd_latent(q, cache, t, length)
        ok()
        ops_ref.check(o, lse, ref)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements; the pages in use lie at both ends."""
    page = 1024
    pages = (1 << 32) // (page * 576) + 40
    cache = torch.empty((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    use = [pages - 1, 0, pages - 2]
    table = ints([use])
    c, r = normal(15, 1, 2500, 512).bfloat16(), normal(16, 1, 2500, 64).bfloat16()
    fa.fa_latent_write(c, r, cache, table)
    out = fa.fa_latent_read(cache, table, out=[torch.empty_like(c), torch.empty_like(r)])
    q = normal(17, 1, 128, 1, 576).bfloat16()
    o, lse = fa.fa_fwd_latent(q, cache, table, ints([2500]))
    ok()
    assert torch.equal(out[0], c) and torch.equal(out[1], r)
    ops_ref.check(o, lse, paged_ref.newest(q, cache, None, table, ints([2500]), SCALE))


def test_two_streams_and_a_graph_at_once():
    cache, table, _, _ = cache_of(2, 3000, 64, "bf16", 18)
    q = normal(19, 2, 128, 1, 576).bfloat16()
    length = ints([3000, 1500])
    ref = fa.fa_fwd_latent(q, cache, table, length)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fa.fa_fwd_latent(q, cache, table, length)
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
    got = [held]
    for _ in range(20):
        got.append(fa.fa_fwd_latent(q, cache, table, length, stream=s1))
        got.append(fa.fa_fwd_latent(q, cache, table, length, stream=s2))
        with torch.cuda.stream(s3):
            graph.replay()
    ok()
    for o, lse in got:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("H,L", [(5, 70), (20, 900), (40, 100), (80, 900), (65, 100)])
def test_rows_of_other_sequences_stay_out(H, L, value):
    """The heads are fewer than a tile (or a pair's two) holds, whose other rows are the
    next sequence's: whatever they are, a row has the same bits."""
    B = 3
    cache, table, _, _ = cache_of(B, L, 16, "bf16", 40)
    length = ints([L, L - 7, L // 3])
    q = normal(41, B, H, 1, 576).bfloat16()
    o, lse = fa.fa_fwd_latent(q, cache, table, length)
    for b in range(B):
        other = torch.full_like(q, value)
        other[b] = q[b]
        o2, lse2 = fa.fa_fwd_latent(other, cache, table, length)
        assert torch.equal(o2[b], o[b]) and torch.equal(lse2[b], lse[b])
    ok()
