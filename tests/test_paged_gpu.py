"""The 16-bit paged cache: rotating write, read back, attention over it, and the run
of them as a server makes it, within the bounds of paged_ref.py."""
import math
import random

import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref
import paged_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


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


def freqs_of(rot):
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return (10000.0 ** (-2.0 * j / rot)).float()


def cache_of(B, L, Hkv, page, D, dt, seed=0):
    """A cache of B sequences of L random tokens and its table; slots past L hold NaN."""
    per = -(-L // page)
    cache = fa.fa_paged_empty(B * per + 2, Hkv, page, D, DT[dt])
    for t in cache:
        t.fill_(math.nan)
    table = table_of(B, per, B * per + 2, seed)
    k, v = (normal(seed + i, B, Hkv, L, D).to(DT[dt]) for i in range(2))
    fa.fa_paged_write(k, v, cache, table)
    ok()
    return cache, table, k, v


# ------------------------------------------------------------ write and read

@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("B,H,Hkv,S,page,D,rot", [
    (1, 1, 1, 1, 16, 64, 64), (2, 6, 3, 17, 16, 128, 128), (3, 2, 2, 130, 64, 64, 32),
    (1, 32, 4, 300, 128, 128, 16), (5, 7, 1, 31, 1024, 128, 96), (2, 4, 4, 9, 16, 64, 48)])
def test_write_rotates_and_reads_back(B, H, Hkv, S, page, D, rot, pairs, dt):
    per = -(-(S + 40) // page)
    cache = [t.fill_(7.0) for t in fa.fa_paged_empty(B * per + 2, Hkv, page, D, DT[dt])]
    table = table_of(B, per, B * per + 2, 1)
    q, k, v = (normal(i, B, n, S, D).to(DT[dt]) for i, n in ((1, H), (2, Hkv), (3, Hkv)))
    start = ints([(37 * b) % 41 for b in range(B)])
    freqs = freqs_of(rot)
    turned = fa.fa_paged_write(k, v, cache, table, start, freqs=freqs, interleaved=pairs, q=q)
    out = [torch.full_like(k, 5.0) for _ in range(2)]
    fa.fa_paged_read(cache, table, start, out=out)
    ok()
    mine = torch.zeros(cache[0].shape[:3], dtype=torch.bool, device="cuda")
    for b in range(B):
        at = int(start[b]) + torch.arange(S, device="cuda")
        paged_ref.close(turned[b], *paged_ref.rotate(q[b], at, freqs, pairs))
        paged_ref.close(out[0][b], *paged_ref.rotate(k[b], at, freqs, pairs))
        assert torch.equal(turned[b, ..., rot:], q[b, ..., rot:])
        assert torch.equal(out[0][b, ..., rot:], k[b, ..., rot:])
        pg = table[b][at // page].long()
        for c, o in zip(cache, out):
            assert torch.equal(c[pg, :, at % page].transpose(0, 1), o[b])
        mine[pg, :, at % page] = True
    assert torch.equal(out[1], v)
    for c in cache:
        assert (c[~mine] == 7.0).all()


@pytest.mark.parametrize("pairs", [False, True])
def test_angles_of_far_positions(pairs):
    """To the last position a table can hold; frequencies from far below a radian to
    more than a turn a position."""
    page, per = 1024, 16384
    table = torch.full((1, per), -1, dtype=torch.int32, device="cuda")
    table[0, -1], table[0, per // 3] = 1, 0
    cache = fa.fa_paged_empty(2, 1, page, 64, torch.float16)
    k = normal(4, 1, 1, 16, 64).half()
    freqs = torch.tensor([1.0, 0.7, 0.31, 1e-3, 1e-6, 3.0, 6.5, 0.0] * 2, device="cuda")
    for first in (2 ** 24 - 16, per // 3 * page + 5):
        out = [torch.empty_like(k) for _ in range(2)]
        fa.fa_paged_write(k, k, cache, table, ints([first]), freqs=freqs, interleaved=pairs)
        fa.fa_paged_read(cache, table, ints([first]), out=out)
        ok()
        at = first + torch.arange(16, device="cuda")
        paged_ref.close(out[0][0], *paged_ref.rotate(k[0], at, freqs, pairs))


def test_starts_counts_and_what_stays_untouched():
    B, H, Hkv, S, page, D = 4, 4, 2, 20, 16, 128
    cache, table, k, v = cache_of(B, 100, Hkv, page, D, "bf16", 2)
    before = [t.clone() for t in cache]
    nk, q = normal(5, B, Hkv, S, D).bfloat16(), normal(6, B, H, S, D).bfloat16()
    start, count = ints([0, 15, 80, 3]), ints([20, 0, 17, 50])
    freqs = freqs_of(D)
    kept = torch.full_like(q, 3.0)
    fa.fa_paged_write(nk, nk, cache, table, start, count, freqs=freqs, q=q, q_out=kept)
    fresh = fa.fa_paged_write(nk, nk, cache, table, start, count, freqs=freqs, q=q)
    out = [torch.full_like(nk, 7.0) for _ in range(2)]
    fa.fa_paged_read(cache, table, start, count, out=out)
    ok()
    touched = torch.zeros(cache[0].shape[:3], dtype=torch.bool, device="cuda")
    for b in range(B):
        n = min(int(count[b]), S)
        at = int(start[b]) + torch.arange(n, device="cuda")
        if n:
            paged_ref.close(out[0][b, :, :n], *paged_ref.rotate(nk[b, :, :n], at, freqs, False))
            paged_ref.close(kept[b, :, :n], *paged_ref.rotate(q[b, :, :n], at, freqs, False))
        assert torch.equal(out[1][b, :, :n], nk[b, :, :n])
        assert (kept[b, :, n:] == 3.0).all() and (fresh[b, :, n:] == 0).all()
        assert torch.equal(fresh[b, :, :n], kept[b, :, :n])
        assert (out[0][b, :, n:] == 7.0).all() and (out[1][b, :, n:] == 7.0).all()
        touched[table[b][at // page].long(), :, at % page] = True
    for old, new in zip(before, cache):
        assert torch.equal(old.view(torch.int16)[~touched], new.view(torch.int16)[~touched])


def test_queries_may_be_rotated_in_place_and_nothing_need_be():
    cache, table, k, v = cache_of(2, 50, 2, 16, 64, "fp16", 7)
    assert torch.equal(paged_ref.sequence(cache[0], table[1], 50), k[1])  # no freqs: as they are
    q = normal(8, 2, 6, 50, 64).half()
    freqs = freqs_of(64)
    want = fa.fa_paged_write(k, v, cache, table, freqs=freqs, interleaved=True, q=q)
    same = fa.fa_paged_write(k, v, cache, table, freqs=freqs, interleaved=True, q=q, q_out=q)
    ok()
    assert same is q and torch.equal(q, want)
    plain = fa.fa_paged_write(k, v, cache, table, q=q)
    ok()
    assert torch.equal(plain, q)


def test_places_that_do_not_exist_are_skipped_and_reported():
    B, page, D = 3, 16, 64
    cache, table, k, v = cache_of(B, 64, 1, page, D, "fp16", 9)
    before = [t.clone() for t in cache]
    bad = table.clone()
    bad[0, 1], bad[1, 0] = -1, cache[0].shape[0]
    new = torch.ones((B, 1, 20, D), dtype=torch.float16, device="cuda")
    fa.fa_paged_write(new, new, cache, bad, ints([16, 0, -20]), ints([16, 16, 20]))
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    fa.fa_paged_write(new, new, cache, bad, ints([64, 64, 2 ** 31 - 1]), None, freqs_of(64), q=new)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    for a, b in zip(before, cache):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    out = [torch.full_like(new, 7.0) for _ in range(2)]
    fa.fa_paged_read(cache, bad, ints([10, 0, 0]), ints([10, 5, 20]), out=out)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    for o, x in zip(out, (k, v)):
        assert (o[0, :, 6:10] == 0).all() and (o[1, :, :5] == 0).all()
        assert torch.equal(o[0, :, :6], x[0, :, 10:16]) and torch.equal(o[2], x[2, :, :20])
        assert (o[0, :, 10:] == 7.0).all()


# ------------------------------------------------------------ attention

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("B,H,Hkv,Sq,L,page", [
    (1, 1, 1, 1, 1, 16), (2, 8, 2, 1, 17, 16), (1, 16, 1, 1, 300, 32), (2, 4, 4, 1, 1000, 64),
    (3, 6, 2, 1, 129, 128), (2, 8, 2, 2, 65, 16), (1, 8, 8, 5, 700, 16), (2, 12, 4, 7, 90, 16),
    (1, 32, 1, 3, 513, 64), (1, 4, 2, 20, 33, 16), (1, 8, 2, 1, 5000, 1024), (1, 2, 1, 40, 8, 16),
    (1, 17, 1, 1, 64, 16), (1, 65, 1, 1, 2000, 16), (2, 16, 1, 13, 1100, 32)])
def test_attention(B, H, Hkv, Sq, L, page, dt, D):
    cache, table, _, _ = cache_of(B, L, Hkv, page, D, dt, 10)
    length = ints([L, max(0, L - 1), L // 2][:B])
    q = normal(11, B, H, Sq, D).to(DT[dt])
    o, lse = fa.fa_fwd_paged(q, cache, table, length)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, *cache, table, length, D ** -0.5))


@pytest.mark.parametrize("cap,mult", [(0.0, 1.0), (30.0, 1.0), (5.0, 4.0), (1e6, 1.0), (1e-6, 1.0)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("D,Sq", [(64, 2), (128, 2), (128, 7)])
def test_cap_and_bias(cap, mult, bias, D, Sq):
    B, H, Hkv, L = 2, 12, 2, 1400
    cache, table, _, _ = cache_of(B, L, Hkv, 16, D, "bf16", 12)
    q = (normal(13, B, H, Sq, D) * mult).bfloat16()
    s = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda") if bias else None
    length = ints([1400, 333])
    o, lse = fa.fa_fwd_paged(q, cache, table, length, scale=0.2, softcap=cap, slopes=s)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, *cache, table, length, 0.2, cap, s))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rise", [1.0, 40.0])
def test_scores_that_rise_and_fall_along_the_keys(rise, dt):
    """The reference maximum moves in many tiles, by a little and by more than fp16
    holds, up and down, for each row at other keys."""
    B, H, L, D = 1, 6, 900, 64
    cache, table, k, v = cache_of(B, L, 1, 16, D, dt, 14)
    at = torch.arange(L, device="cuda")
    k = k.clone()
    k[..., 0] = (at / L * rise).to(DT[dt])
    k[..., 1] = (-at / L * rise).to(DT[dt])
    k[..., 2] = ((at % 97) / 97 * rise).to(DT[dt])
    fa.fa_paged_write(k, v, cache, table)
    q = normal(15, B, H, 1, D)
    for h in range(6):
        q[:, h, :, h % 3] = 8.0 if h < 3 else -8.0
    q = q.to(DT[dt])
    o, lse = fa.fa_fwd_paged(q, cache, table, ints([L]), scale=0.4)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, *cache, table, ints([L]), 0.4))


@pytest.mark.parametrize("D", [64, 128])
def test_lengths_of_zero_and_garbage_behind_the_last_token(D):
    """Slots past the length hold NaN and infinities; unused table entries anything."""
    B, H, Hkv, L = 6, 8, 2, 90
    cache, table, _, _ = cache_of(B, L, Hkv, 16, D, "bf16", 16)
    length = ints([0, 1, 3, 81, 64, 72])
    wide = torch.full((B, 20), -7, dtype=torch.int32, device="cuda")
    wide[:, 15:] = 2 ** 31 - 1
    for b in range(B):
        n = -(-int(length[b]) // 16)
        wide[b, :n] = table[b, :n]
        for pos in range(int(length[b]), 16 * n):
            for i, t in enumerate(cache):
                t[int(table[b, pos // 16]), :, pos % 16] = math.inf if (pos + i) % 2 else math.nan
    for Sq in (1, 3):
        q = normal(17, B, H, Sq, D).bfloat16()
        ref = paged_ref.newest(q, *cache, table, length, D ** -0.5)
        for t in (wide, torch.cat([wide, wide[:, -1:].repeat(1, 100)], 1).contiguous()):
            o, lse = fa.fa_fwd_paged(q, cache, t, length)
            ok()
            ops_ref.check(o, lse, ref)


@pytest.mark.parametrize("value", [1e30, 1e-30, 0.0])
def test_queries_far_from_one(value):
    cache, table, _, _ = cache_of(1, 70, 1, 16, 64, "bf16", 18)
    q = (normal(19, 1, 4, 1, 64) * value).bfloat16()
    sc = min(max(0.125 / value if value else 1.0, 1e-37), 1e37)
    o, lse = fa.fa_fwd_paged(q, cache, table, ints([70]), scale=sc)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, *cache, table, ints([70]), sc))


def test_a_nan_token_reaches_the_rows_that_see_it():
    cache, table, k, v = cache_of(2, 40, 2, 16, 64, "fp16", 20)
    k[0, 1, 5, 3] = math.nan
    fa.fa_paged_write(k, v, cache, table)
    q = normal(21, 2, 4, 1, 64).half()
    o, lse = fa.fa_fwd_paged(q, cache, table, ints([40, 40]))
    ok()
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert o[0, :2].isfinite().all() and o[1].isfinite().all()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_bad_pages_are_not_seen_and_reported(dt):
    cache, table, k, v = cache_of(1, 2000, 1, 16, 128, dt, 22)
    q = normal(23, 1, 2, 1, 128).to(DT[dt])
    for L in (64, 2000):
        bad = table[:, :-(-L // 16)].contiguous()
        bad[0, 1], bad[0, 3], bad[0, -1] = 10 ** 6, -1, cache[0].shape[0]
        o, lse = fa.fa_fwd_paged(q, cache, bad, ints([L]))
        assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
        j = torch.arange(L, device="cuda") // 16
        seen = ((j != 1) & (j != 3) & (j != bad.shape[1] - 1)).view(1, 1, 1, L)
        ops_ref.check(o, lse, paged_ref.attention(q, k[:, :, :L], v[:, :, :L], seen, 128 ** -0.5))
    short = table[:, :4].contiguous()
    fa.fa_fwd_paged(q, cache, short, ints([65]))  # longer than the table
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    fa.fa_fwd_paged(q, cache, table, ints([-1]))
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    ok()


@pytest.mark.parametrize("B,L", [(1, 20000), (2, 3000), (7, 900), (300, 70)])
@pytest.mark.parametrize("rows", [4, 24, 100])
def test_ragged_batches_and_wide_tables(B, L, rows):
    """The keys are dealt by the lengths found, not by the table's room."""
    Hkv, Sq = 2, rows // 4
    cache, table, _, _ = cache_of(B, L, Hkv, 64, 128, "bf16", 24)
    q = normal(25, B, 4 * Hkv, Sq, 128).bfloat16()
    rng = random.Random(B)
    length = ints([rng.choice([0, 1, 63, 64, 65, L // 2, L]) for _ in range(B - 1)] + [L])
    wide = torch.cat([table, torch.full((B, 4000), -1, dtype=torch.int32, device="cuda")],
                     1).contiguous()
    ref = paged_ref.newest(q, *cache, table, length, 128 ** -0.5)
    for t in (table, wide):
        o, lse = fa.fa_fwd_paged(q, cache, t, length)
        ok()
        ops_ref.check(o, lse, ref)


def test_sequences_may_share_pages_for_reading():
    cache, table, _, _ = cache_of(1, 160, 2, 16, 64, "bf16", 26)
    q = normal(27, 3, 4, 1, 64).bfloat16()
    shared = table.repeat(3, 1).contiguous()
    length = ints([160, 100, 160])
    o, lse = fa.fa_fwd_paged(q, cache, shared, length)
    ok()
    ops_ref.check(o, lse, paged_ref.newest(q, *cache, shared, length, 0.125))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes; the pages in use lie at both ends."""
    Hkv, page, D = 8, 1024, 128
    pages = (1 << 32) // (Hkv * page * D * 2) + 40
    cache = [torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    use = [pages - 1, 0, pages - 2]
    table = ints([use])
    q, k, v = (normal(28 + i, 1, n, 2500, D).bfloat16() for i, n in enumerate((16, Hkv, Hkv)))
    freqs = freqs_of(D)
    turned = fa.fa_paged_write(k, v, cache, table, freqs=freqs, q=q)
    out = fa.fa_paged_read(cache, table, out=[torch.empty_like(k), torch.empty_like(v)])
    q1 = turned[:, :, -1:].contiguous()
    o, lse = fa.fa_fwd_paged(q1, cache, table, ints([2500]))
    ok()
    at = torch.arange(2500, device="cuda")
    paged_ref.close(out[0][0], *paged_ref.rotate(k[0], at, freqs, False))
    assert torch.equal(out[1], v)
    small = [t[use].contiguous() for t in cache]
    o2, lse2 = fa.fa_fwd_paged(q1, small, ints([[0, 1, 2]]), ints([2500]))
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ops_ref.check(o, lse, paged_ref.newest(q1, *cache, table, ints([2500]), D ** -0.5))


def test_two_streams_at_once():
    cache, table, _, _ = cache_of(2, 2000, 4, 64, 128, "bf16", 31)
    q = normal(32, 2, 16, 1, 128).bfloat16()
    length = ints([2000, 1500])
    ref = fa.fa_fwd_paged(q, cache, table, length)
    ok()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(30):
        got.append(fa.fa_fwd_paged(q, cache, table, length, stream=s1))
        got.append(fa.fa_fwd_paged(q, cache, table, length, stream=s2))
    ok()
    for o, lse in got:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_captured_attention_without_a_workspace():
    """The graph's own memory holds its parts; the library's is for direct calls."""
    cache, table, _, _ = cache_of(2, 3000, 2, 64, 128, "bf16", 33)
    q = normal(34, 2, 8, 1, 128).bfloat16()
    length = ints([3000, 1111])
    ref = fa.fa_fwd_paged(q, cache, table, length)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fa_fwd_paged(q, cache, table, length)
    fa.fa_release_workspaces()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        direct = fa.fa_fwd_paged(q, cache, table, length)
    ok()
    for o, lse in (got, direct):
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


# ------------------------------------------------------------ together

@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "fp16")])
def test_prompt_decode_and_a_further_chunk(D, dt):
    """A prompt rotated into the cache and through fa_fwd_score; decode steps, captured
    once and replayed as lengths grow; then a chunk over the cache read back."""
    B, H, Hkv, S, page, cap = 2, 8, 2, 150, 16, 30.0
    seeds = iter(range(100, 400))
    n = lambda *s: normal(next(seeds), *s).to(DT[dt])  # noqa: E731
    per = 16
    cache = fa.fa_paged_empty(B * per, Hkv, page, D, DT[dt])
    table = table_of(B, per, B * per, 35)
    freqs = freqs_of(D)
    q, k, v = n(B, H, S, D), n(B, Hkv, S, D), n(B, Hkv, S, D)
    length = ints([S, 101])  # a padded batch: sequence 1 has 101 tokens
    doc = torch.where(torch.arange(S, device="cuda")[None] < length[:, None], 0, -1)
    doc = doc.to(torch.int32).contiguous()
    qr = fa.fa_paged_write(k, v, cache, table, None, length, freqs, q=q)
    kr, vr = (torch.zeros_like(k) for _ in range(2))
    fa.fa_paged_read(cache, table, None, length, out=[kr, vr])
    o, lse = fa.fa_fwd_score(qr, kr, vr, causal=True, softcap=cap, doc_q=doc, doc_k=doc)
    ok()
    seen, dist = ops_ref.score_seen(S, S, True, None, doc, doc)
    u = torch.finfo(DT[dt]).eps / 2
    ops_ref.check(o, lse, ops_ref.attention(qr, kr, vr, seen, D ** -0.5, cap, None, dist, p_step=u))
    # the newest tokens of the prompt by either path
    new = torch.stack([qr[0, :, S - 1:S], qr[1, :, 100:101]])
    o1, l1 = fa.fa_fwd_paged(new.contiguous(), cache, table, length, softcap=cap)
    ok()
    ops_ref.check(o1, l1, paged_ref.newest(new, *cache, table, length, D ** -0.5, cap))

    q1, k1, v1 = n(B, H, 1, D), n(B, Hkv, 1, D), n(B, Hkv, 1, D)
    q1r, o1 = torch.empty_like(q1), torch.empty_like(q1)
    l1 = torch.empty((B, H, 1), device="cuda")

    def step():
        fa.fa_paged_write(k1, v1, cache, table, length, freqs=freqs, q=q1, q_out=q1r)
        length.add_(1)
        fa.fa_fwd_paged(q1r, cache, table, length, softcap=cap, out=o1, lse=l1)

    step()
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for t, heads in ((q1, H), (k1, Hkv), (v1, Hkv)):
            t.copy_(n(B, heads, 1, D))
        was = length.tolist()
        graph.replay()
        ok()
        for b in range(B):
            at = torch.tensor([was[b]], device="cuda")
            paged_ref.close(q1r[b], *paged_ref.rotate(q1[b], at, freqs, False))
            pg, slot = int(table[b, was[b] // page]), was[b] % page
            paged_ref.close(cache[0][pg, :, slot:slot + 1], *paged_ref.rotate(k1[b], at, freqs, False))
        ops_ref.check(o1, l1, paged_ref.newest(q1r, *cache, table, length, D ** -0.5, cap))
    assert length.tolist() == [S + 21, 122]


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("H,Hkv,Sq,L", [(5, 1, 1, 70), (6, 2, 1, 1500), (10, 2, 3, 1500), (20, 1, 1, 900)])
def test_rows_of_other_heads_stay_out(H, Hkv, Sq, L, value):
    """The rows of a head group are fewer than a tile holds, whose others are the next
    group's or sequence's: whatever they are, a row has the same bits."""
    B = 3
    cache, table, _, _ = cache_of(B, L, Hkv, 16, 64, "bf16", 40)
    length = ints([L, L - 7, L // 3])
    q = normal(41, B, H, Sq, 64).bfloat16()
    o, lse = fa.fa_fwd_paged(q, cache, table, length)
    for b in range(B):
        for g in range(Hkv):
            heads = slice(g * H // Hkv, (g + 1) * H // Hkv)
            other = torch.full_like(q, value)
            other[b, heads] = q[b, heads]
            o2, lse2 = fa.fa_fwd_paged(other, cache, table, length)
            assert torch.equal(o2[b, heads], o[b, heads]) and torch.equal(lse2[b, heads], lse[b, heads])
    ok()


def test_copies_that_follow_each_other():
    """A write, a read into a buffer, a write of the buffer and its read, over and over on
    one stream with other values: each sees what the one before it wrote."""
    B, Hkv, S, n = 2, 2, 200, 30
    a, b = (fa.fa_paged_empty(32, Hkv, 16, 64, torch.float16) for _ in range(2))
    table = table_of(B, 13, 32)
    rows = [[normal(50 + 2 * i + j, B, Hkv, S, 64).half() for j in range(2)] for i in range(n)]
    got = [[torch.empty_like(x) for x in r] for r in rows]
    buf = [torch.empty_like(x) for x in rows[0]]
    torch.cuda.synchronize()
    for i in range(n):
        fa.fa_paged_write(*rows[i], a, table)
        fa.fa_paged_read(a, table, out=buf)
        fa.fa_paged_write(*buf, b, table)
        fa.fa_paged_read(b, table, out=got[i])
    ok()
    for r, g in zip(rows, got):
        assert torch.equal(r[0], g[0]) and torch.equal(r[1], g[1])
