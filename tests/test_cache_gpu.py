"""The 4-bit cache: what is written, what it reads back as, attention over it,
and the run of them as a server makes it.  Codes are compared exactly, values
and attention within the bounds of ops_ref.py."""
import math
import random

import pytest
import torch

from attention_forward_gb300 import fa
import ops_ref

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


def cache_of(B, L, Hkv, page, D, dt, seed=0):
    """A cache of B sequences of L random tokens, written by the library, and
    its table; slots past L hold garbage (NaN parameters among it)."""
    per = -(-L // page)
    cache = fa.fa_cache_empty(B * per + 2, Hkv, page, D)
    for t in cache:
        t.view(torch.uint8).fill_(255)  # codes 15, parameters NaN
    table = table_of(B, per, B * per + 2, seed)
    g = torch.Generator("cuda").manual_seed(seed)
    k = torch.randn((B, Hkv, L, D), generator=g, device="cuda").to(DT[dt])
    v = torch.randn((B, Hkv, L, D), generator=g, device="cuda").to(DT[dt])
    fa.fa_cache_write(k, v, cache, table)
    ok()
    return cache, table, k, v


def expect(q, cache, table, length, scale=None, cap=0.0, slopes=None):
    B, H, Sq, D = q.shape
    u = torch.finfo(q.dtype).eps / 2
    outs = []
    for b in range(B):
        n = max(0, int(length[b]))
        if n == 0:
            z = torch.zeros((1, H, Sq, D), dtype=torch.float64, device="cuda")
            outs.append((z, torch.full((1, H, Sq), -math.inf, dtype=torch.float64, device="cuda"),
                         z, z[..., 0]))
            continue
        k = ops_ref.sequence(cache[0], cache[1], table[b], n)[None]
        v = ops_ref.sequence(cache[2], cache[3], table[b], n)[None]
        i = torch.arange(Sq, device="cuda")[:, None] + (n - Sq)
        j = torch.arange(n, device="cuda")[None]
        big = cache[1].float().nan_to_num().abs().amax(tuple(range(cache[1].dim() - 1)))
        sc = scale or D ** -0.5
        x = (q[b].double().abs().sum(-1).amax() * (15 * big[0] + big[1]) * sc).item()
        outs.append(ops_ref.attention(q[b:b + 1], k, v, (j <= i)[None, None], sc, cap, slopes,
                                      (i - j).abs(), p_step=2.0 ** -11, v_step=2.0 ** -11,
                                      x_bound=x))
    return [torch.cat(x) for x in zip(*outs)]


# ------------------------------------------------------------ write and read

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("B,Hkv,S,page", [(1, 1, 1, 16), (2, 3, 17, 16), (3, 2, 130, 64),
                                          (1, 4, 1000, 128), (5, 1, 31, 1024)])
def test_written_codes_are_the_definition_and_read_back(B, Hkv, S, page, dt, D):
    cache, table, k, v = cache_of(B, S, Hkv, page, D, dt, 1)
    at = torch.arange(S, device="cuda")
    out = [torch.full_like(k, 7.0) for _ in range(2)]
    fa.fa_cache_read(cache, table, out=out)
    ok()
    for n, x in enumerate((k, v)):
        codes, params = ops_ref.quantise(x)
        want = ops_ref.pack(codes)
        for b in range(B):
            pg = table[b][at // page].long()
            assert torch.equal(cache[2 * n][pg, :, at % page].transpose(0, 1), want[b])
            assert torch.equal(cache[2 * n + 1][pg, :, at % page].transpose(0, 1), params[b])
        p = params.double()
        val = (codes.double().unflatten(-1, (-1, 32)) * p[..., :1] + p[..., 1:]).flatten(-2)
        u = torch.finfo(x.dtype).eps / 2
        room = (p[..., :1] * 15 + p[..., 1:].abs()).expand(p.shape[:-1] + (32,)).flatten(-2)
        # one rounding to the type, behind one of fp32
        assert ((out[n].double() - val).abs() <= u * val.abs() + 2.0 ** -23 * room).all()
        # half a scale, the parameters' own rounding, and the type's
        far = 0.5 * p[..., :1] + 2.0 ** -10 * (15 * p[..., :1] + p[..., 1:].abs())
        far = far.expand(p.shape[:-1] + (32,)).flatten(-2)
        assert ((out[n].double() - x.double()).abs() <= far + u * val.abs() + 2.0 ** -23 * room).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_ties_constants_extremes_and_nan(dt):
    D, rows = 64, []
    step = torch.arange(64) % 32
    rows.append(step.float() / 2)                     # halves of a scale: exact ties
    rows.append((step.float() - 10) / 2 * 0.25)
    rows.append(torch.full((64,), 3.25))              # one value: scale 0
    rows.append(torch.zeros(64))
    rows.append(torch.linspace(-6e4, 6e4, 64))
    rows.append(torch.linspace(-3e-6, 3e-6, 64))      # scales in fp16's subnormals
    rows.append(torch.where(step == 3, 1e-7, step * 0.1 - 1.5))
    rows.append(torch.linspace(1000, 1001, 64))
    x = torch.stack(rows)[None, None].to(DT[dt]).cuda()
    big = x.clone()
    big[..., 0, 1], big[..., 1, 2], big[..., 2, 40] = math.inf, -math.inf, math.nan
    for y in (x, big):
        cache = fa.fa_cache_empty(1, 1, 16, D)
        table = ints([[0]])
        fa.fa_cache_write(y.contiguous(), x, cache, table)
        ok()
        codes, params = ops_ref.quantise(y[0, 0].nan_to_num(nan=math.nan, posinf=61440.0,
                                                            neginf=-61440.0))
        n = x.shape[2]
        assert torch.equal(cache[0][0, 0, :n], ops_ref.pack(codes))
        assert torch.equal(cache[1][0, 0, :n].nan_to_num(nan=9.0), params.nan_to_num(nan=9.0))
        out = [torch.empty_like(x), torch.empty_like(x)]
        fa.fa_cache_read(cache, table, out=out)
        ok()
        assert torch.equal(out[0].isnan(), torch.isnan(ops_ref.unpack(
            cache[0][0, 0, :n], cache[1][0, 0, :n]))[None, None])
        assert not out[1].isnan().any()


@pytest.mark.parametrize("lo,hi,scale", [
    (-1940.0, -55.15625, 125.625),       # range / 15 = 125.65625, a tie: to even
    (-86.5, 0.365234375, 5.7890625),     # 5.791015625, a tie
    (-34784.0, 1711.0, 2432.0),          # 2433, a tie
    (-61440.0, 61440.0, 8192.0), (-7.5, 7.5, 1.0), (0.0, 2.0 ** -20, 2.0 ** -24)])
def test_scales_are_rounded_to_nearest_even(lo, hi, scale):
    x = torch.full((1, 1, 1, 64), lo, device="cuda")
    x[..., 5] = x[..., 60] = hi
    x = x.half()
    cache = fa.fa_cache_empty(1, 1, 16, 64)
    fa.fa_cache_write(x, x, cache, ints([[0]]))
    ok()
    for params in (cache[1], cache[3]):
        assert params[0, 0, 0].tolist() == [[scale, lo], [scale, lo]]


def test_starts_counts_and_what_stays_untouched():
    B, Hkv, S, page, D = 4, 2, 20, 16, 128
    cache, table, k, v = cache_of(B, 100, Hkv, page, D, "bf16", 2)
    before = [t.clone() for t in cache]
    g = torch.Generator("cuda").manual_seed(3)
    nk = torch.randn((B, Hkv, S, D), generator=g, device="cuda").bfloat16()
    start, count = ints([0, 15, 80, 3]), ints([20, 0, 17, 50])
    fa.fa_cache_write(nk, nk, cache, table, start, count)
    out = [torch.full_like(nk, 7.0) for _ in range(2)]
    fa.fa_cache_read(cache, table, start, count, out=out)
    ok()
    codes, params = ops_ref.quantise(nk)
    val = ops_ref.unpack(ops_ref.pack(codes), params)
    touched = torch.zeros(cache[0].shape[:3], dtype=torch.bool, device="cuda")
    for b in range(B):
        n = min(int(count[b]), S)
        for x in out:
            assert ((x[b, :, :n].double() - val[b, :, :n]).abs() <= 2.0 ** -8 * val[b, :, :n].abs() + 1e-6).all()
            assert (x[b, :, n:] == 7.0).all()
        for i in range(n):
            pos = int(start[b]) + i
            touched[int(table[b, pos // page]), :, pos % page] = True
    for old, new in zip(before, cache):
        assert torch.equal(old.view(torch.uint8)[~touched], new.view(torch.uint8)[~touched])


def test_places_that_do_not_exist_are_skipped_and_reported():
    B, Hkv, page, D = 3, 1, 16, 64
    cache, table, k, v = cache_of(B, 64, Hkv, page, D, "fp16", 4)
    before = [t.clone() for t in cache]
    bad = table.clone()
    bad[0, 1], bad[1, 0] = -1, cache[0].shape[0]
    new = torch.ones((B, Hkv, 20, D), dtype=torch.float16, device="cuda")
    # page -1 and a page past the pool; a position below 0; positions past the table
    fa.fa_cache_write(new, new, cache, bad, ints([16, 0, -20]), ints([16, 16, 20]))
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    fa.fa_cache_write(new, new, cache, bad, ints([64, 64, 2 ** 31 - 1]), None)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    for a, b in zip(before, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = [torch.full_like(new, 7.0) for _ in range(2)]
    fa.fa_cache_read(cache, bad, ints([10, 0, 0]), ints([10, 5, 20]), out=out)
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    assert (out[0][0, :, 6:10] == 0).all() and (out[0][1, :, :5] == 0).all()
    good = [torch.full_like(new, 7.0) for _ in range(2)]
    fa.fa_cache_read(cache, table, ints([10, 0, 0]), ints([6, 0, 20]), out=good)
    ok()
    assert torch.equal(out[0][0, :, :6], good[0][0, :, :6])
    assert torch.equal(out[0][2], good[0][2])
    assert (out[0][0, :, 10:] == 7.0).all()


# ------------------------------------------------------------ attention

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("B,H,Hkv,Sq,L,page", [
    (1, 1, 1, 1, 1, 16), (2, 8, 2, 1, 17, 16), (1, 16, 1, 1, 300, 32), (2, 4, 4, 1, 1000, 64),
    (3, 6, 2, 1, 129, 128), (2, 8, 2, 2, 65, 16), (1, 8, 8, 5, 700, 16), (2, 12, 4, 7, 90, 16),
    (1, 32, 1, 3, 513, 64), (1, 4, 2, 20, 33, 16), (1, 8, 2, 1, 5000, 1024), (1, 2, 1, 40, 8, 16)])
def test_attention(B, H, Hkv, Sq, L, page, dt, D):
    cache, table, _, _ = cache_of(B, L, Hkv, page, D, dt, 5)
    length = ints([L, max(0, L - 1), L // 2][:B])
    q = torch.randn((B, H, Sq, D), generator=torch.Generator("cuda").manual_seed(6),
                    device="cuda").to(DT[dt])
    o, lse = fa.fa_fwd_cache(q, cache, table, length)
    ok()
    ops_ref.check(o, lse, expect(q, cache, table, length))


@pytest.mark.parametrize("cap,mult", [(0.0, 1.0), (30.0, 1.0), (5.0, 4.0), (1e6, 1.0), (1e-6, 1.0)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_cap_and_bias(cap, mult, bias, D):
    B, H, Hkv, Sq, L = 2, 12, 2, 2, 400
    cache, table, _, _ = cache_of(B, L, Hkv, 16, D, "bf16", 7)
    q = (torch.randn((B, H, Sq, D), generator=torch.Generator("cuda").manual_seed(8),
                     device="cuda") * mult).bfloat16()
    s = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda") if bias else None
    length = ints([400, 333])
    o, lse = fa.fa_fwd_cache(q, cache, table, length, scale=0.2, softcap=cap, slopes=s)
    ok()
    ops_ref.check(o, lse, expect(q, cache, table, length, 0.2, cap, s))


def test_lengths_of_zero_and_garbage_behind_the_last_token():
    """Slots past the length hold NaN parameters; unused table entries hold
    anything."""
    B, H, Hkv, L = 4, 8, 2, 90
    cache, table, _, _ = cache_of(B, L, Hkv, 16, 128, "bf16", 9)
    length = ints([0, 1, 3, 81])
    wide = torch.full((B, 20), -7, dtype=torch.int32, device="cuda")
    wide[:, 15:] = 2 ** 31 - 1
    for b in range(B):
        n = -(-int(length[b]) // 16)
        wide[b, :n] = table[b, :n]
        # tokens past the length in the last page become garbage too
        for pos in range(int(length[b]), 16 * n):
            pg = int(table[b, pos // 16])
            for t in cache:
                t[pg, :, pos % 16].view(torch.uint8).fill_(255)
    q = torch.randn((B, H, 3, 128), generator=torch.Generator("cuda").manual_seed(10),
                    device="cuda").bfloat16()
    o, lse = fa.fa_fwd_cache(q, cache, wide, length)
    ok()
    ops_ref.check(o, lse, expect(q, cache, table, length))


@pytest.mark.parametrize("value", [1e30, 1e-30, 0.0])
def test_queries_far_from_one(value):
    cache, table, _, _ = cache_of(1, 70, 1, 16, 64, "bf16", 11)
    q = torch.randn((1, 4, 1, 64), generator=torch.Generator("cuda").manual_seed(12), device="cuda")
    q = (q * value).bfloat16()
    sc = 0.125 / value if value else 1.0
    sc = min(max(sc, 1e-37), 1e37)
    o, lse = fa.fa_fwd_cache(q, cache, table, ints([70]), scale=sc)
    ok()
    ops_ref.check(o, lse, expect(q, cache, table, ints([70]), sc))


def test_a_nan_token_reaches_the_rows_that_see_it():
    cache, table, k, v = cache_of(2, 40, 2, 16, 64, "fp16", 13)
    k[0, 1, 5, 3] = math.nan
    fa.fa_cache_write(k, v, cache, table)
    q = torch.randn((2, 4, 1, 64), generator=torch.Generator("cuda").manual_seed(14),
                    device="cuda").half()
    o, lse = fa.fa_fwd_cache(q, cache, table, ints([40, 40]))
    ok()
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert o[0, :2].isfinite().all() and o[1].isfinite().all()


def test_bad_pages_are_not_seen_and_reported():
    cache, table, _, _ = cache_of(1, 64, 1, 16, 128, "bf16", 15)
    q = torch.randn((1, 2, 1, 128), generator=torch.Generator("cuda").manual_seed(16),
                    device="cuda").bfloat16()
    bad = table.clone()
    bad[0, 1] = 10 ** 6
    o, lse = fa.fa_fwd_cache(q, cache, bad, ints([64]))
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    k = ops_ref.sequence(cache[0], cache[1], table[0], 64)[None]
    v = ops_ref.sequence(cache[2], cache[3], table[0], 64)[None]
    j = torch.arange(64, device="cuda")
    seen = ((j < 16) | (j >= 32)).view(1, 1, 1, 64)
    ops_ref.check(o, lse, ops_ref.attention(q, k, v, seen, 128 ** -0.5, p_step=2.0 ** -11,
                                            v_step=2.0 ** -11, x_bound=60.0))
    fa.fa_fwd_cache(q, cache, table, ints([65]))  # longer than the table
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    fa.fa_fwd_cache(q, cache, table, ints([-1]))
    assert fa.fa_get_device_status() == fa.FA_ERR_INVALID_ARG
    ok()


@pytest.mark.parametrize("B,L", [(1, 20000), (2, 3000), (7, 900), (300, 70)])
@pytest.mark.parametrize("rows", [4, 24])
def test_ragged_batches_and_wide_tables(B, L, rows):
    """The keys are dealt by the lengths found, not by the table's room."""
    Hkv, Sq = 2, rows // 4
    cache, table, _, _ = cache_of(B, L, Hkv, 64, 128, "bf16", 17)
    q = torch.randn((B, 4 * Hkv, Sq, 128), generator=torch.Generator("cuda").manual_seed(18),
                    device="cuda").bfloat16()
    rng = random.Random(B)
    length = ints([rng.choice([0, 1, 63, 64, 65, L // 2, L]) for _ in range(B - 1)] + [L])
    wide = torch.cat([table, torch.full((B, 4000), -1, dtype=torch.int32, device="cuda")],
                     1).contiguous()
    ref = expect(q, cache, table, length)
    for t in (table, wide):
        o, lse = fa.fa_fwd_cache(q, cache, t, length)
        ok()
        ops_ref.check(o, lse, ref)


def test_sequences_may_share_pages_for_reading():
    cache, table, _, _ = cache_of(1, 160, 2, 16, 64, "bf16", 19)
    q = torch.randn((3, 4, 1, 64), generator=torch.Generator("cuda").manual_seed(20),
                    device="cuda").bfloat16()
    shared = table.repeat(3, 1).contiguous()
    length = ints([160, 100, 160])
    o, lse = fa.fa_fwd_cache(q, cache, shared, length)
    ok()
    ops_ref.check(o, lse, expect(q, cache, shared, length))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes; the pages in use lie at both
    ends."""
    Hkv, page, D = 8, 1024, 128
    pages = (1 << 32) // (Hkv * page * D // 2) + 40
    cache = [torch.empty((pages, Hkv, page, D // 2), dtype=torch.uint8, device="cuda"),
             torch.empty((pages, Hkv, page, D // 32, 2), dtype=torch.float16, device="cuda")]
    cache = cache + [torch.empty_like(t) for t in cache]
    table = ints([[pages - 1, 0, pages - 2]])
    g = torch.Generator("cuda").manual_seed(21)
    k = torch.randn((1, Hkv, 2500, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((1, Hkv, 2500, D), generator=g, device="cuda").bfloat16()
    fa.fa_cache_write(k, v, cache, table)
    q = torch.randn((1, 16, 1, D), generator=g, device="cuda").bfloat16()
    o, lse = fa.fa_fwd_cache(q, cache, table, ints([2500]))
    out = fa.fa_cache_read(cache, table, out=[torch.empty_like(k), torch.empty_like(v)])
    ok()
    small = [t[[pages - 1, 0, pages - 2]].contiguous() for t in cache]
    near = ints([[0, 1, 2]])
    o2, lse2 = fa.fa_fwd_cache(q, small, near, ints([2500]))
    out2 = fa.fa_cache_read(small, near, out=[torch.empty_like(k), torch.empty_like(v)])
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(out[0], out2[0]) and torch.equal(out[1], out2[1])
    codes, params = ops_ref.quantise(k)
    val = ops_ref.unpack(ops_ref.pack(codes), params)
    assert ((out[0].double() - val).abs() <= 2.0 ** -8 * val.abs() + 1e-6).all()


def test_two_streams_at_once():
    cache, table, _, _ = cache_of(2, 2000, 4, 64, 128, "bf16", 22)
    q = torch.randn((2, 16, 1, 128), generator=torch.Generator("cuda").manual_seed(23),
                    device="cuda").bfloat16()
    length = ints([2000, 1500])
    ref = fa.fa_fwd_cache(q, cache, table, length)
    ok()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(30):
        got.append(fa.fa_fwd_cache(q, cache, table, length, stream=s1))
        got.append(fa.fa_fwd_cache(q, cache, table, length, stream=s2))
    ok()
    for o, lse in got:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


# ------------------------------------------------------------ together

@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "fp16")])
def test_prompt_decode_and_a_further_chunk(D, dt):
    """A prompt through fa_fwd_score into the cache; decode steps, captured
    once and replayed as lengths grow; then a chunk at full precision over the
    cache read back."""
    B, H, Hkv, S, page, cap = 2, 8, 2, 150, 16, 30.0
    g = torch.Generator("cuda").manual_seed(24)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[dt])  # noqa: E731
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device="cuda")
    per = 16
    cache = fa.fa_cache_empty(B * per, Hkv, page, D)
    table = table_of(B, per, B * per, 25)
    q, k, v = n(B, H, S, D), n(B, Hkv, S, D), n(B, Hkv, S, D)
    length = ints([S, 101])  # a padded batch: sequence 1 has 101 tokens
    pad = torch.arange(S, device="cuda")[None] < length[:, None]
    doc = torch.where(pad, 0, -1).to(torch.int32).contiguous()
    o, lse = fa.fa_fwd_score(q, k, v, causal=True, softcap=cap, slopes=slopes, doc_q=doc, doc_k=doc)
    fa.fa_cache_write(k, v, cache, table, None, length)
    ok()
    seen, dist = ops_ref.score_seen(S, S, True, None, doc, doc)
    u = torch.finfo(DT[dt]).eps / 2
    ops_ref.check(o, lse, ops_ref.attention(q, k, v, seen, D ** -0.5, cap, slopes, dist, p_step=u))

    q1, k1, v1 = n(B, H, 1, D), n(B, Hkv, 1, D), n(B, Hkv, 1, D)
    o1 = torch.empty_like(q1)
    l1 = torch.empty((B, H, 1), device="cuda")
    ws = torch.empty(fa.fa_cache_workspace_bytes(B, H, Hkv, 1, D, page, per) + 256,
                     dtype=torch.uint8, device="cuda")

    def step():
        fa.fa_cache_write(k1, v1, cache, table, length)
        length.add_(1)
        fa.fa_fwd_cache(q1, cache, table, length, softcap=cap, slopes=slopes, workspace=ws,
                        out=o1, lse=l1)

    step()
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        q1.copy_(n(B, H, 1, D))
        k1.copy_(n(B, Hkv, 1, D))
        v1.copy_(n(B, Hkv, 1, D))
        graph.replay()
        ok()
        ops_ref.check(o1, l1, expect(q1, cache, table, length, None, cap, slopes))
    assert length.tolist() == [S + 21, 122]

    C = 40  # the next chunk of sequence 0, over its cache at full precision
    L0 = S + 21
    kf, vf = (torch.zeros((1, Hkv, L0 + C, D), dtype=DT[dt], device="cuda") for _ in range(2))
    part = [torch.empty((1, Hkv, L0, D), dtype=DT[dt], device="cuda") for _ in range(2)]
    fa.fa_cache_read(cache, table[:1].contiguous(), out=part)
    kf[:, :, :L0], vf[:, :, :L0] = part[0], part[1]
    kf[:, :, L0:], vf[:, :, L0:] = n(1, Hkv, C, D), n(1, Hkv, C, D)
    qc = n(1, H, C, D)
    o, lse = fa.fa_fwd_score(qc, kf, vf, causal=True, softcap=cap, slopes=slopes)
    ok()
    seen, dist = ops_ref.score_seen(C, L0 + C, True)
    ops_ref.check(o, lse, ops_ref.attention(qc, kf, vf, seen, D ** -0.5, cap, slopes, dist, p_step=u))


def test_captured_attention_without_a_workspace():
    """The graph's own memory holds its parts; the library's is for direct calls."""
    cache, table, _, _ = cache_of(2, 3000, 2, 64, 128, "bf16", 28)
    q = torch.randn((2, 8, 1, 128), generator=torch.Generator("cuda").manual_seed(29),
                    device="cuda").bfloat16()
    length = ints([3000, 1111])
    ref = fa.fa_fwd_cache(q, cache, table, length)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fa_fwd_cache(q, cache, table, length)
    fa.fa_release_workspaces()
    side = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        direct = fa.fa_fwd_cache(q, cache, table, length)
    ok()
    for o, lse in (got, direct):
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_captured_write_and_read_follow_their_arrays():
    cache, table, k, v = cache_of(2, 40, 2, 16, 64, "bf16", 26)
    start, count = ints([0, 0]), ints([4, 4])
    new = torch.randn((2, 2, 8, 64), generator=torch.Generator("cuda").manual_seed(27),
                      device="cuda").bfloat16()
    out = [torch.zeros_like(new) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_cache_write(new, new, cache, table, start, count)
        fa.fa_cache_read(cache, table, start, count, out=out)
    start.copy_(ints([10, 30]))
    count.copy_(ints([8, 1]))
    graph.replay()
    ok()
    codes, params = ops_ref.quantise(new)
    val = ops_ref.unpack(ops_ref.pack(codes), params)
    for b, n in ((0, 8), (1, 1)):
        assert ((out[0][b, :, :n].double() - val[b, :, :n]).abs()
                <= 2.0 ** -8 * val[b, :, :n].abs() + 1e-6).all()
        assert (out[0][b, :, n:] == 0).all()
