"""Latent attention with its heads expanded, and the run of a latent layer's
operators as a server makes it, within the bounds of paged_ref.py."""
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


def ok():
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


def normal(seed, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def inputs(B, H, Sq, Skv, dt, seed=1):
    return (normal(seed, B, H, Sq, 192).to(DT[dt]), normal(seed + 1, B, H, Skv, 256).to(DT[dt]),
            normal(seed + 2, B, Skv, 64).to(DT[dt]))


def expect(q, kv, k_rope, causal, scale=SCALE):
    B, H, Sq, _ = q.shape
    Skv = kv.shape[2]
    k = torch.cat([kv[..., :128], k_rope[:, None].expand(B, H, Skv, 64)], -1)
    i = torch.arange(Sq, device="cuda")[:, None] + (Skv - Sq)
    j = torch.arange(Skv, device="cuda")[None]
    seen = (j <= i) if causal else torch.ones((Sq, Skv), dtype=torch.bool, device="cuda")
    return paged_ref.attention(q, k, kv[..., 128:], seen[None, None], scale)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,Sq,Skv", [
    (1, 1, 1, 1), (2, 3, 1, 17), (1, 2, 17, 17), (1, 1, 128, 128), (2, 2, 129, 200), (1, 5, 256, 256),
    (1, 3, 300, 300), (2, 4, 509, 1500), (1, 2, 513, 129), (1, 1, 700, 64), (1, 40, 1000, 1000),
    (3, 60, 257, 385), (1, 1, 64, 5000)])
def test_attention(B, H, Sq, Skv, causal, dt):
    """Rows that see nothing (more queries than keys under the mask), odd ends, whole
    and split keys, more items than multiprocessors."""
    x = inputs(B, H, Sq, Skv, dt)
    o, lse = fa.fa_fwd_expanded(*x, causal=causal)
    ok()
    ops_ref.check(o, lse, expect(*x, causal))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
def test_scores_that_rise_along_the_keys(causal, dt):
    q, kv, r = inputs(1, 4, 520, 900, dt, 4)
    at = torch.arange(900, device="cuda")
    r[..., 0], r[..., 1] = (at / 900 * 30).to(DT[dt]), ((at % 200) / 200 * 30).to(DT[dt])
    q[:, ::2, :, 128], q[:, 1::2, :, 129], q[:, 3, :, 128] = 8.0, 8.0, -8.0
    o, lse = fa.fa_fwd_expanded(q, kv, r, causal=causal, scale=0.3)
    ok()
    ops_ref.check(o, lse, expect(q, kv, r, causal, 0.3))


def test_masked_keys_may_hold_anything():
    q, kv, r = inputs(1, 2, 200, 200, "bf16", 7)
    ref = expect(q[:, :, :100], kv[:, :, :100], r[:, :100], True)
    kv[:, :, 100:, :128], r[:, 100:] = math.nan, math.inf
    o, lse = fa.fa_fwd_expanded(q, kv, r, causal=True)
    ok()
    ops_ref.check(o[:, :, :100].contiguous(), lse[:, :, :100].contiguous(), ref)


def test_a_nan_reaches_the_rows_that_see_it():
    q, kv, r = inputs(1, 2, 300, 300, "fp16", 8)
    kv[0, 1, 150, 5] = math.nan
    o, lse = fa.fa_fwd_expanded(q, kv, r, causal=True)
    ok()
    assert o[0, 1, 150:].isnan().all() and lse[0, 1, 150:].isnan().all()
    assert o[0, 0].isfinite().all() and o[0, 1, :150].isfinite().all()


def test_caller_workspace_and_rows_behind_the_outputs():
    """Split and unsplit by the workspace given; what lies behind the outputs stays."""
    q, kv, r = inputs(1, 2, 130, 4000, "bf16", 9)
    need = fa.fa_expanded_workspace_bytes(1, 2, 130, 4000)
    assert need > 0
    ref = expect(q, kv, r, True)
    for size in (need, 256):
        big, tail = torch.full((2 * 130 * 128 + 4096,), 3.0, device="cuda").bfloat16(), 4096
        l_big = torch.full((2 * 130 + 64,), 3.0, device="cuda")
        o, lse = big[:-tail].view(1, 2, 130, 128), l_big[:-64].view(1, 2, 130)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        fa.fa_fwd_expanded(q, kv, r, causal=True, workspace=ws, out=o, lse=lse)
        ok()
        ops_ref.check(o, lse, ref)
        assert (big[-tail:] == 3.0).all() and (l_big[-64:] == 3.0).all()


def test_two_streams_and_graphs_at_once():
    q, kv, r = inputs(1, 4, 300, 3000, "bf16", 10)
    ref = fa.fa_fwd_expanded(q, kv, r, causal=True)
    ok()
    graphs, got = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(fa.fa_fwd_expanded(q, kv, r, causal=True))
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(15):
        for s in streams[:2]:
            got.append(fa.fa_fwd_expanded(q, kv, r, causal=True, stream=s))
        for s, g in zip(streams[2:], graphs):
            with torch.cuda.stream(s):
                g.replay()
    ok()
    for o, lse in got:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


# ------------------------------------------------------------ together

@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_layer_from_prompt_to_decode(dt):
    """A prompt into the latent cache, read back, expanded and attended; a further
    chunk over what is cached; then decode steps in the absorbed form, captured once,
    whose outputs through the value expansion are the expanded form's."""
    B, H, page, per = 2, 6, 16, 24
    seeds = iter(range(100, 999))
    n = lambda *s: normal(next(seeds), *s).to(DT[dt])  # noqa: E731
    wk, wv = (normal(next(seeds), H, 512, 128) / 512 ** 0.5 for _ in range(2))
    j = torch.arange(32, dtype=torch.float64, device="cuda")
    freqs = (10000.0 ** (-j / 32)).float()
    cache = fa.fa_latent_empty(B * per, page, DT[dt])
    order = list(range(B * per))
    random.Random(3).shuffle(order)
    table = ints(order).view(B, per)

    def expanded(c):  # [B, S, 512] -> kv [B, H, S, 256], one product
        w = torch.cat([wk, wv], -1).to(DT[dt])
        return torch.matmul(c[:, None], w[None]).contiguous()

    done = 0
    for S in (200, 57):  # the prompt, then a chunk behind it
        c, r, qr = n(B, S, 512), n(B, S, 64), n(B, H, S, 64)
        q = n(B, H, S, 192)
        start = ints([done] * B)
        fa.fa_latent_write(c, r, cache, table, start, freqs=freqs, interleaved=True, q_rope=qr, q=q)
        done += S
        call, rall = (torch.empty((B, done, w), dtype=DT[dt], device="cuda") for w in (512, 64))
        fa.fa_latent_read(cache, table, out=(call, rall))
        kv = expanded(call)
        o, lse = fa.fa_fwd_expanded(q, kv, rall, causal=True)
        ok()
        at = done - S + torch.arange(S, device="cuda")
        for b in range(B):
            paged_ref.close(q[b, :, :, 128:], *paged_ref.rotate(qr[b], at, freqs, True))
            paged_ref.close(rall[b, done - S:], *paged_ref.rotate(r[b], at, freqs, True))
        assert torch.equal(call[:, done - S:], c)
        ops_ref.check(o, lse, expect(q, kv, rall, True))

    length = ints([done, done])
    c1, r1, qr1 = n(B, 1, 512), n(B, 1, 64), n(B, H, 1, 64)
    qn = n(B, H, 1, 128)
    q1 = torch.zeros((B, H, 1, 576), dtype=DT[dt], device="cuda")
    o1 = torch.empty((B, H, 1, 512), dtype=DT[dt], device="cuda")
    l1 = torch.empty((B, H, 1), device="cuda")

    def step():
        q1[..., :512] = torch.einsum("bhsd,hcd->bhsc", qn, wk.to(DT[dt]))
        fa.fa_latent_write(c1, r1, cache, table, length, freqs=freqs, interleaved=True, q_rope=qr1,
                           q=q1)
        length.add_(1)
        fa.fa_fwd_latent(q1, cache, table, length, out=o1, lse=l1)

    step()
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(10):
        for t in (c1, r1, qr1, qn):
            t.copy_(n(*t.shape))
        graph.replay()
        ok()
        ops_ref.check(o1, l1, paged_ref.newest(q1, cache, None, table, length, SCALE))
    assert length.tolist() == [done + 11] * B

    # the last step in the expanded form: the same scores and outputs, but for the
    # roundings of q W (absorbed) and c W (expanded) to 16 bits and of P and O
    L = done + 11
    call, rall = (torch.empty((B, L, w), dtype=DT[dt], device="cuda") for w in (512, 64))
    fa.fa_latent_read(cache, table, out=(call, rall))
    qe = torch.cat([qn, q1[..., 512:]], -1).contiguous()
    o2, l2 = fa.fa_fwd_expanded(qe, expanded(call), rall, causal=True)
    ok()
    u = torch.finfo(DT[dt]).eps / 2
    wk64, wv64 = wk.to(DT[dt]).double(), wv.to(DT[dt]).double()
    k64 = torch.einsum("bsc,hcd->bhsd", call.double(), wk64)
    q64 = torch.einsum("bhsd,hcd->bhsc", qn.double(), wk64)
    # a score's error by either path: u times the sums that were rounded
    room = (qn.double().abs() @ k64.abs().transpose(2, 3)
            + q64.abs() @ call.double().abs().transpose(1, 2)[:, None]).amax(-1) * SCALE * u
    assert ((l1 - l2).double().abs() <= room + 1e-4).all()
    v64 = torch.einsum("bsc,hcd->bhsd", call.double(), wv64)
    mine = torch.einsum("bhsc,hcd->bhsd", o1.double(), wv64)
    # probabilities off by that at most, and each rounded once; the values (v) and the
    # latent sums (o1) rounded once, the latter through the expansion
    most = v64.abs().amax(2, keepdim=True)
    through = torch.einsum("bhsc,hcd->bhsd", o1.double().abs(), wv64.abs())
    latent_p = torch.einsum("bsc,hcd->bhsd", call.double().abs(), wv64.abs()).amax(2, keepdim=True)
    tol = (4 * room[..., None] + 4 * u) * most + u * through + u * latent_p + 1e-4
    assert ((o2.double() - mine).abs() <= tol).all()
