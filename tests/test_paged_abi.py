"""Refusals of the 16-bit paged caches' calls, before any work is launched, through
the C ABI and the binding (no GPU needed)."""
import ctypes

import pytest
import torch

from attention_forward_gb300 import _build, fa

NAN, INF = float("nan"), float("inf")
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def sizes(a, *names):
    return [a[n] for n in names]


POOL = [
    (dict(pool=0), 1), (dict(pool=8), 1), (dict(table=0), 1), (dict(table=2), 1), (dict(B=0), 1),
    (dict(pages=0), 1), (dict(per=0), 1), (dict(page=8), 1), (dict(page=24), 1), (dict(page=0), 1),
    (dict(page=2048), 1), (dict(page=1024, per=16385), 1), (dict(B=1 << 16), 1),
    (dict(pages=1 << 21, page=1024), 1), (dict(dtype=7), 2)]
ROWS = [(dict(k=0), 1), (dict(k=8), 1), (dict(v=0), 1), (dict(v=8), 1), (dict(S=0), 1),
        (dict(S=(1 << 24) + 1), 1), (dict(start=3), 1), (dict(count=2), 1)]


def base(**kw):
    a = dict(q=256, k=256, v=256, q_out=256, pool=256, table=256, start=None, count=None, freqs=256,
             rot=32, pairs=0, B=2, H=4, Hkv=2, S=3, D=64, width=576, pages=4, page=16, per=2, dtype=1,
             o=256, lse=256, length=256, Sq=1, scale=0.125, cap=0.0, slopes=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", POOL + ROWS + [
    (dict(Hkv=0), 1), (dict(D=96), 2), (dict(q=8), 1), (dict(q_out=8), 1), (dict(q_out=0), 1),
    (dict(H=3), 1), (dict(q=0), 1), (dict(freqs=2), 1), (dict(rot=0), 1), (dict(rot=24), 1),
    (dict(rot=80), 1), (dict(rot=-16), 1), (dict(freqs=None), 1), (dict(pairs=2), 1)])
def test_paged_write_refusals(lib, kw, want):
    a = base(**kw)
    assert lib.fa_paged_write(a["q"], a["k"], a["v"], a["q_out"], a["pool"], a["pool"], a["table"],
                              a["start"], a["count"], a["freqs"], a["rot"], a["pairs"],
                              *sizes(a, "B", "H", "Hkv", "S", "D", "pages", "page", "per", "dtype"),
                              None) == want


@pytest.mark.parametrize("kw,want", POOL + ROWS + [(dict(Hkv=0), 1), (dict(D=96), 2)])
def test_paged_read_refusals(lib, kw, want):
    a = base(**kw)
    assert lib.fa_paged_read(a["pool"], a["pool"], a["table"], a["start"], a["count"], a["k"], a["v"],
                             *sizes(a, "B", "Hkv", "S", "D", "pages", "page", "per", "dtype"),
                             None) == want


ATTEND = [(dict(q=0), 1), (dict(q=8), 1), (dict(o=8), 1), (dict(o=0), 1), (dict(lse=4), 1),
          (dict(length=0), 1), (dict(length=2), 1), (dict(Sq=0), 1), (dict(Sq=257), 1),
          (dict(scale=-1.0), 1), (dict(scale=INF), 1), (dict(scale=NAN), 1), (dict(H=0), 1)]


@pytest.mark.parametrize("kw,want", POOL + ATTEND + [
    (dict(H=3), 1), (dict(Hkv=0), 1), (dict(cap=-0.5), 1), (dict(cap=1e7), 1), (dict(slopes=1), 1),
    (dict(D=576), 2)])
def test_paged_attention_refusals(lib, kw, want):
    a = base(**kw)
    assert lib.fa_fwd_paged(a["q"], a["pool"], a["pool"], a["table"], a["length"], a["o"], a["lse"],
                            *sizes(a, "B", "H", "Hkv", "Sq", "D", "pages", "page", "per"),
                            F(a["scale"]), a["dtype"], F(a["cap"]), a["slopes"], None, 0,
                            None) == want


@pytest.mark.parametrize("kw,want", POOL + ROWS + [
    (dict(q=8), 1), (dict(q_out=8), 1), (dict(q_out=0), 1), (dict(q=0), 1), (dict(freqs=2), 1),
    (dict(H=0), 1), (dict(width=56), 1), (dict(width=196), 1), (dict(width=1 << 17), 1),
    (dict(pairs=-1), 1)])
def test_latent_write_refusals(lib, kw, want):
    a = base(**kw)
    assert lib.fa_latent_write(a["v"], a["k"], a["pool"], a["q"], a["q_out"], a["table"], a["start"],
                               a["count"], a["freqs"], a["pairs"],
                               *sizes(a, "B", "H", "S", "width", "pages", "page", "per", "dtype"),
                               None) == want


@pytest.mark.parametrize("kw,want", POOL + ROWS)
def test_latent_read_refusals(lib, kw, want):
    a = base(**kw)
    assert lib.fa_latent_read(a["pool"], a["table"], a["start"], a["count"], a["v"], a["k"],
                              *sizes(a, "B", "S", "pages", "page", "per", "dtype"), None) == want


@pytest.mark.parametrize("kw,want", POOL + ATTEND)
def test_latent_attention_refusals(lib, kw, want):
    a = base(**kw)
    assert lib.fa_fwd_latent(a["q"], a["pool"], a["table"], a["length"], a["o"], a["lse"],
                             *sizes(a, "B", "H", "Sq", "pages", "page", "per"), F(a["scale"]),
                             a["dtype"], None, 0, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), 1), (dict(q=8), 1), (dict(k=0), 1), (dict(k=8), 1), (dict(v=0), 1), (dict(v=8), 1),
    (dict(o=0), 1), (dict(o=8), 1), (dict(lse=0), 1), (dict(lse=4), 1), (dict(B=0), 1),
    (dict(H=0), 1), (dict(B=1 << 14), 1), (dict(Sq=0), 1), (dict(S=0), 1), (dict(S=(1 << 24) + 1), 1),
    (dict(Sq=(1 << 24) + 1), 1), (dict(scale=0.0), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1),
    (dict(dtype=2), 2), (dict(ws=128), 4)])
def test_expanded_refusals(lib, kw, want):
    a = base(ws=None, **kw) if "ws" not in kw else base(**kw)
    assert lib.fa_fwd_expanded(a["q"], a["v"], a["k"], a["o"], a["lse"], a["B"], a["H"], a["Sq"],
                               a["S"], F(a["scale"]), 1, a["dtype"], a["ws"], 0, None) == want


def test_workspace_sizes():
    assert fa.fa_expanded_workspace_bytes(0, 4, 8, 8) == 0
    assert fa.fa_expanded_workspace_bytes(1, 4, 100, 100) == 0        # one key tile
    assert fa.fa_expanded_workspace_bytes(8, 32, 4096, 4096) == 0     # items enough
    n = fa.fa_expanded_workspace_bytes(1, 4, 100, 16384)
    assert n >= 2 * 4 * 100 * 129 * 4 and n % 256 == 0
    assert fa.fa_paged_workspace_bytes(1, 4, 3, 1, 64, 16, 4) == 0    # refused sizes need none
    assert fa.fa_paged_workspace_bytes(1, 4, 1, 257, 64, 16, 400) == 0
    assert fa.fa_paged_workspace_bytes(1, 4, 1, 1, 64, 16, 4) == 0    # short: not split
    assert fa.fa_latent_workspace_bytes(1, 4, 1, 16, 4) == 0
    n = fa.fa_paged_workspace_bytes(1, 4, 1, 1, 64, 16, 1024)
    assert n >= 2 * 2 * 16 * 65 * 4 and n % 256 == 0
    n = fa.fa_latent_workspace_bytes(1, 4, 1, 16, 1024)
    assert n >= 2 * 2 * 16 * 513 * 4 and n % 256 == 0
    # however long: the parts of what the GPU holds at once
    assert fa.fa_paged_workspace_bytes(64, 32, 8, 1, 64, 16, 1 << 20) <= 2 * 2000 * 16 * 65 * 4
    assert fa.fa_latent_workspace_bytes(64, 128, 1, 16, 1 << 20) <= 2 * 500 * 64 * 513 * 4


LIMIT, PAGE = 2 ** 31 - 256, 1024


@pytest.mark.parametrize("B,H,Hkv,Sq,blocks", [(64, 64, 8, 256, 64 * 8 * 32), (9000, 4, 1, 2, 9000),
                                               (12000, 5, 1, 5, 12000)])
def test_more_chunks_than_are_counted(lib, B, H, Hkv, Sq, blocks):
    most = (LIMIT // blocks - 1) // (PAGE // 64)  # pages
    assert (most + 1) * PAGE <= 1 << 24  # within the table's own limit
    assert fa.fa_paged_workspace_bytes(B, H, Hkv, Sq, 64, PAGE, most) > 0
    assert fa.fa_paged_workspace_bytes(B, H, Hkv, Sq, 64, PAGE, most + 1) == 0
    assert lib.fa_fwd_paged(256, 256, 256, 256, 256, 256, 256, B, H, Hkv, Sq, 64, 4, PAGE, most + 1,
                            F(0.125), 1, F(0.0), None, None, 0, None) == fa.FA_ERR_INVALID_ARG


def test_binding_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    kv, q = torch.zeros(1, 2, 8, 64, dtype=bf), torch.zeros(1, 4, 8, 64, dtype=bf)
    cache = fa.fa_paged_empty(2, 2, 16, 64, device="cpu")
    assert [t.shape for t in cache] == [(2, 2, 16, 64)] * 2 and cache[0].dtype is bf
    latent = fa.fa_latent_empty(2, 16, torch.float16, device="cpu")
    assert latent.shape == (2, 16, 576) and latent.dtype is torch.float16
    table, length = torch.zeros((1, 2), dtype=i32), torch.zeros(1, dtype=i32)
    c, r = torch.zeros(1, 8, 512, dtype=bf), torch.zeros(1, 8, 64, dtype=bf)
    wide = torch.zeros(1, 4, 8, 576, dtype=bf)
    for call in (lambda: fa.fa_paged_write(kv, kv, cache, table),  # not on a GPU
                 lambda: fa.fa_paged_read(cache, table),
                 lambda: fa.fa_paged_read(cache, table, out=[kv, kv]),
                 lambda: fa.fa_fwd_paged(q, cache, table, length),
                 lambda: fa.fa_paged_empty(2, 2, 16, 96),
                 lambda: fa.fa_paged_empty(2, 2, 16, 64, torch.float32),
                 lambda: fa.fa_latent_empty(2, 16, torch.float32),
                 lambda: fa.fa_latent_write(c, r, latent, table),
                 lambda: fa.fa_latent_read(latent, table),
                 lambda: fa.fa_latent_read(latent, table, out=[c, r]),
                 lambda: fa.fa_fwd_latent(q, latent, table, length),
                 lambda: fa.fa_fwd_latent(wide, latent, table, length),
                 lambda: fa.fa_fwd_expanded(torch.zeros(1, 4, 8, 192, dtype=bf),
                                            torch.zeros(1, 4, 8, 256, dtype=bf), r)):
        with pytest.raises(ValueError):
            call()
