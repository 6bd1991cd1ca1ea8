"""Refusals of fa_fwd_score and the 4-bit cache's calls, before any work is
launched, through the C ABI and the binding (no GPU needed)."""
import ctypes

import pytest
import torch

from attention_forward_gb300 import _build, fa


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def score(lib, **kw):
    a = dict(q=256, k=256, v=256, o=256, lse=256, B=1, H=4, Hkv=2, Sq=8, Skv=8, D=64, scale=0.125,
             causal=1, dtype=1, cap=0.0, slopes=None, doc_q=None, doc_k=None, prefix=None,
             ws=None, ws_bytes=0)
    a.update(kw)
    return lib.fa_fwd_score(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["H"], a["Hkv"],
                            a["Sq"], a["Skv"], a["D"], ctypes.c_float(a["scale"]), a["causal"],
                            a["dtype"], ctypes.c_float(a["cap"]), a["slopes"], a["doc_q"],
                            a["doc_k"], a["prefix"], a["ws"], a["ws_bytes"], None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=8), 1), (dict(o=24), 1), (dict(lse=4), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(Hkv=8), 1),
    (dict(Sq=0), 1), (dict(Skv=0), 1), (dict(Skv=(1 << 24) + 1), 1), (dict(B=1 << 14), 1),
    (dict(scale=0.0), 1), (dict(scale=NAN), 1), (dict(cap=-1.0), 1), (dict(cap=NAN), 1),
    (dict(cap=INF), 1), (dict(cap=1e-7), 1), (dict(cap=2e6), 1), (dict(slopes=2), 1),
    (dict(doc_q=256), 1), (dict(doc_k=256), 1), (dict(doc_q=256, doc_k=258), 1),
    (dict(prefix=256, causal=0), 1), (dict(prefix=257), 1), (dict(D=96), 2), (dict(dtype=2), 2),
])
def test_score_refusals(lib, kw, want):
    assert score(lib, **kw) == want


def cache_args(**kw):
    a = dict(k=256, v=256, kc=256, kp=256, vc=256, vp=256, table=256, start=None, count=None, B=2,
             Hkv=2, S=3, D=64, pages=4, page=16, per=2, dtype=1)
    a.update(kw)
    return a


CACHE_REFUSALS = [
    (dict(kc=0), 1), (dict(kp=8), 1), (dict(vc=4), 1), (dict(vp=0), 1), (dict(table=0), 1),
    (dict(table=2), 1), (dict(B=0), 1), (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(per=0), 1),
    (dict(page=8), 1), (dict(page=24), 1), (dict(page=0), 1), (dict(page=2048), 1),
    (dict(page=1024, per=16385), 1), (dict(B=1 << 15, Hkv=2), 1), (dict(D=32), 2),
    (dict(dtype=7), 2),
]


@pytest.mark.parametrize("kw,want", CACHE_REFUSALS + [
    (dict(k=0), 1), (dict(v=8), 1), (dict(S=0), 1), (dict(S=(1 << 24) + 1), 1),
    (dict(start=3), 1), (dict(count=2), 1)])
def test_cache_copy_refusals(lib, kw, want):
    a = cache_args(**kw)
    tail = (a["table"], a["start"], a["count"])
    sizes = (a["B"], a["Hkv"], a["S"], a["D"], a["pages"], a["page"], a["per"], a["dtype"], None)
    pool = (a["kc"], a["kp"], a["vc"], a["vp"])
    assert lib.fa_cache_write(a["k"], a["v"], *pool, *tail, *sizes) == want
    assert lib.fa_cache_read(*pool, *tail, a["k"], a["v"], *sizes) == want


@pytest.mark.parametrize("kw,want", CACHE_REFUSALS + [
    (dict(q=0), 1), (dict(o=8), 1), (dict(lse=4), 1), (dict(length=0), 1), (dict(length=2), 1),
    (dict(H=3), 1), (dict(Sq=0), 1), (dict(Sq=257), 1), (dict(scale=-1.0), 1),
    (dict(scale=INF), 1), (dict(cap=-0.5), 1), (dict(cap=1e7), 1), (dict(slopes=1), 1)])
def test_cache_attention_refusals(lib, kw, want):
    a = dict(cache_args(), q=256, o=256, lse=256, length=256, H=4, Sq=1, scale=0.125,
             cap=0.0, slopes=None)
    a.update(kw)
    got = lib.fa_fwd_cache(a["q"], a["kc"], a["kp"], a["vc"], a["vp"], a["table"], a["length"],
                           a["o"], a["lse"], a["B"], a["H"], a["Hkv"], a["Sq"], a["D"], a["pages"],
                           a["page"], a["per"], ctypes.c_float(a["scale"]), a["dtype"],
                           ctypes.c_float(a["cap"]), a["slopes"], None, 0, None)
    assert got == want


def test_workspace_sizes(lib):
    assert fa.fa_score_workspace_bytes(1, 4, 3, 8, 8, 64) == 0       # refused sizes need none
    assert fa.fa_score_workspace_bytes(1, 4, 2, 8, 8, 64) == 0       # one key tile
    docs = fa.fa_score_workspace_bytes(2, 4, 4, 500, 1000, 64, True)
    assert docs >= 2 * 8 * 12 + 2 * 4 * 8 and docs % 256 == 0
    split = fa.fa_score_workspace_bytes(1, 4, 1, 1, 8192, 128)
    assert split >= 2 * 4 * 129 * 4 and split % 256 == 0
    assert fa.fa_cache_workspace_bytes(1, 4, 3, 1, 64, 16, 4) == 0
    assert fa.fa_cache_workspace_bytes(1, 4, 1, 1, 64, 16, 4) == 0    # short: not split
    n = fa.fa_cache_workspace_bytes(1, 4, 1, 1, 64, 16, 1024)
    assert n >= 2 * 2 * 8 * 65 * 4 and n % 256 == 0
    # however long: the parts of what the GPU holds at once
    assert fa.fa_cache_workspace_bytes(64, 32, 8, 1, 64, 16, 1 << 20) <= 2 * 2000 * 16 * 65 * 4


def test_binding_refusals():
    q = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16)
    kv = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    cache = fa.fa_cache_empty(2, 2, 16, 64, device="cpu")
    assert cache[0].shape == (2, 2, 16, 32) and cache[1].shape == (2, 2, 16, 2, 2)
    table = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_fwd_score(q, kv, kv)  # not on a GPU
    with pytest.raises(ValueError):
        fa.fa_cache_write(kv, kv, cache, table)
    with pytest.raises(ValueError):
        fa.fa_cache_read(cache, table)
    with pytest.raises(ValueError):
        fa.fa_cache_read(cache, table, out=[kv, kv])
    with pytest.raises(ValueError):
        fa.fa_fwd_cache(q, cache, table, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.fa_fwd_cache(q, cache[:2], table, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.fa_cache_empty(2, 2, 16, 96, device="cpu")
